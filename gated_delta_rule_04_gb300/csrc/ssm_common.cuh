// Shared by the kernels of the selective state space mixer (sm_103a).
#pragma once

#include <cuda.h>

#include "kda_common.cuh"

namespace kda {
namespace ssm {

// The tables of a call of a few sequences travel in the kernel arguments; more
// sequences have them built on the device.
constexpr int INLINE_SEQS = 16;
struct InlineMeta {
    int32_t n;                            // 0: the tables in global memory
    int32_t cu[INLINE_SEQS + 1];          // token offsets (below 2^31: checked on the host)
    int32_t coff[INLINE_SEQS + 1];        // first chunk of each sequence (chunked form)
    uint8_t order[INLINE_SEQS];           // longest first
};

// One prefill call, as the kernels see it.  Channels: x (W = H*P) | B (G*N) |
// C (G*N), Cx = W + 2 G N in all; rows of xbc, dt and z are `*_stride`
// elements apart, rows of o packed.
struct PrefillArgs {
    const void *xbc, *dt, *z;
    int64_t xbc_stride, dt_stride, z_stride;
    const float *conv_w, *conv_b, *A_log, *dt_bias, *skip;
    const float* S_in;
    float* S_out;
    const void* ring_in;
    void* ring_out;
    void* o;
    const int64_t* cu;       // device [n_seqs + 1]
    const int32_t* order;    // device [n_seqs], longest first
    int32_t n_seqs, H, G, P, N;
    int64_t T;               // total tokens
    InlineMeta meta;         // instead of cu and order, if meta.n > 0
};
__device__ __forceinline__ int64_t seq_start(const PrefillArgs& g, int n) { return g.meta.n ? g.meta.cu[n] : g.cu[n]; }
__device__ __forceinline__ int seq_at(const PrefillArgs& g, int i) { return g.meta.n ? g.meta.order[i] : g.order[i]; }

struct DecodeArgs {
    const void *xbc, *dt, *z;
    int64_t xbc_stride, dt_stride, z_stride;
    const float *conv_w, *conv_b, *A_log, *dt_bias, *skip;
    const int32_t* slots;
    float* S;
    void* ring;
    void* o;
    float* u;                // workspace [n][Cx] fp32: the conv's outputs (where decode_needs_workspace)
    float2* step;            // workspace [n][H]: dt and the decay
    int32_t n, n_slots, H, G, P, N;
};

// softplus without overflow; exact to fp32 rounding on both sides
__device__ __forceinline__ float softplus(float x) { return x > 20.f ? x : log1pf(expf(x)); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp(x) of a token's decay, x <= 0, next to 1 rounded to nearest: expf's error there has one
// sign, and a state that takes the factor at every token adds it up (3e-5 after 3000 tokens of
// a decay of 1.7e-4 each, 1.3e-6 this way).  The Taylor polynomial of degree 4 leaves 5e-10 of
// the distance from 1; below it a state forgets the errors.  (1 + expm1f(x): the same, fp32
// prompts of 601 tokens x 8 heads 32.5 us, not 30.8.)
__device__ __forceinline__ float decay(float x) {
    if (x <= -1.f / 64) return expf(x);
    const float p = fmaf(fmaf(fmaf(1.f / 24, x, 1.f / 6), x, 0.5f), x, 1.f);
    return fmaf(p, x, 1.f);
}

// SiLU to fp32 rounding, 8 x 2^-24 at any x (zero below -87): these values reach the fp32
// state.  The exponent -x log2(e) = h + t log2(e) in two parts (as Cody and Waite split an
// argument): h rounded, t = -x - h ln(2) what that lost, e^t = 1 + t.  With the rounded
// exponent alone the error grows with |x|, to 2^-18 at -40; expf and a division took 45
// us where this takes 31 (fp32 prompts, 601 tokens x 8 heads).
__device__ __forceinline__ float silu(float x) {
    const float c = fminf(fmaxf(x, -88.f), 88.f), h = c * -1.44269504f;
    float t = fmaf(h, -0.693359375f, -c);                    // ln(2) in a few bits
    t = fmaf(h, 2.12194440e-4f, t);                          // and the rest of it
    const float e = ex2(h);
    return x * rcp(1.f + fmaf(e, t, e));
}

// Two SiLUs, the arithmetic around the special functions packed.  (One
// reciprocal for both denominators saves a special-function operation and
// costs five others; those units are the least used ones here.)
__device__ __forceinline__ float2 silu2(float2 x) {
    constexpr float L = -1.4426950408889634f;
    const float2 t = __fmul2_rn(x, make_float2(L, L));
    const float2 d = __fadd2_rn(make_float2(ex2(t.x), ex2(t.y)), make_float2(1.f, 1.f));
    return __fmul2_rn(x, make_float2(rcp(d.x), rcp(d.y)));
}

// TMA descriptor of T rows of W values of `es` bytes (2: bf16, 4: fp32), `stride`
// values apart: boxes of `rows` rows x `cols` values, zero fill out of bounds.
bool encode_rows(CUtensorMap* m, const void* base, int es, int64_t T, int64_t W, int64_t stride, uint32_t rows, uint32_t cols);

// `status`: the workspace's error word, which the scan clears.
cudaError_t launch_scan(const PrefillArgs& a, int io_bf16, int32_t* status, cudaStream_t s);
cudaError_t launch_ring(const PrefillArgs& a, int io_bf16, cudaStream_t s);
cudaError_t launch_decode(const DecodeArgs& a, int io_bf16, cudaStream_t s);
// Whether a call of n sessions runs in two kernels, through the workspace.
bool decode_needs_workspace(int64_t n, int H, int G, int P, int N);

}  // namespace ssm
}  // namespace kda
