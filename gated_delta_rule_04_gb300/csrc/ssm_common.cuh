// Shared by the kernels of the selective state space mixer (sm_103a).
#pragma once

#include "kda_common.cuh"

namespace kda {
namespace ssm {

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
};

struct DecodeArgs {
    const void *xbc, *dt, *z;
    int64_t xbc_stride, dt_stride, z_stride;
    const float *conv_w, *conv_b, *A_log, *dt_bias, *skip;
    const int32_t* slots;
    float* S;
    void* ring;
    void* o;
    float* u;                // workspace [n][Cx] fp32: the conv's outputs
    int32_t n, n_slots, H, G, P, N;
};

// softplus without overflow; exact to fp32 rounding on both sides
__device__ __forceinline__ float softplus(float x) { return x > 20.f ? x : log1pf(expf(x)); }

// SiLU to fp32 rounding: these values reach the fp32 state
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two SiLUs at once (packed fp32 arithmetic), with one reciprocal of the
// product of the denominators, each at most 1 + 2^60: three special-function
// operations instead of four.  (Below x = -41.6 the result is x 2^-60 instead
// of something smaller still.)
__device__ __forceinline__ float2 silu2(float2 x) {
    constexpr float L = -1.4426950408889634f;
    const float2 t = __fmul2_rn(x, make_float2(L, L));
    const float2 d = __fadd2_rn(make_float2(ex2(fminf(t.x, 60.f)), ex2(fminf(t.y, 60.f))), make_float2(1.f, 1.f));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d.x * d.y));
    return __fmul2_rn(x, __fmul2_rn(make_float2(d.y, d.x), make_float2(r, r)));
}

cudaError_t launch_scan(const PrefillArgs& a, int io_bf16, cudaStream_t s);
cudaError_t launch_ring(const PrefillArgs& a, int io_bf16, cudaStream_t s);
cudaError_t launch_decode(const DecodeArgs& a, int io_bf16, cudaStream_t s);

}  // namespace ssm
}  // namespace kda
