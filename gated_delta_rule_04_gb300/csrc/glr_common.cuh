// Shared by the kernels of the gated linear recurrence (sm_103a).
#pragma once

#include "kda_common.cuh"

namespace kda {
namespace glr {

constexpr int CHUNK = KDA_GLR_CHUNK;
constexpr int INLINE_SEQS = 16;

// The token offsets of a call of few sequences travel in the kernel arguments;
// those of more are built on the device.
struct Offsets {
    int32_t n;                       // sequences
    int32_t cu[INLINE_SEQS + 1];     // where n <= INLINE_SEQS
    const int64_t* d_cu;             // device [n + 1] otherwise
};
__device__ __forceinline__ int64_t seq_start(const Offsets& f, int n) {
    return f.n <= INLINE_SEQS ? f.cu[n] : f.d_cu[n];
}

// One prefill or backward call, as the kernels see it.  Rows of the token
// tensors are `*_s` elements apart, rows of o packed.
struct ScanArgs {
    const void *x, *r, *i, *z;
    int64_t x_s, r_s, i_s, z_s;
    const float *A_log, *r_bias, *i_bias;
    const float* S_in;
    float* S_out;
    float* states;                   // [ceil(T / CHUNK)][C]: written by the prefill, read by the backward pass
    void* o;
    const void* d_o;                 // gradients from here on
    int64_t do_s;
    const float* dS_out;
    void *dx, *dr, *di, *dz;
    int64_t dx_s, dr_s, di_s, dz_s;
    float *dS_in, *dA_log, *dr_bias, *di_bias;
    float* part;                     // workspace: partial sums of the parameters' gradients
    int64_t T;
    int32_t C;
    Offsets f;
};

struct TokenArgs {
    const void *x, *r, *i, *z;
    int64_t x_s, r_s, i_s, z_s;
    const float *A_log, *r_bias, *i_bias;
    const int32_t *path, *path_len;  // NULL: all tokens in order
    const int32_t* slots;
    const float* S_in;
    float* S_out;                    // NULL: the states stay
    void* o;                         // NULL: states only
    int32_t n, n_tokens, max_len, n_slots, C;
};

cudaError_t launch_scan(const ScanArgs& a, int io_bf16, cudaStream_t s);
cudaError_t launch_backward(const ScanArgs& a, int io_bf16, cudaStream_t s);
cudaError_t launch_tokens(const TokenArgs& a, int io_bf16, cudaStream_t s);

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// What a token does to a channel's state: h -> a h + m v x.
struct Step {
    float w, v, la, a, m;
};
__device__ __forceinline__ Step step_of(float r, float i, float neg_ea) {
    Step s;
    s.w = sigmoid(r);
    s.v = sigmoid(i);
    s.la = neg_ea * s.w;
    s.a = expf(s.la);
    s.m = sqrtf(-expm1f(2.f * s.la));
    return s;
}

}  // namespace glr
}  // namespace kda
