// Shared by the kernels of the gated linear recurrence (sm_103a).
#pragma once

#include "kda_common.cuh"

namespace kda {
namespace glr {

constexpr int CHUNK = KDA_GLR_CHUNK;
constexpr int INLINE_SEQS = 16;
constexpr int TILE_C = 64;           // channels of a tile; its tokens are a CHUNK

// The sequences of a call that have tokens, in order.  Few travel in the kernel
// arguments; more are built on the device.
struct Sequences {
    int32_t n;                       // sequences with tokens
    int32_t cu[INLINE_SEQS + 1];     // where n <= INLINE_SEQS: their first tokens, and T
    int32_t id[INLINE_SEQS];         // their rows of S_in and S_out
    const int64_t* d_cu;             // device [n + 1] and [n] otherwise
    const int32_t* d_id;
};
__device__ __forceinline__ int seq_id(const Sequences& f, int s) { return f.n <= INLINE_SEQS ? f.id[s] : f.d_id[s]; }

// One prefill or backward call, as the kernels see it.  Rows of the token
// tensors are `*_s` bytes apart.
struct ScanArgs {
    const void *x, *r, *i, *z;
    uint32_t x_s, r_s, i_s, z_s;
    const float *A_log, *r_bias, *i_bias;
    const float* S_in;
    float* S_out;
    float* states;                   // [ceil(T / CHUNK)][C]: written by the prefill, read by the backward pass
    void* o;
    uint32_t o_s;
    const void* d_o;                 // gradients from here on
    uint32_t do_s;
    const float* dS_out;
    void *dx, *dr, *di, *dz;
    uint32_t dx_s, dr_s, di_s, dz_s;
    float *dS_in, *dA_log, *dr_bias, *di_bias;
    int64_t T;
    int32_t C;
    Sequences f;
    // workspace
    int32_t* status;                 // error word
    float2* gates;                   // [tiles along C][3][TILE_C / 2]: see load_gate
    uint4* borders;                  // [tiles along T]: see borders()
    uint32_t* ticket;                // the next tile to be taken, and behind it
    float* map;                      // [tiles along T][tiles along C][TILE_C][2]
    float* val;                      // [tiles along T][tiles along C][TILE_C]
    size_t empty;                    // 16-byte words, from the ticket on, that are set to EMPTY first
    int32_t alone;                   // the walk's kernel sets up and adds up by itself
    float* part;                     // [tiles along T][3][C]: partial sums of the parameters' gradients
    int32_t tiles_t, tiles_c;
};

struct TokenArgs {
    const void *x, *r, *i, *z;
    uint32_t x_s, r_s, i_s, z_s;     // bytes between rows
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

}  // namespace glr
}  // namespace kda
