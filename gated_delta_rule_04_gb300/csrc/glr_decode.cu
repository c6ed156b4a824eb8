// Tokens of the gated linear recurrence over a pool of states: straight runs of
// 1 to 64 tokens per session, and the accepted paths of a round.  A thread per
// (session, channel) walks the tokens with its state in a register.
#include "glr_common.cuh"

namespace kda {
namespace glr {
namespace {

constexpr int NT = 128;

template <typename TI>
__global__ void __launch_bounds__(NT) token_kernel(const __grid_constant__ TokenArgs g) {
    const int blocks = (g.C + NT - 1) / NT;
    const int n = blockIdx.x / blocks, c = blockIdx.x % blocks * NT + threadIdx.x;
    const int slot = g.slots ? g.slots[n] : n;
    if (slot < 0 || slot >= g.n_slots) return;
    int len = g.n_tokens;
    const int32_t* path = g.path ? g.path + (size_t)n * g.max_len : nullptr;
    if (path) {                                       // a session with an entry out of range is skipped
        len = g.path_len[n];
        if (len < 0 || len > g.max_len) return;
        bool bad = false;
        for (int j = 0; j < len; ++j) bad |= path[j] < 0 || path[j] >= g.n_tokens;
        if (bad) return;
    }
    if (c >= g.C) return;
    const float ea = -expf(g.A_log[c]), rb = g.r_bias ? g.r_bias[c] : 0.f, ib = g.i_bias ? g.i_bias[c] : 0.f;
    float h = g.S_in[(size_t)slot * g.C + c];
    for (int j = 0; j < len; ++j) {
        const int64_t row = (int64_t)n * g.n_tokens + (path ? path[j] : j);
        const Step s = step_of(to_f32(static_cast<const TI*>(g.r)[row * g.r_s + c]) + rb,
                               to_f32(static_cast<const TI*>(g.i)[row * g.i_s + c]) + ib, ea);
        h = fmaf(s.a, h, s.m * s.v * to_f32(static_cast<const TI*>(g.x)[row * g.x_s + c]));
        if (g.o) {
            float o = h;
            if (g.z) {
                const float z = to_f32(static_cast<const TI*>(g.z)[row * g.z_s + c]);
                o *= z * sigmoid(z);
            }
            static_cast<TI*>(g.o)[row * g.C + c] = from_f32<TI>(o);
        }
    }
    if (g.S_out) g.S_out[(size_t)slot * g.C + c] = h;
}

}  // namespace

cudaError_t launch_tokens(const TokenArgs& a, int io_bf16, cudaStream_t s) {
    const unsigned grid = (unsigned)((int64_t)a.n * ((a.C + NT - 1) / NT));
    if (io_bf16) token_kernel<__nv_bfloat16><<<grid, NT, 0, s>>>(a);
    else token_kernel<float><<<grid, NT, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace glr
}  // namespace kda
