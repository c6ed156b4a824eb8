// Prefill of the gated linear recurrence: h_t = a_t h_{t-1} + m_t v_t x_t,
// o_t = h_t SiLU(z_t).  One thread per (sequence, channel), token by token.
#include "glr_common.cuh"

namespace kda {
namespace glr {
namespace {

constexpr int NT = 128;

template <typename TI>
__global__ void __launch_bounds__(NT) scan_kernel(const __grid_constant__ ScanArgs g) {
    const int blocks = (g.C + NT - 1) / NT;
    const int n = blockIdx.x / blocks, c = blockIdx.x % blocks * NT + threadIdx.x;
    if (c >= g.C) return;
    const int64_t t0 = seq_start(g.f, n), t1 = seq_start(g.f, n + 1);
    const float ea = -expf(g.A_log[c]), rb = g.r_bias ? g.r_bias[c] : 0.f, ib = g.i_bias ? g.i_bias[c] : 0.f;
    float h = g.S_in ? g.S_in[(size_t)n * g.C + c] : 0.f;
    for (int64_t t = t0; t < t1; ++t) {
        if (g.states && t % CHUNK == 0) g.states[(size_t)(t / CHUNK) * g.C + c] = h;
        const Step s = step_of(to_f32(static_cast<const TI*>(g.r)[t * g.r_s + c]) + rb,
                               to_f32(static_cast<const TI*>(g.i)[t * g.i_s + c]) + ib, ea);
        h = fmaf(s.a, h, s.m * s.v * to_f32(static_cast<const TI*>(g.x)[t * g.x_s + c]));
        float o = h;
        if (g.z) {
            const float z = to_f32(static_cast<const TI*>(g.z)[t * g.z_s + c]);
            o *= z * sigmoid(z);
        }
        static_cast<TI*>(g.o)[t * g.C + c] = from_f32<TI>(o);
    }
    g.S_out[(size_t)n * g.C + c] = h;
}

}  // namespace

cudaError_t launch_scan(const ScanArgs& a, int io_bf16, cudaStream_t s) {
    const unsigned grid = (unsigned)((int64_t)a.f.n * ((a.C + NT - 1) / NT));
    if (io_bf16) scan_kernel<__nv_bfloat16><<<grid, NT, 0, s>>>(a);
    else scan_kernel<float><<<grid, NT, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace glr
}  // namespace kda
