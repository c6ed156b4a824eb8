// Backward pass of the gated linear recurrence.  With m = sqrt(1 - a^2),
// b = m v x and G = do SiLU(z):
//   g_t = G_t + a_{t+1} g_{t+1}            (the last token: + dS_out)
//   dz = do h SiLU'(z)      dx = g m v      di = g b (1 - v)
//   dla = g (a h_{t-1} - (a / m)^2 b)       dr = dla la (1 - w)
//   dA_log = sum dla la,  dr_bias = sum dr,  di_bias = sum di,  dS_in = a_1 g_1
// One thread per (sequence, channel): the states of 64 tokens are computed again
// from the one the prefill left, then the tokens are walked backwards.
#include "glr_common.cuh"

namespace kda {
namespace glr {
namespace {

constexpr int NT = 128;

template <typename TI>
__global__ void __launch_bounds__(NT) backward_kernel(const __grid_constant__ ScanArgs g) {
    const int blocks = (g.C + NT - 1) / NT;
    const int n = blockIdx.x / blocks, c = blockIdx.x % blocks * NT + threadIdx.x;
    if (c >= g.C) return;
    const int64_t t0 = seq_start(g.f, n), t1 = seq_start(g.f, n + 1);
    const float ea = -expf(g.A_log[c]), rb = g.r_bias ? g.r_bias[c] : 0.f, ib = g.i_bias ? g.i_bias[c] : 0.f;
    float carry = g.dS_out ? g.dS_out[(size_t)n * g.C + c] : 0.f, sA = 0.f, sr = 0.f, si = 0.f;
    float hb[CHUNK];                                  // the states before the tokens of a chunk
    auto at = [&](int64_t t) {
        return step_of(to_f32(static_cast<const TI*>(g.r)[t * g.r_s + c]) + rb,
                       to_f32(static_cast<const TI*>(g.i)[t * g.i_s + c]) + ib, ea);
    };
    for (int64_t end = t1; end > t0;) {
        const int64_t first = (end - 1) / CHUNK * CHUNK, from = first > t0 ? first : t0;
        float h = from == first ? g.states[(size_t)(first / CHUNK) * g.C + c] : g.S_in ? g.S_in[(size_t)n * g.C + c] : 0.f;
        for (int64_t t = from; t < end; ++t) {
            hb[t - first] = h;
            const Step s = at(t);
            h = fmaf(s.a, h, s.m * s.v * to_f32(static_cast<const TI*>(g.x)[t * g.x_s + c]));
        }
        for (int64_t t = end - 1; t >= from; --t) {
            const Step s = at(t);
            const float x = to_f32(static_cast<const TI*>(g.x)[t * g.x_s + c]), b = s.m * s.v * x;
            float G = to_f32(static_cast<const TI*>(g.d_o)[t * g.do_s + c]);
            if (g.z) {
                const float z = to_f32(static_cast<const TI*>(g.z)[t * g.z_s + c]), e = sigmoid(z);
                static_cast<TI*>(g.dz)[t * g.dz_s + c] = from_f32<TI>(G * fmaf(s.a, hb[t - first], b) * e * fmaf(z, 1.f - e, 1.f));
                G *= z * e;
            }
            const float gt = G + carry;
            carry = s.a * gt;
            static_cast<TI*>(g.dx)[t * g.dx_s + c] = from_f32<TI>(gt * s.m * s.v);
            const float di = gt * b * sigmoid(-(to_f32(static_cast<const TI*>(g.i)[t * g.i_s + c]) + ib));
            // (a / m)^2 b la = a^2 v x (la / m), zero where la is
            const float la_m = s.m > 0.f ? s.la / s.m : 0.f;
            const float dA = gt * fmaf(s.a * hb[t - first], s.la, -s.a * s.a * s.v * x * la_m);
            const float dr = dA * sigmoid(-(to_f32(static_cast<const TI*>(g.r)[t * g.r_s + c]) + rb));
            static_cast<TI*>(g.di)[t * g.di_s + c] = from_f32<TI>(di);
            static_cast<TI*>(g.dr)[t * g.dr_s + c] = from_f32<TI>(dr);
            sA += dA;
            sr += dr;
            si += di;
        }
        end = from;
    }
    if (g.dS_in) g.dS_in[(size_t)n * g.C + c] = carry;
    float* p = g.part + (size_t)n * 3 * g.C + c;
    p[0] = sA;
    p[g.C] = sr;
    p[2 * (size_t)g.C] = si;
}

// The sums over the sequences, in their order.
__global__ void __launch_bounds__(NT) params_kernel(const __grid_constant__ ScanArgs g) {
    const int c = blockIdx.x * NT + threadIdx.x;
    if (c >= g.C) return;
    double s[3] = {0.0, 0.0, 0.0};
    for (int n = 0; n < g.f.n; ++n)
        for (int k = 0; k < 3; ++k) s[k] += g.part[((size_t)n * 3 + k) * g.C + c];
    g.dA_log[c] = (float)s[0];
    if (g.dr_bias) g.dr_bias[c] = (float)s[1];
    if (g.di_bias) g.di_bias[c] = (float)s[2];
}

}  // namespace

cudaError_t launch_backward(const ScanArgs& a, int io_bf16, cudaStream_t s) {
    const unsigned blocks = (unsigned)((a.C + NT - 1) / NT);
    const unsigned grid = (unsigned)a.f.n * blocks;
    if (io_bf16) backward_kernel<__nv_bfloat16><<<grid, NT, 0, s>>>(a);
    else backward_kernel<float><<<grid, NT, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    params_kernel<<<blocks, NT, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace glr
}  // namespace kda
