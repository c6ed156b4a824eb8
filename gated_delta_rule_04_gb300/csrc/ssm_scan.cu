// Sequential prefill of the state space mixer on the CUDA cores, in fp32:
// the form for fp32 I/O, whose outputs tensor-core operands of 16 bits would
// not reach.
//
// One CTA per (sequence, head), 256 threads; the N x P fp32 state stays in
// registers over the whole sequence: thread (p, ng) holds the N / NG state
// rows of group ng in column p, so the decay, the rank-one update and the
// readout of a token are two FMAs per state element with the token's B and C
// as shared-memory broadcasts, and no barrier per token.  Tokens go through in
// blocks of TB: conv + SiLU of the block's x, B and C (each thread walks one
// channel through the block, its window in registers), TB steps, then the sum
// over the row groups, the skip and the gate.
#include "ssm_common.cuh"

namespace kda {
namespace ssm {
namespace {

constexpr int NT = 256;
constexpr int TB = 16;   // tokens per block

template <int P, int N>
struct ScanSmem {
    float x[TB][P], B[TB][N], C[TB][N];
    float part[TB][NT / P][P];   // readout partial sums by row group
    float a[TB], dt[TB];
};

template <typename TI, int P, int N>
__global__ void __launch_bounds__(NT) scan_kernel(PrefillArgs g) {
    constexpr int NG = NT / P, RN = N / NG;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    ScanSmem<P, N>& sm = *reinterpret_cast<ScanSmem<P, N>*>(smem_raw);
    const int H = g.H, W = H * P, Cx = W + 2 * g.G * N;
    const int n = g.order[blockIdx.x / H], h = blockIdx.x % H;
    const int grp = h / (H / g.G);
    const int64_t bos = g.cu[n], L = g.cu[n + 1] - bos;
    const int tid = threadIdx.x, p = tid % P, ng = tid / P;
    const size_t soff = ((size_t)n * H + h) * N * P;

    float S[RN];
#pragma unroll
    for (int i = 0; i < RN; ++i) S[i] = g.S_in ? g.S_in[soff + (size_t)(ng * RN + i) * P + p] : 0.f;

    const TI* xbc = static_cast<const TI*>(g.xbc);
    const TI* ring = static_cast<const TI*>(g.ring_in);
    // raw value of channel c at position t of the sequence (t >= -3)
    auto raw = [&](int64_t t, int c) -> float {
        if (t >= 0) return to_f32(xbc[(size_t)(bos + t) * g.xbc_stride + c]);
        return ring ? to_f32(ring[((size_t)n * RING + (t + RING)) * Cx + c]) : 0.f;
    };
    const float eA = expf(g.A_log[h]), dtb = g.dt_bias[h], skip = g.skip ? g.skip[h] : 0.f;

#pragma unroll 1
    for (int64_t t0 = 0; t0 < L; t0 += TB) {
        const int nt = (int)(L - t0 < TB ? L - t0 : TB);
        // ---- conv + SiLU: channel j of x (j < P), B, C
        for (int j = tid; j < P + 2 * N; j += NT) {
            const int c = j < P ? h * P + j : j < P + N ? W + grp * N + (j - P) : W + (g.G + grp) * N + (j - P - N);
            const float4 w = __ldg(reinterpret_cast<const float4*>(g.conv_w) + c);
            const float bias = g.conv_b ? g.conv_b[c] : 0.f;
            float v0 = raw(t0 - 3, c), v1 = raw(t0 - 2, c), v2 = raw(t0 - 1, c);
            float* dst = j < P ? &sm.x[0][j] : j < P + N ? &sm.B[0][j - P] : &sm.C[0][j - P - N];
            const int ld = j < P ? P : N;
            for (int t = 0; t < nt; ++t) {
                const float v3 = raw(t0 + t, c);
                dst[t * ld] = silu(fmaf(w.w, v3, fmaf(w.z, v2, fmaf(w.y, v1, fmaf(w.x, v0, bias)))));
                v0 = v1; v1 = v2; v2 = v3;
            }
        }
        if (tid < nt) {
            const float dt = softplus(to_f32(static_cast<const TI*>(g.dt)[(size_t)(bos + t0 + tid) * g.dt_stride + h]) + dtb);
            sm.dt[tid] = dt;
            sm.a[tid] = expf(-eA * dt);
        }
        __syncthreads();
        // ---- the steps
#pragma unroll 1
        for (int t = 0; t < nt; ++t) {
            const float a = sm.a[t], xd = sm.dt[t] * sm.x[t][p];
            float y0 = 0.f, y1 = 0.f;
#pragma unroll
            for (int i = 0; i < RN; i += 4) {
                const float4 b4 = *reinterpret_cast<const float4*>(&sm.B[t][ng * RN + i]);
                const float4 c4 = *reinterpret_cast<const float4*>(&sm.C[t][ng * RN + i]);
                S[i] = fmaf(a, S[i], b4.x * xd);
                S[i + 1] = fmaf(a, S[i + 1], b4.y * xd);
                S[i + 2] = fmaf(a, S[i + 2], b4.z * xd);
                S[i + 3] = fmaf(a, S[i + 3], b4.w * xd);
                y0 = fmaf(c4.x, S[i], y0);
                y1 = fmaf(c4.y, S[i + 1], y1);
                y0 = fmaf(c4.z, S[i + 2], y0);
                y1 = fmaf(c4.w, S[i + 3], y1);
            }
            sm.part[t][ng][p] = y0 + y1;
        }
        __syncthreads();
        // ---- outputs of the block
        for (int i = tid; i < nt * P; i += NT) {
            const int t = i / P, c = i % P;
            float y = sm.part[t][0][c];
#pragma unroll
            for (int k = 1; k < NG; ++k) y += sm.part[t][k][c];
            y = fmaf(skip, sm.x[t][c], y);
            if (g.z) y *= silu(to_f32(static_cast<const TI*>(g.z)[(size_t)(bos + t0 + t) * g.z_stride + h * P + c]));
            static_cast<TI*>(g.o)[(size_t)(bos + t0 + t) * W + h * P + c] = from_f32<TI>(y);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < RN; ++i) g.S_out[soff + (size_t)(ng * RN + i) * P + p] = S[i];
}

// The last three raw rows of every sequence; a thread owns 16 bytes of
// channels of one sequence and reads all it needs before it writes, so
// ring_out may be ring_in.
template <typename TI>
__global__ void __launch_bounds__(256) ring_kernel(PrefillArgs g) {
    constexpr int V = 16 / sizeof(TI);
    const int Cx = g.H * g.P + 2 * g.G * g.N;
    const int n = blockIdx.y;
    const int c = (blockIdx.x * blockDim.x + threadIdx.x) * V;
    if (c >= Cx) return;
    const int64_t bos = g.cu[n], L = g.cu[n + 1] - bos;
    const TI* xbc = static_cast<const TI*>(g.xbc);
    const TI* rin = static_cast<const TI*>(g.ring_in);
    TI* rout = static_cast<TI*>(g.ring_out);
    uint4 row[RING];
#pragma unroll
    for (int s = 0; s < RING; ++s) {
        const int64_t t = L - RING + s;      // position of ring slot s
        row[s] = t >= 0 ? *reinterpret_cast<const uint4*>(xbc + (size_t)(bos + t) * g.xbc_stride + c)
                 : rin  ? *reinterpret_cast<const uint4*>(rin + ((size_t)n * RING + (t + RING)) * Cx + c)
                        : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int s = 0; s < RING; ++s) *reinterpret_cast<uint4*>(rout + ((size_t)n * RING + s) * Cx + c) = row[s];
}

template <typename TI, int P, int N>
cudaError_t scan(const PrefillArgs& a, cudaStream_t s) {
    const int64_t blocks = (int64_t)a.n_seqs * a.H;
    if (blocks > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
    static_assert(sizeof(ScanSmem<P, N>) <= 48 * 1024, "static shared memory limit");
    scan_kernel<TI, P, N><<<(unsigned)blocks, NT, sizeof(ScanSmem<P, N>), s>>>(a);
    return cudaGetLastError();
}

template <typename TI>
cudaError_t scan_io(const PrefillArgs& a, cudaStream_t s) {
    if (a.P == 64) return a.N == 64 ? scan<TI, 64, 64>(a, s) : scan<TI, 64, 128>(a, s);
    return a.N == 64 ? scan<TI, 128, 64>(a, s) : scan<TI, 128, 128>(a, s);
}

}  // namespace

cudaError_t launch_scan(const PrefillArgs& a, int io_bf16, cudaStream_t s) {
    return io_bf16 ? scan_io<__nv_bfloat16>(a, s) : scan_io<float>(a, s);
}

cudaError_t launch_ring(const PrefillArgs& a, int io_bf16, cudaStream_t s) {
    const int Cx = a.H * a.P + 2 * a.G * a.N, v = io_bf16 ? 8 : 4;
    // (grid.y is limited to 65535 sequences a launch)
    for (int n0 = 0; n0 < a.n_seqs; n0 += 65535) {
        PrefillArgs b = a;
        const size_t row = (size_t)RING * Cx * (io_bf16 ? 2 : 4);
        b.cu = a.cu + n0;
        if (a.ring_in) b.ring_in = static_cast<const char*>(a.ring_in) + n0 * row;
        b.ring_out = static_cast<char*>(a.ring_out) + n0 * row;
        const dim3 grid((Cx / v + 255) / 256, a.n_seqs - n0 < 65535 ? a.n_seqs - n0 : 65535);
        if (io_bf16) ring_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(b);
        else ring_kernel<float><<<grid, 256, 0, s>>>(b);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace ssm
}  // namespace kda
