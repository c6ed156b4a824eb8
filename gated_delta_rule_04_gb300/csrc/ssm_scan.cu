// Sequential prefill of the state space mixer on the CUDA cores, in fp32:
// the form for fp32 I/O, whose outputs tensor-core operands of 16 bits would
// not reach.
//
// One CTA of 256 threads per (sequence, head, PS columns of the head); its
// N x PS part of the fp32 state stays in registers over the whole sequence:
// thread (p, ng) holds N / NG state rows of column p, so a token costs two FMAs
// per state element with its B and C as shared-memory broadcasts, and no
// barrier.  Tokens go through in blocks of TB: conv + SiLU of the block's x, B
// and C (each thread one channel, the next block's raw values already in
// flight), TB steps, then the sum over the row groups, the skip and the gate.
// The walk over a sequence is latency-bound, so few heads run with PS = 16: more
// CTAs of shorter steps, each repeating the conv of B and C (5 sequences of 601
// tokens in all, 8 heads of 64 x 64: 121 us with PS = 64, 69 us with 16); with
// PS = 64 that repetition is gone, which pays once the SMs are full.
#include "ssm_common.cuh"

namespace kda {
namespace ssm {
namespace {

constexpr int NT = 256;
constexpr int TB = 16;   // tokens per block

template <int N, int PS>
struct ScanSmem {
    float x[2][TB][PS], B[2][TB][N], C[2][TB][N];   // two blocks in turn
    float part[TB][NT / PS][PS];   // readout partial sums by row group
    float a[2][TB], dt[2][TB];
};

template <typename TI, int P, int N, int PS>
__global__ void __launch_bounds__(NT) scan_kernel(PrefillArgs g) {
    constexpr int NG = NT / PS, RN = N / NG, SL = P / PS;
    constexpr int CHS = (PS + 2 * N + NT - 1) / NT;      // channels of a thread in the conv
    extern __shared__ __align__(16) unsigned char smem_raw[];
    ScanSmem<N, PS>& sm = *reinterpret_cast<ScanSmem<N, PS>*>(smem_raw);
    const int H = g.H, W = H * P, Cx = W + 2 * g.G * N;
    const int slice = blockIdx.x % SL, h = blockIdx.x / SL % H, n = g.order[blockIdx.x / SL / H];
    const int grp = h / (H / g.G);
    const int64_t bos = g.cu[n], L = g.cu[n + 1] - bos;
    const int tid = threadIdx.x, p = tid % PS, ng = tid / PS;
    const int col0 = h * P + slice * PS;                 // this CTA's first channel of x
    const size_t soff = ((size_t)n * H + h) * N * P + slice * PS;

    float S[RN];
#pragma unroll
    for (int i = 0; i < RN; ++i) S[i] = g.S_in ? g.S_in[soff + (size_t)(ng * RN + i) * P + p] : 0.f;

    const TI* xbc = static_cast<const TI*>(g.xbc);
    const TI* ring = static_cast<const TI*>(g.ring_in);
    // the conv channels of this thread: x of the slice, B, C
    int c[CHS];
    float4 w[CHS];
    float bias[CHS], win[CHS][RING];
#pragma unroll
    for (int k = 0; k < CHS; ++k) {
        const int j = tid + k * NT;
        c[k] = j < PS ? col0 + j : j < PS + N ? W + grp * N + (j - PS) : j < PS + 2 * N ? W + (g.G + grp) * N + (j - PS - N) : -1;
        w[k] = c[k] >= 0 ? __ldg(reinterpret_cast<const float4*>(g.conv_w) + c[k]) : make_float4(0.f, 0.f, 0.f, 0.f);
        bias[k] = c[k] >= 0 && g.conv_b ? g.conv_b[c[k]] : 0.f;
#pragma unroll
        for (int s = 0; s < RING; ++s) win[k][s] = c[k] >= 0 && ring ? to_f32(ring[((size_t)n * RING + s) * Cx + c[k]]) : 0.f;
    }
    const float eA = expf(g.A_log[h]), dtb = g.dt_bias[h], skip = g.skip ? g.skip[h] : 0.f;
    TI raw[CHS][TB], raw_dt = TI(0.f);
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int k = 0; k < CHS; ++k)
#pragma unroll
            for (int t = 0; t < TB; ++t)
                raw[k][t] = c[k] >= 0 && t0 + t < L ? xbc[(size_t)(bos + t0 + t) * g.xbc_stride + c[k]] : TI(0.f);
        if (tid < TB && t0 + tid < L) raw_dt = static_cast<const TI*>(g.dt)[(size_t)(bos + t0 + tid) * g.dt_stride + h];
    };
    load(0);
    int buf = 0;
#pragma unroll 1
    for (int64_t t0 = 0; t0 < L; t0 += TB, buf ^= 1) {
        const int nt = (int)(L - t0 < TB ? L - t0 : TB);
        // ---- conv + SiLU (rows past the sequence: of zeros, not used)
#pragma unroll
        for (int k = 0; k < CHS; ++k) {
            const int j = tid + k * NT;
            float* dst = j < PS ? &sm.x[buf][0][j] : j < PS + N ? &sm.B[buf][0][j - PS] : &sm.C[buf][0][j - PS - N];
            const int ld = j < PS ? PS : N;
            if (c[k] >= 0) {
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    const float v = to_f32(raw[k][t]);
                    dst[t * ld] = silu(fmaf(w[k].w, v, fmaf(w[k].z, win[k][2], fmaf(w[k].y, win[k][1], fmaf(w[k].x, win[k][0], bias[k])))));
                    win[k][0] = win[k][1]; win[k][1] = win[k][2]; win[k][2] = v;
                }
            }
        }
        if (tid < TB) {
            const float dt = softplus(to_f32(raw_dt) + dtb);
            sm.dt[buf][tid] = dt;
            sm.a[buf][tid] = expf(-eA * dt);
        }
        __syncthreads();
        if (t0 + TB < L) load(t0 + TB);
        // ---- the steps
#pragma unroll 4
        for (int t = 0; t < nt; ++t) {
            const float a = sm.a[buf][t], xd = sm.dt[buf][t] * sm.x[buf][t][p];
            float y0 = 0.f, y1 = 0.f;
#pragma unroll
            for (int i = 0; i < RN; i += 4) {
                const float4 b4 = *reinterpret_cast<const float4*>(&sm.B[buf][t][ng * RN + i]);
                const float4 c4 = *reinterpret_cast<const float4*>(&sm.C[buf][t][ng * RN + i]);
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
        // ---- outputs of the block (its buffers are written again behind the next two barriers)
        for (int i = tid; i < nt * PS; i += NT) {
            const int t = i / PS, cc = i % PS;
            float y = sm.part[t][0][cc];
#pragma unroll
            for (int k = 1; k < NG; ++k) y += sm.part[t][k][cc];
            y = fmaf(skip, sm.x[buf][t][cc], y);
            if (g.z) y *= silu(to_f32(static_cast<const TI*>(g.z)[(size_t)(bos + t0 + t) * g.z_stride + col0 + cc]));
            static_cast<TI*>(g.o)[(size_t)(bos + t0 + t) * W + col0 + cc] = from_f32<TI>(y);
        }
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

template <typename TI, int P, int N, int PS>
cudaError_t scan_ps(const PrefillArgs& a, cudaStream_t s) {
    const int64_t blocks = (int64_t)a.n_seqs * a.H * (P / PS);
    if (blocks > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
    constexpr int smem = (int)sizeof(ScanSmem<N, PS>);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(scan_kernel<TI, P, N, PS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    scan_kernel<TI, P, N, PS><<<(unsigned)blocks, NT, smem, s>>>(a);
    return cudaGetLastError();
}

template <typename TI, int P, int N>
cudaError_t scan(const PrefillArgs& a, cudaStream_t s) {
    // narrow slices while their CTAs are at most four to an SM
    return (int64_t)a.n_seqs * a.H * (P / 16) <= 4 * 152 ? scan_ps<TI, P, N, 16>(a, s) : scan_ps<TI, P, N, 64>(a, s);
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
