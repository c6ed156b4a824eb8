// Sequential prefill of the state space mixer on the CUDA cores, in fp32:
// the form for fp32 I/O, whose outputs tensor-core operands of 16 bits would
// not reach.
//
// One CTA per (sequence, head, PS columns of the head); its N x PS part of the
// fp32 state stays in registers over the whole sequence, a block of TB tokens at a
// time.  Four things run side by side on warps of their own, one barrier a block:
// the steps of block b, the sums, skip and gate of block b - 1's outputs, conv +
// SiLU of block b + 1, and the copies (TMA) of the rows of block b + 3 with dt and
// the decays of block b + 2.  In turn on the same threads they took three times as
// long: the walk over a sequence is a chain of latencies.
//
// Few heads run with PS = 16: more CTAs of shorter steps, each repeating the conv
// of B and C; with PS = 64 that repetition is gone, which pays once the SMs are
// full.  5 sequences of 601 tokens in all, 8 heads of 64 x 64, fp32: 35 us (121 with
// PS = 64 and the phases in turn, 69 with PS = 16), 90 ns a token of the longest;
// 5000 tokens x 4 heads of 128 x 128: 0.59 ms.  Bound by shared-memory reads: a step
// reads N values each of B and C for every CP columns, and the conv 7 rows for 4.
#include <limits.h>

#include "ssm_common.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace ssm {
namespace {

constexpr int NG = 16;                            // row groups of the stepping threads
constexpr int STAGES = 4;                         // blocks of raw rows
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;

// Threads by role: NS step, NC convolve, one warp copies, NO write outputs (0: the
// convolving and copying ones do).  A thread holds CP columns for every B or C value
// that it reads.  Narrow: CP = 2 with 4 warps (35 us above; one column with 8 warps
// 49, CP = 4 with 2 warps 49).  Wide: CP = 4 with 8 warps (2048 tokens in 4 sequences,
// 64 heads of 64 x 128, fp32: 0.24 ms; one column 0.47).
template <int PS> struct Roles {
    static constexpr int CP = PS == 16 ? 2 : 4, PQ = PS / CP, NS = PQ * NG, NC = 224, NO = PS == 16 ? 128 : 0;
    static constexpr int NT = NS + NC + 32 + NO;
    static constexpr int IN_WARP = PS == 16 ? 1 : 32 / PQ;   // row groups whose partial sums a warp adds
    static constexpr int PARTS = NG / IN_WARP;
};

// Tensor maps of TB-row boxes: of PS columns of xbc and of z, of N columns of xbc.
struct ScanMaps {
    CUtensorMap x, bc, z;
};

template <typename TI, int N, int PS, int TB>
struct ScanSmem {
    static constexpr int CH = PS + 2 * N;         // conv channels: x of the slice, B, C
    float4 w[CH];
    // row r of the sequence in slot r mod (STAGES TB)
    alignas(128) TI rx[STAGES * TB][PS];
    TI rB[STAGES * TB][N], rC[STAGES * TB][N];
    TI z[STAGES][TB][PS];
    float B[2][TB][N], C[2][TB][N];               // two blocks in turn
    float xd[2][TB][PS];                          // dt x
    float x[3][TB][PS];
    float part[2][TB][Roles<PS>::PARTS][PS];       // readout partial sums
    float a[3][TB], dt[3][TB];
    float bias[CH];
    unsigned long long bar[STAGES];
    int stop;                                     // after a timeout: the block no one begins any more
};

// While block b is stepped, block b - 1's outputs are written, block b + 1 is
// convolved and the rows of block b + 3 are sent for.
template <typename TI, int P, int N, int PS, int TB>
__global__ void __launch_bounds__(Roles<PS>::NT, 2) scan_kernel(const __grid_constant__ PrefillArgs g,
                                                                    const __grid_constant__ ScanMaps maps, int32_t* status) {
    using Smem = ScanSmem<TI, N, PS, TB>;
    using K = Roles<PS>;
    constexpr int NS = K::NS, CP = K::CP, NC = K::NC, RN = N / NG, SL = P / PS, CH = Smem::CH;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    cudaTriggerProgrammaticLaunchCompletion();           // the ring kernel may read beside this one's end
    if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
    const int H = g.H, W = H * P, Cx = W + 2 * g.G * N;
    const int slice = blockIdx.x % SL, h = blockIdx.x / SL % H, n = seq_at(g, blockIdx.x / SL / H);
    const int grp = h / (H / g.G);
    const int64_t bos = seq_start(g, n);
    const uint32_t L = (uint32_t)(seq_start(g, n + 1) - bos);   // (below 2^31)
    const int nb = (int)((L + TB - 1) / TB);
    const int col0 = h * P + slice * PS;                 // this CTA's first channel of x
    const size_t soff = ((size_t)n * H + h) * N * P + slice * PS;
    if (threadIdx.x < NS) {
        // ---- the steps
        const int p = threadIdx.x % K::PQ * CP, ng = threadIdx.x / K::PQ;
        float2 S[CP][RN / 2];                            // two rows of a column
        const size_t at = soff + (size_t)(ng * RN) * P + p;
#pragma unroll
        for (int q = 0; q < CP; ++q)
#pragma unroll
            for (int i = 0; i < RN / 2; ++i)
                S[q][i] = g.S_in ? make_float2(g.S_in[at + (size_t)(2 * i) * P + q], g.S_in[at + (size_t)(2 * i + 1) * P + q])
                                 : make_float2(0.f, 0.f);
        __syncthreads();
        __syncthreads();
        // tokens at a time: their operands are read before the first partial sum is written
        // (a store holds back the loads behind it), as far as registers go
        constexpr int TG = CP * RN <= 8 ? 4 : CP * RN <= 16 ? 2 : 1;
        int b = 0;
#pragma unroll 1
        for (; b < nb && b < *(volatile int*)&sm.stop; ++b) {
            const int buf = b & 1;
            const float *Bs = &sm.B[buf][0][ng * RN], *Cs = &sm.C[buf][0][ng * RN], *xs = &sm.xd[buf][0][p], *as = sm.a[b % 3];
#pragma unroll
            for (int t = 0; t < TB; t += TG) {           // (past the sequence: a = 1, B = xd = 0)
                float4 b4[TG][RN / 4], c4[TG][RN / 4];
                float x[TG][CP], y[TG][CP], a[TG];
#pragma unroll
                for (int e = 0; e < TG; ++e) {
                    a[e] = as[t + e];
#pragma unroll
                    for (int q = 0; q < CP; q += 2) {
                        const float2 x2 = *reinterpret_cast<const float2*>(xs + (t + e) * PS + q);
                        x[e][q] = x2.x;
                        x[e][q + 1] = x2.y;
                    }
#pragma unroll
                    for (int i = 0; i < RN / 4; ++i) {
                        b4[e][i] = *reinterpret_cast<const float4*>(Bs + (t + e) * N + 4 * i);
                        c4[e][i] = *reinterpret_cast<const float4*>(Cs + (t + e) * N + 4 * i);
                    }
                }
#pragma unroll
                for (int e = 0; e < TG; ++e) {
                    const float2 a2 = make_float2(a[e], a[e]);
#pragma unroll
                    for (int q = 0; q < CP; ++q) {
                        const float2 x2 = make_float2(x[e][q], x[e][q]);
                        float2 y2 = make_float2(0.f, 0.f);
#pragma unroll
                        for (int i = 0; i < RN / 4; ++i) {
                            S[q][2 * i] = __ffma2_rn(a2, S[q][2 * i], __fmul2_rn(make_float2(b4[e][i].x, b4[e][i].y), x2));
                            S[q][2 * i + 1] = __ffma2_rn(a2, S[q][2 * i + 1], __fmul2_rn(make_float2(b4[e][i].z, b4[e][i].w), x2));
                            y2 = __ffma2_rn(make_float2(c4[e][i].x, c4[e][i].y), S[q][2 * i], y2);
                            y2 = __ffma2_rn(make_float2(c4[e][i].z, c4[e][i].w), S[q][2 * i + 1], y2);
                        }
                        y[e][q] = y2.x + y2.y;
                    }
                }
#pragma unroll
                for (int e = 0; e < TG; ++e) {
#pragma unroll
                    for (int o = K::PQ; o < K::PQ * K::IN_WARP; o <<= 1)
#pragma unroll
                        for (int q = 0; q < CP; ++q) y[e][q] += __shfl_xor_sync(0xffffffffu, y[e][q], o);
                    if (ng % K::IN_WARP == 0)
#pragma unroll
                        for (int q = 0; q < CP; q += 2)
                            *reinterpret_cast<float2*>(&sm.part[buf][t + e][ng / K::IN_WARP][p + q]) = make_float2(y[e][q], y[e][q + 1]);
                }
            }
            __syncthreads();
        }
        if (b < nb) return;
#pragma unroll
        for (int q = 0; q < CP; ++q)
#pragma unroll
            for (int i = 0; i < RN / 2; ++i) {
                g.S_out[at + (size_t)(2 * i) * P + q] = S[q][i].x;
                g.S_out[at + (size_t)(2 * i + 1) * P + q] = S[q][i].y;
            }
        return;
    }
    // ---- rows, conv and outputs
    const int tid = threadIdx.x - NS, lane = tid - NC, otid = K::NO ? tid - NC - 32 : tid;
    constexpr int OUT = K::NO ? K::NO : NC + 32;         // output threads
    const TI* dts = static_cast<const TI*>(g.dt) + bos * g.dt_stride + h;
    auto channel = [&](int j) { return j < PS ? col0 + j : j < PS + N ? W + grp * N + (j - PS) : W + (g.G + grp) * N + (j - PS - N); };
    auto raw_at = [&](int j) { return j < PS ? &sm.rx[0][j] : j < PS + N ? &sm.rB[0][j - PS] : &sm.rC[0][j - PS - N]; };
    auto raw_ld = [&](int j) { return j < PS ? PS : N; };
    for (int j = tid; j < CH; j += K::NT - NS) {
        const int c = channel(j);
        sm.w[j] = __ldg(reinterpret_cast<const float4*>(g.conv_w) + c);
        sm.bias[j] = g.conv_b ? g.conv_b[c] : 0.f;
#pragma unroll
        for (int s = 0; s < RING; ++s)                   // rows -3 .. -1
            *(raw_at(j) + (STAGES * TB - RING + s) * raw_ld(j)) = g.ring_in ? static_cast<const TI*>(g.ring_in)[((size_t)n * RING + s) * Cx + c] : TI(0.f);
    }
    const float eA = expf(g.A_log[h]), dtb = g.dt_bias[h], skip = g.skip ? g.skip[h] : 0.f;
    // One warp (lane 0 .. 31) sends for the raw rows of block b and z of the block before it, and has dt and
    // the decays ready a block ahead of the conv, which multiplies x by dt.  A tile is one
    // tensor copy; row by row one warp took longer to send than the steps take.  (Rows past
    // the sequence are another's or zeros, and not used.)
    auto bytes = [&](int b) { return (uint32_t)sizeof(TI) * TB * ((b < nb ? CH : 0) + (g.z && b > 0 && b <= nb ? PS : 0)); };
    auto load = [&](int b) {
        const uint32_t bar = ptx::smem_u32(&sm.bar[b % STAGES]), all = bytes(b);
        if (lane != 0 || all == 0) return;
        ptx::mbar_expect_tx(bar, all);
        const int at = b % STAGES * TB;
        if (b < nb) {
            const int t = (int)(bos + (uint32_t)b * TB);
            ptx::tma_load_2d(ptx::smem_u32(&sm.rx[at][0]), &maps.x, col0, t, bar);
            ptx::tma_load_2d(ptx::smem_u32(&sm.rB[at][0]), &maps.bc, W + grp * N, t, bar);
            ptx::tma_load_2d(ptx::smem_u32(&sm.rC[at][0]), &maps.bc, W + (g.G + grp) * N, t, bar);
        }
        if (g.z && b > 0) ptx::tma_load_2d(ptx::smem_u32(&sm.z[(b - 1) % STAGES][0][0]), &maps.z, col0, (int)(bos + (uint32_t)(b - 1) * TB), bar);
    };
    // false when the copies of a block did not arrive in time
    auto landed = [&](int b) {
        return bytes(b) == 0 || ptx::mbar_wait(ptx::smem_u32(&sm.bar[b % STAGES]), (uint32_t)(b / STAGES) & 1u, WAIT_LIMIT_NS);
    };
    TI raw_dt = TI(0.f);
    auto load_dt = [&](int b) {
        const uint32_t t = (uint32_t)b * TB + lane;
        if (lane < TB && t < L) raw_dt = dts[t * g.dt_stride];
    };
    auto steps = [&](int b) {
        if (lane < TB) {
            const bool in = (uint32_t)b * TB + lane < L;
            const float dt = in ? softplus(to_f32(raw_dt) + dtb) : 0.f;
            sm.dt[b % 3][lane] = dt;
            sm.a[b % 3][lane] = in ? decay(-eA * dt) : 1.f;
        }
    };
    // conv: items of four tokens of a channel, all of a thread's read before the first is
    // written; past the sequence zeros
    constexpr int ITEMS = CH * (TB / 4), MINE = (ITEMS + NC - 1) / NC;
    auto conv = [&](int b) {
        const int buf = b & 1;
        float v[MINE][4 + RING];
#pragma unroll
        for (int k = 0; k < MINE; ++k) {
            const int i = min(tid + k * NC, ITEMS - 1), j = i % CH, t0 = i / CH * 4, ld = raw_ld(j);
            const TI* src = raw_at(j);
#pragma unroll
            for (int e = 0; e < 4 + RING; ++e) v[k][e] = to_f32(src[((b * TB + t0 + e - RING) & (STAGES * TB - 1)) * ld]);
        }
#pragma unroll
        for (int k = 0; k < MINE; ++k) {
            const int i = min(tid + k * NC, ITEMS - 1), j = i % CH, t0 = i / CH * 4, ld = raw_ld(j);
            const float4 w = sm.w[j];
            const float bias = sm.bias[j];
            float u[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u[t] = silu(fmaf(w.w, v[k][t + 3], fmaf(w.z, v[k][t + 2], fmaf(w.y, v[k][t + 1], fmaf(w.x, v[k][t], bias)))));
                if ((uint32_t)b * TB + t0 + t >= L) u[t] = 0.f;
            }
            if (tid + k * NC >= ITEMS) break;
            if (j < PS) {
                const float4 d4 = *reinterpret_cast<const float4*>(&sm.dt[b % 3][t0]);
                sm.xd[buf][t0][j] = d4.x * u[0];
                sm.xd[buf][t0 + 1][j] = d4.y * u[1];
                sm.xd[buf][t0 + 2][j] = d4.z * u[2];
                sm.xd[buf][t0 + 3][j] = d4.w * u[3];
            }
            float* dst = j < PS ? &sm.x[b % 3][t0][j] : j < PS + N ? &sm.B[buf][t0][j - PS] : &sm.C[buf][t0][j - PS - N];
#pragma unroll
            for (int t = 0; t < 4; ++t) dst[t * ld] = u[t];
        }
    };
    auto output = [&](int b) {
        for (int i = otid; i < TB * PS; i += OUT) {
            const int tl = i / PS, cc = i % PS;
            const uint32_t t = (uint32_t)b * TB + tl;
            if (t >= L) break;
            float y = sm.part[b & 1][tl][0][cc];
#pragma unroll
            for (int q = 1; q < K::PARTS; ++q) y += sm.part[b & 1][tl][q][cc];
            y = fmaf(skip, sm.x[b % 3][tl][cc], y);
            if (g.z) y *= silu(to_f32(sm.z[b % STAGES][tl][cc]));
            static_cast<TI*>(g.o)[(size_t)(bos + t) * W + col0 + cc] = from_f32<TI>(y);
        }
    };
    static_assert((STAGES & (STAGES - 1)) == 0 && (TB & (TB - 1)) == 0, "row slots by mask");
    const bool sends = lane >= 0 && lane < 32, convolves = tid < NC, writes = otid >= 0 && otid < OUT;
    if (sends) {
        if (lane == 0) {
            for (int i = 0; i < STAGES; ++i) ptx::mbar_init(ptx::smem_u32(&sm.bar[i]), 1);
            ptx::fence_mbar_init();
            sm.stop = INT_MAX;
        }
        __syncwarp();
        load_dt(0);
        load(0);
        load(1);
        load(2);
        steps(0);
        load_dt(1);
        if (!landed(0)) sm.stop = 0;
    }
    __syncthreads();
    if (sends) {
        steps(1);
        load_dt(2);
        if (!landed(1)) sm.stop = 0;
    } else if (convolves) {
        conv(0);
    }
    ptx::fence_async_smem();                             // rows -3 .. -1 lie where block 3 goes
    __syncthreads();
    int b = 0;
#pragma unroll 1
    for (; b < nb && b < *(volatile int*)&sm.stop; ++b) {
        if (sends) load(b + 3);
        if (writes && b > 0) output(b - 1);
        if (sends) {
            steps(b + 2);
            load_dt(b + 3);
            if (!landed(b + 2)) sm.stop = b + 1;         // (and z of block b + 1)
        } else if (convolves && b + 1 < nb) {
            conv(b + 1);
        }
        __syncthreads();
    }
    if (b == nb) {
        if (writes && nb > 0) output(nb - 1);
    } else if (lane == 0) {
        atomicExch(status, ERR_TIMEOUT);
        for (int k = b; k < b + 3; ++k) landed(k);       // copies in flight land before the CTA leaves
    }
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
    const int64_t bos = seq_start(g, n), L = seq_start(g, n + 1) - bos;
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
    cudaGridDependencySynchronize();                     // the scan has read ring_in
#pragma unroll
    for (int s = 0; s < RING; ++s) *reinterpret_cast<uint4*>(rout + ((size_t)n * RING + s) * Cx + c) = row[s];
}

template <typename TI, int P, int N, int PS>
cudaError_t scan_ps(const PrefillArgs& a, int32_t* status, cudaStream_t s) {
    constexpr int TB = PS == 16 && N == 64 ? 16 : 8;
    const int64_t blocks = (int64_t)a.n_seqs * a.H * (P / PS);
    if (blocks > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
    constexpr int smem = (int)sizeof(ScanSmem<TI, N, PS, TB>);
    static_assert(smem <= 113 * 1024, "two CTAs per SM");
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(scan_kernel<TI, P, N, PS, TB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    ScanMaps m{};
    const int64_t W = (int64_t)a.H * P, Cx = W + 2 * (int64_t)a.G * N;
    if (a.T > 0 && (!encode_rows(&m.x, a.xbc, sizeof(TI), a.T, Cx, a.xbc_stride, TB, PS) ||
                    !encode_rows(&m.bc, a.xbc, sizeof(TI), a.T, Cx, a.xbc_stride, TB, N) ||
                    (a.z && !encode_rows(&m.z, a.z, sizeof(TI), a.T, W, a.z_stride, TB, PS))))
        return cudaErrorInvalidValue;
    scan_kernel<TI, P, N, PS, TB><<<(unsigned)blocks, Roles<PS>::NT, smem, s>>>(a, m, status);
    return cudaGetLastError();
}

template <typename TI, int P, int N>
cudaError_t scan(const PrefillArgs& a, int32_t* status, cudaStream_t s) {
    // narrow slices while their CTAs are at most four to an SM
    return (int64_t)a.n_seqs * a.H * (P / 16) <= 4 * 152 ? scan_ps<TI, P, N, 16>(a, status, s) : scan_ps<TI, P, N, 64>(a, status, s);
}

template <typename TI>
cudaError_t scan_io(const PrefillArgs& a, int32_t* status, cudaStream_t s) {
    if (a.P == 64) return a.N == 64 ? scan<TI, 64, 64>(a, status, s) : scan<TI, 64, 128>(a, status, s);
    return a.N == 64 ? scan<TI, 128, 64>(a, status, s) : scan<TI, 128, 128>(a, status, s);
}

}  // namespace

cudaError_t launch_scan(const PrefillArgs& a, int io_bf16, int32_t* status, cudaStream_t s) {
    return io_bf16 ? scan_io<__nv_bfloat16>(a, status, s) : scan_io<float>(a, status, s);
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
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = grid;
        cfg.blockDim = dim3(256);
        cfg.stream = s;
        cudaLaunchAttribute at{};
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        const cudaError_t e = io_bf16 ? cudaLaunchKernelEx(&cfg, ring_kernel<__nv_bfloat16>, b) : cudaLaunchKernelEx(&cfg, ring_kernel<float>, b);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace ssm
}  // namespace kda
