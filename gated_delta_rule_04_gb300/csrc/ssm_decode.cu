// One token per session of the state space mixer, state and ring updated in
// place:  S = a S + dt B x^T,  y = S^T C + D x,  o = y SiLU(z).
//
// The state moves through HBM once in each direction and bounds the call; a
// session's conv channels are 1 to 3 % of its state.  B and C of a group are
// shared by its heads, and their ring is rolled in place, so it may be written
// only when every head's CTA has read it:
//   - fused_kernel, for calls whose states are small enough that latency counts:
//     the heads of a (session, group) are one thread-block cluster (up to 16 CTAs of
//     one or two heads).  Every CTA convolves the group's B and C for itself (6 KiB
//     from L2 beside a 32 KiB state) and its own heads' x, and a cluster barrier
//     stands between the last read of that ring and its write.  One launch of 5 us
//     takes a single session's call from 19 to 14 us as the caller sees it;
//   - otherwise conv_kernel takes every channel of every session through the conv
//     into the workspace, with the heads' steps and decays, and rolls the ring, and
//     state_kernel streams the states: persistent CTAs, the next state's 16 to 64 KiB prefetched into L2, the first
//     one read while conv_kernel still runs.  256 sessions x 64 heads: 219 us
//     fused, 192 us this way.
#include <algorithm>
#include <atomic>

#include "ssm_common.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace ssm {
namespace {

constexpr int NT = 256;
// Resident CTAs of the state kernel.  256 sessions x 64 heads of 128 x 64: 244 us with
// two, 204 with three, 192 with four, 211 with six.  (Heads of 128 x 128 hold twice the state a
// thread and spill 176 bytes of it: 128 sessions x 64 heads 240 to 247 us, of the same bytes.)
constexpr int PER_SM = 4;

template <typename TI>
__global__ void __launch_bounds__(NT) conv_kernel(DecodeArgs g) {
    constexpr int V = 16 / sizeof(TI);   // channels per thread
    const int Cx = g.H * g.P + 2 * g.G * g.N;
    const int per = Cx / V;
    const int64_t id = (int64_t)blockIdx.x * NT + threadIdx.x, channels = (int64_t)g.n * per;
    cudaTriggerProgrammaticLaunchCompletion();   // the state kernel's first loads may start
    if (id >= channels) {                        // the threads behind the channels: a session's head each
        if (id >= channels + (int64_t)g.n * g.H) return;
        const int n = (int)((id - channels) / g.H), h = (int)((id - channels) % g.H);
        const float dt = softplus(to_f32(static_cast<const TI*>(g.dt)[(size_t)n * g.dt_stride + h]) + g.dt_bias[h]);
        g.step[id - channels] = make_float2(dt, decay(-expf(g.A_log[h]) * dt));
        return;
    }
    const int n = (int)(id / per), c = (int)(id % per) * V;
    const int slot = g.slots ? g.slots[n] : n;
    if (slot < 0 || slot >= g.n_slots) return;
    TI* ring = static_cast<TI*>(g.ring) + (size_t)slot * RING * Cx + c;
    union Row { uint4 u; TI v[V]; } r[4];
#pragma unroll
    for (int s = 0; s < RING; ++s) r[s].u = *reinterpret_cast<const uint4*>(ring + (size_t)s * Cx);
    r[3].u = *reinterpret_cast<const uint4*>(static_cast<const TI*>(g.xbc) + (size_t)n * g.xbc_stride + c);
    float y[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(g.conv_w) + c + i);
        const float b = g.conv_b ? __ldg(g.conv_b + c + i) : 0.f;
        y[i] = silu(fmaf(w.w, to_f32(r[3].v[i]), fmaf(w.z, to_f32(r[2].v[i]), fmaf(w.y, to_f32(r[1].v[i]),
                    fmaf(w.x, to_f32(r[0].v[i]), b)))));
    }
    float4* dst = reinterpret_cast<float4*>(g.u + (size_t)n * Cx + c);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
#pragma unroll
    for (int s = 0; s < RING; ++s) *reinterpret_cast<uint4*>(ring + (size_t)s * Cx) = r[s + 1].u;
}

// Thread (rg, cq): state rows rg, rg + RG, ..., columns 4 cq .. 4 cq + 3.
// Persistent CTAs walk the (session, head) items; the next item's state goes to
// L2 while this one computes.
template <typename TI, int P, int N>
__global__ void __launch_bounds__(NT, PER_SM) state_kernel(DecodeArgs g) {
    constexpr int CQ = P / 4, RG = NT / CQ, RN = N / RG;
    __shared__ float4 part[2][NT / 32][CQ];
    const int H = g.H, W = H * P, Cx = W + 2 * g.G * N;
    const int tid = threadIdx.x, cq = tid % CQ, rg = tid / CQ;
    const uint32_t items = (uint32_t)g.n * H;
    int next_slot = g.slots ? g.slots[blockIdx.x / H] : blockIdx.x / H;
    int buf = 0;
#pragma unroll 1
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int n = item / H, h = item % H;
        const int slot = next_slot;
        if (item + gridDim.x < items) {
            const int nn = (item + gridDim.x) / H, nh = (item + gridDim.x) % H;
            next_slot = g.slots ? g.slots[nn] : nn;
            if (tid == 0 && next_slot >= 0 && next_slot < g.n_slots)
                ptx::bulk_prefetch_l2(g.S + ((size_t)next_slot * H + nh) * N * P, N * P * 4);
        }
        if (slot < 0 || slot >= g.n_slots) continue;
        float4* Sg = reinterpret_cast<float4*>(g.S + ((size_t)slot * H + h) * N * P) + tid;
        float4 S[RN];
#pragma unroll
        for (int i = 0; i < RN; ++i) S[i] = __ldcs(Sg + i * NT);
        const float* u = g.u + (size_t)n * Cx;
        const int grp = h / (H / g.G);
        cudaGridDependencySynchronize();   // u is there (at once from the second item on)
        const float2 step = g.step[item];
        const float dt = step.x, a = step.y;
        const float4 x4 = *reinterpret_cast<const float4*>(u + h * P + 4 * cq);
        const float4 xd = make_float4(dt * x4.x, dt * x4.y, dt * x4.z, dt * x4.w);
        const float* B = u + W + grp * N;
        const float* C = B + g.G * N;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < RN; ++i) {
            const float b = B[rg + i * RG], c = C[rg + i * RG];
            S[i].x = fmaf(a, S[i].x, b * xd.x); S[i].y = fmaf(a, S[i].y, b * xd.y);
            S[i].z = fmaf(a, S[i].z, b * xd.z); S[i].w = fmaf(a, S[i].w, b * xd.w);
            __stcs(Sg + i * NT, S[i]);
            y.x = fmaf(c, S[i].x, y.x); y.y = fmaf(c, S[i].y, y.y);
            y.z = fmaf(c, S[i].z, y.z); y.w = fmaf(c, S[i].w, y.w);
        }
        if (CQ == 16) {   // two row groups share a warp
            y.x += __shfl_xor_sync(0xffffffffu, y.x, 16); y.y += __shfl_xor_sync(0xffffffffu, y.y, 16);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, 16); y.w += __shfl_xor_sync(0xffffffffu, y.w, 16);
        }
        if ((tid & 31) < CQ) part[buf][tid >> 5][cq] = y;
        __syncthreads();   // (two buffers: the one read here is written again behind the next barrier)
        if (tid < P) {
            const float* pf = reinterpret_cast<const float*>(part[buf]);
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < NT / 32; ++k) s += pf[k * P + tid];
            if (g.skip) s = fmaf(g.skip[h], u[h * P + tid], s);
            if (g.z) s *= silu(to_f32(static_cast<const TI*>(g.z)[(size_t)n * g.z_stride + h * P + tid]));
            static_cast<TI*>(g.o)[(size_t)n * W + h * P + tid] = from_f32<TI>(s);
        }
        buf ^= 1;
    }
}

// The state step of one head by a CTA: thread (rg, cq) holds state rows rg,
// rg + RG, ... and columns 4 cq .. 4 cq + 3.  Returns y's partial sums in `part`.
template <int P, int N>
struct Tile {
    static constexpr int CQ = P / 4, RG = NT / CQ, RN = N / RG;
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <typename TI, int P, int N>
__global__ void __launch_bounds__(NT) fused_kernel(DecodeArgs g, int cs) {
    using T = Tile<P, N>;
    constexpr int CQ = T::CQ, RG = T::RG, RN = T::RN;
    __shared__ float sBC[2 * N], sx[2][P];
    __shared__ float4 part[NT / 32][CQ];
    const int H = g.H, G = g.G, HG = H / G, W = H * P, Cx = W + 2 * G * N;
    const int rank = blockIdx.x % cs;
    const int64_t unit = blockIdx.x / cs;                // (session, group)
    const int n = (int)(unit / G), grp = (int)(unit % G);
    const int tid = threadIdx.x, cq = tid % CQ, rg = tid / CQ;
    const int slot = g.slots ? g.slots[n] : n;
    if (slot < 0 || slot >= g.n_slots) return;           // (the whole cluster: one session)
    // this CTA's heads: rank and rank + cs of the group
    const int heads = rank >= HG ? 0 : rank + cs < HG ? 2 : 1, h0 = grp * HG + rank;
    float4 S[RN];
    float4* Sg = reinterpret_cast<float4*>(g.S + ((size_t)slot * H + h0) * N * P) + tid;
    if (heads > 0) {
#pragma unroll
        for (int i = 0; i < RN; ++i) S[i] = __ldcs(Sg + i * NT);
    }
    TI* ring = static_cast<TI*>(g.ring) + (size_t)slot * RING * Cx;
    const TI* row = static_cast<const TI*>(g.xbc) + (size_t)n * g.xbc_stride;
    auto conv = [&](int c, TI (&r)[4]) -> float {
#pragma unroll
        for (int s = 0; s < RING; ++s) r[s] = ring[(size_t)s * Cx + c];
        r[3] = row[c];
        const float4 w = __ldg(reinterpret_cast<const float4*>(g.conv_w) + c);
        const float b = g.conv_b ? __ldg(g.conv_b + c) : 0.f;
        return silu(fmaf(w.w, to_f32(r[3]), fmaf(w.z, to_f32(r[2]), fmaf(w.y, to_f32(r[1]), fmaf(w.x, to_f32(r[0]), b)))));
    };
    // B | C of the group (every CTA), x of this CTA's heads (whose ring it owns)
    TI rb[4];
    const int cb = W + (tid < N ? grp * N + tid : G * N + grp * N + tid - N);
    if (tid < 2 * N) sBC[tid] = conv(cb, rb);
    const int hx = tid / P;
    if (hx < heads) {
        TI rx[4];
        const int c = (h0 + hx * cs) * P + tid % P;
        sx[hx][tid % P] = conv(c, rx);
#pragma unroll
        for (int s = 0; s < RING; ++s) ring[(size_t)s * Cx + c] = rx[s + 1];
    }
    __syncthreads();
    cluster_arrive();                                    // this CTA has read the group's ring
#pragma unroll 1
    for (int x = 0; x < heads; ++x) {
        const int h = h0 + x * cs;
        const float dt = softplus(to_f32(static_cast<const TI*>(g.dt)[(size_t)n * g.dt_stride + h]) + g.dt_bias[h]);
        const float a = decay(-expf(g.A_log[h]) * dt);
        const float4 x4 = *reinterpret_cast<const float4*>(&sx[x][4 * cq]);
        const float4 xd = make_float4(dt * x4.x, dt * x4.y, dt * x4.z, dt * x4.w);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < RN; ++i) {
            const float b = sBC[rg + i * RG], c = sBC[N + rg + i * RG];
            S[i].x = fmaf(a, S[i].x, b * xd.x); S[i].y = fmaf(a, S[i].y, b * xd.y);
            S[i].z = fmaf(a, S[i].z, b * xd.z); S[i].w = fmaf(a, S[i].w, b * xd.w);
            __stcs(Sg + i * NT, S[i]);
            y.x = fmaf(c, S[i].x, y.x); y.y = fmaf(c, S[i].y, y.y);
            y.z = fmaf(c, S[i].z, y.z); y.w = fmaf(c, S[i].w, y.w);
        }
        if (x + 1 < heads) {
            Sg += (size_t)cs * N * P / 4;
#pragma unroll
            for (int i = 0; i < RN; ++i) S[i] = __ldcs(Sg + i * NT);
        }
        if (CQ == 16) {   // two row groups share a warp
            y.x += __shfl_xor_sync(0xffffffffu, y.x, 16); y.y += __shfl_xor_sync(0xffffffffu, y.y, 16);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, 16); y.w += __shfl_xor_sync(0xffffffffu, y.w, 16);
        }
        if ((tid & 31) < CQ) part[tid >> 5][cq] = y;
        __syncthreads();
        if (tid < P) {
            const float* pf = reinterpret_cast<const float*>(part);
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < NT / 32; ++k) s += pf[k * P + tid];
            if (g.skip) s = fmaf(g.skip[h], sx[x][tid], s);
            if (g.z) s *= silu(to_f32(static_cast<const TI*>(g.z)[(size_t)n * g.z_stride + h * P + tid]));
            static_cast<TI*>(g.o)[(size_t)n * W + h * P + tid] = from_f32<TI>(s);
        }
        __syncthreads();
    }
    cluster_wait();
    if (rank == 0 && tid < 2 * N) {
#pragma unroll
        for (int s = 0; s < RING; ++s) ring[(size_t)s * Cx + cb] = rb[s + 1];
    }
}

// Cluster size of the fused kernel for a group of HG heads: a power of two up
// to 16, at most two heads a CTA; 0: the group is too large for it.
int cluster_size(int HG) {
    int cs = 1;
    while (cs < HG && cs < 16) cs *= 2;
    return HG <= 2 * cs ? cs : 0;
}

// The cluster size a call runs the fused kernel with, or 0.  Up to 32 MB of
// states (5 us at HBM rate) a call costs less than its second launch.
int fused_cluster(int64_t n, int H, int G, int P, int N) {
    return n * H * N * P * 4 <= ((int64_t)32 << 20) ? cluster_size(H / G) : 0;
}

template <typename TI, int P, int N>
cudaError_t fused(const DecodeArgs& a, int cs, cudaStream_t s) {
    auto k = fused_kernel<TI, P, N>;
    if (cs > 8) {   // 16 CTAs are beyond the portable size (set once per device)
        static std::atomic<uint64_t> done{0};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
        if (!(done.load() & bit)) {
            e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            done.fetch_or(bit);
        }
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)a.n * a.G * cs));
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a, cs);
}

template <typename TI, int P, int N>
cudaError_t state(const DecodeArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>((int64_t)a.n * a.H, 152 * PER_SM));
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, state_kernel<TI, P, N>, a);
}

template <typename TI>
cudaError_t decode(const DecodeArgs& a, cudaStream_t s) {
    if (const int cs = fused_cluster(a.n, a.H, a.G, a.P, a.N)) {
        if (a.P == 64) return a.N == 64 ? fused<TI, 64, 64>(a, cs, s) : fused<TI, 64, 128>(a, cs, s);
        return a.N == 64 ? fused<TI, 128, 64>(a, cs, s) : fused<TI, 128, 128>(a, cs, s);
    }
    const int64_t per = (int64_t)(a.H * a.P + 2 * a.G * a.N) / (16 / sizeof(TI));
    conv_kernel<TI><<<(unsigned)((a.n * (per + a.H) + NT - 1) / NT), NT, 0, s>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (a.P == 64) return a.N == 64 ? state<TI, 64, 64>(a, s) : state<TI, 64, 128>(a, s);
    return a.N == 64 ? state<TI, 128, 64>(a, s) : state<TI, 128, 128>(a, s);
}

}  // namespace

bool decode_needs_workspace(int64_t n, int H, int G, int P, int N) { return fused_cluster(n, H, G, P, N) == 0; }

cudaError_t launch_decode(const DecodeArgs& a, int io_bf16, cudaStream_t s) {
    return io_bf16 ? decode<__nv_bfloat16>(a, s) : decode<float>(a, s);
}

}  // namespace ssm
}  // namespace kda
