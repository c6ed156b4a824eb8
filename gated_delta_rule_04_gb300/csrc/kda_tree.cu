// A tree of drafted tokens against the KDA state (kda_decode_tree), and the
// state after an accepted path through it (kda_tree_commit).
//
// The step of a path's last token r from the state S0 under the root, with
// Gam_r the sum of the gate g over the path (per channel) and anc(r) the nodes
// above r, unrolls to
//   u_r = beta_r (v_r - (k_r e^{Gam_r})^T S0 - sum_{s in anc(r)} A_rs u_s)
//   o_r = (q_r e^{Gam_r})^T S0 + sum_{s in anc(r) or s = r} P_rs u_s
//   A_rs = sum_c k_rc k_sc e^{Gam_rc - Gam_sc},  P_rs the same with q_r
// so one read of S0 serves every node of the tree, where a walk would carry a
// 64 KiB state per branch.  Gam falls along a path: every exponent here is
// <= 0 and no factor leaves fp32's range, with either gate.  Parents come
// before children, so the solve for u runs over the nodes in order.
//
// The tree kernel keeps fp32 throughout; one CTA per (session, head), 256
// threads.
#include <algorithm>
#include <atomic>

#include "kda_common.cuh"

namespace kda {
namespace {

constexpr int NT = 256;

struct TreeSmemHead {
    unsigned long long anc[KDA_TREE_MAX_NODES];   // ancestors of a node, itself included; 0: unused node
    int win[KDA_TREE_MAX_NODES][CONV_K];          // its conv window, oldest first: node, or -1 - j for the j-th newest ring row
    float beta[KDA_TREE_MAX_NODES];
};

// The path above node r: its ancestor set and conv window.  False when a link
// is not a parent (below -1 or not below its child).
__device__ __forceinline__ bool walk_up(const int32_t* par, int r, unsigned long long* anc, int (&win)[CONV_K]) {
    unsigned long long m = 1ull << r;
    int filled = CONV_K - 1;
    win[filled] = r;
    for (int x = r;;) {
        const int p = par[x];
        if (p < -1 || p >= x) return false;
        if (p < 0) break;
        m |= 1ull << p;
        if (filled > 0) win[--filled] = p;
        x = p;
    }
    for (int j = 0; filled > 0; ++j) win[--filled] = -1 - j;
    *anc = m;
    return true;
}

template <typename TI>
__global__ void __launch_bounds__(NT) tree_kernel(TreeArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    TreeSmemHead& hd = *reinterpret_cast<TreeSmemHead*>(smem_raw);
    const int R = a.n_nodes, H = a.H, W = H * D;
    float* kk = reinterpret_cast<float*>(smem_raw + sizeof(TreeSmemHead));   // [R][128] k^, then k^ e^Gam
    float* qq = kk + R * D;                                                  // [R][128] q^, then q^ e^Gam
    float* gam = qq + R * D;                                                 // [R][128] Gam, then q^ e^Gam S0
    float* uu = gam + R * D;                                                 // [R][128] v, then u
    float* A = uu + R * D;                                                   // [R][R]
    float* Pm = A + R * R;                                                   // [R][R]
    __shared__ int32_t par[KDA_TREE_MAX_NODES];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = blockIdx.x / H, h = blockIdx.x % H;
    const int slot = a.slots ? a.slots[n] : n;
    if (slot < 0 || slot >= a.n_slots) return;
    const size_t row0 = (size_t)n * R;

    if (tid < R) par[tid] = a.parents[row0 + tid];
    __syncthreads();
    if (tid < R) {
        int win[CONV_K];
        unsigned long long m = 0;
        if (!walk_up(par, tid, &m, win)) {
            m = 0;
            for (int j = 0; j < CONV_K; ++j) win[j] = tid;   // (in range; the node is not computed further)
        }
        hd.anc[tid] = m;
        for (int j = 0; j < CONV_K; ++j) hd.win[tid][j] = win[j];
        hd.beta[tid] = sigmoid_fast(to_f32(static_cast<const TI*>(a.b)[(row0 + tid) * H + h]));
    }
    __syncthreads();

    // ---- conv + SiLU, gate: a thread owns a channel
    const int i = tid & (D - 1), half = tid >> 7, c = h * D + i;
    {
        const TI* ring = static_cast<const TI*>(a.ring) + (size_t)slot * 3 * RING * W + c;
        const TI* src[3] = {static_cast<const TI*>(a.q) + row0 * W + c, static_cast<const TI*>(a.k) + row0 * W + c,
                            static_cast<const TI*>(a.v) + row0 * W + c};
        float* dst[3] = {qq, kk, uu};
        for (int p = 0; p < 3; ++p) {
            const float4 w = __ldg(reinterpret_cast<const float4*>(a.conv_w + ((size_t)p * W + c) * CONV_K));
            const float wt[4] = {w.x, w.y, w.z, w.w};
            for (int r = half; r < R; r += 2) {
                float y = 0.f;
#pragma unroll
                for (int j = 0; j < CONV_K; ++j) {
                    const int x = hd.win[r][j];
                    const TI raw = x >= 0 ? src[p][(size_t)x * W] : ring[((size_t)p * RING + (RING + x)) * W];
                    y = fmaf(wt[j], to_f32(raw), y);
                }
                dst[p][r * D + i] = silu_fast(y);
            }
        }
        const float eA = expf(a.A_log[h]), dtb = a.dt_bias[c];
        const TI* z = static_cast<const TI*>(a.z) + row0 * W + c;
        for (int r = half; r < R; r += 2) gam[r * D + i] = decay_gate(a.gate_kind, a.lb, eA, to_f32(z[(size_t)r * W]) + dtb);
    }
    __syncthreads();
    // ---- Gam along the paths (threads 0-127), L2 norms (a warp per node)
    if (half == 0) {
        for (int r = 0; r < R; ++r) {
            const int p = par[r];
            if (hd.anc[r] && p >= 0) gam[r * D + i] += gam[p * D + i];
        }
    }
    for (int r = warp; r < R; r += NT / 32) {
        float4 q4 = *reinterpret_cast<const float4*>(qq + r * D + 4 * lane);
        float4 k4 = *reinterpret_cast<const float4*>(kk + r * D + 4 * lane);
        const float sq = warp_sum(q4.x * q4.x + q4.y * q4.y + q4.z * q4.z + q4.w * q4.w);
        const float sk = warp_sum(k4.x * k4.x + k4.y * k4.y + k4.z * k4.z + k4.w * k4.w);
        const float rq = rsqrtf(sq + a.l2_eps) * a.q_scale, rk = rsqrtf(sk + a.l2_eps);
        *reinterpret_cast<float4*>(qq + r * D + 4 * lane) = make_float4(q4.x * rq, q4.y * rq, q4.z * rq, q4.w * rq);
        *reinterpret_cast<float4*>(kk + r * D + 4 * lane) = make_float4(k4.x * rk, k4.y * rk, k4.z * rk, k4.w * rk);
    }
    __syncthreads();
    // ---- A and P: a warp per row, four channels per lane
    for (int r = warp; r < R; r += NT / 32) {
        const float4 q4 = *reinterpret_cast<const float4*>(qq + r * D + 4 * lane);
        const float4 k4 = *reinterpret_cast<const float4*>(kk + r * D + 4 * lane);
        const float4 g4 = *reinterpret_cast<const float4*>(gam + r * D + 4 * lane);
        for (unsigned long long m = hd.anc[r]; m; m &= m - 1) {
            const int s = __ffsll(m) - 1;
            const float4 ks = *reinterpret_cast<const float4*>(kk + s * D + 4 * lane);
            const float4 gs = *reinterpret_cast<const float4*>(gam + s * D + 4 * lane);
            const float e0 = ks.x * __expf(g4.x - gs.x), e1 = ks.y * __expf(g4.y - gs.y);
            const float e2 = ks.z * __expf(g4.z - gs.z), e3 = ks.w * __expf(g4.w - gs.w);
            const float sa = warp_sum(k4.x * e0 + k4.y * e1 + k4.z * e2 + k4.w * e3);
            const float sp = warp_sum(q4.x * e0 + q4.y * e1 + q4.z * e2 + q4.w * e3);
            if (lane == 0) {
                A[r * R + s] = sa;
                Pm[r * R + s] = sp;
            }
        }
    }
    __syncthreads();
    for (int x = tid; x < R * D; x += NT) {
        const float e = __expf(gam[x]);
        kk[x] *= e;
        qq[x] *= e;
    }
    __syncthreads();
    // ---- rows times S0: threads 0-127 take the k rows, 128-255 the q rows; a thread
    // owns a value column and 16 nodes a pass
    {
        const float* S0 = a.S + ((size_t)slot * H + h) * D * D + i;
        const float* rows = half == 0 ? kk : qq;
        for (int r0 = 0; r0 < R; r0 += 16) {
            float acc[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) acc[x] = 0.f;
#pragma unroll 1
            for (int ch = 0; ch < D; ch += 4) {
                const float s0 = __ldg(S0 + ch * D), s1 = __ldg(S0 + (ch + 1) * D), s2 = __ldg(S0 + (ch + 2) * D),
                            s3 = __ldg(S0 + (ch + 3) * D);
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int r = min(r0 + x, R - 1);
                    const float4 w = *reinterpret_cast<const float4*>(rows + r * D + ch);
                    acc[x] = fmaf(w.x, s0, fmaf(w.y, s1, fmaf(w.z, s2, fmaf(w.w, s3, acc[x]))));
                }
            }
#pragma unroll
            for (int x = 0; x < 16; ++x) {
                const int r = r0 + x;
                if (r >= R) continue;
                if (half == 0) uu[r * D + i] = hd.beta[r] * (uu[r * D + i] - acc[x]);
                else gam[r * D + i] = acc[x];
            }
        }
    }
    __syncthreads();
    // ---- u over the nodes in order: a thread owns a value column
    if (half == 0) {
        for (int r = 0; r < R; ++r) {
            const unsigned long long self = hd.anc[r];
            if (!self) continue;
            float t = 0.f;
            for (unsigned long long m = self & ~(1ull << r); m; m &= m - 1) {
                const int s = __ffsll(m) - 1;
                t = fmaf(A[r * R + s], uu[s * D + i], t);
            }
            uu[r * D + i] = fmaf(-hd.beta[r], t, uu[r * D + i]);
        }
    }
    __syncthreads();
    // ---- o, RMSNormGated: a warp per node, four channels per lane
    for (int r = warp; r < R; r += NT / 32) {
        if (!hd.anc[r]) continue;
        float4 o4 = *reinterpret_cast<const float4*>(gam + r * D + 4 * lane);
        for (unsigned long long m = hd.anc[r]; m; m &= m - 1) {
            const int s = __ffsll(m) - 1;
            const float w = Pm[r * R + s];
            const float4 u4 = *reinterpret_cast<const float4*>(uu + s * D + 4 * lane);
            o4.x = fmaf(w, u4.x, o4.x); o4.y = fmaf(w, u4.y, o4.y);
            o4.z = fmaf(w, u4.z, o4.z); o4.w = fmaf(w, u4.w, o4.w);
        }
        const float ss = warp_sum(o4.x * o4.x + o4.y * o4.y + o4.z * o4.z + o4.w * o4.w);
        const float rs = rsqrtf(ss * (1.0f / D) + a.norm_eps);
        const float ov[4] = {o4.x, o4.y, o4.z, o4.w};
        const size_t at = (row0 + r) * W + (size_t)h * D + 4 * lane;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float gt = to_f32(static_cast<const TI*>(a.gout)[at + m]);
            static_cast<TI*>(a.o)[at + m] = from_f32<TI>(ov[m] * rs * a.norm_w[4 * lane + m] * sigmoid_fast(gt));
        }
    }
}

size_t tree_smem(int R) { return sizeof(TreeSmemHead) + sizeof(float) * ((size_t)4 * R * D + (size_t)2 * R * R); }

// Opts a kernel into `bytes` of dynamic shared memory, once per device.
cudaError_t opt_in(const void* f, size_t bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit && (done.load() & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) done.fetch_or(bit);
    return e;
}

// ---- commit --------------------------------------------------------------------
// The decode step over the path's tokens, the state in registers between
// them (warp w: key rows 16w .. 16w+15, lane l: columns 4l .. 4l+3): one read
// and one write of the state, which bounds the kernel.  Tokens go through the
// conv, gate and norm in groups of CG.
constexpr int CG = 8;

struct CommitSmem {
    float kc[CG][D], va[CG][D], e[CG][D], kh[CG][D], av[CG][D];
    float beta[CG];
    float red[NT / 32][D];
    float d[D];
    int path[KDA_TREE_MAX_NODES];
    int bad;
};

template <typename TI>
__global__ void __launch_bounds__(NT, 2) commit_kernel(CommitArgs a) {
    __shared__ CommitSmem sm;
    const int H = a.H, W = H * D;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = blockIdx.x / H, h = blockIdx.x % H;
    const int slot = a.slots ? a.slots[n] : n;
    if (slot < 0 || slot >= a.n_slots) return;
    const int len = a.path_len[n];
    if (len < 0 || len > a.max_len) return;
    if (len == 0 && a.S_in == a.S_out && a.ring_in == a.ring_out) return;
    const float* Sg_in = a.S_in + ((size_t)slot * H + h) * D * D;
    float4 Sr[16];
#pragma unroll
    for (int r = 0; r < 16; ++r)
        Sr[r] = __ldcs(reinterpret_cast<const float4*>(Sg_in + (size_t)(16 * warp + r) * D) + lane);
    if (tid == 0) sm.bad = 0;
    __syncthreads();
    if (tid < len) {
        const int node = a.path[(size_t)n * a.max_len + tid];
        sm.path[tid] = node;
        if (node < 0 || node >= a.n_nodes) sm.bad = 1;
    }
    __syncthreads();
    if (sm.bad) return;

    const int i = tid & (D - 1), half = tid >> 7, c = h * D + i;
    const size_t row0 = (size_t)n * a.n_nodes;
    const TI* ring = static_cast<const TI*>(a.ring_in) + (size_t)slot * 3 * RING * W + c;
    const TI* plane[3] = {static_cast<const TI*>(a.q) + row0 * W + c, static_cast<const TI*>(a.k) + row0 * W + c,
                          static_cast<const TI*>(a.v) + row0 * W + c};
    // raw row of plane p at position t of the path (t < 0: the ring)
    auto raw = [&](int p, int t) -> TI {
        return t >= 0 ? plane[p][(size_t)sm.path[t] * W] : ring[((size_t)p * RING + (RING + t)) * W];
    };
    const int p = 1 + half;   // threads 0-127 own a channel of k, 128-255 of v and the gate
    const float4 w = __ldg(reinterpret_cast<const float4*>(a.conv_w + ((size_t)p * W + c) * CONV_K));
    const float eA = expf(a.A_log[h]), dtb = a.dt_bias[c];

#pragma unroll 1
    for (int g0 = 0; g0 < len; g0 += CG) {
        const int ng = min(CG, len - g0);
        for (int t = 0; t < ng; ++t) {
            const int x = g0 + t;
            float y = w.x * to_f32(raw(p, x - 3));
            y = fmaf(w.y, to_f32(raw(p, x - 2)), y);
            y = fmaf(w.z, to_f32(raw(p, x - 1)), y);
            y = fmaf(w.w, to_f32(raw(p, x)), y);
            y = silu_fast(y);
            if (half == 0) {
                sm.kc[t][i] = y;
            } else {
                sm.va[t][i] = y;
                const float z = to_f32(static_cast<const TI*>(a.z)[(row0 + sm.path[x]) * W + c]);
                sm.e[t][i] = __expf(decay_gate(a.gate_kind, a.lb, eA, z + dtb));
            }
        }
        if (tid < ng) sm.beta[tid] = sigmoid_fast(to_f32(static_cast<const TI*>(a.b)[(row0 + sm.path[g0 + tid]) * H + h]));
        __syncthreads();
        if (warp < ng) {
            const float4 k4 = *reinterpret_cast<const float4*>(&sm.kc[warp][4 * lane]);
            const float4 e4 = *reinterpret_cast<const float4*>(&sm.e[warp][4 * lane]);
            const float rk = rsqrtf(warp_sum(k4.x * k4.x + k4.y * k4.y + k4.z * k4.z + k4.w * k4.w) + a.l2_eps);
            const float4 kh = make_float4(k4.x * rk, k4.y * rk, k4.z * rk, k4.w * rk);
            *reinterpret_cast<float4*>(&sm.kh[warp][4 * lane]) = kh;
            *reinterpret_cast<float4*>(&sm.av[warp][4 * lane]) = make_float4(e4.x * kh.x, e4.y * kh.y, e4.z * kh.z, e4.w * kh.w);
        }
        __syncthreads();
#pragma unroll 1
        for (int t = 0; t < ng; ++t) {
            float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float ar = sm.av[t][16 * warp + r];
                u.x = fmaf(ar, Sr[r].x, u.x); u.y = fmaf(ar, Sr[r].y, u.y);
                u.z = fmaf(ar, Sr[r].z, u.z); u.w = fmaf(ar, Sr[r].w, u.w);
            }
            *reinterpret_cast<float4*>(&sm.red[warp][4 * lane]) = u;
            __syncthreads();
            if (tid < D) {
                float uj = 0.f;
#pragma unroll
                for (int k = 0; k < NT / 32; ++k) uj += sm.red[k][tid];
                sm.d[tid] = sm.beta[t] * (sm.va[t][tid] - uj);
            }
            __syncthreads();
            const float4 d4 = *reinterpret_cast<const float4*>(&sm.d[4 * lane]);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const float er = sm.e[t][16 * warp + r], kr = sm.kh[t][16 * warp + r];
                Sr[r].x = fmaf(er, Sr[r].x, kr * d4.x); Sr[r].y = fmaf(er, Sr[r].y, kr * d4.y);
                Sr[r].z = fmaf(er, Sr[r].z, kr * d4.z); Sr[r].w = fmaf(er, Sr[r].w, kr * d4.w);
            }
        }
        __syncthreads();   // the group's vectors are rewritten
    }
    float* Sg_out = a.S_out + ((size_t)slot * H + h) * D * D;
#pragma unroll
    for (int r = 0; r < 16; ++r) __stcs(reinterpret_cast<float4*>(Sg_out + (size_t)(16 * warp + r) * D) + lane, Sr[r]);

    // ring: the last three raw rows of ring | path, of every plane (every read of the
    // input ring by the conv is behind the barriers above; a thread owns its channel)
    TI* rout = static_cast<TI*>(a.ring_out) + (size_t)slot * 3 * RING * W + c;
    for (int pl = half; pl < 3; pl += 2) {
        TI row[RING];
#pragma unroll
        for (int s = 0; s < RING; ++s) row[s] = raw(pl, len - RING + s);
#pragma unroll
        for (int s = 0; s < RING; ++s) rout[((size_t)pl * RING + s) * W] = row[s];
    }
}

}  // namespace

cudaError_t launch_tree(const TreeArgs& a, int io_bf16, cudaStream_t s) {
    const size_t bytes = tree_smem(a.n_nodes);
    const int64_t blocks = (int64_t)a.n * a.H;
    static std::atomic<uint64_t> done[2];
    const void* f = io_bf16 ? (const void*)tree_kernel<__nv_bfloat16> : (const void*)tree_kernel<float>;
    const cudaError_t e = opt_in(f, tree_smem(KDA_TREE_MAX_NODES), done[io_bf16 ? 1 : 0]);
    if (e != cudaSuccess) return e;
    if (io_bf16) tree_kernel<__nv_bfloat16><<<(unsigned)blocks, NT, bytes, s>>>(a);
    else tree_kernel<float><<<(unsigned)blocks, NT, bytes, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_commit(const CommitArgs& a, int io_bf16, cudaStream_t s) {
    const unsigned blocks = (unsigned)((int64_t)a.n * a.H);
    if (io_bf16) commit_kernel<__nv_bfloat16><<<blocks, NT, 0, s>>>(a);
    else commit_kernel<float><<<blocks, NT, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
