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
// <= 0 and no factor leaves fp32's range, with either gate.  Nodes of one depth
// do not see one another, so the solve for u runs depth by depth.
//
// Tree kernel: one CTA per SM (two for trees of up to 32 nodes) walks the
// (session, head) items; an item's phases are
//   1. the nodes' raw rows to shared memory as fp32, the state to registers;
//   2. conv + SiLU and the gate, a thread per channel pair and plane, 16 nodes at
//      a time; a node's window holds only nodes above it, so the planes are
//      convolved in place, the last nodes first; L2 norms, a warp per node;
//   3. A and P, a warp per node walking up its path: the factor
//      e^{Gam_r - Gam_s} is the running product of e^{g} over the nodes passed, so
//      a pair costs no exponential, and at the root it is e^{Gam_r};
//   4. [K e^Gam; Q e^Gam] S0 on the tensor cores, transposed: A = S0^T in
//      tensor memory (lane = value), B = the rows, N = 2 x nodes, K = keys.  At 64
//      nodes these products are 80 % of the item's arithmetic, and 8.5 us of
//      fp32 FMAs per SM; as three tcgen05 products of fp16 pairs (hi hi, hi lo,
//      lo hi: 22-bit operands, so that fp32 outputs hold too) under 1 us.  S0 is
//      scaled by an exact power of two per value, the rows by 2^8;
//   5. u depth by depth, a warp per node; o, RMSNormGated, a warp per node.
// While an item computes, the next one's state and rows go to L2.
//
// 64 trees of 64 nodes, 32 heads: 336 us, where reading each state and row once
// takes 51.  One CTA fits an SM (200 KB of planes at 64 nodes), so its phases
// follow one another: of 47 thousand cycles an item, loads take 9, the conv 8.5, A
// and P 8, the solve 6, the outputs 6; some 16 thousand are shared-memory bandwidth (48 % of it).
// The first kernel, fp32 throughout and a thread per channel, took 2345 us, tensor
// cores for phase 4 and running products for phase 3 566, the conv in pairs and the
// solve by depth 357, a warp per node in it and the prefetch during the MMAs 336.
// One tree of 16 nodes: 13 us.
#include <stddef.h>

#include <algorithm>
#include <atomic>

#include "kda_chunk_layout.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace {

constexpr int NT = 256;                     // commit kernel
constexpr int RMAX = KDA_TREE_MAX_NODES;
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr uint32_t TM_HI = 0, TM_LO = 64, TM_D = 128, TMEM_COLS = 256;
// of the fp16 rows, so that their low halves are normal: unit vectors, k^ and q^ alike (q_scale,
// which may be of any size, multiplies the outputs)
constexpr float ROW_SCALE = 256.f;

struct TreeHead {
    float beta[RMAX];
    int32_t par[RMAX];
    int32_t depth[RMAX];                    // nodes on the path, itself included; 0: unused node
    alignas(16) int32_t win[RMAX][CONV_K];  // conv window, oldest first: node, or -1 - j for the j-th newest ring row
    float smax[4][D];                       // column maxima of |S0| by key part
    uint8_t order[RMAX];                    // nodes by depth (unused ones first)
    int32_t level[RMAX + 1];                // level[l]: nodes of a depth below l (l >= 1)
    alignas(16) uint8_t path[RMAX][RMAX];   // node, parent, grandparent, ..., then the padding row (read in fours)
    unsigned long long bar;
    uint32_t tmem;
    int32_t bad;
};

static_assert(offsetof(TreeHead, path) % 16 == 0 && offsetof(TreeHead, win) % 16 == 0 && offsetof(TreeHead, bar) % 8 == 0,
              "vector accesses");

// Shared memory of a tree of R nodes (rows padded to Rp, a multiple of 8).
struct TreeMap {
    uint32_t hi, lo, k, q, v, ap, total;
    __host__ __device__ explicit TreeMap(int Rp) {
        const uint32_t plane = (uint32_t)Rp * D * 4;
        hi = (sizeof(TreeHead) + 1023) / 1024 * 1024;   // fp16 [2 panels][2 Rp rows][64 keys], rows k | q
        lo = hi + plane;                    // the same of the low halves; before that fp32 [Rp][128] e^g
        // k, q, v: the ring's three rows before row 0 (row -1 the newest); e^g, k, v: row Rp,
        // where a path's padding points (e^g = 1, k = u = 0)
        k = lo + plane + (RING + 1) * D * 4;    // fp32 [Rp + 1][128] raw k, then k^
        q = k + plane + (RING + 1) * D * 4;     // raw q, then q^, then (q e^Gam)^T S0
        v = q + plane + (RING + 1) * D * 4;     // raw v, then v, then u
        ap = v + plane + D * 4;             //                     // fp32 [Rp][2][Rp] A, then P of a node and the d-th node of its path
        total = ap + (uint32_t)Rp * Rp * 8 + 1024;
    }
};

__device__ __forceinline__ uint32_t pack2_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// fp16 pairs (hi, lo) of two values
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack2_f16(a, b);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = pack2_f16(a - f.x, b - f.y);
}

// The path above node r and its conv window; 0 when a link of it is not a
// parent (below -1 or not below its child).
__device__ __forceinline__ int walk_up(const int32_t* par, int r, int Rp, uint8_t* path, int32_t* win) {
    int n = 0;
    for (int x = 0; x < RMAX; x += 8) *reinterpret_cast<uint2*>(path + x) = make_uint2(0x01010101u * (uint32_t)Rp, 0x01010101u * (uint32_t)Rp);
    for (int x = r;;) {
        path[n] = (uint8_t)x;
        if (n < CONV_K) win[CONV_K - 1 - n] = x;
        ++n;
        const int p = par[x];
        if (p < -1 || p >= x) return 0;
        if (p < 0) break;
        x = p;
    }
    for (int i = n; i < CONV_K; ++i) win[CONV_K - 1 - i] = n - 1 - i;   // -1, -2, -3 past the root
    return n;
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Sums of eight values over the warp; lanes 4 i .. 4 i + 3 return value i.
__device__ __forceinline__ float warp_sum8(float (&v)[8], int lane) {
#pragma unroll
    for (int w = 4, o = 16; w > 0; w >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float send = up ? v[i] : v[i + w], keep = up ? v[i + w] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// 16 bytes of a raw row as fp32.
template <typename TI>
__device__ __forceinline__ void to_rows(float* dst, uint4 u) {
    if constexpr (sizeof(TI) == 4) {
        *reinterpret_cast<uint4*>(dst) = u;
    } else {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
        const float2 a = __bfloat1622float2(h[0]), b = __bfloat1622float2(h[1]), c = __bfloat1622float2(h[2]), d = __bfloat1622float2(h[3]);
        reinterpret_cast<float4*>(dst)[0] = make_float4(a.x, a.y, b.x, b.y);
        reinterpret_cast<float4*>(dst)[1] = make_float4(c.x, c.y, d.x, d.y);
    }
}

// Four elements of a row as fp32 (16-byte or 8-byte aligned).
template <typename TI>
__device__ __forceinline__ float4 load4(const TI* p) {
    if constexpr (sizeof(TI) == 4) {
        return *reinterpret_cast<const float4*>(p);
    } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
}

template <typename TI, int THREADS>
__global__ void __launch_bounds__(THREADS, 512 / THREADS) tree_kernel(TreeArgs a) {
    constexpr int NW = THREADS / 32, KP = THREADS / 128, KEYS = D / KP;   // warps; key parts and keys of a part
    constexpr int NODES = THREADS / 8, ROWS = NODES / NW;                // most nodes, and of a warp (4)
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = ptx::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    unsigned char* sb = smem_raw + (base - raw);
    TreeHead& hd = *reinterpret_cast<TreeHead*>(sb);
    const int R = a.n_nodes, H = a.H, W = H * D, Rp = (R + 7) / 8 * 8;
    const TreeMap map(Rp);
    float* kk = reinterpret_cast<float*>(sb + map.k);
    float* qq = reinterpret_cast<float*>(sb + map.q);
    float* vv = reinterpret_cast<float*>(sb + map.v);
    float* eg = reinterpret_cast<float*>(sb + map.lo);
    float* ap = reinterpret_cast<float*>(sb + map.ap);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t bar = ptx::smem_u32(&hd.bar);
    if (warp == 0) {
        ptx::tmem_alloc(ptx::smem_u32(&hd.tmem), TMEM_COLS);
        ptx::tmem_relinquish();
    }
    if (tid == 0) {
        ptx::mbar_init(bar, 1);
        ptx::fence_mbar_init();
        hd.bad = 0;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = hd.tmem;
    const int quarter = warp & 3, part = warp >> 2;      // TMEM lane quarter; key part
    const uint32_t tlane = tmem + ((uint32_t)(32 * quarter) << 16);
    const int j = 32 * quarter + lane;                   // value column = TMEM lane
    const int i = tid & (D - 1);                         // channel of the conv phase

    const uint32_t items = (uint32_t)a.n * H;            // (below 2^31: checked on the host)
    uint32_t phase = 0;
    uint32_t item = blockIdx.x;
    auto slot_of = [&](uint32_t it) { return it >= items ? -1 : a.slots ? a.slots[it / H] : (int)(it / H); };
    int next_slot = slot_of(item);
#pragma unroll 1
    for (; item < items; item += gridDim.x) {
        const int n = (int)(item / H), h = (int)(item % H), slot = next_slot;
        next_slot = slot_of(item + gridDim.x);
        if (slot < 0 || slot >= a.n_slots) continue;
        const size_t row0 = (size_t)n * R;
        const int c = h * D + i;
        if (tid == 0 && item == blockIdx.x) ptx::bulk_prefetch_l2(a.S + ((size_t)slot * H + h) * D * D, D * D * 4);

        // ---- 1. raw rows into shared memory, then the state into registers (which would not
        // hold both at once)
        {
            constexpr int E = 16 / sizeof(TI), CH = D / E;   // elements and chunks of 16 bytes
            const size_t off = row0 * W + (size_t)h * D;
            const TI* src[4] = {static_cast<const TI*>(a.q) + off, static_cast<const TI*>(a.k) + off, static_cast<const TI*>(a.v) + off,
                                static_cast<const TI*>(a.z) + off};
            float* dst[4] = {qq, kk, vv, eg};
            // (a chunk of each plane in flight per thread: with two the registers spill)
#pragma unroll 1
            for (int x = tid; x < R * CH; x += THREADS) {
                uint4 u[4];
#pragma unroll
                for (int p = 0; p < 4; ++p) u[p] = __ldg(reinterpret_cast<const uint4*>(src[p] + (size_t)(x / CH) * W) + x % CH);
#pragma unroll
                for (int p = 0; p < 4; ++p) to_rows<TI>(dst[p] + x * E, u[p]);
            }
        }
        float S[KEYS];
        {
            const float* S0 = a.S + ((size_t)slot * H + h) * D * D + (size_t)(KEYS * part) * D + j;
#pragma unroll
            for (int x = 0; x < KEYS; ++x) S[x] = __ldg(S0 + (size_t)x * D);
        }
        if (tid < R) hd.par[tid] = a.parents[row0 + tid];
        // the ring's rows and the padding row; the conv weights of this thread's plane and channels
        {
            constexpr int NR = (3 * RING + KP - 1) / KP;     // ring rows of this thread's channel
            const TI* src = static_cast<const TI*>(a.ring) + (size_t)slot * 3 * RING * W + c;
            TI v[NR];
#pragma unroll
            for (int x = 0; x < NR; ++x)
                if (KP * x + (tid >> 7) < 3 * RING) v[x] = src[(size_t)(KP * x + (tid >> 7)) * W];
#pragma unroll
            for (int x = 0; x < NR; ++x) {
                const int y = KP * x + (tid >> 7), p = y / RING, s = y % RING;
                if (y < 3 * RING) (p == 0 ? qq : p == 1 ? kk : vv)[(s - RING) * D + i] = to_f32(v[x]);
            }
        }
        if (tid < D) {
            eg[Rp * D + tid] = 1.f;
            kk[Rp * D + tid] = 0.f;
            vv[Rp * D + tid] = 0.f;
        }
        const int pl = (tid >> 6) & 3, cpair = 2 * (tid & 63), node0 = 32 * (tid >> 8);
        const int c2 = h * D + cpair;
        float2 cw[CONV_K];
        if (pl < 3) {
            const float4* w = reinterpret_cast<const float4*>(a.conv_w + ((size_t)pl * W + c2) * CONV_K);
            const float4 wa = __ldg(w), wb = __ldg(w + 1);
            cw[0] = make_float2(wa.x, wb.x); cw[1] = make_float2(wa.y, wb.y);
            cw[2] = make_float2(wa.z, wb.z); cw[3] = make_float2(wa.w, wb.w);
        } else {
            cw[0] = *reinterpret_cast<const float2*>(a.dt_bias + c2);
            cw[1] = make_float2(expf(a.A_log[h]), 0.f);
        }
        __syncthreads();
        if (tid < R) {
            int win[CONV_K] = {0, 0, 0, 0};
            hd.depth[tid] = walk_up(hd.par, tid, Rp, hd.path[tid], win);
            for (int x = 0; x < CONV_K; ++x) hd.win[tid][x] = win[x];
            hd.beta[tid] = sigmoid_fast(to_f32(static_cast<const TI*>(a.b)[(row0 + tid) * H + h]));
        }
        {
            float m = 0.f;
#pragma unroll
            for (int x = 0; x < KEYS; ++x) m = fmaxf(m, fabsf(S[x]));
            hd.smax[part][j] = m;
        }
        __syncthreads();
        // S0^T to tensor memory as fp16 pairs, each value column scaled into [1, 2)
        float unscale;                                       // of D's lane
        {
            float m = hd.smax[0][j];
#pragma unroll
            for (int x = 1; x < KP; ++x) m = fmaxf(m, hd.smax[x][j]);
            int e = (int)((__float_as_uint(m) >> 23) & 255u) - 127;
            e = e < -100 ? -100 : e > 100 ? 100 : e;
            const float f = __uint_as_float((uint32_t)(127 - e) << 23);
            unscale = __uint_as_float((uint32_t)(127 + e) << 23) * (1.f / ROW_SCALE);
#pragma unroll
            for (int g = 0; g < KEYS / 32; ++g) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int x = 0; x < 16; ++x) split2(S[32 * g + 2 * x] * f, S[32 * g + 2 * x + 1] * f, hi[x], lo[x]);
                ptx::tmem_st16u(tlane + TM_HI + KEYS / 2 * part + 16 * g, hi);
                ptx::tmem_st16u(tlane + TM_LO + KEYS / 2 * part + 16 * g, lo);
            }
            ptx::tmem_wait_st();
        }
        // ---- 2. conv + SiLU and e^g, in place: a thread owns a plane's channel pair and takes 16
        // nodes at a time, the last ones first, every window read before they are written
        {
            float* plane = (pl == 0 ? qq : pl == 1 ? kk : pl == 2 ? vv : eg) + cpair;
            auto at = [&](int r) { return *reinterpret_cast<const float2*>(plane + r * D); };
            float2 y[16];
            auto compute = [&](int r0) {
                if (r0 >= R) return;
                if (pl < 3) {
#pragma unroll
                    for (int m = 0; m < 16; ++m) {
                        const int4 w = *reinterpret_cast<const int4*>(hd.win[min(r0 + m, R - 1)]);
                        y[m] = __fmul2_rn(cw[0], at(w.x));
                        y[m] = __ffma2_rn(cw[1], at(w.y), y[m]);
                        y[m] = __ffma2_rn(cw[2], at(w.z), y[m]);
                        y[m] = __ffma2_rn(cw[3], at(w.w), y[m]);
                        if ((m & 3) == 3) asm volatile("" ::: "memory");   // (all windows at once would spill)
                    }
#pragma unroll
                    for (int m = 0; m < 16; ++m) y[m] = make_float2(silu_fast(y[m].x), silu_fast(y[m].y));
                } else {
#pragma unroll
                    for (int m = 0; m < 16; ++m) y[m] = __fadd2_rn(at(min(r0 + m, R - 1)), cw[0]);
                    if (a.gate_kind == KDA_GATE_BOUNDED) {
#pragma unroll
                        for (int m = 0; m < 16; ++m)
                            y[m] = make_float2(__expf(a.lb * sigmoid_fast(cw[1].x * y[m].x)), __expf(a.lb * sigmoid_fast(cw[1].x * y[m].y)));
                    } else {
#pragma unroll
                        for (int m = 0; m < 16; ++m)
                            y[m] = make_float2(__expf(decay_gate(1, 0.f, cw[1].x, y[m].x)), __expf(decay_gate(1, 0.f, cw[1].x, y[m].y)));
                    }
                }
            };
            auto store = [&](int r0) {
#pragma unroll
                for (int m = 0; m < 16; ++m)
                    if (r0 + m < R) *reinterpret_cast<float2*>(plane + (r0 + m) * D) = y[m];
            };
            // (with two thread groups to a plane the lower nodes are written only after the
            // upper ones' windows, which hold them, are read)
#pragma unroll 1
            for (int b = 16; b >= 0; b -= 16) {
                compute(node0 + b);
                if (THREADS == 512 && node0 == 0 && b) __syncthreads();
                store(node0 + b);
            }
            if (THREADS == 512 && node0 != 0) __syncthreads();
        }
        // the nodes by depth, for the solve
        if (tid >= THREADS - RMAX) {
            const int r = tid - (THREADS - RMAX);
            int below = 0, rank = 0;                         // nodes of a depth up to r; r's place
            const int mine = r < R ? hd.depth[r] : 0;
            for (int x = 0; x < R; ++x) {
                const int d = hd.depth[x];
                below += d <= r;
                rank += d < mine || (d == mine && x < r);
            }
            hd.level[r + 1] = below;
            if (r < R) hd.order[rank] = (uint8_t)r;
        }
        __syncthreads();
        for (int r0 = warp; r0 < R; r0 += 4 * NW) {          // four rows a pass
            float4 q4[4], k4[4];
            float v[8];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int r = min(r0 + x * NW, R - 1);
                q4[x] = *reinterpret_cast<const float4*>(qq + r * D + 4 * lane);
                k4[x] = *reinterpret_cast<const float4*>(kk + r * D + 4 * lane);
                v[2 * x] = q4[x].x * q4[x].x + q4[x].y * q4[x].y + q4[x].z * q4[x].z + q4[x].w * q4[x].w;
                v[2 * x + 1] = k4[x].x * k4[x].x + k4[x].y * k4[x].y + k4[x].z * k4[x].z + k4[x].w * k4[x].w;
            }
            const float sum = warp_sum8(v, lane);
            const float rn = rsqrtf(sum + a.l2_eps);
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int r = r0 + x * NW;
                const float rq = __shfl_sync(0xffffffffu, rn, 8 * x), rk = __shfl_sync(0xffffffffu, rn, 8 * x + 4);
                if (r >= R) continue;
                *reinterpret_cast<float4*>(qq + r * D + 4 * lane) = make_float4(q4[x].x * rq, q4[x].y * rq, q4[x].z * rq, q4[x].w * rq);
                *reinterpret_cast<float4*>(kk + r * D + 4 * lane) = make_float4(k4[x].x * rk, k4[x].y * rk, k4[x].z * rk, k4[x].w * rk);
            }
        }
        __syncthreads();
        // ---- 3. A and P along the paths, and the rows e^Gam k^, e^Gam q^
        uint32_t lo_k[ROWS][2], lo_q[ROWS][2];
        const uint32_t panel = 2 * (uint32_t)Rp * 128;       // bytes of 64 keys of the 2 Rp rows
        auto row_off = [&](int row) {                        // 8 bytes: keys 4 lane .. 4 lane + 3 of a row
            return (4 * lane >= 64 ? panel : 0u) + (uint32_t)row * 128 + ((((4 * lane & 63) >> 3) ^ (row & 7)) << 4) + (lane & 1) * 8;
        };
#pragma unroll
        for (int x = 0; x < ROWS; ++x) {
            const int r = warp + x * NW;
            const int depth = r < R ? hd.depth[r] : 0;
            lo_k[x][0] = lo_k[x][1] = lo_q[x][0] = lo_q[x][1] = 0;
            if (depth == 0) continue;
            const float4 q4 = *reinterpret_cast<const float4*>(qq + r * D + 4 * lane);
            const float4 k4 = *reinterpret_cast<const float4*>(kk + r * D + 4 * lane);
            const float2 qa = make_float2(q4.x, q4.y), qb = make_float2(q4.z, q4.w), ka = make_float2(k4.x, k4.y), kb = make_float2(k4.z, k4.w);
            float2 wa = make_float2(1.f, 1.f), wb = wa;      // e^{Gam_r - Gam_s}
            for (int d0 = 0; d0 < depth; d0 += 4) {
                float v[8];
                const uint32_t p4 = *reinterpret_cast<const uint32_t*>(hd.path[r] + d0);
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    const int s = p4 >> (8 * d) & 255u;
                    const float4 ks = *reinterpret_cast<const float4*>(kk + s * D + 4 * lane);
                    const float4 es = *reinterpret_cast<const float4*>(eg + s * D + 4 * lane);
                    const float2 xa = __fmul2_rn(make_float2(ks.x, ks.y), wa), xb = __fmul2_rn(make_float2(ks.z, ks.w), wb);
                    const float2 sa = __ffma2_rn(ka, xa, __fmul2_rn(kb, xb)), sp = __ffma2_rn(qa, xa, __fmul2_rn(qb, xb));
                    v[2 * d] = sa.x + sa.y;
                    v[2 * d + 1] = sp.x + sp.y;
                    wa = __fmul2_rn(wa, make_float2(es.x, es.y));
                    wb = __fmul2_rn(wb, make_float2(es.z, es.w));
                }
                const float sum = warp_sum8(v, lane);
                const int d = d0 + (lane >> 3);              // values 2 d, 2 d + 1: A and P (0 past the root)
                if ((lane & 3) == 0) ap[(2 * r + ((lane >> 2) & 1)) * Rp + d] = sum;
            }
            const float2 sc = make_float2(ROW_SCALE, ROW_SCALE);
            wa = __fmul2_rn(wa, sc);
            wb = __fmul2_rn(wb, sc);
            uint32_t h0, h1;
            split2(ka.x * wa.x, ka.y * wa.y, h0, lo_k[x][0]);
            split2(kb.x * wb.x, kb.y * wb.y, h1, lo_k[x][1]);
            *reinterpret_cast<uint2*>(sb + map.hi + row_off(r)) = make_uint2(h0, h1);
            split2(qa.x * wa.x, qa.y * wa.y, h0, lo_q[x][0]);
            split2(qb.x * wb.x, qb.y * wb.y, h1, lo_q[x][1]);
            *reinterpret_cast<uint2*>(sb + map.hi + row_off(Rp + r)) = make_uint2(h0, h1);
        }
        __syncthreads();                                     // e^g is read: its place takes the low halves
#pragma unroll
        for (int x = 0; x < ROWS; ++x) {
            const int r = warp + x * NW;
            if (r >= R) continue;
            *reinterpret_cast<uint2*>(sb + map.lo + row_off(r)) = make_uint2(lo_k[x][0], lo_k[x][1]);
            *reinterpret_cast<uint2*>(sb + map.lo + row_off(Rp + r)) = make_uint2(lo_q[x][0], lo_q[x][1]);
        }
        ptx::fence_async_smem();
        ptx::tc_fence_before();
        __syncthreads();
        ptx::tc_fence_after();
        // ---- 4. D = S0^T [K e^Gam; Q e^Gam]^T
        if (tid == 0) {
            const uint32_t idesc = ptx::idesc_f16_f32(128, 2 * Rp);
#pragma unroll
            for (int term = 0; term < 3; ++term) {           // hi hi, hi lo, lo hi
                const uint64_t db = ptx::sdesc_sw128(base + (term == 1 ? map.lo : map.hi));
#pragma unroll
                for (int x = 0; x < D / 16; ++x)
                    ptx::mma_f16_ta(tmem + TM_D, tmem + (term == 2 ? TM_LO : TM_HI) + 8 * x, db + (x >> 2) * (panel / 16) + (x & 3) * 2, idesc,
                                    term > 0 || x > 0);
            }
            ptx::mma_commit(bar);
        }
        if (next_slot >= 0 && next_slot < a.n_slots) {       // the next item's state and rows into L2
            const uint32_t nx = item + gridDim.x;
            const int nn = (int)(nx / H), nh = (int)(nx % H);
            if (tid == 0) ptx::bulk_prefetch_l2(a.S + ((size_t)next_slot * H + nh) * D * D, D * D * 4);
            constexpr int LINES = D * sizeof(TI) / 128;      // 128-byte lines of a row
            for (int x = tid; x < 5 * R * LINES; x += THREADS) {
                const int pl = x / (R * LINES), r = x / LINES % R;
                const void* rows = pl == 0 ? a.q : pl == 1 ? a.k : pl == 2 ? a.v : pl == 3 ? a.z : a.gout;
                prefetch_l2(static_cast<const char*>(rows) + (((size_t)nn * R + r) * W + (size_t)nh * D) * sizeof(TI) + x % LINES * 128);
            }
        }
        if (!ptx::mbar_wait(bar, phase, WAIT_LIMIT_NS)) hd.bad = 1;
        phase ^= 1u;
        __syncthreads();
        if (hd.bad) break;
        ptx::tc_fence_after();
        // ---- 5. right sides of the solve, (q e^Gam)^T S0: lane = value, 8 columns at a time
        for (int col = 8 * part; col < 2 * Rp; col += 8 * KP) {
            float f[8];
            ptx::tmem_ld8(tlane + TM_D + col, f);
            if (col < Rp) {
                float v[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) v[x] = vv[min(col + x, R - 1) * D + j];
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (col + x < R) vv[(col + x) * D + j] = hd.beta[col + x] * fmaf(-unscale, f[x], v[x]);
            } else {
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (col - Rp + x < R) qq[(col - Rp + x) * D + j] = f[x] * unscale;
            }
        }
        ptx::tc_fence_before();
        __syncthreads();
        // u depth by depth, a warp per node (nodes of one depth do not see one another)
        for (int l = 2; l <= RMAX; ++l) {
            const int k0 = hd.level[l], k1 = l < RMAX ? hd.level[l + 1] : R;
            if (k0 >= R) break;
            for (int k = k0 + warp; k < k1; k += NW) {
                const int r = hd.order[k];
                const uint8_t* path = hd.path[r];
                const float* A = ap + 2 * r * Rp;
                float4* row = reinterpret_cast<float4*>(vv + r * D + 4 * lane);
                const float4 self = *row;
                const float beta = hd.beta[r];
                float2 ta = make_float2(0.f, 0.f), tb = ta;
#pragma unroll 2
                for (int d = 0; d < l; d += 4) {             // (d = 0, the node itself, is left out)
                    const uint32_t p4 = *reinterpret_cast<const uint32_t*>(path + d);
                    const float4 a4 = *reinterpret_cast<const float4*>(A + d);
                    const float av[4] = {d ? a4.x : 0.f, a4.y, a4.z, a4.w};
                    float4 u[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) u[m] = *reinterpret_cast<const float4*>(vv + (p4 >> (8 * m) & 255u) * D + 4 * lane);
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const float2 a2 = make_float2(av[m], av[m]);
                        ta = __ffma2_rn(a2, make_float2(u[m].x, u[m].y), ta);
                        tb = __ffma2_rn(a2, make_float2(u[m].z, u[m].w), tb);
                    }
                }
                *row = make_float4(fmaf(-beta, ta.x, self.x), fmaf(-beta, ta.y, self.y), fmaf(-beta, tb.x, self.z), fmaf(-beta, tb.y, self.w));
            }
            __syncthreads();
        }
        // gate logits of this warp's rows, in flight during the sums
        float4 gt[ROWS];
#pragma unroll
        for (int x = 0; x < ROWS; ++x)
            if (warp + x * NW < R) gt[x] = load4(static_cast<const TI*>(a.gout) + (row0 + warp + x * NW) * W + (size_t)h * D + 4 * lane);
        const float4 nw = __ldg(reinterpret_cast<const float4*>(a.norm_w) + lane);
        float4 o4[ROWS];
        float ss[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < ROWS; ++x) {
            const int r = warp + x * NW;
            const int depth = r < R ? hd.depth[r] : 0;
            if (depth == 0) continue;
            const float* Pr = ap + (2 * r + 1) * Rp;
            o4[x] = *reinterpret_cast<const float4*>(qq + r * D + 4 * lane);
#pragma unroll 2
            for (int d = 0; d < depth; d += 4) {
                const uint32_t p4 = *reinterpret_cast<const uint32_t*>(hd.path[r] + d);
                const float4 w4 = *reinterpret_cast<const float4*>(Pr + d);
                const float wd[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const float4 u4 = *reinterpret_cast<const float4*>(vv + (p4 >> (8 * m) & 255u) * D + 4 * lane);
                    o4[x].x = fmaf(wd[m], u4.x, o4[x].x); o4[x].y = fmaf(wd[m], u4.y, o4[x].y);
                    o4[x].z = fmaf(wd[m], u4.z, o4[x].z); o4[x].w = fmaf(wd[m], u4.w, o4[x].w);
                }
            }
            o4[x].x *= a.q_scale; o4[x].y *= a.q_scale; o4[x].z *= a.q_scale; o4[x].w *= a.q_scale;
            ss[x] = o4[x].x * o4[x].x + o4[x].y * o4[x].y + o4[x].z * o4[x].z + o4[x].w * o4[x].w;
        }
        const float rms = rsqrtf(warp_sum8(ss, lane) * (1.0f / D) + a.norm_eps);
#pragma unroll
        for (int x = 0; x < ROWS; ++x) {
            const int r = warp + x * NW;
            const float rs = __shfl_sync(0xffffffffu, rms, 4 * x);
            if (r >= R || hd.depth[r] == 0) continue;
            const float y0 = o4[x].x * rs * nw.x * sigmoid_fast(gt[x].x), y1 = o4[x].y * rs * nw.y * sigmoid_fast(gt[x].y);
            const float y2 = o4[x].z * rs * nw.z * sigmoid_fast(gt[x].z), y3 = o4[x].w * rs * nw.w * sigmoid_fast(gt[x].w);
            const size_t at = (row0 + r) * W + (size_t)h * D + 4 * lane;
            if constexpr (sizeof(TI) == 4) {
                *reinterpret_cast<float4*>(static_cast<TI*>(a.o) + at) = make_float4(y0, y1, y2, y3);
            } else {
                const __nv_bfloat162 b0 = __floats2bfloat162_rn(y0, y1), b1 = __floats2bfloat162_rn(y2, y3);
                *reinterpret_cast<uint2*>(static_cast<TI*>(a.o) + at) =
                    make_uint2(*reinterpret_cast<const uint32_t*>(&b0), *reinterpret_cast<const uint32_t*>(&b1));
            }
        }
        __syncthreads();                                     // the next item's rows replace this one's
    }
    if (hd.bad) {
        // the bounded wait gave up: no row of this item and of the CTA's later ones passes
        // for a result
        for (; item < items; item += gridDim.x) {
            const int n = (int)(item / H), h = (int)(item % H), slot = a.slots ? a.slots[n] : n;
            if (slot < 0 || slot >= a.n_slots) continue;
            for (int x = tid; x < R * D; x += THREADS)
                static_cast<TI*>(a.o)[((size_t)n * R + x / D) * W + (size_t)h * D + x % D] = from_f32<TI>(__int_as_float(0x7fc00000));
        }
        if (tid == 0) ptx::mbar_wait(bar, phase ^ 1u, WAIT_LIMIT_NS);   // the MMAs finish before their TMEM is freed
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TMEM_COLS);
    }
}

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

// SMs of the current device, looked up once per device.
int sm_count() {
    static std::atomic<int> cache[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 152;
    if (dev < 64 && (sms = cache[dev].load()) > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0) sms = 152;
    if (dev < 64) cache[dev].store(sms);
    return sms;
}

// ---- commit --------------------------------------------------------------------
// The decode step over the path's tokens, the state in registers between
// them (warp w: key rows 16w .. 16w+15, lane l: columns 4l .. 4l+3): one read
// and one write of the state, which bounds the kernel.  Tokens go through the
// conv, gate and norm in groups of CG.  256 sessions x 32 heads, paths of up to 6:
// 219 us, 78 % of the measured copy rate (a CTA an item 278 us, path and ring read
// when they are needed 226); the rest is two barriers a token and the walk from conv
// to state within an item, which two CTAs an SM overlap.
constexpr int CG = 8;

struct CommitSmem {
    alignas(16) float kc[CG][D], va[CG][D], e[CG][D], kh[CG][D], av[CG][D];
    alignas(16) float beta[CG];
    float red[NT / 32][D];
    float d[D];
    int path[KDA_TREE_MAX_NODES];
};

// Persistent CTAs: while an item computes, the next one's state goes to L2.
template <typename TI>
__global__ void __launch_bounds__(NT, 2) commit_kernel(CommitArgs a) {
    __shared__ CommitSmem sm;
    const int H = a.H, W = H * D;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int i = tid & (D - 1), half = tid >> 7;
    const uint32_t items = (uint32_t)a.n * H;   // (below 2^31: checked on the host)
    // slot, length and path (a node a thread) are read an item ahead: the addresses of the
    // state and of the rows wait for them
    int next_slot = a.slots ? a.slots[blockIdx.x / H] : blockIdx.x / H, next_len = a.path_len[blockIdx.x / H];
    auto path_at = [&](int nn) { return tid < next_len && next_len <= a.max_len ? a.path[(size_t)nn * a.max_len + tid] : 0; };
    int next_node = path_at(blockIdx.x / H);
#pragma unroll 1
    for (uint32_t item = blockIdx.x; item < items; item += gridDim.x) {
        const int n = (int)(item / H), h = (int)(item % H), c = h * D + i;
        const int slot = next_slot, len = next_len, node = next_node;
        if (item + gridDim.x < items) {
            const int nn = (int)((item + gridDim.x) / H), nh = (int)((item + gridDim.x) % H);
            next_slot = a.slots ? a.slots[nn] : nn;
            next_len = a.path_len[nn];
            next_node = path_at(nn);
            if (tid == 0 && next_slot >= 0 && next_slot < a.n_slots)
                ptx::bulk_prefetch_l2(a.S_in + ((size_t)next_slot * H + nh) * D * D, D * D * 4);
        }
        if (slot < 0 || slot >= a.n_slots) continue;
        if (len < 0 || len > a.max_len) continue;
        if (len == 0 && a.S_in == a.S_out && a.ring_in == a.ring_out) continue;
        const float* Sg_in = a.S_in + ((size_t)slot * H + h) * D * D;
        float4 Sr[16];
#pragma unroll
        for (int r = 0; r < 16; ++r)
            Sr[r] = __ldcs(reinterpret_cast<const float4*>(Sg_in + (size_t)(16 * warp + r) * D) + lane);
        // rows of the next item's path and ring into L2 (behind this state's loads, whose
        // latency covers the path's)
        if (item + gridDim.x < items && next_slot >= 0 && next_slot < a.n_slots) {
            constexpr int LINES = D * sizeof(TI) / 128;
            const int nn = (int)((item + gridDim.x) / H), nh = (int)((item + gridDim.x) % H);
            if (tid < next_len && next_len <= a.max_len) {
                if (next_node >= 0 && next_node < a.n_nodes) {
                    const size_t off = (((size_t)nn * a.n_nodes + next_node) * W + (size_t)nh * D) * sizeof(TI);
#pragma unroll
                    for (int x = 0; x < LINES; ++x) {
                        prefetch_l2(static_cast<const char*>(a.k) + off + 128 * x);
                        prefetch_l2(static_cast<const char*>(a.v) + off + 128 * x);
                        prefetch_l2(static_cast<const char*>(a.z) + off + 128 * x);
                    }
                }
            } else if (tid >= NT - 3 * RING * LINES) {
                const int x = tid - (NT - 3 * RING * LINES);
                prefetch_l2(static_cast<const char*>(a.ring_in) +
                            (((size_t)next_slot * 3 * RING + x / LINES) * W + (size_t)nh * D) * sizeof(TI) + x % LINES * 128);
            }
        }
        bool bad = false;
        if (tid < len) {
            sm.path[tid] = node;
            bad = node < 0 || node >= a.n_nodes;
        }
        if (__syncthreads_or(bad)) continue;

        const size_t row0 = (size_t)n * a.n_nodes;
        const TI* ring = static_cast<const TI*>(a.ring_in) + (size_t)slot * 3 * RING * W + c;
        const TI* plane[3] = {static_cast<const TI*>(a.q) + row0 * W + c, static_cast<const TI*>(a.k) + row0 * W + c,
                              static_cast<const TI*>(a.v) + row0 * W + c};
        // raw row of plane p at position t of the path (t < 0: the ring)
        auto raw = [&](int p, int t) -> TI {
            const TI* src = t >= 0 ? plane[p] + (size_t)sm.path[t] * W : ring + ((size_t)p * RING + (RING + t)) * W;
            return *src;
        };
        // the new ring: the last three raw rows of ring | path, of every plane
        TI tail[2][RING];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int s = 0; s < RING; ++s) tail[k][s] = half + 2 * k < 3 ? raw(half + 2 * k, len - RING + s) : TI(0.f);
        const int p = 1 + half;   // threads 0-127 own a channel of k, 128-255 of v and the gate
        const float4 w = __ldg(reinterpret_cast<const float4*>(a.conv_w + ((size_t)p * W + c) * CONV_K));
        const float eA = expf(a.A_log[h]), dtb = a.dt_bias[c];

#pragma unroll 1
        for (int g0 = 0; g0 < len; g0 += CG) {
            const int ng = min(CG, len - g0);
            // the group's raw rows and gate logits, all in flight at once
            TI xs[CG + RING], zs[CG];
#pragma unroll
            for (int t = 0; t < CG + RING; ++t) xs[t] = t < ng + RING ? raw(p, g0 + t - RING) : TI(0.f);
#pragma unroll
            for (int t = 0; t < CG; ++t)
                zs[t] = half && t < ng ? static_cast<const TI*>(a.z)[(row0 + sm.path[g0 + t]) * W + c] : TI(0.f);
            TI bl = TI(0.f);
            if (tid < ng) bl = static_cast<const TI*>(a.b)[(row0 + sm.path[g0 + tid]) * H + h];
#pragma unroll
            for (int t = 0; t < CG; ++t) {
                if (t >= ng) break;
                float y = w.x * to_f32(xs[t]);
                y = fmaf(w.y, to_f32(xs[t + 1]), y);
                y = fmaf(w.z, to_f32(xs[t + 2]), y);
                y = fmaf(w.w, to_f32(xs[t + 3]), y);
                y = silu_fast(y);
                if (half == 0) {
                    sm.kc[t][i] = y;
                } else {
                    sm.va[t][i] = y;
                    sm.e[t][i] = __expf(decay_gate(a.gate_kind, a.lb, eA, to_f32(zs[t]) + dtb));
                }
            }
            if (tid < ng) sm.beta[tid] = sigmoid_fast(to_f32(bl));
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
                float2 u01 = make_float2(0.f, 0.f), u23 = u01;
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const float4 a4 = *reinterpret_cast<const float4*>(&sm.av[t][16 * warp + r]);
                    const float ar[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const float2 aa = make_float2(ar[m], ar[m]);
                        u01 = __ffma2_rn(aa, make_float2(Sr[r + m].x, Sr[r + m].y), u01);
                        u23 = __ffma2_rn(aa, make_float2(Sr[r + m].z, Sr[r + m].w), u23);
                    }
                }
                *reinterpret_cast<float4*>(&sm.red[warp][4 * lane]) = make_float4(u01.x, u01.y, u23.x, u23.y);
                __syncthreads();
                if (tid < D) {
                    float uj = 0.f;
#pragma unroll
                    for (int k = 0; k < NT / 32; ++k) uj += sm.red[k][tid];
                    sm.d[tid] = sm.beta[t] * (sm.va[t][tid] - uj);
                }
                __syncthreads();
                const float4 d4 = *reinterpret_cast<const float4*>(&sm.d[4 * lane]);
                const float2 d01 = make_float2(d4.x, d4.y), d23 = make_float2(d4.z, d4.w);
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const float4 e4 = *reinterpret_cast<const float4*>(&sm.e[t][16 * warp + r]);
                    const float4 k4 = *reinterpret_cast<const float4*>(&sm.kh[t][16 * warp + r]);
                    const float er[4] = {e4.x, e4.y, e4.z, e4.w}, kr[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const float2 ee = make_float2(er[m], er[m]), kk = make_float2(kr[m], kr[m]);
                        const float2 s01 = __ffma2_rn(ee, make_float2(Sr[r + m].x, Sr[r + m].y), __fmul2_rn(kk, d01));
                        const float2 s23 = __ffma2_rn(ee, make_float2(Sr[r + m].z, Sr[r + m].w), __fmul2_rn(kk, d23));
                        Sr[r + m] = make_float4(s01.x, s01.y, s23.x, s23.y);
                    }
                }
            }
            __syncthreads();   // the group's vectors are rewritten
        }
        float* Sg_out = a.S_out + ((size_t)slot * H + h) * D * D;
#pragma unroll
        for (int r = 0; r < 16; ++r) __stcs(reinterpret_cast<float4*>(Sg_out + (size_t)(16 * warp + r) * D) + lane, Sr[r]);

        // (a thread has read all three of its channel, and every conv's read of the input ring is
        // behind the barriers above; without tokens there was none)
        TI* rout = static_cast<TI*>(a.ring_out) + (size_t)slot * 3 * RING * W + c;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int s = 0; s < RING; ++s)
                if (half + 2 * k < 3) rout[((size_t)(half + 2 * k) * RING + s) * W] = tail[k][s];
        __syncthreads();       // the next item's path replaces this one's
    }
}

}  // namespace

namespace {

template <typename TI, int THREADS>
cudaError_t tree(const TreeArgs& a, cudaStream_t s) {
    static std::atomic<uint64_t> done;
    const int Rp = (a.n_nodes + 7) / 8 * 8;
    // up to 32 nodes two CTAs share an SM
    constexpr int most = THREADS == 256 ? 32 : RMAX;
    cudaError_t e = opt_in((const void*)tree_kernel<TI, THREADS>, TreeMap(most).total, done);
    if (e != cudaSuccess) return e;
    const int64_t items = (int64_t)a.n * a.H, ctas = 512 / THREADS * (int64_t)sm_count();
    tree_kernel<TI, THREADS><<<(unsigned)std::min(items, ctas), THREADS, TreeMap(Rp).total, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree(const TreeArgs& a, int io_bf16, cudaStream_t s) {
    if (a.n_nodes <= 32) return io_bf16 ? tree<__nv_bfloat16, 256>(a, s) : tree<float, 256>(a, s);
    return io_bf16 ? tree<__nv_bfloat16, 512>(a, s) : tree<float, 512>(a, s);
}

cudaError_t launch_commit(const CommitArgs& a, int io_bf16, cudaStream_t s) {
    const unsigned blocks = (unsigned)std::min<int64_t>((int64_t)a.n * a.H, 2 * (int64_t)sm_count());
    if (io_bf16) commit_kernel<__nv_bfloat16><<<blocks, NT, 0, s>>>(a);
    else commit_kernel<float><<<blocks, NT, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kda
