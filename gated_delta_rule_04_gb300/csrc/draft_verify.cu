// Verification of a round's drafted tokens: the accepted path through each
// session's nodes and the token that follows it.
//
// A cluster of 1 to 16 CTAs per session.  Every warp of it walks alike: lane j
// holds nodes j and 32 + j with the target's and the drafter's probability of their
// token, so that the tests of one parent are a few ballots.  What bounds the call
// is the row behind the last accepted node: V values of p, and of q where a child was
// refused, read once; each warp of the cluster sums a piece of it.  A row is
// also summed where a refused child leaves siblings to be tested.  The token is found
// by halves: CTA, warp, then the warp's piece once more from L2.
//
// Sums are in pairs of floats (Knuth's two-sum, Dekker's products: 48 bits) within
// a thread and in 64 bits between threads: next to a random border, in a sum
// over 10^5 entries, a 32-bit sum would take another token in one session of 30, and
// this GPU adds 2 doubles a cycle and SM, where the rows arrive at 3 pairs.
#include <atomic>

#include "draft_verify.cuh"

namespace kda {
namespace {

constexpr int NT = 256, WARPS = NT / 32, MAX_CTAS = 16, SMS = 152;
constexpr uint32_t FULL = 0xffffffffu;

__device__ __forceinline__ float clean(float v) { return v > 0.f && v <= 3.402823466e38f ? v : 0.f; }

// A sum as two floats; adding is exact but for the rounding of `lo`.
struct Sum {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
        hi = s;
    }
    __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

// The coefficient c of W = max(p - c q, 0).
struct Coef {
    double c = 0.0;
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void set(double v) {
        c = v;
        hi = (float)v;
        lo = (float)(v - (double)hi);
    }
};
enum Kind { P_ONLY, ONE, ANY };      // c = 0, c = 1 (the first refusal), any

// Adds W of one token: p - c q as a pair of floats, where above zero.
template <int KIND> __device__ __forceinline__ void add_w(Sum& s, const Coef& k, float p, float q) {
    p = clean(p);
    if (KIND == P_ONLY) {
        s.add(p);
        return;
    }
    q = clean(q);
    float m = q, e = 0.f;                             // c q = m + e
    if (KIND == ANY) {
        m = __fmul_rn(k.hi, q);
        e = __fmaf_rn(k.lo, q, __fmaf_rn(k.hi, q, -m));
    }
    const float d = __fsub_rn(p, m), b = __fsub_rn(d, p);
    const float r = __fsub_rn(__fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(m, b)), e);
    if (__fadd_rn(d, r) > 0.f) {
        s.add(d);
        s.lo = __fadd_rn(s.lo, r);
    }
}

template <typename TP> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ float get(const uint4& u, int i) { return __uint_as_float((&u.x)[i]); }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ float get(const uint4& u, int i) {
        const uint32_t w = (&u.x)[i / 2];
        return __uint_as_float(i % 2 ? w & 0xffff0000u : w << 16);
    }
};

// A row (pair) cut into pieces, one for each warp of the cluster: piece i is [lo(i), hi(i)); all
// but the first begin on 16 bytes where p and q allow it.
template <typename TP> struct Row {
    const TP *p, *q;
    int V, size, head;               // head: elements before the first 16-byte boundary, -1: p and q lie differently
    __device__ __forceinline__ Row(const TP* p_, const TP* q_, int V_, int pieces) : p(p_), q(q_), V(V_) {
        const uint32_t at = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15;
        head = q && ((uint32_t)reinterpret_cast<uintptr_t>(q) & 15) != at ? -1 : (int)((16 - at) % 16 / sizeof(TP));
        const int unit = 32 * Vec<TP>::N, each = (V + pieces - 1) / pieces;
        size = (each + unit - 1) / unit * unit;
    }
    __device__ __forceinline__ int begin(int i) const { return i == 0 ? 0 : (int)min((int64_t)V, (int64_t)i * size + max(head, 0)); }
    __device__ __forceinline__ int end(int i, int pieces) const { return i + 1 == pieces ? V : begin(i + 1); }
};

// The lane's share of the sum of W over [a, b): 16 bytes at a time from the first boundary on.
template <int KIND, typename TP>
__device__ __forceinline__ void sum_piece(Sum& s, const Coef& k, const Row<TP>& r, int a, int b) {
    constexpr int N = Vec<TP>::N, U = 4;
    const int lane = threadIdx.x & 31;
    if (r.head >= 0) {
        const int va = a == 0 ? min(r.head, b) : a, nv = (b - va) / N, vb = va + nv * N;
        if (lane < va - a) add_w<KIND>(s, k, to_f32(r.p[a + lane]), KIND ? to_f32(r.q[a + lane]) : 0.f);
        if (lane < b - vb) add_w<KIND>(s, k, to_f32(r.p[vb + lane]), KIND ? to_f32(r.q[vb + lane]) : 0.f);
        const uint4* pv = reinterpret_cast<const uint4*>(r.p + va);
        const uint4* qv = KIND ? reinterpret_cast<const uint4*>(r.q + va) : nullptr;
        for (int i = lane; i < nv; i += 32 * U) {
            uint4 x[U], y[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = i + 32 * u < nv;
                x[u] = in ? __ldcs(pv + i + 32 * u) : make_uint4(0, 0, 0, 0);
                if (KIND) y[u] = in ? __ldcs(qv + i + 32 * u) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < N; ++j) add_w<KIND>(s, k, Vec<TP>::get(x[u], j), KIND ? Vec<TP>::get(y[u], j) : 0.f);
        }
    } else {
        constexpr int E = 2 * U;
        for (int i = a + lane; i < b; i += 32 * E) {
            float x[E], y[E];
#pragma unroll
            for (int u = 0; u < E; ++u) {
                const bool in = i + 32 * u < b;
                x[u] = in ? to_f32(r.p[i + 32 * u]) : 0.f;
                y[u] = KIND && in ? to_f32(r.q[i + 32 * u]) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < E; ++u) add_w<KIND>(s, k, x[u], y[u]);
        }
    }
}

__device__ __forceinline__ double shfl_up(double v, int d) { return __shfl_up_sync(FULL, v, d); }
// Inclusive sums over the lanes.
__device__ __forceinline__ double scan(double v, int lanes) {
    const int lane = threadIdx.x & 31;
    for (int d = 1; d < lanes; d <<= 1) {
        const double u = shfl_up(v, d);
        if (lane >= d) v += u;
    }
    return v;
}
// The first lane whose inclusive sum is above the goal, or (rounding) the last with a share; -1: none has one.
__device__ __forceinline__ int pick(double incl, double share, double goal) {
    const uint32_t over = __ballot_sync(FULL, share > 0.0 && incl > goal), any = __ballot_sync(FULL, share > 0.0);
    return over ? __ffs(over) - 1 : any ? 31 - __clz(any) : -1;
}

template <typename TP>
__global__ void __launch_bounds__(NT) verify_kernel(const __grid_constant__ VerifyArgs g, int ctas) {
    __shared__ double wsum[WARPS], slots[2][MAX_CTAS], twarp[WARPS];
    __shared__ int best, last;
    const int s = blockIdx.x / ctas, rank = blockIdx.x % ctas, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int R = g.R, V = g.V, pieces = ctas * WARPS;
    auto p_row = [&](int r) -> const TP* {
        if (r >= 0) return static_cast<const TP*>(g.p) + s * g.p_ss + r * g.p_rs;
        return g.p_last ? static_cast<const TP*>(g.p_last) + s * g.pl_s : nullptr;
    };
    auto q_row = [&](int r) -> const TP* {
        if (!g.q) return nullptr;
        if (r >= 0) return static_cast<const TP*>(g.q) + s * g.q_ss + r * g.q_rs;
        return g.q_last ? static_cast<const TP*>(g.q_last) + s * g.ql_s : nullptr;
    };
    const bool hot = g.q == nullptr;                  // chosen tokens: q is one at the child's own
    // the lane's two nodes; an entry that leaves one out makes its parent -2
    int tok[2], par[2];
    float u[2], pt[2], qt[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = lane + 32 * h;
        tok[h] = -1;
        par[h] = -2;
        u[h] = pt[h] = qt[h] = 0.f;
        if (r < R) {
            tok[h] = g.tokens[(size_t)s * R + r];
            par[h] = g.parents[(size_t)s * R + r];
            u[h] = g.u[(size_t)s * R + r];
            if (par[h] < -1 || par[h] >= r || tok[h] < 0 || tok[h] >= V) par[h] = -2;
            if (par[h] >= -1 && p_row(par[h])) {
                pt[h] = clean(to_f32(p_row(par[h])[tok[h]]));
                qt[h] = hot ? 1.f : clean(to_f32(q_row(par[h])[tok[h]]));
            }
        }
    }
    auto nodes = [&](bool a, bool b) { return (uint64_t)__ballot_sync(FULL, a) | (uint64_t)__ballot_sync(FULL, b) << 32; };
    auto of = [&](auto (&v)[2], int r) { return __shfl_sync(FULL, r < 32 ? v[0] : v[1], r & 31); };
    // accepted as the first child that its parent tests (c = 0, T = 1)
    auto first_test = [&](int h) { return pt[h] > 0.f && (double)u[h] * (double)qt[h] < (double)pt[h]; };
    const uint64_t at_once = nodes(first_test(0), first_test(1));

    // W of the current node: all CTAs and warps alike
    int cur = -1, len = 0, turn = 0;
    Coef c;
    double T = 1.0;
    uint64_t refused = 0;                             // (chosen tokens) those that left something out of W
    double mine = 0.0, incl = 0.0;                    // a pass's sum of CTA `lane`, and the inclusive ones
    auto pass = [&]() -> double {                     // sums W over the row; leaves wsum, mine and incl
        const Row<TP> row(p_row(cur), c.c > 0.0 ? q_row(cur) : nullptr, V, pieces);
        const int piece = rank * WARPS + warp, a = row.begin(piece), b = row.end(piece, pieces);
        Sum sum;
        if (c.c == 0.0) sum_piece<P_ONLY>(sum, c, row, a, b);
        else if (c.c == 1.0) sum_piece<ONE>(sum, c, row, a, b);
        else sum_piece<ANY>(sum, c, row, a, b);
#pragma unroll
        for (int h = 0; h < 2; ++h)                   // (p is what was added: the sum stays exact)
            if ((refused >> (lane + 32 * h) & 1) && tok[h] >= a && tok[h] < b) sum.add(-pt[h]);
        double v = sum.value();
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(FULL, v, d);
        if (lane == 0) wsum[warp] = v;
        __syncthreads();
        const int buf = turn++ & 1;
        if (warp == 0) {
            v = scan(lane < WARPS ? wsum[lane] : 0.0, WARPS);
            v = __shfl_sync(FULL, v, WARPS - 1);
            if (lane < ctas) {
                uint32_t at = (uint32_t)__cvta_generic_to_shared(&slots[buf][rank]);
                asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(at) : "r"(lane));
                asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(at), "d"(v) : "memory");
            }
        }
        asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
        mine = lane < ctas ? slots[buf][lane] : 0.0;
        incl = scan(mine, MAX_CTAS);
        return __shfl_sync(FULL, incl, MAX_CTAS - 1);
    };

    while (len < g.max_len) {
        uint64_t left = nodes(par[0] == cur, par[1] == cur);
        int to = -1;
        bool first = true;
        while (left) {
            const int r = __ffsll((long long)left) - 1;
            left &= left - 1;
            if (p_row(cur) == nullptr) {              // the token that was chosen already
                to = r;
                break;
            }
            double w = (double)of(pt, r);
            if (first) {
                if (at_once >> r & 1) to = r;
            } else {
                const double q = (double)of(qt, r);
                if (hot) {
                    const int x = of(tok, r);
                    if (refused & nodes(tok[0] == x, tok[1] == x)) w = 0.0;
                } else {
                    w = fmax(w - c.c * q, 0.0);
                }
                if (w > 0.0 && (double)of(u, r) * T * q < w) to = r;
            }
            if (to >= 0) break;
            first = false;
            if (hot) {
                T -= w;
                if (w > 0.0) refused |= (uint64_t)1 << r;
            } else {
                c.set(c.c + T);
                if (left) T = pass();
            }
        }
        if (to < 0) break;
        if (rank == 0 && tid == 0) g.path[(size_t)s * g.max_len + len] = to;
        ++len;
        cur = to;
        c.set(0.0);
        T = 1.0;
        refused = 0;
    }
    if (rank == 0) {
        for (int j = len + tid; j < g.max_len; j += NT) g.path[(size_t)s * g.max_len + j] = -1;
        if (tid == 0) g.path_len[s] = len;
    }
    if (p_row(cur) == nullptr) {                      // not even the chosen token is there
        if (rank == 0 && tid == 0) g.next[s] = -1;
        return;
    }
    double total = pass();
    if (!(total > 0.0) && (c.c > 0.0 || refused)) {   // nothing is left: p itself
        c.set(0.0);
        refused = 0;
        total = pass();
    }
    const double goal = (double)g.u_next[s] * total;
    const int owner = pick(incl, mine, goal);
    if (owner < 0) {
        if (rank == 0 && tid == 0) g.next[s] = -1;
        return;
    }
    if (owner != rank) return;
    // the warp's piece that holds the token, once more: a few neighbouring entries a thread
    double base = __shfl_sync(FULL, incl - mine, owner);
    {
        const double w = lane < WARPS ? wsum[lane] : 0.0, in = scan(w, WARPS);
        const int at = pick(base + in, w, goal);
        base += __shfl_sync(FULL, in - w, at);
        const Row<TP> row(p_row(cur), c.c > 0.0 ? q_row(cur) : nullptr, V, pieces);
        const int a = row.begin(rank * WARPS + at), b = row.end(rank * WARPS + at, pieces), per = (b - a + NT - 1) / NT;
        const int y0 = (int)min((int64_t)b, a + (int64_t)tid * per), y1 = min(b, y0 + per);
        auto entry = [&](int y) -> double {           // W(y)
            for (uint64_t m = refused; m; m &= m - 1)
                if (g.tokens[(size_t)s * R + __ffsll((long long)m) - 1] == y) return 0.0;
            Sum e;
            const float p = to_f32(row.p[y]);
            if (c.c == 0.0) add_w<P_ONLY>(e, c, p, 0.f);
            else add_w<ANY>(e, c, p, to_f32(row.q[y]));
            return e.value();
        };
        double v = 0.0;
        for (int y = y0; y < y1; ++y) v += entry(y);
        double in2 = scan(v, 32);
        if (lane == 31) twarp[warp] = in2;
        if (tid == 0) {
            best = NT;
            last = -1;
        }
        __syncthreads();
        for (int k = 0; k < warp; ++k) base += twarp[k];
        if (v > 0.0) {
            if (base + in2 > goal) atomicMin(&best, tid);
            atomicMax(&last, tid);
        }
        __syncthreads();
        if (tid == (best < NT ? best : last)) {
            double run = base + (in2 - v);
            int next = -1;
            for (int y = y0; y < y1; ++y) {
                const double x = entry(y);
                if (!(x > 0.0)) continue;
                next = y;
                run += x;
                if (run > goal) break;
            }
            g.next[s] = next;
        }
        if (tid == 0 && best == NT && last < 0) g.next[s] = -1;   // (not with a positive sum)
    }
}

template <typename TP> cudaError_t verify(const VerifyArgs& a, int ctas, cudaStream_t s) {
    auto k = verify_kernel<TP>;
    if (ctas > 8) {                                   // 16 CTAs are beyond the portable size (set once per device)
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
    cfg.gridDim = dim3((unsigned)((int64_t)a.n * ctas));
    cfg.blockDim = dim3(NT);
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a, ctas);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int io_bf16, cudaStream_t s) {
    // CTAs a session: enough for four an SM, while each warp's piece is at least 512 bytes
    int ctas = 1;
    const int64_t bytes = (int64_t)a.V * (io_bf16 ? 2 : 4);
    while (ctas < MAX_CTAS && (int64_t)a.n * ctas < 4 * SMS && bytes >= (int64_t)ctas * 2 * WARPS * 512) ctas *= 2;
    return io_bf16 ? verify<__nv_bfloat16>(a, ctas, s) : verify<float>(a, ctas, s);
}

}  // namespace kda

using namespace kda;

extern "C" kda_status kda_draft_verify(int32_t dtype, int32_t n_sessions, int32_t n_nodes, int32_t vocab, const void* p,
                                       int64_t p_session_stride, int64_t p_row_stride, const void* p_last,
                                       int64_t p_last_stride, const void* q, int64_t q_session_stride,
                                       int64_t q_row_stride, const void* q_last, int64_t q_last_stride,
                                       const int32_t* tokens, const int32_t* parents, const float* u,
                                       const float* u_next, int32_t max_len, int32_t* path, int32_t* path_len,
                                       int32_t* next_token, void* stream) {
    if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARG;
    if (n_sessions < 0 || n_nodes < 1 || n_nodes > KDA_TREE_MAX_NODES || vocab < 1 || max_len < 1 ||
        max_len > KDA_TREE_MAX_NODES)
        return KDA_ERR_INVALID_ARG;
    if (vocab > (1 << 30)) return KDA_ERR_UNSUPPORTED;
    if (n_sessions == 0) return KDA_OK;
    const uintptr_t es = dtype == KDA_DTYPE_BF16 ? 2 : 4;
    auto bad = [](const void* x, uintptr_t align) { return (reinterpret_cast<uintptr_t>(x) & (align - 1)) != 0; };
    if (!p || !tokens || !parents || !u || !u_next || !path || !path_len || !next_token) return KDA_ERR_INVALID_ARG;
    if (bad(p, es) || bad(p_last, es) || bad(q, es) || bad(q_last, es) || bad(tokens, 4) || bad(parents, 4) || bad(u, 4) ||
        bad(u_next, 4) || bad(path, 4) || bad(path_len, 4) || bad(next_token, 4))
        return KDA_ERR_INVALID_ARG;
    if ((q_last != nullptr) != (p_last != nullptr && q != nullptr)) return KDA_ERR_INVALID_ARG;
    // rows may share memory (one distribution for all), but not run backwards
    if (p_session_stride < 0 || p_row_stride < 0 || p_last_stride < 0 || q_session_stride < 0 || q_row_stride < 0 ||
        q_last_stride < 0)
        return KDA_ERR_INVALID_ARG;
    VerifyArgs a{p, p_last, q, q_last, p_session_stride, p_row_stride, p_last_stride, q_session_stride, q_row_stride,
                 q_last_stride, tokens, parents, u, u_next, path, path_len, next_token, n_sessions, n_nodes, vocab, max_len};
    return launch_verify(a, dtype == KDA_DTYPE_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
