// Verification of a round's drafted tokens: the accepted path through each
// session's nodes and the token that follows it.
//
// A cluster of 1 to 16 CTAs per session.  The first warp of each walks alike: lane
// j holds nodes j and 32 + j with the target's and the drafter's probability of their
// token, so that the tests of one parent are a few ballots.  What bounds the call
// is the row behind the last accepted node: V values of p, and of q where a child was
// refused, read once; each warp of the cluster sums a piece of it.  A row is
// also summed where a refused child leaves siblings to be tested; then the sums' way
// through the cluster (a word from each CTA to each, counted by a barrier) is
// what counts.  The token is found level by level: CTA, warp, part of its piece, then the
// part's entries once more from L2.
//
// Sums, borders and tests are pairs of floats (two-sums and products of Knuth and Dekker): next to a
// random border, in a sum over 10^5 entries, a 32-bit sum would take another token in one
// session of 30, and this GPU adds 2 doubles a cycle and SM where the rows arrive at 3 pairs; each
// operation on doubles also holds a warp up for 64 cycles and more.  A lane adds n entries to a pair of which the
// second float's last place is 2^-48 of the sum: at most n^1/2 2^-49 or so off (softmax rows on the CPU: 2^-45 over
// 4096), all lanes' sum less: 2^-48 of a row of 2^20 entries in one CTA.
//
// 256 sessions x 5 nodes x 131072, fp32: 48 us in a graph, 51 to 54 a call (4.6 TB/s of a copy's 6.8; memory
// 57 %, issue slots 40 %): the pass over the rows takes about two thirds, the tests before it and the exchange and
// search behind it the rest, in all sessions at about the same time.  1 x 6 nodes 9.0 us, a chain of latencies.
#include <limits.h>

#include <atomic>

#include "draft_verify.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace {

constexpr int MAX_CTAS = 16, SMS = 152;
constexpr int DEPTH = 3;             // steps of copies on their way, of 32 bytes of p and of q a thread
constexpr uint32_t FULL = 0xffffffffu;
constexpr int PARTS = 8;             // of a piece, whose sums are kept for the search
constexpr int MARKED = 2048;         // a piece longer than this keeps them
constexpr int STAGED = 22;           // entries a thread that the token is found in without another read
constexpr int LOOSE = 8;             // entries a lane and step where rows lie off 16 bytes
constexpr uint64_t WAIT_NS = 2000000000ull;   // the limit of a wait for the other CTAs' sums
constexpr uint64_t DRAIN_NS = 100000;         // a store to another CTA's shared memory has arrived long before

__device__ __forceinline__ float clean(float v) { return v > 0.f && v <= 3.402823466e38f ? v : 0.f; }

__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.f, -1.f), a); }

// A sum as two floats.
struct Sum {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x, float rest = 0.f) {
        const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
        const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b));
        lo = __fadd_rn(__fadd_rn(lo, rest), e);       // (the same whichever of two sums is added to the other)
        hi = s;
    }
    __device__ __forceinline__ void add(const Sum& o) { add(o.hi, o.lo); }
    __device__ __forceinline__ void sub(const Sum& o) { add(-o.hi, -o.lo); }
    // hi to be the sum to its own digits: behind a difference lo can be as large.
    __device__ __forceinline__ void settle() {
        const float s = __fadd_rn(hi, lo), b = __fsub_rn(s, hi);
        lo = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(lo, b));
        hi = s;
    }
    __device__ __forceinline__ bool positive() const { return hi + lo > 0.f; }
};
__device__ __forceinline__ Sum sum_of(float hi, float lo) {
    Sum s;
    s.hi = hi;
    s.lo = lo;
    return s;
}
__device__ __forceinline__ Sum sum_of(float2 x) { return sum_of(x.x, x.y); }
// Whether a > b: where the large parts are near, their difference is exact.
__device__ __forceinline__ bool above(const Sum& a, const Sum& b) { return (a.hi - b.hi) + (a.lo - b.lo) > 0.f; }
__device__ __forceinline__ Sum times(float u, const Sum& t) {
    const float m = __fmul_rn(u, t.hi);
    return sum_of(m, __fmaf_rn(u, t.lo, __fmaf_rn(u, t.hi, -m)));
}
__device__ __forceinline__ Sum times(const Sum& u, const Sum& t) {
    Sum r = times(u.hi, t);
    r.lo = __fmaf_rn(u.lo, t.hi, r.lo);
    return r;
}
__device__ __forceinline__ Sum shfl(const Sum& s, int lane) { return sum_of(__shfl_sync(FULL, s.hi, lane), __shfl_sync(FULL, s.lo, lane)); }
__device__ __forceinline__ Sum shfl_xor(Sum s, int d) {
    Sum o;
    o.hi = __shfl_xor_sync(FULL, s.hi, d);
    o.lo = __shfl_xor_sync(FULL, s.lo, d);
    return o;
}
// Over all lanes, the same bits in each.
__device__ __forceinline__ Sum warp_sum(Sum s) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const Sum o = shfl_xor(s, d);
        s.add(o.hi, o.lo);
    }
    s.settle();
    return s;
}

// The coefficient c of W = max(p - c q, 0).
struct Coef {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(const Sum& t) {
        Sum v;
        v.hi = hi;
        v.lo = lo;
        v.add(t);
        v.settle();
        hi = v.hi;
        lo = v.lo;
    }
    __device__ __forceinline__ int kind() const { return hi == 0.f ? 0 : hi == 1.f && lo == 0.f ? 1 : 2; }
};
enum Kind { P_ONLY, ONE, ANY };      // c = 0, c = 1 (the first refusal), any

// W of one token as two floats, p and q finite and not negative: p - c q with c q = m + e, m <= p, so that p - m is
// d + r exactly (Dekker).  Where the product is above p, by however little, e takes r below -d: W is then zero.
template <int KIND> __device__ __forceinline__ void w_of(const Coef& k, float p, float q, float& d, float& r) {
    const float m = fminf(KIND == ANY ? __fmul_rn(k.hi, q) : q, p);
    d = __fsub_rn(p, m);
    r = __fsub_rn(__fsub_rn(p, d), m);
    if (KIND == ANY) r = fmaxf(__fsub_rn(r, __fmaf_rn(k.lo, q, __fmaf_rn(k.hi, q, -m))), -d);
}

// A lane's sums of W, of two tokens at a time side by side, for values that are neither negative nor infinite nor
// NaN: `most` is the largest of their words, and if it is none of a finite number's the piece is summed again
// with cleaned values.
struct Pairs {
    float2 hi = make_float2(0.f, 0.f), lo = hi;
    uint32_t most = 0;
    template <int KIND> __device__ __forceinline__ void add(const Coef& k, float2 p, float2 q) {
        if (KIND == P_ONLY) {
            most = __vimax3_u32(most, __float_as_uint(p.x), __float_as_uint(p.y));
        } else {
            most = __vimax3_u32(most, __float_as_uint(p.x), __float_as_uint(q.x));
            most = __vimax3_u32(most, __float_as_uint(p.y), __float_as_uint(q.y));
        }
        float2 d = p;
        if (KIND == ONE) {
            const float2 m = make_float2(fminf(q.x, p.x), fminf(q.y, p.y));
            d = sub2(p, m);
            lo = add2(lo, sub2(sub2(p, d), m));
        } else if (KIND == ANY) {
            const float2 h = make_float2(k.hi, k.hi), v = __fmul2_rn(h, q);   // (as w_of)
            const float2 m = make_float2(fminf(v.x, p.x), fminf(v.y, p.y));
            const float2 e = __ffma2_rn(make_float2(k.lo, k.lo), q, __ffma2_rn(h, q, __fmul2_rn(m, make_float2(-1.f, -1.f))));
            d = sub2(p, m);
            const float2 r = sub2(sub2(sub2(p, d), m), e);
            lo = add2(lo, make_float2(fmaxf(r.x, -d.x), fmaxf(r.y, -d.y)));
        }
        const float2 s = add2(hi, d), b = sub2(s, hi);
        lo = add2(lo, add2(sub2(hi, sub2(s, b)), sub2(d, b)));
        hi = s;
    }
    // hi to be the sums to their own digits.  Between, lo is added up in plain fp32: were it never taken in, it
    // would outgrow its digits over thousands of entries a lane.
    __device__ __forceinline__ void settle() {
        const float2 s = add2(hi, lo), b = sub2(s, hi);
        lo = add2(sub2(hi, sub2(s, b)), sub2(lo, b));
        hi = s;
    }
    __device__ __forceinline__ bool good() const { return most <= 0x7f7fffffu; }
};

template <typename TP> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ float2 pair(const uint4& u, int i) {
        return make_float2(__uint_as_float((&u.x)[2 * i]), __uint_as_float((&u.x)[2 * i + 1]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ float2 pair(const uint4& u, int i) {
        const uint32_t w = (&u.x)[i];
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
};

// A row (pair) cut into pieces, one for each warp of the cluster: piece i is [begin(i), end(i)); all
// but the first begin on 16 bytes where p and q allow it.
template <typename TP> struct Row {
    const TP *p, *q;
    int V, size, head;               // head: elements before the first 16-byte boundary, -1: p and q lie differently
    __device__ __forceinline__ Row(const TP* p_, const TP* q_, int V_, int pieces) : p(p_), q(q_), V(V_) {
        const uint32_t at = (uint32_t)reinterpret_cast<uintptr_t>(p) & 15;
        head = q && ((uint32_t)reinterpret_cast<uintptr_t>(q) & 15) != at ? -1 : (int)((16 - at) % 16 / sizeof(TP));
        const int unit = 64 * Vec<TP>::N, each = (V + pieces - 1) / pieces;
        size = (each + unit - 1) / unit * unit;
    }
    __device__ __forceinline__ int begin(int i) const { return i == 0 ? 0 : (int)min((int64_t)V, (int64_t)i * size + max(head, 0)); }
    __device__ __forceinline__ int end(int i, int pieces) const { return i + 1 == pieces ? V : begin(i + 1); }
};

// A piece [a, b) in at most 8 parts of whole steps of the loop that sums it: part i ends at end(i).
struct Parts {
    int va, b, size;                 // the loop's first element, behind the piece's head
    template <typename TP> __device__ __forceinline__ Parts(const Row<TP>& r, int a, int b_) : b(b_) {
        constexpr int N = Vec<TP>::N;
        va = r.head < 0 ? a : min(b, a + ((r.head - a) & (N - 1)));
        const int unit = r.head < 0 ? 32 * LOOSE : 64 * N;
        size = ((b - va + unit - 1) / unit + PARTS - 1) / PARTS * unit;
    }
    __device__ __forceinline__ int end(int i) const { return i + 1 == PARTS ? b : (int)min((int64_t)b, va + (int64_t)(i + 1) * size); }
    __device__ __forceinline__ int begin(int i, int a) const { return i == 0 ? a : end(i - 1); }
};

// The lane's share of the sum of W over [a, b): 16 bytes at a time from the first boundary on.  With `marks`,
// the warp's sums up to the end of each part are left there.  `there`: the pass before was over the same rows,
// and a piece that fits the ring is still in it.  (Chosen tokens) the n_gone tokens `gone` count as zero: next
// to what they hold the rest may be less than a sum's rounding, so they are never in it.
template <int KIND, int NT, typename TP>
__device__ __forceinline__ Sum sum_piece(const Coef& k, const Row<TP>& r, int a, int b, uint4* ring, float2* marks,
                                         bool there, const int* gone, int n_gone) {
    constexpr int N = Vec<TP>::N;
    const int lane = threadIdx.x & 31;
    const Parts parts(r, a, b);
    const int va = parts.va;
    uint64_t inside = 0;                              // of them, those in this piece: few warps have any
    if (KIND == P_ONLY && n_gone > 0) {
        auto in = [&](int j) { return j < n_gone && gone[j] >= a && gone[j] < b; };
        inside = (uint64_t)__ballot_sync(FULL, in(lane)) | (uint64_t)__ballot_sync(FULL, in(lane + 32)) << 32;
    }
    auto is_gone = [&](int y) {
        bool is = false;
        for (uint64_t w = inside; w; w &= w - 1) is |= gone[__ffsll((long long)w) - 1] == y;
        return is;
    };
    Pairs s;
    auto so_far = [&]() {
        Sum t;
        t.add(s.hi.x, s.lo.x);
        t.add(s.hi.y, s.lo.y);
        return t;
    };
    auto mark = [&](int i, Sum t) {
        t = warp_sum(t);
        if (lane == 0) marks[i] = make_float2(t.hi, t.lo);
    };
    int part = 0;
    if (r.head >= 0) {
        const int nv = (b - va) / N, vb = va + nv * N;
        // the head's and the tail's entries, a lane each (at most N - 1 of either)
        const int edge = lane < va - a ? a + lane : lane >= 16 && lane - 16 < b - vb ? vb + lane - 16 : -1;
        const float pe = edge >= 0 && !is_gone(edge) ? to_f32(r.p[edge]) : 0.f, qe = KIND && edge >= 0 ? to_f32(r.q[edge]) : 0.f;
        // Steps of two pieces of 16 bytes a lane, copied DEPTH ahead of the sum; a lane reads what it copied, so
        // nothing waits for another.  Behind the last piece a step is filled up with zeros.
        const int steps = (nv + 63) / 64;
        const uint32_t slot = ptx::smem_u32(ring + threadIdx.x);   // [DEPTH][2][p, q][NT]
        const uint4 *pn = reinterpret_cast<const uint4*>(r.p + va) + lane, *qn = KIND ? reinterpret_cast<const uint4*>(r.q + va) + lane : nullptr;
        int ahead = lane;                             // the lane's next piece
        auto copy = [&](int to, const uint4* from, bool in) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot + to * NT * 16), "l"(from), "r"(in ? 16 : 0) : "memory");
        };
        auto issue = [&](int st, bool step) {
            if (step) {
                const bool in0 = ahead < nv, in1 = ahead + 32 < nv;
                copy(st * 4, in0 ? pn : reinterpret_cast<const uint4*>(r.p + va), in0);
                copy(st * 4 + 2, in1 ? pn + 32 : reinterpret_cast<const uint4*>(r.p + va), in1);
                if (KIND) {
                    copy(st * 4 + 1, in0 ? qn : reinterpret_cast<const uint4*>(r.q + va), in0);
                    copy(st * 4 + 3, in1 ? qn + 32 : reinterpret_cast<const uint4*>(r.q + va), in1);
                    qn += 64;
                }
                pn += 64;
                ahead += 64;
            }
            ptx::cp_async_commit();
        };
        auto add = [&](const uint4& x, const uint4& y) {
#pragma unroll
            for (int j = 0; j < N / 2; ++j)
                s.add<KIND>(k, Vec<TP>::pair(x, j), KIND ? Vec<TP>::pair(y, j) : make_float2(0.f, 0.f));
        };
        // Sets those of a step to zero where it lies copied, by the lane that reads them.
        auto take_out = [&](int st, int step) {
            for (uint64_t w = inside; w; w &= w - 1) {
                const int e = gone[__ffsll((long long)w) - 1] - va;
                if (e < 0 || e >= nv * N || e / (64 * N) != step || (e / N & 31) != lane) continue;
                unsigned char* z = reinterpret_cast<unsigned char*>(ring + threadIdx.x + (st * 4 + (e / (32 * N) & 1) * 2) * NT) +
                                   e % N * (int)sizeof(TP);
                for (int j = 0; j < (int)sizeof(TP); ++j) z[j] = 0;
            }
        };
#pragma unroll
        for (int st = 0; st < DEPTH; ++st) issue(st, st < steps && !(there && steps <= DEPTH));
        // (the head belongs to the first part, the tail to the last)
        s.add<KIND>(k, make_float2(lane < 16 ? pe : 0.f, 0.f), make_float2(lane < 16 ? qe : 0.f, 0.f));
        const int each = marks ? parts.size / (64 * N) : INT_MAX;
        int left = each;
        for (int i = 0; i < steps;) {
#pragma unroll
            for (int st = 0; st < DEPTH; ++st) {
                if (i == steps) break;
                asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
                if (KIND == P_ONLY && inside) take_out(st, i);
                const uint4* const at = ring + threadIdx.x + st * 4 * NT;
                add(at[0], KIND ? at[NT] : at[0]);
                add(at[2 * NT], KIND ? at[3 * NT] : at[0]);
                ++i;
                issue(st, i - 1 + DEPTH < steps);
                if (--left == 0 && parts.end(part) < b) {   // (the tail's entries may be a part of their own)
                    mark(part++, so_far());
                    left = each;
                }
            }
            s.settle();
        }
        s.add<KIND>(k, make_float2(lane < 16 ? 0.f : pe, 0.f), make_float2(lane < 16 ? 0.f : qe, 0.f));
    } else {
        for (int i0 = a; i0 < b; i0 += 32 * LOOSE) {
            const int i = i0 + lane;
            float x[LOOSE], y[LOOSE];
#pragma unroll
            for (int u = 0; u < LOOSE; ++u) {
                const bool in = i + 32 * u < b;
                x[u] = in ? to_f32(r.p[i + 32 * u]) : 0.f;
                y[u] = KIND && in ? to_f32(r.q[i + 32 * u]) : 0.f;
            }
#pragma unroll
            for (int u = 0; u < LOOSE; u += 2) s.add<KIND>(k, make_float2(x[u], x[u + 1]), make_float2(y[u], y[u + 1]));
            s.settle();
            if (marks && i0 + 32 * LOOSE == parts.end(part)) mark(part++, so_far());
        }
    }
    Sum t = so_far();
    // an infinity, a NaN or a minus somewhere: once more, counted as zero
    if (__any_sync(FULL, !s.good())) {
        t = Sum{};
        int y = a;
        for (part = 0; part < PARTS; ++part) {
            const int end = parts.end(part);
            for (; y < end; y += 32) {
                float d = 0.f, e = 0.f;
                if (y + lane < end && !is_gone(y + lane)) w_of<ANY>(k, clean(to_f32(r.p[y + lane])), KIND ? clean(to_f32(r.q[y + lane])) : 0.f, d, e);
                t.add(d, e);
                t.settle();
            }
            y = end;
            if (marks) mark(part, t);
        }
    } else if (marks) {
        for (; part < PARTS; ++part) mark(part, t);
    }
    return t;
}

// Inclusive sums over the first `lanes` lanes.
__device__ __forceinline__ Sum scan(Sum v, int lanes) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < lanes; d <<= 1) {
        const float hi = __shfl_up_sync(FULL, v.hi, d), lo = __shfl_up_sync(FULL, v.lo, d);
        if (lane >= d) v.add(hi, lo);
    }
    return v;
}

// The first lane with a share whose inclusive sum (behind base) is above the goal, or (rounding) the last with a share; -1: none has one.
__device__ __forceinline__ int pick(Sum base, const Sum& incl, const Sum& share, const Sum& goal) {
    base.add(incl);
    const uint32_t any = __ballot_sync(FULL, share.positive()), over = __ballot_sync(FULL, above(base, goal)) & any;
    return over ? __ffs(over) - 1 : any ? 31 - __clz(any) : -1;
}

// What the first warp asks of the others.
enum Ask { SUM, SEARCH, END };
struct Order {
    int ask, then;                   // SUM or END; behind the sum: SUM (another one), SEARCH or END
    int cur, refused, last;          // the current node; tokens refused there, taken out of W; a search follows
    float2 c;
    int a, b;                        // (SEARCH) where the token is, in the part that
    int whole;                       // the sums gave (0), the whole row (1), or p itself (2); 3: found
    Sum base, goal;                  // the sum before that, and the one to be passed
    int tok[KDA_TREE_MAX_NODES];
};

template <typename TP, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) verify_kernel(const __grid_constant__ VerifyArgs g, int ctas) {
    constexpr int WARPS = NT / 32;
    extern __shared__ __align__(16) uint4 ring[];     // sum_piece's copies
    __shared__ __align__(16) unsigned char order_smem[sizeof(Order)];
    Order& order = *reinterpret_cast<Order*>(order_smem);
    __shared__ float2 wsum[WARPS], slots[2][MAX_CTAS];
    __shared__ uint64_t bars[2];
    __shared__ uint32_t given_up;                     // a CTA of the session waited in vain
    __shared__ float2 psum[WARPS][PARTS];
    const int s = blockIdx.x / ctas, rank = blockIdx.x % ctas, tid = threadIdx.x, lane = tid % 32;
    // (the same in all lanes, which the compiler cannot see from tid / 32: what the first warp alone does, with its
    // many shuffles and ballots, then needs no code for lanes that part ways: 256 sessions 49.5 us for 54.7, 37 of 23 nodes 25 for 29)
    const int warp = __shfl_sync(FULL, tid / 32, 0);
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
    if (tid == 0) {
        ptx::mbar_init(ptx::smem_u32(&bars[0]), 1);
        ptx::mbar_init(ptx::smem_u32(&bars[1]), 1);
        ptx::fence_mbar_init();
        given_up = 0;
    }
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // (the barriers are there; waited for below)

    // ---- the first warp: tests, and what a sum over the row comes to
    const bool hot = g.q == nullptr;                  // chosen tokens: q is one at the child's own
    int tok[2] = {-1, -1}, par[2] = {-2, -2};         // the lane's two nodes; parent -2: left out
    float u[2] = {0.f, 0.f}, pt[2] = {0.f, 0.f}, qt[2] = {0.f, 0.f};
    uint64_t at_once = 0;                             // accepted as the first child that its parent tests (c = 0, T = 1)
    auto nodes = [&](bool a, bool b) { return (uint64_t)__ballot_sync(FULL, a) | (uint64_t)__ballot_sync(FULL, b) << 32; };
    auto of = [&](auto (&v)[2], int r) { return __shfl_sync(FULL, r < 32 ? v[0] : v[1], r & 31); };
    if (warp == 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = lane + 32 * h;
            if (r < R) {
                tok[h] = g.tokens[(size_t)s * R + r];
                par[h] = g.parents[(size_t)s * R + r];
                u[h] = g.u[(size_t)s * R + r];
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = lane + 32 * h;
            if (par[h] < -1 || par[h] >= r || tok[h] < 0 || tok[h] >= V) par[h] = -2;
            if (par[h] >= -1 && p_row(par[h])) {
                pt[h] = clean(to_f32(p_row(par[h])[tok[h]]));
                qt[h] = hot ? 1.f : clean(to_f32(q_row(par[h])[tok[h]]));
            }
        }
        auto first_test = [&](int h) { return pt[h] > 0.f && above(sum_of(pt[h], 0.f), times(u[h], sum_of(qt[h], 0.f))); };
        at_once = nodes(first_test(0), first_test(1));
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");

    int cur = -1, len = 0;
    uint32_t turn = 0;
    uint64_t children = 0, refused = 0;               // to be tested at cur; (chosen tokens) refused, taken out of W
    bool first = true, arrived = true, ending = false, dead = false;
    Coef c;
    Sum T = sum_of(1.f, 0.f), total;
    Sum share;                                        // the sum of CTA `lane`

    // Goes on with the tests until a sum is needed: true, or the walk has ended: false.
    auto go = [&]() -> bool {
        for (;;) {
            if (arrived) {
                if (len == g.max_len) return false;
                children = nodes(par[0] == cur, par[1] == cur);
                arrived = false;
            }
            if (!children) return false;
            const int r = __ffsll((long long)children) - 1;
            children &= children - 1;
            bool yes = false;
            Sum w;
            if (p_row(cur) == nullptr) {              // the token that was chosen already
                yes = true;
            } else if (first) {
                w.hi = of(pt, r);
                yes = at_once >> r & 1;
            } else {
                const float p = of(pt, r), q = of(qt, r);
                if (hot) {
                    const int x = of(tok, r);
                    w.hi = refused & nodes(tok[0] == x, tok[1] == x) ? 0.f : p;
                } else {
                    w_of<ANY>(c, p, q, w.hi, w.lo);
                }
                yes = w.positive() && above(w, times(times(of(u, r), sum_of(q, 0.f)), T));
            }
            if (yes) {
                if (rank == 0 && lane == 0) g.path[(size_t)s * g.max_len + len] = r;
                ++len;
                cur = r;
                c = Coef{};
                T = sum_of(1.f, 0.f);
                refused = 0;
                first = arrived = true;
                continue;
            }
            first = false;
            if (hot) {
                T.sub(w);
                T.settle();
                if (w.positive()) refused |= (uint64_t)1 << r;
            } else {
                c.add(T);
                if (children) return true;
            }
        }
    };
    // This CTA's sum to all, all CTAs' sums here: `share` and their `total`.
    auto exchange = [&]() {
        const int buf = turn & 1;
        Sum v;
        if (lane < WARPS) v = sum_of(wsum[lane]);
        v = warp_sum(v);
        if (ctas > 1) {
            const uint32_t bar = ptx::smem_u32(&bars[buf]);
            if (lane == 0) ptx::mbar_expect_tx(bar, ctas * 8);
            __syncwarp();
            if (lane < ctas) {
                uint32_t to = ptx::smem_u32(&slots[buf][rank]), tobar = bar;
                asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(to) : "r"(lane));
                asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(tobar) : "r"(lane));
                asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];"
                             ::"r"(to), "f"(v.hi), "f"(v.lo), "r"(tobar) : "memory");
            }
            const bool there = ptx::mbar_wait(bar, turn >> 1 & 1, g.wait_ns);
            dead = __any_sync(FULL, !there);          // gives up: see below
            v = lane < ctas ? sum_of(slots[buf][lane]) : Sum{};
            ++turn;
        } else if (lane > 0) {
            v = Sum{};
        }
        share = v;
        total = warp_sum(v);
    };

    int node_before = INT_MIN;                        // whose p and q the pass before went over
    for (;;) {
        if (warp == 0) {
            if (!ending && !go()) ending = true;
            if (lane == 0) {
                order.ask = ending && p_row(cur) == nullptr ? END : SUM;   // (END: not even the chosen token is there)
                order.cur = cur;
                order.c = make_float2(c.hi, c.lo);
                order.refused = 0;
                order.last = ending;
            }
            __syncwarp();
            if (refused) {                            // a list of the tokens, in the order of the nodes
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = lane + 32 * h;
                    if (refused >> r & 1) {
                        const int at = __popcll(refused & (((uint64_t)1 << r) - 1));
                        order.tok[at] = tok[h];
                    }
                }
                if (lane == 0) order.refused = __popcll(refused);
            }
        }
        __syncthreads();
        if (order.ask == END) break;
        const int node = order.cur;
        Coef k;
        k.hi = order.c.x;
        k.lo = order.c.y;
        const Row<TP> row(p_row(node), k.kind() ? q_row(node) : nullptr, V, pieces);
        {
            const int a = row.begin(rank * WARPS + warp), b = row.end(rank * WARPS + warp, pieces);
            const bool there = node == node_before && k.kind();      // (a refusal more at the same node: both rows again)
            node_before = k.kind() ? node : INT_MIN;
            float2* const marks = order.last && b - a > MARKED ? psum[warp] : nullptr;
            Sum sum = k.kind() == P_ONLY ? sum_piece<P_ONLY, NT>(k, row, a, b, ring, marks, there, order.tok, order.refused)
                    : k.kind() == ONE ? sum_piece<ONE, NT>(k, row, a, b, ring, marks, there, order.tok, 0)
                                      : sum_piece<ANY, NT>(k, row, a, b, ring, marks, there, order.tok, 0);
            sum = warp_sum(sum);
            if (lane == 0) wsum[warp] = make_float2(sum.hi, sum.lo);
        }
        __syncthreads();
        if (warp == 0) {
            exchange();
            int then = SUM;
            if (dead) {
                then = END;                           // no sum, no further test: the others will wait in vain too, or are done
            } else if (!ending) {
                T = total;
            } else if (!total.positive() && (k.kind() || refused)) {
                c = Coef{};                           // nothing is left: p itself
                refused = 0;
            } else {
                const Sum goal = times(g.u_next[s], total), incl = scan(share, MAX_CTAS);
                const int owner = pick(Sum{}, incl, share, goal);
                then = END;
                if (owner < 0) {
                    if (rank == 0 && lane == 0) g.next[s] = -1;
                } else if (owner == rank) {           // the warp whose piece holds the token
                    Sum before = incl;
                    before.sub(share);
                    Sum base = shfl(before, owner);
                    const Sum mine = lane < WARPS ? sum_of(wsum[lane]) : Sum{};
                    const Sum in = scan(mine, WARPS);
                    const int at = max(pick(base, in, mine, goal), 0);
                    before = in;
                    before.sub(mine);
                    base.add(shfl(before, at));
                    then = SEARCH;
                    if (lane == 0) {
                        order.goal = goal;
                        order.whole = 0;
                    }
                    const Row<TP> row(p_row(cur), c.kind() ? q_row(cur) : nullptr, V, pieces);
                    int a = row.begin(rank * WARPS + at), b = row.end(rank * WARPS + at, pieces);
                    if (b - a > MARKED) {             // and the part of it: lane i has the sum up to the end of part i
                        const Parts parts(row, a, b);
                        const Sum up_to = lane < PARTS ? sum_of(psum[at][lane]) : Sum{};
                        before = shfl(up_to, max(lane - 1, 0));
                        if (lane == 0) before = Sum{};
                        Sum part = up_to;
                        part.sub(before);
                        part.settle();
                        const int i = max(pick(base, up_to, lane < PARTS ? part : Sum{}, goal), 0);
                        base.add(shfl(before, i));
                        b = parts.end(i);
                        a = parts.begin(i, a);
                    }
                    if (lane == 0) {
                        order.a = a;
                        order.b = b;
                        order.base = base;
                    }
                }
            }
            if (lane == 0) order.then = then;
        }
        __syncthreads();
        if (order.then == END) break;
        if (order.then == SUM) continue;
        // That part once more: while it is long, a warp's share of it; then its W in shared memory (where
        // the copies were), so that of reads in a row, 1 to 3 us each while others sum, there is one.  Where
        // rounding (of the difference of two marks) led to a part with nothing in it, the whole row; if
        // that has nothing, p itself.
        for (int whole = order.whole; whole < 3;) {
            const TP* const q = whole == 2 ? nullptr : row.q;
            const int out = whole == 2 ? 0 : order.refused;
            auto entry = [&](int y, bool in, float& d, float& r) {    // W(y)
                w_of<ANY>(k, in ? clean(to_f32(row.p[y])) : 0.f, in && q ? clean(to_f32(q[y])) : 0.f, d, r);
                for (int j = 0; j < out; ++j)
                    if (order.tok[j] == y) d = r = 0.f;
            };
            for (bool sum = whole > 0; sum || order.b - order.a > STAGED * NT; sum = false) {   // (sum: the row's comes first)
                const int a = order.a, b = order.b, size = (int)(((int64_t)b - a + WARPS * 32 - 1) / (WARPS * 32)) * 32;
                const int from = (int)min((int64_t)b, a + (int64_t)warp * size), to = (int)min((int64_t)b, (int64_t)from + size);
                Sum v;
                for (int y0 = from; y0 < to; y0 += 32 * 4) {
                    float d[4], r[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) entry(y0 + 32 * e + lane, y0 + 32 * e + lane < to, d[e], r[e]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v.add(d[e], r[e]);
                    v.settle();
                }
                v = warp_sum(v);
                if (lane == 0) wsum[warp] = make_float2(v.hi, v.lo);
                __syncthreads();
                if (warp == 0) {
                    const Sum mine = lane < WARPS ? sum_of(wsum[lane]) : Sum{};
                    const Sum in = scan(mine, WARPS), goal = sum ? times(g.u_next[s], shfl(in, WARPS - 1)) : order.goal;
                    const int at = max(pick(order.base, in, mine, goal), 0);
                    __syncwarp();
                    if (lane == at) {
                        order.a = (int)min((int64_t)b, a + (int64_t)at * size);
                        order.b = (int)min((int64_t)b, (int64_t)order.a + size);
                        order.base.add(in);
                        order.base.sub(mine);
                        order.goal = goal;
                    }
                }
                __syncthreads();
            }
            float2* const W = reinterpret_cast<float2*>(ring);        // [STAGED * NT], then a thread's sums each
            float4* const sums = reinterpret_cast<float4*>(W + STAGED * NT);
            static_assert(DEPTH * 4 * 16 >= STAGED * 8 + 16, "they fit where the copies were");
            const int a = order.a, n = order.b - a, per = (n + NT - 1) / NT | 1;   // neighbouring entries a thread (odd: banks)
            for (int y0 = tid; y0 < n; y0 += 8 * NT) {
                float d[8], r[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) entry(a + y0 + e * NT, y0 + e * NT < n, d[e], r[e]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (y0 + e * NT < n) W[y0 + e * NT] = make_float2(d[e], r[e]);
            }
            __syncthreads();
            Sum one;
            for (int y = tid * per; y < min(n, tid * per + per); ++y) one.add(W[y].x, W[y].y);
            const Sum up_to = scan(one, 32);
            sums[tid] = make_float4(up_to.hi, up_to.lo, one.hi, one.lo);
            if (lane == 31) wsum[warp] = make_float2(up_to.hi, up_to.lo);
            __syncthreads();
            int found = -1;
            if (warp == 0) {
                const Sum mine = lane < WARPS ? sum_of(wsum[lane]) : Sum{};
                const Sum goal = order.goal;
                Sum base = order.base, before = scan(mine, WARPS);
                int at = max(pick(base, before, mine, goal), 0);           // the warp,
                before.sub(mine);
                base.add(shfl(before, at));
                at = at * 32;
                const float4 t = sums[at + lane];
                const Sum share = sum_of(t.z, t.w);
                before = sum_of(t.x, t.y);
                const int from = max(pick(base, before, share, goal), 0);  // its lane,
                before.sub(share);
                base.add(shfl(before, from));
                const int y = (at + from) * per + lane;
                const Sum v = lane < per && y < n ? sum_of(W[y]) : Sum{};
                const int k0 = pick(base, scan(v, 32), v, goal);           // and its entry
                if (k0 >= 0) found = a + (at + from) * per + k0;
            }
            __syncthreads();                          // (all have read what changes now)
            if (tid == 0) {
                if (found >= 0 || whole == 2) g.next[s] = found;
                order.whole = found >= 0 ? 3 : whole + 1;
                order.a = 0;
                order.b = V;
                order.base = Sum{};
            }
            __syncthreads();
            whole = order.whole;
        }
        break;
    }
    if (warp == 0 && rank == 0) {
        for (int j = len + lane; j < g.max_len; j += 32) g.path[(size_t)s * g.max_len + j] = -1;
        if (lane == 0) {
            g.path_len[s] = len;
            if (p_row(cur) == nullptr) g.next[s] = -1;
        }
    }
    if (warp == 0 && dead && lane < ctas) {           // all of them know
        uint32_t to = ptx::smem_u32(&given_up);
        asm volatile("mapa.shared::cluster.u32 %0, %0, %1;\n st.shared::cluster.u32 [%0], %2;" : "+r"(to) : "r"(lane), "r"(1) : "memory");
    }
    __syncwarp();
    // no CTA leaves while another may still write to it
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (given_up) {                                   // whatever token another CTA found: it is not valid
        if (rank == 0 && tid == 0) g.next[s] = -1;
        // sums that nobody waited for may be on their way here
        for (const uint64_t t0 = ptx::globaltimer_ns(); ptx::globaltimer_ns() - t0 < DRAIN_NS;) {}
    }
}

template <typename TP, int NT> cudaError_t verify(const VerifyArgs& a, int ctas, cudaStream_t s) {
    auto k = verify_kernel<TP, NT>;
    constexpr int RING_BYTES = DEPTH * 4 * NT * 16;
    static std::atomic<uint64_t> done{0};             // (set once per device)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(done.load() & bit)) {                       // 16 CTAs are beyond the portable size
        e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, RING_BYTES);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((int64_t)a.n * ctas));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = RING_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a, ctas);
}

// CTAs a session: as many as all run at once (1024 threads an SM), while each warp's piece is at least 512
// bytes.
template <typename TP, int NT> cudaError_t verify(const VerifyArgs& a, cudaStream_t s) {
    int ctas = 1;
    const int64_t bytes = (int64_t)a.V * (int)sizeof(TP);
    while (ctas < MAX_CTAS && (int64_t)a.n * ctas * 2 <= 1024 / NT * SMS && bytes >= (int64_t)ctas * 2 * (NT / 32) * 512) ctas *= 2;
    return verify<TP, NT>(a, ctas, s);
}
template <typename TP> cudaError_t verify(const VerifyArgs& a, cudaStream_t s) {
    // CTAs of 4 warps where they fill the SMs: more evenly
    return (int64_t)a.n * MAX_CTAS > 4 * SMS ? verify<TP, 128>(a, s) : verify<TP, 256>(a, s);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int io_bf16, cudaStream_t s) {
    return io_bf16 ? verify<__nv_bfloat16>(a, s) : verify<float>(a, s);
}

}  // namespace kda

using namespace kda;

static kda_status draft_verify(int32_t dtype, int32_t n_sessions, int32_t n_nodes, int32_t vocab, const void* p,
                               int64_t p_session_stride, int64_t p_row_stride, const void* p_last,
                               int64_t p_last_stride, const void* q, int64_t q_session_stride,
                               int64_t q_row_stride, const void* q_last, int64_t q_last_stride,
                               const int32_t* tokens, const int32_t* parents, const float* u,
                               const float* u_next, int32_t max_len, int32_t* path, int32_t* path_len,
                               int32_t* next_token, void* stream, uint64_t wait_ns) {
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
                 q_last_stride, tokens, parents, u, u_next, path, path_len, next_token, n_sessions, n_nodes, vocab, max_len, wait_ns};
    return launch_verify(a, dtype == KDA_DTYPE_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" {

kda_status kda_draft_verify(int32_t dtype, int32_t n_sessions, int32_t n_nodes, int32_t vocab, const void* p,
                            int64_t p_session_stride, int64_t p_row_stride, const void* p_last, int64_t p_last_stride,
                            const void* q, int64_t q_session_stride, int64_t q_row_stride, const void* q_last,
                            int64_t q_last_stride, const int32_t* tokens, const int32_t* parents, const float* u,
                            const float* u_next, int32_t max_len, int32_t* path, int32_t* path_len, int32_t* next_token,
                            void* stream) {
    return draft_verify(dtype, n_sessions, n_nodes, vocab, p, p_session_stride, p_row_stride, p_last, p_last_stride, q,
                        q_session_stride, q_row_stride, q_last, q_last_stride, tokens, parents, u, u_next, max_len, path,
                        path_len, next_token, stream, WAIT_NS);
}

// As kda_draft_verify with another limit of the waits between a session's CTAs, for tests (the interface has none).
kda_status kda_draft_verify_wait(int32_t dtype, int32_t n_sessions, int32_t n_nodes, int32_t vocab, const void* p,
                                 int64_t p_session_stride, int64_t p_row_stride, const void* p_last, int64_t p_last_stride,
                                 const void* q, int64_t q_session_stride, int64_t q_row_stride, const void* q_last,
                                 int64_t q_last_stride, const int32_t* tokens, const int32_t* parents, const float* u,
                                 const float* u_next, int32_t max_len, int32_t* path, int32_t* path_len, int32_t* next_token,
                                 void* stream, uint64_t wait_ns) {
    return draft_verify(dtype, n_sessions, n_nodes, vocab, p, p_session_stride, p_row_stride, p_last, p_last_stride, q,
                        q_session_stride, q_row_stride, q_last, q_last_stride, tokens, parents, u, u_next, max_len, path,
                        path_len, next_token, stream, wait_ns);
}

}  // extern "C"
