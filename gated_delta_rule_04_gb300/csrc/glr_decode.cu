// Tokens of the gated linear recurrence over a pool of states: straight runs of
// 1 to 64 tokens per session, and the accepted paths of a round.  A thread holds
// the states of V neighbouring channels and walks the tokens.  The rows move once and bound
// the call: a thread copies its share of the next 3 tokens' into shared memory
// while it computes.  256 rounds of 5 tokens x 8192 channels, bf16: 22 us in a graph (4.2 TB/s of a
// copy's 6.8; with the next token's rows in registers instead 23), one token 2.5 us.
#include <type_traits>

#include "glr_math.cuh"

namespace kda {
namespace glr {
namespace {

constexpr int NT = 128, DEPTH = 3;

template <int BYTES> struct Word;
template <> struct Word<2> { using T = uint16_t; };
template <> struct Word<4> { using T = uint32_t; };
template <> struct Word<8> { using T = uint2; };
template <> struct Word<16> { using T = uint4; };

// V neighbouring values as pairs (V = 1: the second of the pair is zero).
template <typename TI, int V> struct Values {
    static constexpr int PAIRS = (V + 1) / 2;
    union Raw {
        typename Word<V * sizeof(TI)>::T w;
        TI v[V];
        __device__ Raw() {}
    };
    static __device__ __forceinline__ void load(Raw& r, const void* base, int64_t at) {
        r.w = *reinterpret_cast<const typename Word<V * sizeof(TI)>::T*>(static_cast<const TI*>(base) + at);
    }
    // Into the thread's own place in shared memory.
    static __device__ __forceinline__ void copy(typename Word<V * sizeof(TI)>::T* to, const char* from) {
        constexpr int BYTES = V * (int)sizeof(TI);
        const uint32_t at = (uint32_t)__cvta_generic_to_shared(to);
        if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
        else if constexpr (BYTES >= 4) asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
        else *to = *reinterpret_cast<const typename Word<BYTES>::T*>(from);
    }
    static __device__ __forceinline__ float2 pair(const Raw& r, int p) {
        if constexpr (sizeof(TI) == 2 && V > 1) {     // (by words: an instruction a value)
            const uint32_t u = reinterpret_cast<const uint32_t*>(&r.w)[p];
            return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
        }
        return make_float2(to_f32(r.v[2 * p]), 2 * p + 1 < V ? to_f32(r.v[2 * p + 1 < V ? 2 * p + 1 : 0]) : 0.f);
    }
    static __device__ __forceinline__ void store(void* base, int64_t at, const float2 (&x)[PAIRS]) {
        Raw r;
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            if constexpr (sizeof(TI) == 2 && V > 1) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[p].x, x[p].y);
                reinterpret_cast<uint32_t*>(&r.w)[p] = reinterpret_cast<const uint32_t&>(b);
            } else {
                r.v[2 * p] = from_f32<TI>(x[p].x);
                if (2 * p + 1 < V) r.v[2 * p + 1 < V ? 2 * p + 1 : 0] = from_f32<TI>(x[p].y);
            }
        }
        *reinterpret_cast<typename Word<V * sizeof(TI)>::T*>(static_cast<TI*>(base) + at) = r.w;
    }
};

// V neighbouring numbers of an fp32 tensor as pairs (NULL: zeros).
template <int V> __device__ __forceinline__ void load_f32(const float* base, size_t at, float2 (&x)[(V + 1) / 2]) {
    constexpr int W = V < 4 ? V : 4;
#pragma unroll
    for (int q = 0; q < V / W; ++q) {
        typename Values<float, W>::Raw r;
        if (base) Values<float, W>::load(r, base, at + W * q);
#pragma unroll
        for (int p = 0; p < (W + 1) / 2; ++p) x[q * W / 2 + p] = base ? Values<float, W>::pair(r, p) : f2(0.f);
    }
}

template <typename TI, int V>
__global__ void __launch_bounds__(NT, 7) token_kernel(const __grid_constant__ TokenArgs g, int blocks) {
    using X = Values<TI, V>;
    constexpr int PAIRS = X::PAIRS;
    __shared__ __align__(16) typename Word<V * sizeof(TI)>::T ring[DEPTH][4][NT];
    const int n = blockIdx.x / blocks, c = (blockIdx.x % blocks * blockDim.x + threadIdx.x) * V, lane = threadIdx.x & 31;
    const int slot = g.slots ? g.slots[n] : n;
    int len = g.n_tokens, p1 = 0, p2 = 0;
    if (g.path) {                                     // lane j has the path's tokens j and 32 + j
        len = g.path_len[n];
        const int32_t* path = g.path + (size_t)n * g.max_len;
        if (lane < g.max_len) p1 = path[lane];
        if (lane + 32 < g.max_len) p2 = path[lane + 32];
        bool bad = len < 0 || len > g.max_len;
        bad |= lane < len && (p1 < 0 || p1 >= g.n_tokens);
        bad |= lane + 32 < len && (p2 < 0 || p2 >= g.n_tokens);
        if (__any_sync(0xffffffffu, bad)) return;     // the session is skipped (by every warp alike)
    }
    if (slot < 0 || slot >= g.n_slots) return;
    const bool in = c < g.C;
    float2 h[PAIRS];
    Gate k[PAIRS];
    bool wide = false;
    if (in) {
        float2 A[PAIRS], rb[PAIRS], ib[PAIRS];
        load_f32<V>(g.S_in, (size_t)slot * g.C + c, h);
        load_f32<V>(g.A_log, c, A);
        load_f32<V>(g.r_bias, c, rb);
        load_f32<V>(g.i_bias, c, ib);
#pragma unroll
        for (int p = 0; p < PAIRS; ++p) {
            // (V = 1: the second of the pair is no channel, and asks for no exponential)
            k[p] = Gate{make_float2(-expf(A[p].x), V > 1 ? -expf(A[p].y) : 0.f), mul2(rb[p], f2(-LOG2E)), mul2(ib[p], f2(-LOG2E))};
            wide |= !(k[p].ea.x >= -NEAR && k[p].ea.y >= -NEAR);
        }
    }
    wide = __any_sync(0xffffffffu, wide);
    const int64_t row0 = (int64_t)n * g.n_tokens;
    auto node_of = [&](int j) {
        return !g.path ? j : j < 32 ? __shfl_sync(0xffffffffu, p1, j) : __shfl_sync(0xffffffffu, p2, j - 32);
    };
    auto start = [&](const void* base, uint32_t stride) { return static_cast<const char*>(base) + row0 * stride + (int64_t)c * (int)sizeof(TI); };
    const char *xp = start(g.x, g.x_s), *rp = start(g.r, g.r_s), *ip = start(g.i, g.i_s), *zp = start(g.z, g.z_s);
    auto issue = [&](int j) {                         // (a thread reads what it copied: nothing waits for another)
        if (j < len) {
            const uint64_t node = (uint32_t)node_of(j);
            if (in) {
                X::copy(&ring[j % DEPTH][0][threadIdx.x], xp + node * g.x_s);
                X::copy(&ring[j % DEPTH][1][threadIdx.x], rp + node * g.r_s);
                X::copy(&ring[j % DEPTH][2][threadIdx.x], ip + node * g.i_s);
                if (g.z) X::copy(&ring[j % DEPTH][3][threadIdx.x], zp + node * g.z_s);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int j = 0; j < DEPTH; ++j) issue(j);
    char* const op = static_cast<char*>(g.o) + (row0 * g.C + c) * (int64_t)sizeof(TI);
    for (int j = 0; j < len; ++j) {
        asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
        const int node = node_of(j);
        if (in) {
            typename X::Raw x, r, i, z;
            x.w = ring[j % DEPTH][0][threadIdx.x];
            r.w = ring[j % DEPTH][1][threadIdx.x];
            i.w = ring[j % DEPTH][2][threadIdx.x];
            if (g.z) z.w = ring[j % DEPTH][3][threadIdx.x];
            float2 o[PAIRS];
            auto token = [&](auto w) {
#pragma unroll
                for (int p = 0; p < PAIRS; ++p) {
                    const Step s = step_of<decltype(w)::value>(k[p], X::pair(x, p), X::pair(r, p), X::pair(i, p));
                    h[p] = fma2(s.a, h[p], s.b);
                    o[p] = g.z ? mul2(h[p], silu(X::pair(z, p))) : h[p];
                }
            };
            if (wide) token(std::true_type{});
            else token(std::false_type{});
            if (g.o) X::store(op + (uint64_t)(uint32_t)node * ((uint32_t)g.C * (uint32_t)sizeof(TI)), 0, o);
        }
        issue(j + DEPTH);
    }
    if (in && g.S_out) {
        const size_t at = (size_t)slot * g.C + c;
        if constexpr (V == 8) {
            const float2 lo[2] = {h[0], h[1]}, hi[2] = {h[2], h[3]};
            Values<float, 4>::store(g.S_out, at, lo);
            Values<float, 4>::store(g.S_out, at + 4, hi);
        } else {
            Values<float, V>::store(g.S_out, at, h);
        }
    }
}

template <typename TI, int V>
cudaError_t tokens(const TokenArgs& a, cudaStream_t s) {
    const int64_t per = ((int64_t)a.C + V - 1) / V;
    const int nt = (int)(per < NT ? (per + 31) / 32 * 32 : NT), blocks = (int)((per + nt - 1) / nt);
    token_kernel<TI, V><<<(unsigned)((int64_t)a.n * blocks), nt, 0, s>>>(a, blocks);
    return cudaGetLastError();
}

// The most neighbouring channels (1, 2, 4, 8) that every row, state and parameter can be taken by.
int widest(const TokenArgs& a, int es) {
    uint64_t rows = 0, states = 0;                    // the addresses and strides, or'ed
    auto row = [&](const void* p, uint64_t stride) {
        if (p) rows |= reinterpret_cast<uintptr_t>(p) | stride;
    };
    row(a.x, a.x_s); row(a.r, a.r_s); row(a.i, a.i_s); row(a.z, a.z_s); row(a.o, (uint64_t)a.C * es);
    for (const float* p : {a.S_in, (const float*)a.S_out, a.A_log, a.r_bias, a.i_bias}) states |= reinterpret_cast<uintptr_t>(p);
    int v = 16 / es;
    while (v > 1 && (rows % (v * es) != 0 || states % ((v < 4 ? v : 4) * 4) != 0 || a.C % v != 0)) v /= 2;
    return v;
}

}  // namespace

cudaError_t launch_tokens(const TokenArgs& a, int io_bf16, cudaStream_t s) {
    int v = widest(a, io_bf16 ? 2 : 4);
    // few sessions: pairs, as many threads as there are
    while (v > 2 && (int64_t)a.n * a.C / v < SMS * 256) v /= 2;
    if (!io_bf16)
        return v == 4 ? tokens<float, 4>(a, s) : v == 2 ? tokens<float, 2>(a, s) : tokens<float, 1>(a, s);
    return v == 8 ? tokens<__nv_bfloat16, 8>(a, s) : v == 4 ? tokens<__nv_bfloat16, 4>(a, s)
         : v == 2 ? tokens<__nv_bfloat16, 2>(a, s) : tokens<__nv_bfloat16, 1>(a, s);
}

}  // namespace glr
}  // namespace kda
