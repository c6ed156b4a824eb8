// What the prefill and the backward pass of the gated linear recurrence share:
// the tiles of 64 tokens x 64 channels and their loads, the sequence
// borders inside a tile, and the walk along the tiles.
#pragma once

#include <algorithm>

#include "glr_math.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace glr {

constexpr int NT = 256;              // threads of a tile: 8 warps of 8 tokens, a lane 2 channels
constexpr int WARPS = NT / 32;
constexpr int SUB = CHUNK / WARPS;   // tokens of a warp
static_assert(TILE_C == 64 && SUB == 8, "lanes hold channel pairs, warps 8 tokens");

// ---- tiles in shared memory -------------------------------------------------------------
// How rows are copied: 16 bytes at a time, 4 bytes at a time, or (16-bit elements whose rows
// start on odd ones) 4 bytes at a time from the word that holds the row's first element.
enum Mode { M16 = 0, M4 = 1, MODD = 2 };

template <typename TI, int MODE> struct Rows {
    static constexpr int PITCH = TILE_C * (int)sizeof(TI) + (MODE == MODD ? 4 : 0);
    static constexpr int BYTES = CHUNK * PITCH;

    // Starts the copies of tile rows t0 .. t0 + 63 (those below T), channels c0 .. c0 + 63 (those below C).
    static __device__ __forceinline__ void load(unsigned char* dst, const void* base, int64_t stride, int64_t t0, int c0,
                                                const ScanArgs& g) {
        const uint32_t s = ptx::smem_u32(dst);
        constexpr int ES = sizeof(TI), PIECE = MODE == M16 ? 16 : 4, PER = (PITCH + PIECE - 1) / PIECE;
        constexpr int ALL = CHUNK * PER;
        static_assert(MODE == MODD || PITCH % PIECE == 0, "whole pieces");
#pragma unroll 4
        for (int k = threadIdx.x; k < ALL; k += NT) {
            const int row = k / PER, piece = k % PER;
            const int64_t t = t0 + row;
            const char* p = static_cast<const char*>(base) + ((t < g.T ? t : 0) * stride + c0) * ES;
            int bytes = (g.C - c0) * ES;                        // of the row, from c0 on
            if (MODE == MODD) {
                const int odd = (int)(reinterpret_cast<uintptr_t>(p) & 2);
                p -= odd;
                bytes += odd;
            }
            bytes = t < g.T ? min(max(bytes - piece * PIECE, 0), PIECE) : 0;
            if (bytes > 0) p += piece * PIECE;                  // (an address is formed in bounds only)
            if (MODE == M16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s + row * PITCH + piece * PIECE), "l"(p), "r"(bytes) : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(s + row * PITCH + piece * PIECE), "l"(p), "r"(bytes) : "memory");
        }
    }

    // Whether the first element of row t0 (channel c0) is the second of its word, and how that changes by row.
    struct Odd {
        int first, step;
    };
    static __device__ __forceinline__ Odd odd(const void* base, int64_t stride, int64_t t0, int c0) {
        if (MODE != MODD) return Odd{0, 0};
        return Odd{(int)((reinterpret_cast<uintptr_t>(base) >> 1) + (uintptr_t)(t0 * stride + c0)) & 1, (int)(stride & 1)};
    }
    // The lane's channel pair of a row.
    static __device__ __forceinline__ float2 get(const unsigned char* tile, int row, Odd odd) {
        const unsigned char* p = tile + row * PITCH;
        const int lane = threadIdx.x & 31;
        if constexpr (sizeof(TI) == 4) {
            return reinterpret_cast<const float2*>(p)[lane];
        } else {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(p) + lane;
            uint32_t u = w[0];
            if (MODE == MODD && ((odd.first + row * odd.step) & 1)) u = __funnelshift_r(u, w[1], 16);
            return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
        }
    }
};
static_assert(Rows<float, M16>::PITCH == 256 && Rows<__nv_bfloat16, MODD>::PITCH == 132, "");

// The copies that rows of `es`-byte elements take, and whether channel pairs can be stored as one.
inline int row_mode(const void* base, int64_t stride, int es) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(base) | (uintptr_t)(stride * es);
    return p % 16 == 0 ? M16 : p % 4 == 0 ? M4 : MODD;
}
inline bool row_pairs(const void* base, int64_t stride, int es) {
    return (reinterpret_cast<uintptr_t>(base) | (uintptr_t)(stride * es)) % (2 * es) == 0;
}

// Stores a lane's pair at channel c of row t; `pairs`: every row's pairs lie on their size.
template <typename TI>
__device__ __forceinline__ void put(void* base, int64_t stride, int64_t t, int c, int C, bool pairs, float2 v) {
    TI* p = static_cast<TI*>(base) + t * stride + c;
    if (pairs) {                                                // (C may be odd: the last pair's second channel)
        if (c + 1 < C) {
            if constexpr (sizeof(TI) == 4) *reinterpret_cast<float2*>(p) = v;
            else *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
            return;
        }
        if (c < C) p[0] = from_f32<TI>(v.x);
        return;
    }
    if (c < C) p[0] = from_f32<TI>(v.x);
    if (c + 1 < C) p[1] = from_f32<TI>(v.y);
}

// ---- sequence borders -------------------------------------------------------------------
// Of the warp's 8 tokens from t on: which begin a sequence, which end one, and the sequence
// of the first (each start adds one).  Warp-uniform.
struct Borders {
    uint32_t start, end;
    int seq;
};
__device__ __forceinline__ Borders borders(const ScanArgs& g, int tile_t, int64_t t) {
    const int lane = threadIdx.x & 31, n = g.f.n;
    int s0 = 0;
    int64_t c1 = INT64_MAX, c2 = INT64_MAX, c0 = 0;            // starts of sequences s0 + 1 + lane, s0 + 33 + lane, s0
    if (n <= INLINE_SEQS) {
        if (lane < n) c1 = g.f.cu[1 + lane];
    } else {
        s0 = g.f.d_tile[tile_t];
        c0 = g.f.d_cu[s0];
        if (s0 + 1 + lane <= n) c1 = g.f.d_cu[s0 + 1 + lane];
        if (s0 + 33 + lane <= n) c2 = g.f.d_cu[s0 + 33 + lane];
    }
    auto of = [&](int64_t x) {                                  // the sequence of token x of this tile, or before / behind it
        int s = s0 + __popc(__ballot_sync(0xffffffffu, c1 <= x)) - (x < c0 ? 1 : 0);
        if (n > INLINE_SEQS) s += __popc(__ballot_sync(0xffffffffu, c2 <= x));
        return s;
    };
    Borders b{0, 0, 0};
    int prev = of(t - 1);
    if (t == 0) prev = -1;
    int cur = of(t);
    b.seq = cur;
#pragma unroll
    for (int j = 0; j < SUB; ++j) {
        const int next = of(t + j + 1);
        if (t + j < g.T) {
            b.start |= (cur != prev ? 1u : 0u) << j;
            b.end |= (next != cur ? 1u : 0u) << j;
        }
        prev = cur;
        cur = next;
    }
    return b;
}

// ---- the walk along the tiles -------------------------------------------------------------
// Tiles are taken in the order of a ticket, all of one place along T before the next, so a
// tile's predecessors have been taken, by CTAs that are running, and every wait ends.  A
// tile publishes its map h -> A h + B, looks back over at most 32 predecessors for
// the nearest one whose outgoing value is known, and applies the maps in between in their order:
// the same operations in any timing, so results do not depend on it.
constexpr uint64_t WAIT_NS = 2000000000ull;

__device__ __forceinline__ int ld_acquire(const int32_t* p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_release(int32_t* p, int v) {
    asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
constexpr int HAS_MAP = 1, HAS_VALUE = 2;

// By one whole warp.  order: the tile's place in the walk (0: the first).  Returns the value
// that comes into the tile.
__device__ __forceinline__ float2 walk(const ScanArgs& g, int order, int tile_c, float2 A, float2 B) {
    const int lane = threadIdx.x & 31;
    auto slot = [&](int o) { return (size_t)o * g.tiles_c + tile_c; };
    const size_t me = slot(order);
    float2* pre = reinterpret_cast<float2*>(g.pre) + me * (TILE_C / 2) + lane;
    const bool anew = A.x < 0.f;                                // (both channels: borders are the tokens')
    float2 in = f2(0.f);
    if (anew) {
        *pre = B;
        __syncwarp();
        if (lane == 0) {
            __threadfence();
            st_release(g.flags + me, HAS_VALUE);
        }
    } else {
        reinterpret_cast<float4*>(g.agg)[me * (TILE_C / 2) + lane] = make_float4(A.x, B.x, A.y, B.y);
        __syncwarp();
        if (lane == 0) {
            __threadfence();
            st_release(g.flags + me, HAS_MAP);
        }
    }
    if (order == 0) return in;
    // the nearest predecessor with a value, all maps in between known
    uint64_t begin = 0;
    int back;
    for (uint32_t turn = 1;; ++turn) {
        const int o = order - 1 - lane;
        const int f = o >= 0 ? ld_acquire(g.flags + slot(o)) : 0;
        const uint32_t value = __ballot_sync(0xffffffffu, f == HAS_VALUE), none = __ballot_sync(0xffffffffu, f == 0);
        back = __ffs(value) - 1;
        if (back >= 0 && (none & ((1u << back) - 1)) == 0) break;
        if (turn % 64 == 0) {
            const uint64_t now = ptx::globaltimer_ns();
            if (begin == 0) begin = now;
            if (__any_sync(0xffffffffu, now - begin > WAIT_NS)) {   // gives up: the error word, and NaN from here on
                if (lane == 0) atomicExch(g.status, ERR_TIMEOUT);
                back = -1;
                break;
            }
        }
    }
    __syncwarp();
    if (back < 0) {
        in = f2(__int_as_float(0x7fffffff));
    } else {
        in = __ldcg(reinterpret_cast<const float2*>(g.pre) + slot(order - 1 - back) * (TILE_C / 2) + lane);
#pragma unroll 4
        for (int k = back - 1; k >= 0; --k) {
            const float4 m = __ldcg(reinterpret_cast<const float4*>(g.agg) + slot(order - 1 - k) * (TILE_C / 2) + lane);
            in = make_float2(fmaf(m.x, in.x, m.y), fmaf(m.z, in.y, m.w));
        }
    }
    if (!anew) {
        *pre = make_float2(fmaf(A.x, in.x, B.x), fmaf(A.y, in.y, B.y));
        __syncwarp();
        if (lane == 0) {
            __threadfence();
            st_release(g.flags + me, HAS_VALUE);
        }
    }
    return in;
}

}  // namespace glr
}  // namespace kda
