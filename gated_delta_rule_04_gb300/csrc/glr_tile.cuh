// What the prefill and the backward pass of the gated linear recurrence share:
// the tiles of 64 tokens x 64 channels and their loads, the sequence
// borders inside a tile, and the walk along the tiles.
#pragma once

#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "glr_math.cuh"
#include "ssm_common.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace glr {

constexpr int NT = 256;              // threads of a tile: 8 warps of 8 tokens, a lane 2 channels
constexpr int WARPS = NT / 32;
constexpr int SUB = CHUNK / WARPS;   // tokens of a warp
static_assert(TILE_C == 64 && SUB == 8, "lanes hold channel pairs, warps 8 tokens");

// ---- tiles in shared memory -------------------------------------------------------------
// How rows are copied: a tile by one tensor copy (rows on 16 bytes, at least a tile's channels), 4
// bytes at a time, or (16-bit elements whose rows may start on odd ones) 4 bytes at a time from
// the word that holds the row's first element.
enum Mode { MTMA = 0, M4 = 1, MODD = 2 };
constexpr int MAX_TENSORS = 5;
struct alignas(128) Maps {           // of the tensors, in boxes of a tile; zero fill out of bounds
    CUtensorMap m[MAX_TENSORS];
};

// A warp's 8 rows of one tensor's tile.  Where the tile is no tensor copy, each warp copies, waits for and reads its own.
template <typename TI, int MODE> struct Rows {
    static constexpr int ES = sizeof(TI);
    static constexpr int PITCH = TILE_C * ES + (MODE == MODD ? 4 : 0);
    static constexpr int BYTES = SUB * PITCH, TILE = CHUNK * PITCH;

    template <int N> static __device__ __forceinline__ void copy(uint32_t dst, const char* p, int bytes) {
        if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(bytes) : "memory");
        else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(p), "r"(bytes) : "memory");
    }

    // (not MTMA) Starts the copies of rows t .. t + rows - 1 (`stride` bytes apart), channels c0 .. c0 + cols - 1;
    // the rest becomes zero.  MODD: a row's words from the one that holds its first element; the 33rd
    // of them, whose first half is the row's last element, comes by `last_word`.
    static __device__ __forceinline__ void load(uint32_t dst, const void* base, uint32_t stride, int t, int c0, int rows, int cols) {
        const int lane = threadIdx.x & 31;
        const char* const first = static_cast<const char*>(base);
        constexpr int PER = TILE_C * ES / 128;                  // words of a row, a lane
        const char* p = first + (uint64_t)(uint32_t)t * stride + (uint32_t)(c0 * ES) + lane * 4;
        dst += lane * 4;
        if (rows >= SUB && cols == TILE_C) {
#pragma unroll
            for (int k = 0; k < SUB; ++k) {
#pragma unroll
                for (int w = 0; w < PER; ++w)
                    copy<4>(dst + k * PITCH + w * 128, (MODE == MODD ? down(p) : p) + w * 128, 4);
                p += stride;
            }
            return;
        }
#pragma unroll 1
        for (int k = 0; k < SUB; ++k) {
            const int odd = MODE == MODD ? (int)(reinterpret_cast<uintptr_t>(p) & 2) : 0;
            const int bytes = k < rows ? cols * ES + odd : 0;
#pragma unroll
            for (int w = 0; w < PER; ++w) {
                const int n = min(max(bytes - (lane + 32 * w) * 4, 0), 4);
                copy<4>(dst + k * PITCH + w * 128, n > 0 ? p - odd + w * 128 : down(first), n);
            }
            p += stride;
        }
    }
    static __device__ __forceinline__ const char* down(const char* p) {   // to the word
        return reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)3);
    }
    // (MODD) The 33rd word of a row, a lane each for 8 rows of four tensors (`base` and `stride` by lane / 8).
    static __device__ __forceinline__ void last_word(uint32_t dst, const void* base, uint32_t stride, int t, int c0, int rows, int cols) {
        const int row = threadIdx.x & 7;
        const char* p = static_cast<const char*>(base) + (uint64_t)(uint32_t)(t + row) * stride + (uint32_t)((c0 + TILE_C) * ES);
        const bool in = base != nullptr && row < rows && cols == TILE_C && (reinterpret_cast<uintptr_t>(p) & 2) != 0;
        // (the word before p's holds the row's last element as its first half: p is the half behind it)
        if (in) copy<4>(dst + row * PITCH + TILE_C * ES, p - 2, 2);
    }

    // Whether the first element of row t (channel c0) is the second of its word, and how that changes by row.
    struct Odd {
        uint32_t first, step;
    };
    static __device__ __forceinline__ Odd odd(const void* base, uint32_t stride, int t, int c0) {
        if (MODE != MODD) return Odd{0, 0};
        return Odd{(uint32_t)reinterpret_cast<uintptr_t>(base) + (uint32_t)t * stride + (uint32_t)c0 * ES, stride};
    }
    // The lane's channel pair of a row.
    static __device__ __forceinline__ float2 get(const unsigned char* rows, int row, Odd odd) {
        const unsigned char* p = rows + row * PITCH;
        const int lane = threadIdx.x & 31;
        if constexpr (ES == 4) {
            return reinterpret_cast<const float2*>(p)[lane];
        } else {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(p) + lane;
            uint32_t u = w[0];
            if (MODE == MODD && ((odd.first + row * odd.step) & 2)) u = __funnelshift_r(u, w[1], 16);
            return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
        }
    }
    // The lane's pair of numbers in the place of a row's pairs of two tensors, read before (in MODD, whose
    // pairs lie across words, by all lanes).
    static __device__ __forceinline__ void keep(unsigned char* rows1, unsigned char* rows2, int row, float2 v) {
        const int lane = threadIdx.x & 31;
        if constexpr (ES == 4) {
            reinterpret_cast<float2*>(rows1 + row * PITCH)[lane] = v;
        } else {
            if (MODE == MODD) __syncwarp();
            reinterpret_cast<float*>(rows1 + row * PITCH)[lane] = v.x;
            reinterpret_cast<float*>(rows2 + row * PITCH)[lane] = v.y;
        }
    }
    static __device__ __forceinline__ float2 kept(const unsigned char* rows1, const unsigned char* rows2, int row) {
        const int lane = threadIdx.x & 31;
        if constexpr (ES == 4) return reinterpret_cast<const float2*>(rows1 + row * PITCH)[lane];
        return make_float2(reinterpret_cast<const float*>(rows1 + row * PITCH)[lane], reinterpret_cast<const float*>(rows2 + row * PITCH)[lane]);
    }
};
static_assert(Rows<float, MTMA>::PITCH == 256 && Rows<__nv_bfloat16, MODD>::PITCH == 132, "");

// The copies that rows take, and whether channel pairs of `es`-byte elements can be stored as one.
inline int row_mode(const void* base, uint32_t stride, int C) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(base) | stride;
    return p % 16 == 0 && C >= TILE_C ? MTMA : p % 4 == 0 ? M4 : MODD;
}
inline bool encode(CUtensorMap* m, const void* base, uint32_t stride, int es, const ScanArgs& a) {
    return ssm::encode_rows(m, base, es, a.T, a.C, stride / es, CHUNK, TILE_C);
}
inline bool row_pairs(const void* base, uint32_t stride, int es) {
    return (reinterpret_cast<uintptr_t>(base) | stride) % (2 * es) == 0;
}

// Stores a lane's pair at p; `left` channels are left of the row, `pair`: both go as one.
template <typename TI> __device__ __forceinline__ void put(TI* p, int left, bool pair, float2 v) {
    if (pair) {
        if constexpr (sizeof(TI) == 4) *reinterpret_cast<float2*>(p) = v;
        else *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
        return;
    }
    if (left > 0) p[0] = from_f32<TI>(v.x);
    if (left > 1) p[1] = from_f32<TI>(v.y);
}
// Row t of a tensor whose rows are `stride` bytes apart, from channel c on.
template <typename TI> __device__ __forceinline__ char* row_at(const void* base, uint32_t stride, int t, int c) {
    return static_cast<char*>(const_cast<void*>(base)) + (uint64_t)(uint32_t)t * stride + (int64_t)c * (int)sizeof(TI);
}
template <typename TI> __device__ __forceinline__ void put(char* p, int left, bool pair, float2 v) {
    put(reinterpret_cast<TI*>(p), left, pair, v);
}
// The lane's pair of row `row` of an fp32 tensor [rows][C] (NULL: zero), or its place.
__device__ __forceinline__ float2 pair_at(const float* p, size_t row, int c, int C) {
    float2 h = f2(0.f);
    if (p && c < C) h.x = p[row * C + c];
    if (p && c + 1 < C) h.y = p[row * C + c + 1];
    return h;
}

// ---- sequence borders -------------------------------------------------------------------
// Of the warp's 8 tokens from t on: which begin a sequence, which end one, and the sequence
// of the first (each start adds one).  Warp-uniform.  From a table by tile, made once: a bit for each of
// its tokens that begins a sequence, the sequence of its first token, and whether the next tile begins
// with one.
struct Borders {
    uint32_t start, end;
    int seq;
};
__device__ __forceinline__ Borders borders(const ScanArgs& g, const uint4& tile, int t) {
    const int at = t % CHUNK, rows = (int)g.T - t;
    const uint64_t starts = tile.x | (uint64_t)tile.y << 32;
    const uint32_t after = at + SUB < CHUNK ? (uint32_t)(starts >> (at + SUB)) & 1u : tile.w;
    Borders b;
    b.start = (uint32_t)(starts >> at) & ((1u << SUB) - 1);
    b.end = b.start >> 1 | after << (SUB - 1);
    if (rows > 0 && rows <= SUB) b.end |= 1u << (rows - 1);
    b.seq = (int)tile.z + __popcll(starts & (((uint64_t)2 << at) - 2));
    return b;
}
// Makes it, by all warps of the grid.
__device__ __forceinline__ void make_borders(const ScanArgs& g, size_t warp, size_t warps) {
    const int lane = threadIdx.x & 31, n = g.f.n;
    auto start = [&](int s) -> int64_t { return (uint32_t)s >= (uint32_t)n ? INT64_MAX : n <= INLINE_SEQS ? (int64_t)g.f.cu[s] : g.f.d_cu[s]; };
    for (size_t tt = warp; tt < (size_t)g.tiles_t; tt += warps) {
        const int64_t t0 = (int64_t)tt * CHUNK;
        int lo = 0, hi = n - 1;                                // the last sequence that begins at or before t0
        while (lo < hi) {
            const int mid = hi - (hi - lo) / 2;
            if (start(mid) <= t0) lo = mid; else hi = mid - 1;
        }
        const int64_t c1 = start((int)((uint32_t)lo + 1 + lane)) - t0, c2 = start((int)((uint32_t)lo + 33 + lane)) - t0;
        const uint64_t bits = (c1 < CHUNK ? (uint64_t)1 << c1 : 0) | (c2 < CHUNK ? (uint64_t)1 << c2 : 0);
        const uint32_t first = start(lo) == t0 ? 1u : 0u;
        const uint4 b = make_uint4(__reduce_or_sync(0xffffffffu, (uint32_t)bits) | first,
                                   __reduce_or_sync(0xffffffffu, (uint32_t)(bits >> 32)), (uint32_t)lo,
                                   __any_sync(0xffffffffu, c1 == CHUNK || c2 == CHUNK) ? 1u : 0u);
        if (lane == 0) g.borders[tt] = b;
    }
}

// ---- the walk along the tiles -------------------------------------------------------------
// Tiles are taken in the order of a ticket, all of one place along T before the next, so a
// tile's predecessors have been taken, by CTAs that are running, and every wait ends.  A tile
// publishes its map h -> A h + B, then looks back for the nearest of BACK predecessors whose
// outgoing value is known, and applies the maps in between in their order.  How far back a value
// was found changes neither the maps nor their order, so results do not depend on the timing.
// Maps and values are their own flags: the words are set to EMPTY, a NaN that is never
// published, before the first tile, and a reader takes each as soon as it is another one, so no
// fence stands between a tile and the next.  (With flags beside them, two fences and one
// more read: 5 us more a tile.)
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr uint32_t EMPTY = 0xffffffffu;

__device__ __forceinline__ uint32_t word_of(float x) {
    const uint32_t u = __float_as_uint(x);
    return u == EMPTY ? 0x7fffffffu : u;
}
__device__ __forceinline__ void publish(float* p, float2 v) {
    asm volatile("st.relaxed.gpu.global.v2.b32 [%0], {%1, %2};" ::"l"(p), "r"(word_of(v.x)), "r"(word_of(v.y)) : "memory");
}
__device__ __forceinline__ void publish(float* p, float2 A, float2 B) {
    asm volatile("st.relaxed.gpu.global.v4.b32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(word_of(A.x)), "r"(word_of(B.x)),
                 "r"(word_of(A.y)), "r"(word_of(B.y)) : "memory");
}
__device__ __forceinline__ uint2 peek2(const float* p) {
    uint2 v;
    asm volatile("ld.relaxed.gpu.global.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ uint4 peek4(const float* p) {
    uint4 v;
    asm volatile("ld.relaxed.gpu.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// By one whole warp.  order: the tile's place in the walk (0: the first).
__device__ __forceinline__ size_t walk_place(const ScanArgs& g, int order, int tile_c) {
    return ((size_t)order * g.tiles_c + tile_c) * TILE_C + 2 * (threadIdx.x & 31);
}
// First: the tile's map, or (it begins anew, in all channels: borders are the tokens') its value.
__device__ __forceinline__ void walk_map(const ScanArgs& g, int order, int tile_c, float2 A, float2 B) {
    const size_t me = walk_place(g, order, tile_c);
    if (A.x < 0.f) publish(g.val + me, B);
    else publish(g.map + 2 * me, A, B);
}
// Then: the value that comes into the tile, returned, and the one that leaves it.
template <int BACK> __device__ __forceinline__ float2 walk_back(const ScanArgs& g, int order, int tile_c, float2 A, float2 B) {
    const int lane = threadIdx.x & 31;
    const size_t me = walk_place(g, order, tile_c);
    const size_t step = (size_t)g.tiles_c * TILE_C;
    float2 in = f2(0.f);
    if (order == 0) return in;
    bool done = false;
    uint64_t begin = 0;
    for (uint32_t turn = 1;; ++turn) {
        if (!done) {
            uint2 v[BACK];
            uint4 m[BACK - 1];
#pragma unroll
            for (int k = 0; k < BACK; ++k) {
                v[k] = make_uint2(EMPTY, EMPTY);
                if (k < order) v[k] = peek2(g.val + me - (k + 1) * step);
                if (k + 1 < BACK) {
                    m[k] = make_uint4(EMPTY, EMPTY, EMPTY, EMPTY);
                    if (k < order) m[k] = peek4(g.map + 2 * (me - (k + 1) * step));
                }
            }
            int from = -1;
            bool maps = true;                                   // of the tiles nearer than k
#pragma unroll
            for (int k = 0; k < BACK; ++k) {
                if (from < 0 && maps && v[k].x != EMPTY && v[k].y != EMPTY) {
                    from = k;
                    in = make_float2(__uint_as_float(v[k].x), __uint_as_float(v[k].y));
                }
                if (k + 1 < BACK) maps = maps && m[k].x != EMPTY && m[k].y != EMPTY && m[k].z != EMPTY && m[k].w != EMPTY;
            }
            done = from >= 0;
#pragma unroll
            for (int k = BACK - 2; k >= 0; --k)
                if (k < from) in = make_float2(fmaf(__uint_as_float(m[k].x), in.x, __uint_as_float(m[k].y)),
                                               fmaf(__uint_as_float(m[k].z), in.y, __uint_as_float(m[k].w)));
        }
        if (__all_sync(0xffffffffu, done)) break;
        if (turn % 64 == 0) {
            const uint64_t now = ptx::globaltimer_ns();
            if (begin == 0) begin = now;
            if (__any_sync(0xffffffffu, now - begin > WAIT_NS)) {   // gives up: the error word, and NaN from here on
                if (lane == 0) atomicExch(g.status, ERR_TIMEOUT);
                in = f2(__int_as_float(0x7fffffff));
                break;
            }
        }
    }
    if (!(A.x < 0.f)) publish(g.val + me, make_float2(fmaf(A.x, in.x, B.x), fmaf(A.y, in.y, B.y)));
    return in;
}

// The next tile: its place in the walk and its column, -1 behind the last (the counter starts at EMPTY, like
// everything else that is set before the first tile).
__device__ __forceinline__ uint32_t take_ticket(const ScanArgs& g) { return atomicAdd(g.ticket, 1u); }
__device__ __forceinline__ int2 place_of(const ScanArgs& g, uint32_t ticket) {
    const uint32_t k = ticket + 1u;
    if (k >= (uint32_t)g.tiles_t * (uint32_t)g.tiles_c) return make_int2(-1, 0);
    return make_int2((int)(k / (uint32_t)g.tiles_c), (int)(k % (uint32_t)g.tiles_c));
}

// What a walk finds in its workspace: a cleared error word, ticket, maps and values EMPTY, the gates' table and
// that of the tiles' borders.  By all threads of the grid.
__device__ __forceinline__ void set_up(const ScanArgs& g) {
    const size_t id = (size_t)blockIdx.x * blockDim.x + threadIdx.x, all = (size_t)gridDim.x * blockDim.x;
    if (id == 0) *g.status = ERR_NONE;
    uint4* w = reinterpret_cast<uint4*>(g.ticket);
    for (size_t k = id; k < g.empty; k += all) w[k] = make_uint4(EMPTY, EMPTY, EMPTY, EMPTY);
    for (size_t k = id; k < (size_t)g.tiles_c * (TILE_C / 2); k += all) {
        const Gate q = make_gate(g, (int)k * 2);
        float2* p = g.gates + k / (TILE_C / 2) * (3 * TILE_C / 2) + k % (TILE_C / 2);
        p[0] = q.ea;
        p[TILE_C / 2] = q.rb;
        p[TILE_C] = q.ib;
    }
    make_borders(g, id / 32, all / 32);
}
// At the start of a walk: it sets up by itself, or a kernel before it has.
__device__ __forceinline__ void begin(const ScanArgs& g) {
    if (g.alone) {
        set_up(g);
        cooperative_groups::this_grid().sync();
    } else {
        cudaGridDependencySynchronize();
    }
}
// The lane's gate constants of tile column tc, from the table.
__device__ __forceinline__ Gate load_gate(const ScanArgs& g, int tc) {
    const float2* p = g.gates + (size_t)tc * (3 * TILE_C / 2) + (threadIdx.x & 31);
    return Gate{p[0], p[TILE_C / 2], p[TILE_C]};
}

// Waits for a phase of a barrier of this CTA; past a limit of turns (each waits a while itself) the error word
// is set.
__device__ __forceinline__ void wait_or(const ScanArgs& g, uint32_t bar, uint32_t parity) {
    for (uint32_t turn = 0; !ptx::mbar_try_wait(bar, parity);)
        if (++turn >> 24) {
            atomicExch(g.status, ERR_TIMEOUT);
            break;
        }
}
__device__ __forceinline__ void bar_arrive(int id, int threads) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ __forceinline__ void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// Launches a walk with a CTA for each of its tiles, but no more than run at once.  Up to four such rounds
// the kernel does everything (as a cooperative launch, whose CTAs may wait for all others): a
// launch more takes the host 6 us, and the GPU is done sooner (601 tokens x 512: 22 us a call
// for 24, backward 777 x 321: 45 for 53).  Otherwise `before` is a kernel of its own
// that sets up, and the walk starts beside its end: many CTAs that wait for all others, and
// few that add up, cost the GPU more (backward 32768 x 4096: 600 us for 543).
__global__ void __launch_bounds__(256) setup_kernel(const __grid_constant__ ScanArgs g);
template <typename... Rest>
cudaError_t launch_walk(void (*k)(ScanArgs, Rest...), std::atomic<int> (&most)[64], ScanArgs a, int threads, size_t smem,
                        cudaStream_t s, bool* alone, Rest... rest) {
    int dev = 0, blocks = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64) blocks = most[dev].load();
    if (blocks == 0) {                               // (once per kernel and device)
        int sms = 0, per = 0;
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, k, threads, smem);
        if (e != cudaSuccess) return e;
        blocks = sms * per;
        if (blocks < 1) return cudaErrorLaunchOutOfResources;
        if (dev < 64) most[dev].store(blocks);
    }
    const int64_t tiles = (int64_t)a.tiles_t * a.tiles_c;
    a.alone = *alone = tiles <= 4 * (int64_t)blocks;
    if (!a.alone) {
        const size_t work = std::max({a.empty, (size_t)a.tiles_c * (TILE_C / 2), (size_t)a.tiles_t});
        setup_kernel<<<(unsigned)std::min<size_t>((work + 255) / 256, SMS * 8), 256, 0, s>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::min<int64_t>(tiles, blocks));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    if (a.alone) {
        at.id = cudaLaunchAttributeCooperative;
        at.val.cooperative = 1;
    } else {
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a, rest...);
}

}  // namespace glr
}  // namespace kda
