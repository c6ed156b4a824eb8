// Prefill of the gated linear recurrence: h_t = a_t h_{t-1} + m_t v_t x_t,
// o_t = h_t SiLU(z_t), with m = sqrt(1 - a^2).
//
// One pass over the data.  Tiles of 64 tokens x 64 channels lie in shared memory
// in their own type, copied two tiles ahead; a thread holds 8 tokens of 2
// channels, computes their a and b = m v x once, and the map h -> A h + B of its
// run.  Two more warps compose the maps and walk along the tiles (glr_tile.cuh) for the
// value that comes in, while those 8 are at the next tile's maps; the second
// sweep over the 8 tokens is one multiply-add a token and the output gate.
// Sequences lie anywhere in the tiles: a token that begins one starts its run
// anew from S_in.
//
// 16384 tokens x 4096, bf16: 141 us (4.8 TB/s of a copy's 6.8), 65273 x 8192: 960 (5.6).
// No unit is near its peak: memory 61 %, the exponentials' unit 55 %, issue slots 54 %; without
// arithmetic, loads or walk alone it is 139, 132 or 139 us of then 145, without all three 90.  Two CTAs an
// SM (f32: one) are what the registers of a tile's pending sweep leave.
#include <type_traits>

#include "glr_tile.cuh"

namespace kda {
namespace glr {
namespace {

constexpr int ALL = NT + 64;         // 8 warps that compute, two that walk
constexpr int MEET = NT + 32;        // the computing ones and one that walks
// Named barriers, two each: READY, a tile's maps are there; COME, its warps' first values are.  (The second
// also keeps the computing warps together: they share what they fetch of the code.  With an
// mbarrier instead, which does not, 198 us for 189 at 16384 tokens x 4096.)  FREE: its rows have been read.
constexpr int READY = 1, COME = 3, FREE = 5;
constexpr int RING = 4;              // tiles whose places are known

// What a warp keeps of a tile between its two sweeps.
struct Pending {
    float2 a[SUB], b[SUB];
    Borders bd;
    int tt, tc;
};

template <typename TI, int MODE, bool GATED, int PER_SM>
__global__ void __launch_bounds__(ALL, PER_SM)
    scan_kernel(const __grid_constant__ ScanArgs g, const __grid_constant__ Maps maps, bool pairs) {
    using R = Rows<TI, MODE>;
    constexpr int STAGES = 3, TENSORS = GATED ? 4 : 3, STAGE_BYTES = TENSORS * R::TILE;
    extern __shared__ __align__(128) unsigned char rows_smem[];    // [STAGES][x, r, i, z][CHUNK]
    __shared__ int2 tk[RING];                        // the tiles' places: order and column, -1 behind the last
    __shared__ float2 sG[RING][3][32];               // and gate constants
    __shared__ uint4 sBd[RING];                      // and borders
    __shared__ float2 sA[2][WARPS][32], sB[2][WARPS][32], sIn[2][WARPS][32];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    auto place_gates = [&](int slot, const Gate& k) {
        sG[slot][0][lane] = k.ea;
        sG[slot][1][lane] = k.rb;
        sG[slot][2][lane] = k.ib;
    };
    auto borders_of = [&](int2 tile) { return g.borders[max(tile.x, 0)]; };
    __shared__ uint64_t landed[STAGES];              // (MTMA) a tile's rows are there
    const uint32_t bars = ptx::smem_u32(landed);
    if (tid == 0) {
        for (int k = 0; k < STAGES; ++k) ptx::mbar_init(bars + 8 * k, 1);
        ptx::fence_mbar_init();
    }
    begin(g);
    if (tid == 0)
        for (int k = 0; k < STAGES; ++k) tk[k] = place_of(g, take_ticket(g));
    __syncthreads();
    auto load_tile = [&](int stage, int k) {         // (MTMA) by one thread
        const int2 tile = tk[k % RING];
        if (tile.x < 0) return;
        const uint32_t s = ptx::smem_u32(rows_smem) + stage * STAGE_BYTES, bar = bars + 8 * stage;
        ptx::mbar_expect_tx(bar, STAGE_BYTES);
#pragma unroll
        for (int m = 0; m < TENSORS; ++m) ptx::tma_load_2d(s + m * R::TILE, &maps.m[m], tile.y * TILE_C, tile.x * CHUNK, bar);
    };

    // The walks, even tiles' by one warp and odd ones' by the other (one warp for all was what the others
    // waited for: 151 us for 145 at 16384 tokens x 4096): maps of the tile's warps in, their first
    // values out.
    // (The shuffle tells the compiler that the lanes go together: 1 to 2 % at 65273 x 8192.)
    if (__shfl_sync(0xffffffffu, warp, 0) >= WARPS) {
        const int buf = warp - WARPS;
        if (MODE == MTMA && tid == NT)
            for (int k = 0; k < STAGES; ++k) load_tile(k, k);
        place_gates(buf, load_gate(g, tk[buf].y));
        if (lane == 0) sBd[buf] = borders_of(tk[buf]);
        __syncthreads();
        for (int k = buf;; k += 2) {
            bar_sync(READY + buf, MEET);
            const int2 tile = tk[k % RING], second = tk[(k + 2) % RING];
            if (tile.x < 0) return;
            const Gate q = load_gate(g, second.y);   // of the tile after the next
            const uint4 bd = borders_of(second);
            float2 At = sA[buf][0][lane], Bt = sB[buf][0][lane];
#pragma unroll
            for (int w = 1; w < WARPS; ++w) {
                const float2 A = sA[buf][w][lane], B = sB[buf][w][lane];
                Bt = apply(A, B, Bt);
                At = A.x < 0.f ? A : At.x < 0.f ? At : mul2(At, A);
            }
            walk_map(g, tile.x, tile.y, At, Bt);
            // (where there are few columns, and so many tiles of each under way, 8 predecessors: 32768 tokens x 512
            // channels 64 us for 97, but 16384 x 4096 158 for 139)
            float2 h = g.tiles_c <= 8 ? walk_back<8>(g, tile.x, tile.y, At, Bt) : walk_back<3>(g, tile.x, tile.y, At, Bt);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) {
                sIn[buf][w][lane] = h;
                h = apply(sA[buf][w][lane], sB[buf][w][lane], h);
            }
            place_gates((k + 2) % RING, q);
            if (lane == 0) sBd[(k + 2) % RING] = bd;
            bar_arrive(COME + buf, MEET);
            if (MODE == MTMA) {                      // tile k + 3 in the place of this one
                bar_sync(FREE + buf, MEET);
                if (lane == 0) load_tile(k % STAGES, k + STAGES);
            }
        }
    }

    unsigned char* const mine = rows_smem + warp * R::BYTES;
    const uint32_t mine_u = ptx::smem_u32(mine);
    uint32_t phases = 0;
    auto issue = [&](int stage, int k) {
        if constexpr (MODE != MTMA) {
            __syncwarp();                            // (a lane's copies come where others have read)
            const int2 tile = tk[k % RING];
            if (tile.x >= 0) {
                const int t = tile.x * CHUNK + warp * SUB, c0 = tile.y * TILE_C;
                const int rows = (int)g.T - t, cols = min(TILE_C, g.C - c0);
                const uint32_t s = mine_u + stage * STAGE_BYTES;
                R::load(s, g.x, g.x_s, t, c0, rows, cols);
                R::load(s + R::TILE, g.r, g.r_s, t, c0, rows, cols);
                R::load(s + 2 * R::TILE, g.i, g.i_s, t, c0, rows, cols);
                if (GATED) R::load(s + 3 * R::TILE, g.z, g.z_s, t, c0, rows, cols);
                if (MODE == MODD) {
                    const int m = lane / 8;
                    R::last_word(s + m * R::TILE, m == 0 ? g.x : m == 1 ? g.r : m == 2 ? g.i : GATED ? g.z : nullptr,
                                 m == 0 ? g.x_s : m == 1 ? g.r_s : m == 2 ? g.i_s : g.z_s, t, c0, rows, cols);
                }
            }
            ptx::cp_async_commit();
        }
    };
    auto wait_rows = [&](int stage) {
        if constexpr (MODE == MTMA) {
            wait_or(g, bars + 8 * stage, phases >> stage & 1);
            phases ^= 1u << stage;
        } else {
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
        }
    };
    auto seq_of = [&](const Borders& bd, int j) { return (size_t)seq_id(g.f, bd.seq + __popc((bd.start >> 1) & ((1u << j) - 1))); };

    // a and b of the warp's tokens, and its map
    auto first_sweep = [&](Pending& p, int stage, int slot, int buf) {
        p.tt = tk[slot].x;
        p.tc = tk[slot].y;
        const Gate k{sG[slot][0][lane], sG[slot][1][lane], sG[slot][2][lane]};
        const int t = p.tt * CHUNK + warp * SUB, c0 = p.tc * TILE_C, c = c0 + 2 * lane;
        p.bd = borders(g, sBd[slot], t);
        wait_rows(stage);
        const unsigned char* s = mine + stage * STAGE_BYTES;
        const typename R::Odd ox = R::odd(g.x, g.x_s, t, c0), orr = R::odd(g.r, g.r_s, t, c0), oi = R::odd(g.i, g.i_s, t, c0);
        float2 A = f2(1.f), B = f2(0.f);
        auto token = [&](int j, auto wide) {
            const Step st = step_of<decltype(wide)::value>(k, R::get(s, j, ox), R::get(s + R::TILE, j, orr),
                                                           R::get(s + 2 * R::TILE, j, oi));
            p.a[j] = st.a;
            p.b[j] = st.b;
        };
        if (any_wide(k)) {
#pragma unroll
            for (int j = 0; j < SUB; ++j) token(j, std::true_type{});
        } else {
#pragma unroll
            for (int j = 0; j < SUB; ++j) token(j, std::false_type{});
        }
        if (p.bd.start == 0) {
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                A = mul2(A, p.a[j]);
                B = fma2(p.a[j], B, p.b[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                if (p.bd.start >> j & 1) {           // (S_out, written in second sweeps, may be S_in: read here only)
                    const float2 h = pair_at(g.S_in, seq_of(p.bd, j), c, g.C);
                    if (j == 0 && warp == 0 && g.states) put(g.states + (size_t)p.tt * g.C + c, g.C - c, false, h);
                    p.b[j] = fma2(p.a[j], h, p.b[j]);
                    A = f2(-1.f);
                    B = p.b[j];
                } else {
                    A = A.x < 0.f ? A : mul2(A, p.a[j]);
                    B = fma2(p.a[j], B, p.b[j]);
                }
            }
        }
        sA[buf][warp][lane] = A;
        sB[buf][warp][lane] = B;
        bar_arrive(READY + buf, MEET);
    };
    // Where a border lies in a warp's tokens the second sweep takes other code, not at hand in the instruction
    // cache: it is short (a loop that stays one) and passes the states through shared memory, in the place
    // of the rows of x (and r), done with.  (16384 x 4096 in 128 sequences 191 us for 232.)
    auto place = [&](int stage, int j) {
        constexpr int PER = R::BYTES / 256;
        return reinterpret_cast<float2*>(mine + stage * STAGE_BYTES + j / PER * R::TILE + j % PER * 256 + lane * 8);
    };
    // the states and outputs of a tile, once its first value is there
    auto second_sweep = [&](const Pending& p, int stage, int buf) {
        const int t = p.tt * CHUNK + warp * SUB, c0 = p.tc * TILE_C, c = c0 + 2 * lane, left = g.C - c, rows = (int)g.T - t;
        const unsigned char* s = mine + stage * STAGE_BYTES + 3 * R::TILE;
        const typename R::Odd oz = R::odd(g.z, g.z_s, t, c0);
        char* o = row_at<TI>(g.o, g.o_s, t, c);
        const bool pair = pairs && left > 1, whole = pairs && c0 + TILE_C <= g.C && rows >= SUB && (p.bd.start | p.bd.end) == 0;
        bar_sync(COME + buf, MEET);
        float2 h = sIn[buf][warp][lane];
        if (g.states && warp == 0 && !(p.bd.start & 1)) put(g.states + (size_t)p.tt * g.C + c, left, false, h);
        if (__shfl_sync(0xffffffffu, (int)whole, 0)) {   // (as above: 959 us for 964)
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                h = fma2(p.a[j], h, p.b[j]);
                put<TI>(o, 2, true, GATED ? mul2(h, silu(R::get(s, j, oz))) : h);
                o += g.o_s;
            }
        } else {
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                h = p.bd.start >> j & 1 ? p.b[j] : fma2(p.a[j], h, p.b[j]);
                *place(stage, j) = h;
            }
#pragma unroll 1
            for (int j = 0; j < SUB && j < rows; ++j) {
                h = *place(stage, j);
                put<TI>(o, left, pair, GATED ? mul2(h, silu(R::get(s, j, oz))) : h);
                o += g.o_s;
                if (p.bd.end >> j & 1) put(g.S_out + seq_of(p.bd, j) * g.C + c, left, false, h);
            }
            __syncwarp();
            if (MODE == MTMA) ptx::fence_async_smem();   // (the next rows come here)
        }
    };

    // Tile k's second sweep follows the first of tile k + 1, so the walk has the time of a whole
    // tile; then the rows of tile k + 3 take the place of its own.
    for (int k = 0; k < STAGES; ++k) issue(k, k);
    uint32_t ticket = 0;                             // of tile k + 3, taken an iteration ahead
    if (tid == 0) ticket = take_ticket(g);
    __syncthreads();                                 // (the first tiles' gate constants)
    Pending p[2];
    int stage = 0;
    if (tk[0].x >= 0) first_sweep(p[0], 0, 0, 0);
    else bar_arrive(READY, MEET);
    for (int k0 = 0;; k0 += 2) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {       // tile k in p[half], tile k + 1 in p[half ^ 1]
            const int k = k0 + half, after = stage + 1 == STAGES ? 0 : stage + 1;
            if (tk[k % RING].x < 0) {                // no more: the other walk ends too
                bar_arrive(READY + (half ^ 1), MEET);
                return;
            }
            if (tid == 0) {
                tk[(k + 3) % RING] = place_of(g, ticket);
                ticket = take_ticket(g);
            }
            if (tk[(k + 1) % RING].x >= 0) first_sweep(p[half ^ 1], after, (k + 1) % RING, half ^ 1);
            else bar_arrive(READY + (half ^ 1), MEET);
            second_sweep(p[half], stage, half);
            if (MODE == MTMA) bar_arrive(FREE + half, MEET);
            issue(stage, k + STAGES);
            stage = after;
        }
    }
}

template <typename TI, int MODE, bool GATED>
cudaError_t scan(const ScanArgs& a, bool pairs, cudaStream_t s) {
    Maps maps;
    if (MODE == MTMA) {
        constexpr int es = sizeof(TI);
        if (!encode(&maps.m[0], a.x, a.x_s, es, a) || !encode(&maps.m[1], a.r, a.r_s, es, a) ||
            !encode(&maps.m[2], a.i, a.i_s, es, a) || (GATED && !encode(&maps.m[3], a.z, a.z_s, es, a)))
            return cudaErrorUnknown;
    }
    constexpr int PER_SM = sizeof(TI) == 2 ? 2 : 1;
    auto k = scan_kernel<TI, MODE, GATED, PER_SM>;
    constexpr int SMEM = 3 * (GATED ? 4 : 3) * Rows<TI, MODE>::TILE;
    static std::atomic<int> most[64];
    bool alone;
    return launch_walk(k, most, a, ALL, SMEM, s, &alone, maps, pairs);
}

template <typename TI, int MODE> cudaError_t scan(const ScanArgs& a, bool pairs, cudaStream_t s) {
    return a.z ? scan<TI, MODE, true>(a, pairs, s) : scan<TI, MODE, false>(a, pairs, s);
}

}  // namespace

__global__ void __launch_bounds__(256) setup_kernel(const __grid_constant__ ScanArgs g) {
    cudaTriggerProgrammaticLaunchCompletion();
    set_up(g);
}

cudaError_t launch_scan(const ScanArgs& a, int io_bf16, cudaStream_t s) {
    const int es = io_bf16 ? 2 : 4;
    const int mode = std::max({row_mode(a.x, a.x_s, a.C), row_mode(a.r, a.r_s, a.C), row_mode(a.i, a.i_s, a.C),
                               a.z ? row_mode(a.z, a.z_s, a.C) : 0});
    const bool pairs = row_pairs(a.o, a.o_s, es);
    if (!io_bf16) return mode == MTMA ? scan<float, MTMA>(a, pairs, s) : scan<float, M4>(a, pairs, s);
    return mode == MTMA ? scan<__nv_bfloat16, MTMA>(a, pairs, s)
         : mode == M4 ? scan<__nv_bfloat16, M4>(a, pairs, s) : scan<__nv_bfloat16, MODD>(a, pairs, s);
}

}  // namespace glr
}  // namespace kda
