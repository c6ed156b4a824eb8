// Backward pass of the gated linear recurrence.  With m = sqrt(1 - a^2),
// b = m v x and G = do SiLU(z):
//   g_t = G_t + a_{t+1} g_{t+1}            (the last token of a sequence: + dS_out)
//   dz = do h SiLU'(z)      dx = g m v      di = g b (1 - v)
//   dla = g (a h_{t-1} - (a / m)^2 b)       dr = dla la (1 - w)
//   dA_log = sum dla la,  dr_bias = sum dr,  di_bias = sum di,  dS_in = a_1 g_1
//
// The prefill's tiles (glr_scan.cu), walked from the last to the first.  The
// states of a tile come from the one the prefill left at its first token: a
// thread's forward run meets the earlier warps' maps in shared memory and waits
// for nothing, while one warp walks along the tiles for the gradient a g that comes
// in from the right.  What the gates give is computed once and held in
// registers between the sweeps.  Sums over the tokens go to the workspace by tile
// and are added up in order when all tiles are done.
//
// 16384 tokens x 4096, bf16: 264 us (4.6 TB/s of a copy's 6.8), 32768 x 4096: 484 to 490 (5.0).  Issue
// slots 57 %, memory 61 %: with two CTAs of 8 warps an SM (registers) one other CTA covers the
// waits at a barrier.  Without the walk 253 us of then 292, without arithmetic 251, without the stores 195.
#include <type_traits>

#include "glr_tile.cuh"

namespace kda {
namespace glr {
namespace {

enum { OUT_X = 1, OUT_R = 2, OUT_I = 4, OUT_Z = 8 };   // gradients whose rows take pairs

// The parameters' gradients: the tiles' sums, added up in order with the error of each
// addition kept (Knuth's two-sum).  A CTA takes 32 channels of one gradient, its 8 warps every
// eighth tile.
__device__ __forceinline__ void add_up(const ScanArgs& g, float2 (&part)[WARPS][32]) {
    const int w = threadIdx.x / 32, lane = threadIdx.x % 32, units = (g.C + 31) / 32 * 3;
    for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int c = unit / 3 * 32 + lane, q = unit % 3;
        float* out = q == 0 ? g.dA_log : q == 1 ? g.dr_bias : g.di_bias;
        if (out == nullptr) continue;
        float s = 0.f, err = 0.f;
        auto add = [&](float x) {
            const float n = __fadd_rn(s, x), b = __fsub_rn(n, s);
            err += __fadd_rn(__fsub_rn(s, __fsub_rn(n, b)), __fsub_rn(x, b));
            s = n;
        };
        if (c < g.C) {
#pragma unroll 16
            for (int tt = w; tt < g.tiles_t; tt += WARPS) add(__ldcg(g.part + ((size_t)tt * 3 + q) * g.C + c));
        }
        part[w][lane] = make_float2(s, err);
        __syncthreads();
        if (w == 0 && c < g.C) {
            for (int u = 1; u < WARPS; ++u) {
                add(part[u][lane].x);
                err += part[u][lane].y;
            }
            out[c] = s + err;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(NT) add_up_kernel(const __grid_constant__ ScanArgs g) {
    __shared__ float2 part[WARPS][32];
    add_up(g, part);
}

template <typename TI, int MODE, bool GATED, int STAGES, int PER_SM>
__global__ void __launch_bounds__(NT, PER_SM)
    backward_kernel(const __grid_constant__ ScanArgs g, const __grid_constant__ Maps maps, int pairs) {
    using R = Rows<TI, MODE>;
    constexpr int TENSORS = GATED ? 5 : 4, STAGE_BYTES = TENSORS * R::TILE;
    extern __shared__ __align__(128) unsigned char rows_smem[];    // [STAGES][x, r, i, do, z][CHUNK]
    __shared__ int2 tk[STAGES];
    __shared__ __align__(16) float2 sG[STAGES][3][32];             // the tiles' gate constants
    __shared__ uint4 sBd[STAGES];                                  // and borders
    __shared__ uint64_t landed[STAGES];                            // (MTMA) a tile's rows and these are there
    __shared__ float2 sA[WARPS][32], sB[WARPS][32], sAr[WARPS][32], sBr[WARPS][32];   // maps forwards and backwards
    __shared__ float2 sIn[32], sH[STAGES][32], sums[3][WARPS][32];
    const int tid = threadIdx.x, lane = tid % 32;
    // (the same in all lanes, which the compiler cannot see from tid / 32: 492 us for 546 at 32768 x 4096)
    const int warp = __shfl_sync(0xffffffffu, tid / 32, 0);
    unsigned char* const mine = rows_smem + warp * R::BYTES;
    const uint32_t bars = ptx::smem_u32(landed);
    uint32_t phases = 0;
    // (MTMA) The tile's rows and gate constants, by one thread.
    auto load_tile = [&](int stage) {
        const int2 tile = tk[stage];
        if (tile.x < 0) return;
        const uint32_t s = ptx::smem_u32(rows_smem) + stage * STAGE_BYTES, bar = bars + 8 * stage;
        ptx::mbar_expect_tx(bar, STAGE_BYTES + sizeof sG[0] + sizeof sBd[0]);
#pragma unroll
        for (int m = 0; m < TENSORS; ++m)
            ptx::tma_load_2d(s + m * R::TILE, &maps.m[m], tile.y * TILE_C, (g.tiles_t - 1 - tile.x) * CHUNK, bar);
        ptx::bulk_g2s(ptx::smem_u32(&sBd[stage]), g.borders + (g.tiles_t - 1 - tile.x), sizeof sBd[0], bar);
        ptx::bulk_g2s(ptx::smem_u32(&sG[stage][0][0]), g.gates + (size_t)tile.y * (3 * TILE_C / 2), sizeof sG[0], bar);
    };
    // Each warp: its own rows (not MTMA); the last warp: the tile's first state.
    auto issue = [&](int stage) {
        const int2 tile = tk[stage];
        if (tile.x >= 0) {
            const int tt = g.tiles_t - 1 - tile.x, t = tt * CHUNK + warp * SUB, c0 = tile.y * TILE_C;
            const int rows = (int)g.T - t, cols = min(TILE_C, g.C - c0);
            if constexpr (MODE != MTMA) {
                __syncwarp();                        // (a lane's copies come where others have read)
                const uint32_t s = ptx::smem_u32(mine) + stage * STAGE_BYTES;
                R::load(s, g.x, g.x_s, t, c0, rows, cols);
                R::load(s + R::TILE, g.r, g.r_s, t, c0, rows, cols);
                R::load(s + 2 * R::TILE, g.i, g.i_s, t, c0, rows, cols);
                R::load(s + 3 * R::TILE, g.d_o, g.do_s, t, c0, rows, cols);
                if (GATED) R::load(s + 4 * R::TILE, g.z, g.z_s, t, c0, rows, cols);
                if (MODE == MODD) {
                    const int m = lane / 8;
                    R::last_word(s + m * R::TILE, m == 0 ? g.x : m == 1 ? g.r : m == 2 ? g.i : g.d_o,
                                 m == 0 ? g.x_s : m == 1 ? g.r_s : m == 2 ? g.i_s : g.do_s, t, c0, rows, cols);
                    if (GATED && m == 0) R::last_word(s + 4 * R::TILE, g.z, g.z_s, t, c0, rows, cols);
                }
            }
            if (warp == WARPS - 1) {
                const uint32_t h = ptx::smem_u32(&sH[stage][0]);
                const float* p = g.states + (size_t)tt * g.C + c0;
#pragma unroll
                for (int k = lane; k < TILE_C; k += 32)
                    R::template copy<4>(h + k * 4, reinterpret_cast<const char*>(k < cols ? p + k : g.states), k < cols ? 4 : 0);
            }
        }
        ptx::cp_async_commit();
    };
    if (tid == 0) {
        for (int k = 0; k < STAGES; ++k) ptx::mbar_init(bars + 8 * k, 1);
        ptx::fence_mbar_init();
    }
    begin(g);
    if (tid == 0)
        for (int k = 0; k < STAGES; ++k) tk[k] = place_of(g, take_ticket(g));
    __syncthreads();
    if (MODE == MTMA && tid == NT - 1) {
        asm volatile("fence.proxy.async;" ::: "memory");           // (the constants were written by ordinary stores)
        for (int k = 0; k < STAGES; ++k) load_tile(k);
    }
    for (int k = 0; k < STAGES; ++k) issue(k);

    for (int stage = 0;; stage = stage + 1 == STAGES ? 0 : stage + 1) {
        const int order = tk[stage].x, tc = tk[stage].y, tt = g.tiles_t - 1 - order;
        if (order < 0) break;
        const int t = tt * CHUNK + warp * SUB, c0 = tc * TILE_C, c = c0 + 2 * lane, rows = (int)g.T - t, left = g.C - c;
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        __syncwarp();
        if (MODE == MTMA) {
            wait_or(g, bars + 8 * stage, phases >> stage & 1);
            phases ^= 1u << stage;
        }
        const Borders bd = borders(g, MODE == MTMA ? sBd[stage] : g.borders[tt], t);
        auto seq_of = [&](int j) { return (size_t)seq_id(g.f, bd.seq + __popc((bd.start >> 1) & ((1u << j) - 1))); };
        const Gate k = MODE == MTMA ? Gate{sG[stage][0][lane], sG[stage][1][lane], sG[stage][2][lane]} : load_gate(g, tc);

        unsigned char* const s = mine + stage * STAGE_BYTES;
        const typename R::Odd ox = R::odd(g.x, g.x_s, t, c0), orr = R::odd(g.r, g.r_s, t, c0), oi = R::odd(g.i, g.i_s, t, c0),
                              od = R::odd(g.d_o, g.do_s, t, c0), oz = R::odd(g.z, g.z_s, t, c0);
        auto x_of = [&](int j) { return R::get(s, j, ox); };
        auto r_of = [&](int j) { return fma2(R::get(s + R::TILE, j, orr), f2(-LOG2E), k.rb); };
        // Of each token: a, w, -E = -m v, x (1 - v), K = a (v / m) x, -G.  States and gradients run with
        // the sign changed, as -E and -G lead to them; what is stored has two such factors.
        float2 a[SUB], w[SUB], nE[SUB], xv[SUB], K[SUB], nG[SUB];
        float2 A = f2(1.f), nB = f2(0.f);
        auto token = [&](int j, auto wide) {
            w[j] = sigmoid_of(r_of(j));
            const float2 ei = ex2_most(fma2(R::get(s + 2 * R::TILE, j, oi), f2(-LOG2E), k.ib)), di = add2(ei, f2(1.f));
            const float2 v = make_float2(rcp(di.x), rcp(di.y)), x = x_of(j);
            xv[j] = mul2(x, mul2(ei, v));
            float2 nm2;
            decay_of<decltype(wide)::value>(mul2(k.ea, w[j]), a[j], nm2);
            const float2 iv = mul2(inv_root(nm2), v);
            nE[j] = mul2(nm2, iv);
            K[j] = mul2(mul2(a[j], iv), x);
            const float2 dO = R::get(s + 3 * R::TILE, j, od);
            if (GATED) {
                const float2 z = R::get(s + 4 * R::TILE, j, oz), tz = mul2(z, f2(-LOG2E));
                const float2 dd = fma2(make_float2(ex2(tz.x), ex2(tz.y)), f2(-1.f), f2(-1.f)), ne = make_float2(rcp(dd.x), rcp(dd.y));
                nG[j] = mul2(dO, mul2(z, ne));
                // -do SiLU'(z), for dz = do SiLU'(z) h
                R::keep(s + 3 * R::TILE, s + 4 * R::TILE, j, mul2(dO, mul2(ne, fma2(z, add2(ne, f2(1.f)), f2(1.f)))));
            } else {
                nG[j] = mul2(dO, f2(-1.f));
            }
        };
        if (any_wide(k)) {
#pragma unroll
            for (int j = 0; j < SUB; ++j) token(j, std::true_type{});
        } else {
#pragma unroll
            for (int j = 0; j < SUB; ++j) token(j, std::false_type{});
        }
        float2 Ar = f2(1.f), nBr = f2(0.f);
        const bool plain = (bd.start | bd.end) == 0;
        if (plain) {
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                A = mul2(A, a[j]);
                nB = fma2(a[j], nB, mul2(nE[j], x_of(j)));
            }
            Ar = A;
#pragma unroll
            for (int j = SUB - 1; j >= 0; --j) nBr = mul2(a[j], add2(nG[j], nBr));
        } else {
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                const float2 nb = mul2(nE[j], x_of(j));
                if (bd.start >> j & 1) {
                    A = f2(-1.f);
                    nB = fma2(a[j], neg2(pair_at(g.S_in, seq_of(j), c, g.C)), nb);
                } else {
                    A = A.x < 0.f ? A : mul2(A, a[j]);
                    nB = fma2(a[j], nB, nb);
                }
            }
#pragma unroll
            for (int j = SUB - 1; j >= 0; --j) {
                if (bd.end >> j & 1) {
                    Ar = f2(-1.f);
                    nBr = neg2(pair_at(g.dS_out, seq_of(j), c, g.C));
                } else if (Ar.x >= 0.f) {
                    Ar = mul2(Ar, a[j]);
                }
                nBr = mul2(a[j], add2(nG[j], nBr));
            }
        }
        sA[warp][lane] = A;
        sB[warp][lane] = nB;
        sAr[warp][lane] = Ar;
        sBr[warp][lane] = nBr;
        __syncthreads();
        float2 nh = neg2(sH[stage][lane]);
        if (warp == 0) {
            Ar = sAr[WARPS - 1][lane];
            nBr = sBr[WARPS - 1][lane];
#pragma unroll
            for (int u = WARPS - 2; u >= 0; --u) {
                const float2 Aw = sAr[u][lane], Bw = sBr[u][lane];
                nBr = apply(Aw, Bw, nBr);
                Ar = Aw.x < 0.f ? Aw : Ar.x < 0.f ? Ar : mul2(Ar, Aw);
            }
            walk_map(g, order, tc, Ar, nBr);
        } else if (tid == 32) {
            tk[stage] = place_of(g, take_ticket(g));
        }
        for (int u = 0; u < warp; ++u) nh = apply(sA[u][lane], sB[u][lane], nh);
        const bool full = pairs == (GATED ? OUT_X | OUT_R | OUT_I | OUT_Z : OUT_X | OUT_R | OUT_I) && c0 + TILE_C <= g.C;
        const bool whole = __shfl_sync(0xffffffffu, (int)(plain && full && rows >= SUB), 0);   // (as `warp`: 484 us for 496)
        char* dz = GATED ? row_at<TI>(g.dz, g.dz_s, t, c) : nullptr;
        auto forward = [&](auto fast) {              // K becomes -dA_log / g
            constexpr bool FAST = decltype(fast)::value;
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                if (!FAST && (bd.start >> j & 1)) nh = neg2(pair_at(g.S_in, seq_of(j), c, g.C));
                K[j] = mul2(mul2(mul2(k.ea, w[j]), a[j]), add2(K[j], nh));
                nh = fma2(nE[j], x_of(j), mul2(a[j], nh));
                if (GATED && (FAST || j < rows))
                    put<TI>(dz, FAST ? 2 : left, FAST || ((pairs & OUT_Z) && left > 1),
                            mul2(R::kept(s + 3 * R::TILE, s + 4 * R::TILE, j), nh));
                if (GATED) dz += g.dz_s;
            }
        };
        if (whole) forward(std::true_type{});
        else forward(std::false_type{});
        // (the first warp's own states come before its look back: by then the value is mostly there)
        if (warp == 0) sIn[lane] = walk_back<3>(g, order, tc, Ar, nBr);   // (8 cost registers: 612 us for then 545)
        __syncthreads();
        float2 carry = sIn[lane], sa = f2(0.f), sr = f2(0.f), si = f2(0.f);
        for (int u = WARPS - 1; u > warp; --u) carry = apply(sAr[u][lane], sBr[u][lane], carry);
        char *dx = row_at<TI>(g.dx, g.dx_s, t + SUB - 1, c), *dr = row_at<TI>(g.dr, g.dr_s, t + SUB - 1, c),
             *di = row_at<TI>(g.di, g.di_s, t + SUB - 1, c);
        auto backward = [&](auto fast) {
            constexpr bool FAST = decltype(fast)::value;
#pragma unroll
            for (int j = SUB - 1; j >= 0; --j) {
                if (!FAST && (bd.end >> j & 1)) carry = neg2(pair_at(g.dS_out, seq_of(j), c, g.C));
                const float2 ng = add2(nG[j], carry), gx = mul2(ng, nE[j]), gi = mul2(gx, xv[j]), gA = mul2(ng, K[j]);
                carry = mul2(a[j], ng);
                const float2 gr = mul2(gA, mul2(ex2_most(r_of(j)), w[j]));
                if (FAST || j < rows) {
                    put<TI>(dx, FAST ? 2 : left, FAST || ((pairs & OUT_X) && left > 1), gx);
                    put<TI>(dr, FAST ? 2 : left, FAST || ((pairs & OUT_R) && left > 1), gr);
                    put<TI>(di, FAST ? 2 : left, FAST || ((pairs & OUT_I) && left > 1), gi);
                    sa = add2(sa, gA);
                    sr = add2(sr, gr);
                    si = add2(si, gi);
                }
                dx -= g.dx_s;
                dr -= g.dr_s;
                di -= g.di_s;
                if (!FAST && g.dS_in && (bd.start >> j & 1)) put(g.dS_in + seq_of(j) * g.C + c, left, false, neg2(carry));
            }
        };
        if (whole) backward(std::true_type{});
        else backward(std::false_type{});
        issue(stage);                                // (the warp has read its rows, and all of them the state)
        if (MODE == MTMA) ptx::fence_async_smem();   // (it has also written on them)
        sums[0][warp][lane] = sa;
        sums[1][warp][lane] = sr;
        sums[2][warp][lane] = si;
        __syncthreads();
        if (MODE == MTMA && tid == NT - 1) load_tile(stage);
        if (tid < 96) {
            const int q = tid / 32;
            float2 sum = sums[q][0][lane];
#pragma unroll
            for (int u = 1; u < WARPS; ++u) sum = add2(sum, sums[q][u][lane]);
            put(g.part + ((size_t)tt * 3 + q) * g.C + c, left, false, sum);
        }
    }
    if (g.alone) {
        cooperative_groups::this_grid().sync();
        add_up(g, sums[0]);
    }
}

template <typename TI, int MODE, bool GATED>
cudaError_t backward(const ScanArgs& a, int pairs, cudaStream_t s) {
    Maps maps;
    if (MODE == MTMA) {
        constexpr int es = sizeof(TI);
        if (!encode(&maps.m[0], a.x, a.x_s, es, a) || !encode(&maps.m[1], a.r, a.r_s, es, a) ||
            !encode(&maps.m[2], a.i, a.i_s, es, a) || !encode(&maps.m[3], a.d_o, a.do_s, es, a) ||
            (GATED && !encode(&maps.m[4], a.z, a.z_s, es, a)))
            return cudaErrorUnknown;
    }
    constexpr int STAGES = sizeof(TI) == 2 ? 2 : 1, PER_SM = 2;
    auto k = backward_kernel<TI, MODE, GATED, STAGES, PER_SM>;
    constexpr int SMEM = STAGES * (GATED ? 5 : 4) * Rows<TI, MODE>::TILE;
    static std::atomic<int> most[64];
    bool alone;
    const cudaError_t e = launch_walk(k, most, a, NT, SMEM, s, &alone, maps, pairs);
    if (e != cudaSuccess || alone) return e;
    add_up_kernel<<<(unsigned)((a.C + 31) / 32 * 3), NT, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename TI, int MODE> cudaError_t backward(const ScanArgs& a, int pairs, cudaStream_t s) {
    return a.z ? backward<TI, MODE, true>(a, pairs, s) : backward<TI, MODE, false>(a, pairs, s);
}

}  // namespace

cudaError_t launch_backward(const ScanArgs& a, int io_bf16, cudaStream_t s) {
    const int es = io_bf16 ? 2 : 4;
    const int mode = std::max({row_mode(a.x, a.x_s, a.C), row_mode(a.r, a.r_s, a.C), row_mode(a.i, a.i_s, a.C),
                               row_mode(a.d_o, a.do_s, a.C), a.z ? row_mode(a.z, a.z_s, a.C) : 0});
    const int pairs = (row_pairs(a.dx, a.dx_s, es) ? OUT_X : 0) | (row_pairs(a.dr, a.dr_s, es) ? OUT_R : 0) |
                      (row_pairs(a.di, a.di_s, es) ? OUT_I : 0) | (a.z && row_pairs(a.dz, a.dz_s, es) ? OUT_Z : 0);
    if (!io_bf16) return mode == MTMA ? backward<float, MTMA>(a, pairs, s) : backward<float, M4>(a, pairs, s);
    return mode == MTMA ? backward<__nv_bfloat16, MTMA>(a, pairs, s)
         : mode == M4 ? backward<__nv_bfloat16, M4>(a, pairs, s) : backward<__nv_bfloat16, MODD>(a, pairs, s);
}

}  // namespace glr
}  // namespace kda
