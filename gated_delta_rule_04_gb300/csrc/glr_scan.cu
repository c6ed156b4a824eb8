// Prefill of the gated linear recurrence: h_t = a_t h_{t-1} + m_t v_t x_t,
// o_t = h_t SiLU(z_t), with m = sqrt(1 - a^2).
//
// One pass over the data.  Tiles of 64 tokens x 64 channels lie in shared memory
// in their own type, copied some tiles ahead; a thread holds 8 tokens of 2
// channels, computes their a and b = m v x once, and the map h -> A h + B of its
// run.  The maps meet in shared memory, the tile's value comes from the walk along
// the tiles (glr_tile.cuh), and the second sweep over the 8 tokens is one multiply-add
// a token and the output gate.  Sequences lie anywhere in the tiles: a token
// that begins one starts its run anew from S_in.
#include <atomic>
#include <type_traits>

#include "glr_tile.cuh"

namespace kda {
namespace glr {
namespace {

template <typename TI, int MODE, int STAGES, int PER_SM>
__global__ void __launch_bounds__(NT, PER_SM) scan_kernel(const __grid_constant__ ScanArgs g, bool pairs) {
    using R = Rows<TI, MODE>;
    extern __shared__ __align__(128) unsigned char rows_smem[];    // [WARPS][STAGES][x, r, i, z]
    __shared__ uint32_t tk[STAGES];
    __shared__ float2 sA[2][WARPS][32], sB[2][WARPS][32], sIn[2][32];
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const uint32_t tiles = (uint32_t)g.tiles_t * (uint32_t)g.tiles_c;
    unsigned char* const mine = rows_smem + warp * STAGES * 4 * R::BYTES;
    const uint32_t mine_u = ptx::smem_u32(mine);
    auto issue = [&](int stage, uint32_t tile) {
        if (tile < tiles) {
            const int64_t t = (int64_t)(tile / g.tiles_c) * CHUNK + warp * SUB;
            const int c0 = (int)(tile % g.tiles_c) * TILE_C;
            const int rows = (int)min((int64_t)SUB, g.T - t), cols = min(TILE_C, g.C - c0);
            const uint32_t s = mine_u + stage * 4 * R::BYTES;
            R::load(s, g.x, g.x_s, t, c0, rows, cols);
            R::load(s + R::BYTES, g.r, g.r_s, t, c0, rows, cols);
            R::load(s + 2 * R::BYTES, g.i, g.i_s, t, c0, rows, cols);
            if (g.z) R::load(s + 3 * R::BYTES, g.z, g.z_s, t, c0, rows, cols);
        }
        ptx::cp_async_commit();
    };
    if (tid == 0)
        for (int k = 0; k < STAGES; ++k) tk[k] = next_ticket(g);
    __syncthreads();
    if (tk[0] == 0 && tid == 0) *g.status = ERR_NONE;
    for (int k = 0; k < STAGES; ++k) issue(k, tk[k]);

    int buf = 0;
    for (int stage = 0;; stage = stage + 1 == STAGES ? 0 : stage + 1, buf ^= 1) {
        const uint32_t tile = tk[stage];
        if (tile >= tiles) break;                    // (tickets only grow)
        const int tt = tile / g.tiles_c, tc = tile % g.tiles_c;
        const int64_t t = (int64_t)tt * CHUNK + warp * SUB;
        const int c0 = tc * TILE_C, c = c0 + 2 * lane, rows = (int)min((int64_t)SUB, g.T - t);
        const Gate k = load_gate(g, c);
        const Borders bd = borders(g, tt, t);
        auto seq_of = [&](int j) { return (size_t)seq_id(g.f, bd.seq + __popc((bd.start >> 1) & ((1u << j) - 1))); };
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        __syncwarp();

        const unsigned char* s = mine + stage * 4 * R::BYTES;
        float2 a[SUB], b[SUB], A = f2(1.f), B = f2(0.f), first = f2(0.f);
        const typename R::Odd ox = R::odd(g.x, g.x_s, t, c0), orr = R::odd(g.r, g.r_s, t, c0), oi = R::odd(g.i, g.i_s, t, c0);
        auto token = [&](int j, auto wide) {
            const Step st = step_of<decltype(wide)::value>(k, R::get(s, j, ox), R::get(s + R::BYTES, j, orr),
                                                           R::get(s + 2 * R::BYTES, j, oi));
            a[j] = st.a;
            b[j] = st.b;
        };
        if (any_wide(k)) {
#pragma unroll
            for (int j = 0; j < SUB; ++j) token(j, std::true_type{});
        } else {
#pragma unroll
            for (int j = 0; j < SUB; ++j) token(j, std::false_type{});
        }
        if (bd.start == 0) {
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                A = mul2(A, a[j]);
                B = fma2(a[j], B, b[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                if (bd.start >> j & 1) {
                    const float2 h = pair_at(g.S_in, seq_of(j), c, g.C);   // (S_out, written behind the barriers, may be S_in)
                    if (j == 0) first = h;
                    b[j] = fma2(a[j], h, b[j]);
                    A = f2(-1.f);
                    B = b[j];
                } else {
                    A = A.x < 0.f ? A : mul2(A, a[j]);
                    B = fma2(a[j], B, b[j]);
                }
            }
        }
        sA[buf][warp][lane] = A;
        sB[buf][warp][lane] = B;
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int w = 1; w < WARPS; ++w) {
                const float2 Aw = sA[buf][w][lane], Bw = sB[buf][w][lane];
                B = apply(Aw, Bw, B);
                A = Aw.x < 0.f ? Aw : A.x < 0.f ? A : mul2(A, Aw);
            }
            sIn[buf][lane] = walk(g, tt, tc, A, B);
        } else if (tid == 32) {
            tk[stage] = next_ticket(g);
        }
        float2 gate[SUB];
        if (g.z) {
            const typename R::Odd oz = R::odd(g.z, g.z_s, t, c0);
#pragma unroll
            for (int j = 0; j < SUB; ++j) gate[j] = silu(R::get(s + 3 * R::BYTES, j, oz));
        }
        __syncthreads();
        issue(stage, tk[stage]);                     // (the warp has read its rows)
        float2 h = sIn[buf][lane];
        if (g.states && warp == 0) put(g.states + (size_t)tt * g.C + c, g.C - c, false, bd.start & 1 ? first : h);
        for (int w = 0; w < warp; ++w) h = apply(sA[buf][w][lane], sB[buf][w][lane], h);
        TI* o = static_cast<TI*>(g.o) + t * g.C + c;
        const bool pair = pairs && c + 1 < g.C;
        if ((bd.start | bd.end) == 0 && rows == SUB) {
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                h = fma2(a[j], h, b[j]);
                put(o, g.C - c, pair, g.z ? mul2(h, gate[j]) : h);
                o += g.C;
            }
        } else {
#pragma unroll
            for (int j = 0; j < SUB; ++j) {
                h = bd.start >> j & 1 ? b[j] : fma2(a[j], h, b[j]);
                if (j < rows) put(o, g.C - c, pair, g.z ? mul2(h, gate[j]) : h);
                if (bd.end >> j & 1) put(g.S_out + seq_of(j) * g.C + c, g.C - c, false, h);
                o += g.C;
            }
        }
    }
}

template <typename TI, int MODE>
cudaError_t scan(const ScanArgs& a, bool pairs, cudaStream_t s) {
    constexpr int STAGES = sizeof(TI) == 2 ? 2 : 1, PER_SM = 3;
    auto k = scan_kernel<TI, MODE, STAGES, PER_SM>;
    constexpr int SMEM = WARPS * STAGES * 4 * Rows<TI, MODE>::BYTES;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> done{0};            // (set once per device)
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(done.load() & bit)) {
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit);
    }
    const int64_t tiles = (int64_t)a.tiles_t * a.tiles_c;
    k<<<(unsigned)(tiles < SMS * PER_SM ? tiles : SMS * PER_SM), NT, SMEM, s>>>(a, pairs);
    return cudaGetLastError();
}

// The first sequence of each tile along T: the last one that begins at or before its first token.
__global__ void __launch_bounds__(NT) tile_table_kernel(const int64_t* cu, int n, int32_t* table, int tiles) {
    const int tt = blockIdx.x * NT + threadIdx.x;
    if (tt >= tiles) return;
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= (int64_t)tt * CHUNK) lo = mid; else hi = mid - 1;
    }
    table[tt] = lo;
}

}  // namespace

cudaError_t launch_tile_table(const int64_t* d_cu, int32_t n, int32_t* d_tile, int32_t tiles_t, cudaStream_t s) {
    tile_table_kernel<<<(unsigned)((tiles_t + NT - 1) / NT), NT, 0, s>>>(d_cu, n, d_tile, tiles_t);
    return cudaGetLastError();
}

cudaError_t launch_scan(const ScanArgs& a, int io_bf16, cudaStream_t s) {
    const int es = io_bf16 ? 2 : 4;
    const int mode = std::max({row_mode(a.x, a.x_s, es), row_mode(a.r, a.r_s, es), row_mode(a.i, a.i_s, es),
                               a.z ? row_mode(a.z, a.z_s, es) : 0});
    const bool pairs = row_pairs(a.o, a.C, es);
    if (!io_bf16) return mode == M16 ? scan<float, M16>(a, pairs, s) : scan<float, M4>(a, pairs, s);
    return mode == M16 ? scan<__nv_bfloat16, M16>(a, pairs, s)
         : mode == M4 ? scan<__nv_bfloat16, M4>(a, pairs, s) : scan<__nv_bfloat16, MODD>(a, pairs, s);
}

}  // namespace glr
}  // namespace kda
