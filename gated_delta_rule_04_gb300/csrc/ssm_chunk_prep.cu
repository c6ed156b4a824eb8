// Chunk preparation of the state space mixer's chunked prefill: everything of
// a 64-token chunk that its heads share, and the steps' cumulative decays.
//
// Blocks (chunk, group): conv + SiLU of the group's B and C, their tiles in
// the consumer's layout and G = C B^T on the tensor cores (tcgen05, M = 128:
// rows 64-127 read the memory behind the 64 rows of C, their lanes of the
// result are not used).  A record is 56 KiB at N = 128 and serves every head
// of the group, so its conv and its G are computed once instead of per head.
// The other blocks (chunk, 32 heads): dt = softplus(.), its cumulative sum
// times -exp(A_log) in log2 units, a warp per head.
//
// B reaches the fp32 state, whose error the operands' rounding would set: B'
// goes out as an fp16 pair (22 bits).  C and G reach bf16 outputs only and are
// rounded once to fp16's 11 bits; bf16's 8 would be as coarse as the output.
//
// 32768 tokens, 96 heads, 8 groups, N = 128: 155 us for 218 MB of records and 0.15
// GB of inputs, 0.35 of the measured copy rate.  Bound by latency: two blocks of 16
// warps an SM issue 44 % of the time, the rest is raw rows (each thread's 16 in
// flight at once) and the barriers of a short block (a block alone takes 4.8 us, 1.9 of
// them conv).  A thread per channel with 256-thread blocks took 205 us.
#include <type_traits>

#include "ssm_chunk.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace ssm {
namespace {

constexpr int NT = 512;
constexpr int HB = 32;                     // heads of a step block: two a warp
constexpr uint32_t TMEM_COLS = 64;
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr float LOG2E = 1.4426950408889634f;

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ void steps(const ChunkArgs& a, const ChunkDesc d, int chunk, int hb, float (*sdt)[HB + 1]) {
    const PrefillArgs& g = a.g;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const __nv_bfloat16* dts = static_cast<const __nv_bfloat16*>(g.dt);
    const int h_base = hb * HB, heads = min(HB, g.H - h_base);
    // dt of every (token, head): rows of the block's heads, read side by side
    for (int i = threadIdx.x; i < CHUNK_T * HB; i += NT) {
        const int t = i / HB, hh = i % HB;
        if (hh < heads)
            sdt[t][hh] = t < d.len ? softplus(to_f32(dts[(int64_t)(d.t0 + t) * g.dt_stride + h_base + hh]) + g.dt_bias[h_base + hh]) : 0.f;
    }
    __syncthreads();
    for (int hh = warp; hh < heads; hh += NT / 32) {
        const int h = h_base + hh;
        const float k = -expf(g.A_log[h]) * LOG2E;
        float dt[2], l[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            dt[j] = sdt[2 * lane + j][hh];
            l[j] = 2 * lane + j < d.len ? k * dt[j] : 0.f;   // (k may be infinite: past the sequence nothing decays)
        }
        const float c0 = fmaxf(l[0], LAM_MIN), c1 = fmaxf(l[1], LAM_MIN);
        // inclusive prefix (plain and clamped) and suffix sums of the lanes' pairs
        float pre = l[0] + l[1], cl = c0 + c1, suf = pre, top = fmaxf(dt[0], dt[1]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float u = __shfl_up_sync(0xffffffffu, pre, o), v = __shfl_up_sync(0xffffffffu, cl, o);
            const float w = __shfl_down_sync(0xffffffffu, suf, o);
            if (lane >= o) {
                pre += u;
                cl += v;
            }
            if (lane + o < 32) suf += w;
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
        float pb = __shfl_up_sync(0xffffffffu, pre, 1), cb = __shfl_up_sync(0xffffffffu, cl, 1);
        float sa = __shfl_down_sync(0xffffffffu, suf, 1);
        if (lane == 0) pb = cb = 0.f;
        if (lane == 31) sa = 0.f;
        const float end = __shfl_sync(0xffffffffu, pre, 31);
        float* out = a.step + ((size_t)chunk * g.H + h) * STEP_FLOATS;
        *reinterpret_cast<float2*>(out + 2 * lane) = make_float2(cb + c0, cb + c0 + c1);
        // (an infinite step leaves the others of the chunk no scale: NaN for all of them)
        if (!(top <= 3.4e38f)) dt[0] = dt[1] = __int_as_float(0x7fc00000);
        *reinterpret_cast<float2*>(out + ST_DT + 2 * lane) = make_float2(dt[0], dt[1]);
        const float w0 = ex2(l[1] + sa) * dt[0], w1 = ex2(sa) * dt[1];
        float wsum = w0 + w1;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, o);
        out[ST_W + w_at(2 * lane)] = w0;
        out[ST_W + w_at(2 * lane + 1)] = w1;
        *reinterpret_cast<float2*>(out + ST_EL + 2 * lane) = make_float2(ex2(pb + l[0]), ex2(pb + l[0] + l[1]));
        if (lane == 0)
            *reinterpret_cast<float4*>(out + ST_DEC) = make_float4(ex2(end), __int_as_float(expo(top)), end, fmaxf(wsum, pow2n(-40)));
    }
}

template <int N>
__global__ void __launch_bounds__(NT, 2) prep_kernel(const __grid_constant__ ChunkArgs a) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ float wmax[NT / 32];
    __shared__ __align__(8) unsigned long long bar;
    __shared__ uint32_t tmem_slot;
    const PrefillArgs& g = a.g;
    // the blocks of one chunk side by side: their pieces of a projection row are neighbours
    const int chunk = blockIdx.x / a.prep_blocks, grp = blockIdx.x % a.prep_blocks;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = ERR_NONE;   // this call's timeouts only
    const ChunkDesc d = chunk_desc(a, chunk);
    if (grp >= g.G) {
        cudaTriggerProgrammaticLaunchCompletion();
        steps(a, d, chunk, grp - g.G, reinterpret_cast<float (*)[HB + 1]>(smem_raw));
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t raw = ptx::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    unsigned char* sC = smem_raw + (base - raw);
    unsigned char* sB = sC + (N / 64) * 8192;
    const uint32_t bar_a = ptx::smem_u32(&bar);
    if (warp == 0) {
        ptx::tmem_alloc(ptx::smem_u32(&tmem_slot), TMEM_COLS);
        ptx::tmem_relinquish();
        // The next launch's CTAs may start now, and not before this block has its tensor memory: one
        // that shared the SM would take all of it and then wait for this launch to end.  A block
        // counts from its first thread that gets here on, so this warp says it, behind its
        // allocation.  (Registers keep the two apart as well: 512 x 64 and 640 x 96 exceed an SM's.)
        cudaTriggerProgrammaticLaunchCompletion();
    }
    if (tid == 0) {
        ptx::mbar_init(bar_a, 1);
        ptx::fence_mbar_init();
    }

    // ---- conv + SiLU: a thread owns a pair of neighbouring channels of B or C for TP
    // tokens, in packed fp32 pairs
    constexpr int PARTS = NT / N, TP = CHUNK_T / PARTS;
    const int cp = tid % N, part = tid / N;
    const bool is_c = cp >= N / 2;
    const int n = 2 * (is_c ? cp - N / 2 : cp);
    const int W = g.H * g.P, Cx = W + 2 * g.G * N;
    const int c = W + (is_c ? g.G * N : 0) + grp * N + n;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(g.xbc) + c;
    const float4 wa = __ldg(reinterpret_cast<const float4*>(g.conv_w) + c), wb = __ldg(reinterpret_cast<const float4*>(g.conv_w) + c + 1);
    const float2 w0 = make_float2(wa.x, wb.x), w1 = make_float2(wa.y, wb.y), w2 = make_float2(wa.z, wb.z), w3 = make_float2(wa.w, wb.w);
    const float2 bias = g.conv_b ? *reinterpret_cast<const float2*>(g.conv_b + c) : make_float2(0.f, 0.f);
    auto load = [](const __nv_bfloat16* p) { return *reinterpret_cast<const __nv_bfloat162*>(p); };
    float2 v[TP];
    // rows of a chunk that is full need no tests (almost every chunk)
    auto conv = [&](auto full_c) {
        constexpr bool FULL = decltype(full_c)::value;
        const int t0 = part * TP;                            // first token of this thread in the chunk
        const __nv_bfloat16* row = x + (int64_t)(d.t0 + t0) * g.xbc_stride;
        __nv_bfloat162 r[TP];
#pragma unroll
        for (int t = 0; t < TP; ++t, row += g.xbc_stride)
            r[t] = FULL || t0 + t < d.len ? load(row) : __floats2bfloat162_rn(0.f, 0.f);
        // the three rows before: of this sequence (a chunk's first token sits at a multiple
        // of 64), or at its start of the ring
        float2 h[RING];
        row = x + (int64_t)(d.t0 + t0 - RING) * g.xbc_stride;
        const __nv_bfloat16* ring = g.ring_in ? static_cast<const __nv_bfloat16*>(g.ring_in) + (size_t)d.seq * RING * Cx + c : nullptr;
#pragma unroll
        for (int j = 0; j < RING; ++j, row += g.xbc_stride) {
            if (t0 > 0 || d.pos > 0) h[j] = FULL || t0 + j - RING < d.len ? __bfloat1622float2(load(row)) : make_float2(0.f, 0.f);
            else h[j] = ring ? __bfloat1622float2(load(ring + (size_t)j * Cx)) : make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int t = 0; t < TP; ++t) {
            const float2 x3 = __bfloat1622float2(r[t]);
            v[t] = silu2(__ffma2_rn(w3, x3, __ffma2_rn(w2, h[2], __ffma2_rn(w1, h[1], __ffma2_rn(w0, h[0], bias)))));
            if (!FULL && t0 + t >= d.len) v[t] = make_float2(0.f, 0.f);
            h[0] = h[1]; h[1] = h[2]; h[2] = x3;
        }
    };
    if (d.len == CHUNK_T) conv(std::true_type{});
    else conv(std::false_type{});
    float m = 0.f;
#pragma unroll
    for (int t = 0; t < TP; ++t) m = fmaxf(m, fmaxf(fabsf(v[t].x), fabsf(v[t].y)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) wmax[warp] = m;
    __syncthreads();
    float mb = 0.f, mc = 0.f;
#pragma unroll
    for (int k = 0; k < NT / 32; ++k) {
        if ((32 * k) % N >= N / 2) mc = fmaxf(mc, wmax[k]);
        else mb = fmaxf(mb, wmax[k]);
    }
    const int eb = expo(mb), ec = expo(mc);
    if (tid == 0) a.scale[(size_t)chunk * g.G + grp] = make_int4(eb, ec, 0, 0);
    // an infinity leaves no scale for the rest of its tile: all of it NaN, rather than
    // finite rows that lost their digits
    const float top = is_c ? mc : mb, s = top <= 3.4e38f ? pow2(is_c ? C_TOP - ec : B_TOP - eb) : __int_as_float(0x7fc00000);
    unsigned char* tile = is_c ? sC : sB;
#pragma unroll
    for (int t = 0; t < TP; ++t) {
        v[t] = __fmul2_rn(v[t], make_float2(s, s));
        *reinterpret_cast<uint32_t*>(tile + sw128_off(part * TP + t, n, CHUNK_T)) = pack2(v[t].x, v[t].y);
    }
    unsigned char* rec = a.rec + ((size_t)chunk * g.G + grp) * Rec<N>::BYTES;
    ptx::fence_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    if (tid == 0) {
#pragma unroll
        for (int kk = 0; kk < N / 16; ++kk) {
            const uint32_t off = (kk >> 2) * 8192 + (kk & 3) * 32;
            ptx::mma_f16(tmem, ptx::sdesc_sw128(base + off), ptx::sdesc_sw128(base + (N / 64) * 8192 + off),
                         ptx::idesc_f16_f32(128, 64), kk > 0);
        }
        ptx::mma_commit(bar_a);
    }
    // ---- B^T hi and lo from registers, the C tile as it lies in shared memory
    if (!is_c) {
#pragma unroll
        for (int row = 0; row < 2; ++row)
#pragma unroll
            for (int q = 0; q < TP / 8; ++q) {
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 p0 = v[8 * q + 2 * e], p1 = v[8 * q + 2 * e + 1];
                    const float x0 = row ? p0.y : p0.x, x1 = row ? p1.y : p1.x;
                    hi[e] = pack2(x0, x1);
                    const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi[e]));
                    lo[e] = pack2(x0 - back.x, x1 - back.y);
                }
                const uint32_t off = sw128_off(n + row, part * TP + 8 * q, N);
                *reinterpret_cast<uint4*>(rec + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                *reinterpret_cast<uint4*>(rec + Rec<N>::OFF_LO + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
    }
    for (int i = tid; i < (N / 64) * 512; i += NT)
        reinterpret_cast<uint4*>(rec + Rec<N>::OFF_C)[i] = reinterpret_cast<const uint4*>(sC)[i];
    // ---- G: rows 0-63 from TMEM lanes 0-63 (warps 0 and 1; the others are done)
    if (warp < 2) {
        const bool ok = ptx::mbar_wait(bar_a, 0, WAIT_LIMIT_NS);
        ptx::tc_fence_after();
        if (ok) {
            const int row = 32 * warp + lane;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float f[32];
                ptx::tmem_ld32(tmem + ((uint32_t)(32 * warp) << 16) + 32 * j, f);
#pragma unroll
                for (int x = 0; x < 32; ++x) f[x] *= pow2(G_TOP - C_TOP - B_TOP);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (4 * j + q <= row >> 3)
                        *reinterpret_cast<uint4*>(rec + Rec<N>::OFF_G + sw128_off(row, 32 * j + 8 * q, CHUNK_T)) =
                            make_uint4(pack2(f[8 * q], f[8 * q + 1]), pack2(f[8 * q + 2], f[8 * q + 3]),
                                       pack2(f[8 * q + 4], f[8 * q + 5]), pack2(f[8 * q + 6], f[8 * q + 7]));
            }
        } else if (tid == 0) {
            atomicExch(a.status, ERR_TIMEOUT);
            ptx::mbar_wait(bar_a, 0, WAIT_LIMIT_NS);   // the MMAs finish before their TMEM is freed
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TMEM_COLS);
    }
}

}  // namespace

cudaError_t launch_chunk_prep(const ChunkArgs& a, cudaStream_t s) {
    if (a.n_chunks == 0) return cudaSuccess;
    ChunkArgs b = a;
    b.prep_blocks = a.g.G + (a.g.H + HB - 1) / HB;
    const int64_t grid = (int64_t)a.n_chunks * b.prep_blocks;
    if (grid > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
    const size_t smem = (size_t)(a.g.N / 64) * 16384 + 1024;
    static_assert(sizeof(float) * CHUNK_T * (HB + 1) <= 16384 + 1024, "the step blocks' tile");
    if (a.g.N == 64) prep_kernel<64><<<(unsigned)grid, NT, smem, s>>>(b);
    else prep_kernel<128><<<(unsigned)grid, NT, smem, s>>>(b);
    return cudaGetLastError();
}

}  // namespace ssm
}  // namespace kda
