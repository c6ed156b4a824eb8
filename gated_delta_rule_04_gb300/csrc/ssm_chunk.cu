// Chunked prefill of the state space mixer on the 5th-generation tensor cores
// (tcgen05, accumulators in tensor memory), conv, scan, skip and gate in one
// pass over x, z and o.
//
// One CTA walks the 64-token chunks of one unit: 128 channels of x, i.e. two
// heads of 64 or one of 128, of one group.  With lam the chunk's cumulative
// log2 decay of a head (lam <= 0, falling), S the state at the chunk start
// (transposed: lane = channel, column = state index), per chunk
//   Y^T   = X^T M^T + (S^T C^T) 2^lam_t         M_ts = G_ts 2^(lam_t - lam_s) dt_s
//                                               (s <= t; + D on the diagonal)
//   S^T   = 2^lam_63 S^T + (X 2^(lam_63 - lam_s) dt_s)^T B
// Unlike the delta rule nothing here solves for the update, so the chain from
// chunk to chunk is one decay and one accumulating MMA.  Everything has M = 128
// (the unit's channels), and the channel-side operands are MMA operands in
// tensor memory: a thread convolves its channel's tokens in registers and
// stores the packed row, with no shared-memory tile for x.
//   inter  DI = S^T C^T          A = S^T (fp16, TMEM), B = C      N = 64
//   intra  D_h = X^T M_h^T       A = X (fp16, TMEM),  B = M_h     N = 64, per head (the
//                                rows of the other head are computed and not used: an
//                                M = 64 MMA takes as long)
//   state  S^T += X~^T B         A = X~ hi/lo (fp16, TMEM), B = B^T hi/lo, N = state width;
//                                hi*hi + hi*lo + lo*hi, since S is an fp32 result
// Operands are fp16 with exact power-of-two scales, so that they keep 11 bits
// (22 in pairs) whatever the size of the inputs: B and C by chunk (from the
// preparation), X by channel and chunk, dt by head and chunk, S by channel from
// a running upper bound of its row.  Each lies as far up fp16's range as its sums allow, so
// that a token may be small beside the largest of its chunk.  The scales leave again where a thread
// holds its own channel: in the decay of S and in the readout of Y.
//
// Warp roles.  Warps 0-7 (X group; warp % 4 = lane quarter, warp / 4 = token
// half): conv, operands, S; the two warps of a quarter meet once a chunk, for the
// maxima that set X's scale.  Warps 8-15 (Y group): the readout, Y through a
// shared-memory tile to rows, gate, store.  Warps 17-19: M of the next chunk.  Warp
// 16 issues the MMAs and the loads.  All hand-offs are mbarriers; x, the step records and the
// group records arrive by TMA and bulk copies, x two chunks ahead.  Every wait is
// bounded: on timeout the kernel reports it in the workspace's error word, lets its
// copies and MMAs land, frees its tensor memory and returns.
//
// Few units leave SMs idle, so long sequences are cut into pieces that run side
// by side.  A walk over S alone (LITE: no S copy, no M, no Y) takes 0.65 of a full
// one and gives a piece's end state from a zero start; a piece's true start is
// composed from the pieces before it when it begins.  The first piece needs no
// start, so it is walked in full beside those.
//
// Measured: a full walk takes 2.3 us a chunk and a lite one 1.6 (64 tokens x 128
// channels, N = 128), i.e. 32768 tokens x 96 heads of 64 in 0.54 ms.  No unit is
// near its limit (issue slots 62 %, shared memory 47 %, tensor cores 30 %, L2 22 %);
// four chains of about that length run against each other: the X group's arithmetic
// on 64 x 128 values (conv, SiLU, scaling, three fp16 packings) with the S row, M
// behind its record, and MMAs -> readout -> next MMAs.  From 4.4 us it came there by
// x through registers rather than a shared tile, M and the readout off the X group,
// packed fp32 pairs, one exponential per piece of M, and the loads on the issuing
// thread, behind the MMAs.  Eight more X warps changed nothing, nor did the S row on
// the Y group's.
#include "ssm_chunk.cuh"
#include "tc_ptx.cuh"

namespace kda {
namespace ssm {
namespace {

constexpr int NT = 640;                    // 8 X warps, 8 Y warps, one issuing warp, 3 M warps
// register split: 96 a thread at launch (65536 / 640, in eights of a warp's share); the
// other groups give to the X group (Y 96 and 64 for the last warpgroup spill in M:
// 32768 tokens x 96 heads 0.80 ms, this way 0.77)
constexpr int REG_LAUNCH = 96, REG_X = 112, REG_Y = 88, REG_ISSUE = 80;
static_assert(256 * REG_X + 256 * REG_Y + 128 * REG_ISSUE <= NT * REG_LAUNCH && REG_X % 8 == 0,
              "the split must fit the launch's registers, or setmaxnreg.inc waits forever");
static_assert(REG_X > REG_LAUNCH && REG_Y < REG_LAUNCH && REG_ISSUE < REG_LAUNCH && REG_ISSUE >= 24,
              "setmaxnreg.inc takes no smaller count than the current one, .dec no larger");
constexpr int NX = 256, NY = 256;
constexpr int NM = 96;                     // M threads: warps 17-19
constexpr int BAR_X = 1, BAR_Y = 2, BAR_M = 3, BAR_PAIR = 4;   // named barriers (BAR_PAIR + lane quarter)
constexpr uint32_t TM_S = 0, TM_SH = 128, TM_XF = 192, TM_XH = 224, TM_XL = 256, TM_DI = 288, TM_D = 352;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;
constexpr int LDYS = 132;
constexpr uint32_t ROW = 256;              // bytes of a unit's 128 channels
constexpr uint32_t X_SLOT = 67 * ROW;
constexpr uint32_t STEP_BYTES = STEP_FLOATS * 4;
constexpr uint32_t STEP_SLOT = 2 * STEP_BYTES + 16;   // two heads' step records, the group's scales

// A slot is refilled for chunk c + 2 when the X group is done with chunk c and the
// Y group with the decays of chunk c - 1; M is at chunk c or c + 1.
constexpr int NSTEP = 3;

template <int P, int N>
struct Map {                               // shared memory, from a 1 KiB aligned base
    static constexpr int U = 128 / P;      // heads per unit
    static constexpr uint32_t REC = 0;                                // 2 group records
    static constexpr uint32_t M = REC + 2 * Rec<N>::BYTES;            // fp16 [2 buffers][U][64 t][64 s]
    static constexpr uint32_t X = M + 2 * U * 8192;                   // 2 raw x tiles [67][128] bf16
    static constexpr uint32_t Y = X + 2 * X_SLOT;                     // fp32 [64 t][LDYS]
    static constexpr uint32_t STEP = Y + 64 * LDYS * 4;               // NSTEP step slots
    static constexpr uint32_t SX = STEP + NSTEP * STEP_SLOT;          // fp32 [3][128] scale of D_h by channel
    static constexpr uint32_t SI = SX + 3 * 512;                      // fp32 [3][128] scale of DI
    static constexpr uint32_t XM = SI + 3 * 512;                      // fp32 [2 chunks][2][128] row maxima by token half
    static constexpr uint32_t BAR = XM + 2048;
    static constexpr uint32_t BYTES = BAR + 256 + 1024;
    static_assert(REC % 1024 == 0 && M % 1024 == 0 && X % 128 == 0 && STEP % 16 == 0 && STEP_SLOT % 16 == 0 && BAR % 8 == 0, "");
    static_assert(BYTES <= 232448 && 2 * BYTES > 233472, "one CTA per SM (it takes all of the tensor memory)");
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Waits for a phase; false after the limit or once another thread gave up.
__device__ __forceinline__ bool wait_or_abort(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    // (a suspended thread takes no issue slots from the warps at work)
    if (ptx::mbar_try_wait_sleep(bar, parity, 1000)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait_sleep(bar, parity, 1000)) {
        if (*abort_flag) return false;
        if (ptx::globaltimer_ns() - t0 > WAIT_LIMIT_NS) {
            *abort_flag = 1;
            return false;
        }
    }
    return true;
}

// The exponent by which M is scaled down: |G'| <= 512 N / 128, dt < 2^(edt + 1), and D on the
// diagonal, if there is one, so that |M'| < 2^10 + 2^9; M_TOP more and it fills fp16's range, for
// the tokens whose row is small.
constexpr int M_TOP = 5, X_TOP = 14;       // (X by channel, below 2^(X_TOP + 1): their products are summed in fp32)
__device__ __forceinline__ int m_exponent(int edt, int eb, int ec, float skip) {
    const int e = edt + eb + ec, es = expo(fabsf(skip)) - 8;
    return skip == 0.f || e > es ? e : es;
}

// The exponent by which a state row of at most `bound` is scaled down, to below 2^14.  It
// takes the whole range of a state (products of inputs, not an input): fp16 holds the
// row up to 2^115, 2^-100 is far below what an fp32 state of such inputs resolves.
__device__ __forceinline__ int state_exponent(float bound) {
    const int e = (int)((__float_as_uint(bound) >> 23) & 255u) - 127 - 13;
    return e < -100 ? -100 : e > 100 ? 100 : e;
}

// One piece of a sequence's chunks for one unit.  LITE: its end state from a zero start only.
template <int P, int N, bool LITE>
__device__ __forceinline__ void walk(const ChunkArgs& a, const int unit, const int seq, const int piece) {
    using L = Map<P, N>;
    constexpr int U = L::U;
    extern __shared__ unsigned char smem_raw[];
    const PrefillArgs& g = a.g;
    const int64_t bos = seq_start(g, seq), len_seq = seq_start(g, seq + 1) - bos;
    const int64_t nc_seq = first_chunk(a, seq + 1) - first_chunk(a, seq);
    const int64_t first = piece == 0 ? 0 : a.lp0 + (int64_t)(piece - 1) * a.lp;   // first chunk in the sequence
    const int64_t most = piece == 0 ? a.lp0 : a.lp;
    const bool last_piece = first + most >= nc_seq;
    if (first > 0 && first >= nc_seq) return;
    if (LITE && last_piece) return;
    const int nc = (int)(nc_seq - first < most ? nc_seq - first : most);
    const int64_t chunk0 = first_chunk(a, seq) + first;                // in the chunk table
    const int HG = g.H / g.G, grp = unit / a.upg, h0 = grp * HG + (unit % a.upg) * U;
    const int nh = min(U, (grp + 1) * HG - h0);                        // heads of this unit
    const int c0 = h0 * P, W = g.H * P, Cx = W + 2 * g.G * N;

    const uint32_t raw = ptx::smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    unsigned char* sb = smem_raw + (base - raw);
    const uint32_t bars = base + L::BAR;
    const uint32_t b_x = bars, b_step = bars + 16, b_rec = bars + 56, b_m = bars + 72;   // [2], [NSTEP], [2], [2]
    const uint32_t b_xready = bars + 88, b_done = bars + 96, b_dfree = bars + 104, b_drain = bars + 112, b_sdone = bars + 120, b_mfree = bars + 128;   // b_mfree: [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sb + L::BAR + 160);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sb + L::BAR + 164);
    volatile int* issued = reinterpret_cast<volatile int*>(sb + L::BAR + 168);   // loads issued: [0] x and steps, [1] records
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 16) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), TMEM_COLS);
        ptx::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(b_x + 8 * i, 1);
            ptx::mbar_init(b_rec + 8 * i, 1);
            ptx::mbar_init(b_m + 8 * i, 1);
            ptx::mbar_init(b_mfree + 8 * i, 1);
        }
        for (int i = 0; i < NSTEP; ++i) ptx::mbar_init(b_step + 8 * i, 1);
        ptx::mbar_init(b_xready, NX / 32);
        ptx::mbar_init(b_done, 1);
        ptx::mbar_init(b_dfree, NY / 32);
        ptx::mbar_init(b_drain, 1);
        ptx::mbar_init(b_sdone, 1);
        *abort_flag = 0;
        issued[0] = issued[1] = 0;
        ptx::fence_mbar_init();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int quarter = warp & 3, half = (warp >> 2) & 1;
    const uint32_t tlane = tmem + ((uint32_t)(32 * quarter) << 16);

    // x tile of chunk c; its step records and scales
    auto load_x = [&](int c) {
        const uint32_t bx = b_x + 8 * (c & 1);
        const int64_t t0 = bos + (first + c) * CHUNK_T;
        const uint32_t dst = base + L::X + (c & 1) * X_SLOT;
        if (first + c > 0) {
            ptx::mbar_expect_tx(bx, (CHUNK_T + RING) * ROW);
            ptx::tma_load_2d(dst, &a.map67, c0, (int)(t0 - RING), bx);
        } else {                               // the sequence's first rows: no rows before them
            ptx::mbar_expect_tx(bx, CHUNK_T * ROW);
            ptx::tma_load_2d(dst + RING * ROW, &a.map64, c0, (int)t0, bx);
        }
        issued[0] = c + 1;
    };
    auto load_step = [&](int c) {
        const uint32_t bs = b_step + 8 * (c % NSTEP);
        const uint32_t sdst = base + L::STEP + (c % NSTEP) * STEP_SLOT;
        ptx::mbar_expect_tx(bs, nh * STEP_BYTES + 16);
        ptx::bulk_g2s(sdst, a.step + ((size_t)(chunk0 + c) * g.H + h0) * STEP_FLOATS, nh * STEP_BYTES, bs);
        ptx::bulk_g2s(sdst + 2 * STEP_BYTES, a.scale + (size_t)(chunk0 + c) * g.G + grp, 16, bs);
    };
    auto load_rec = [&](int c) {
        const uint32_t bar = b_rec + 8 * (c & 1);
        const uint32_t bytes = LITE ? Rec<N>::OFF_C : Rec<N>::BYTES;
        const unsigned char* src = a.rec + ((size_t)(chunk0 + c) * g.G + grp) * Rec<N>::BYTES;
        ptx::mbar_expect_tx(bar, bytes);
        ptx::bulk_g2s(base + L::REC + (c & 1) * Rec<N>::BYTES, src, bytes / 2, bar);
        ptx::bulk_g2s(base + L::REC + (c & 1) * Rec<N>::BYTES + bytes / 2, src + bytes / 2, bytes / 2, bar);
        issued[1] = c + 1;
    };
    auto step_of = [&](int c, int hh) { return reinterpret_cast<const float*>(sb + L::STEP + (c % NSTEP) * STEP_SLOT + hh * STEP_BYTES); };
    auto scale_of = [&](int c) { return *reinterpret_cast<const int2*>(sb + L::STEP + (c % NSTEP) * STEP_SLOT + 2 * STEP_BYTES); };

    if (warp < 8) {
        // ================================ X group ================================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_X));
        if (piece > 0) cudaGridDependencySynchronize();      // (end states of the pieces before)
        const int ch = 32 * quarter + lane;                  // channel of the unit = TMEM lane
        const int hh = min(ch / P, nh - 1), h = h0 + hh;     // its head (a channel past the group: computed, never stored)
        const bool valid = ch < nh * P;
        const int p = ch % P;
        const float4 w = __ldg(reinterpret_cast<const float4*>(g.conv_w) + c0 + ch);
        const float bias = g.conv_b ? g.conv_b[c0 + ch] : 0.f;
        const float2 w0 = make_float2(w.x, w.x), w1 = make_float2(w.y, w.y), w2 = make_float2(w.z, w.z), w3 = make_float2(w.w, w.w);
        const float2 bias2 = make_float2(bias, bias);
        const float skip = g.skip ? g.skip[h] : 0.f;
        float* xm = reinterpret_cast<float*>(sb + L::XM);
        float* sSX = reinterpret_cast<float*>(sb + L::SX);
        float* sSI = reinterpret_cast<float*>(sb + L::SI);
        const size_t state = (size_t)N * P;

        // ---- starting state: the caller's for the first piece; later ones compose the
        // end states of the pieces before them (zero in the lite pass)
        const float* start = piece == 0 && nc > 0 && g.S_in ? g.S_in + ((size_t)seq * g.H + h) * state + p : nullptr;
        const float* loc = a.local + ((size_t)seq * a.np * g.H + h) * state + p;
        const float* ltot = a.ltot + (size_t)seq * a.np * g.H + h;
        constexpr int NH = N / 2;                            // state columns of this thread
        float sbound = 0.f;
#pragma unroll 1
        for (int j = 0; j < NH; j += 32) {
            float v[32];
            // (columns inside, pieces outside: 32 loads in flight)
            auto read = [&](const float* src, float decay) {
#pragma unroll
                for (int x = 0; x < 32; ++x) v[x] = fmaf(decay, v[x], src[(size_t)(NH * half + j + x) * P]);
            };
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = 0.f;
            if (valid && !LITE && start) read(start, 0.f);
            if (valid && !LITE)
                for (int q = 0; q < piece; ++q) read(loc + (size_t)q * g.H * state, q ? ex2(ltot[(size_t)q * g.H]) : 0.f);
#pragma unroll
            for (int x = 0; x < 32; ++x) sbound = fmaxf(sbound, fabsf(v[x]));
            ptx::tmem_st32(tlane + TM_S + NH * half + j, v);
        }
        xm[128 * half + ch] = sbound;
        ptx::bar_sync_or(BAR_X, NX, false);
        sbound = fmaxf(xm[ch], xm[128 + ch]);
        ptx::bar_sync_or(BAR_X, NX, false);
        int so = state_exponent(2.f * sbound);               // S = S' 2^so, |S'| < 2^14
        {
            // (an infinite state value leaves the rest of its channel no scale: NaN for all of it)
            const float f = sbound <= 3.4e38f ? pow2(-so) : __int_as_float(0x7fc00000);
#pragma unroll 1
            for (int j = 0; j < NH; j += 32) {
                float v[32];
                ptx::tmem_ld32(tlane + TM_S + NH * half + j, v);
#pragma unroll
                for (int x = 0; x < 32; ++x) v[x] *= f;
                ptx::tmem_st32(tlane + TM_S + NH * half + j, v);
            }
        }
        // the ring's three rows of this channel, for the sequence's first chunk
        float r0 = 0.f, r1 = 0.f, r2 = 0.f;
        if (first == 0 && half == 0 && g.ring_in) {
            const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(g.ring_in) + (size_t)seq * RING * Cx + c0 + ch;
            r0 = to_f32(r[0]); r1 = to_f32(r[Cx]); r2 = to_f32(r[2 * (size_t)Cx]);
        }
        // The ring of this unit's channels and, by a group's first unit, of its B and C: the
        // sequence's last three raw rows, older slots moved up when it has fewer.  The first
        // piece does it: no other CTA of this launch reads those entries of ring_in, so
        // ring_out may be ring_in.
        if (!LITE && first == 0 && g.ring_out && half == 0) {
            cudaGridDependencySynchronize();
            const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(g.xbc);
            const __nv_bfloat16* rin = static_cast<const __nv_bfloat16*>(g.ring_in);
            __nv_bfloat16* rout = static_cast<__nv_bfloat16*>(g.ring_out) + (size_t)seq * RING * Cx;
            auto carry = [&](int cc) {
                __nv_bfloat16 row[RING];
#pragma unroll
                for (int s = 0; s < RING; ++s) {
                    const int64_t t = len_seq - RING + s;
                    row[s] = t >= 0 ? x[(bos + t) * g.xbc_stride + cc]
                             : rin  ? rin[((size_t)seq * RING + t + RING) * Cx + cc] : __nv_bfloat16(0.f);
                }
#pragma unroll
                for (int s = 0; s < RING; ++s) rout[(size_t)s * Cx + cc] = row[s];
            };
            if (valid) carry(c0 + ch);
            if (unit % a.upg == 0)
                for (int x2 = ch; x2 < 2 * N; x2 += 128) carry(W + (x2 < N ? grp * N + x2 : g.G * N + grp * N + x2 - N));
        }
        float lsum = 0.f;
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
            const int b3 = c % 3;
            bool bad = !wait_or_abort(b_step + 8 * (c % NSTEP), (uint32_t)(c / NSTEP) & 1u, abort_flag);
            bad = !wait_or_abort(b_x + 8 * (c & 1), (uint32_t)(c >> 1) & 1u, abort_flag) || bad;
            const int64_t rem = len_seq - (first + c) * CHUNK_T;
            const int len = rem < CHUNK_T ? (int)rem : CHUNK_T;
            // ---- conv + SiLU of this channel's 32 tokens, t and t + 16 as a packed pair
            float2 v[16];
            {
                const __nv_bfloat16* xt = reinterpret_cast<const __nv_bfloat16*>(sb + L::X + (c & 1) * X_SLOT) + 32 * half * 128 + ch;
                auto pair = [&](int t) { return make_float2(to_f32(xt[(t + RING) * 128]), to_f32(xt[(t + RING + 16) * 128])); };
                float2 x0 = pair(-3), x1 = pair(-2), x2 = pair(-1);
                if (first + c == 0 && half == 0) {
                    x0.x = r0; x1.x = r1; x2.x = r2;
                }
#pragma unroll
                for (int t = 0; t < 16; ++t) {
                    const float2 x3 = pair(t);
                    v[t] = __ffma2_rn(w0, x0, bias2);
                    v[t] = __ffma2_rn(w1, x1, v[t]);
                    v[t] = __ffma2_rn(w2, x2, v[t]);
                    v[t] = __ffma2_rn(w3, x3, v[t]);
                    x0 = x1; x1 = x2; x2 = x3;
                }
            }
            // rows past the sequence hold whatever lies there
            if (len < CHUNK_T) {
#pragma unroll
                for (int t = 0; t < 16; ++t) {
                    if (32 * half + t >= len) v[t].x = 0.f;
                    if (32 * half + t + 16 >= len) v[t].y = 0.f;
                }
            }
            float m = 0.f;
#pragma unroll
            for (int t = 0; t < 16; ++t) v[t] = silu2(v[t]);
#pragma unroll
            for (int t = 0; t < 16; ++t) m = fmaxf(m, fmaxf(fabsf(v[t].x), fabsf(v[t].y)));
            float* xmc = xm + 256 * (c & 1);
            xmc[128 * half + ch] = m;
            // the two warps of a lane quarter exchange their maxima; nothing else ties the X
            // warps together within a chunk
            if (ptx::bar_sync_or(BAR_PAIR + quarter, 64, bad)) break;
            // ---- scales
            const float* st = step_of(c, hh);
            const float lend = st[ST_LOG], dec = st[ST_DEC];
            const int edt = __float_as_int(st[ST_EDT]);
            const int2 ebc = scale_of(c);
            const int ex = expo(fmaxf(xmc[ch], xmc[128 + ch]));
            // of |S| after this chunk.  (The weights' sum knows the decay: 64 times the largest dt is
            // 2^9 more for a head that forgets a token within 10, digits that its state then lacks.)
            const float bound = fmaf(dec, sbound, pow2n(2 + ex + ebc.x) * st[ST_WSUM]);
            const int sn = state_exponent(bound);
            if (half == 0 && !LITE) {
                // (products, so that they are infinite or zero past fp32's range: |em| <= 120, |so| <= 100)
                sSX[b3 * 128 + ch] = pow2n(m_exponent(edt, ebc.x, ebc.y, skip) - M_TOP) * pow2n(ex - X_TOP);
                sSI[b3 * 128 + ch] = pow2n(so) * pow2n(ebc.y - C_TOP);
            }
            // ---- operand rows of this half's tokens
            uint32_t xf[16], xh[16], xl[16];
            {
                const float xs = pow2n(X_TOP - ex), kx = pow2(ebc.x - B_TOP - sn);
                const float2 xs2 = make_float2(xs, xs), kx2 = make_float2(kx, kx);
                const float4* wt = reinterpret_cast<const float4*>(st + ST_W + 32 * half);
                // fp16 pairs hold tokens (t, t + 1): column t / 2 from the low halves, 8 + t / 2 from the high
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float4 w4 = wt[q];
                    const float2 ya = __fmul2_rn(v[2 * q], __fmul2_rn(make_float2(w4.x, w4.y), kx2));
                    const float2 yb = __fmul2_rn(v[2 * q + 1], __fmul2_rn(make_float2(w4.z, w4.w), kx2));
                    xh[q] = pack2(ya.x, yb.x);
                    xh[8 + q] = pack2(ya.y, yb.y);
                    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&xh[q]));
                    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&xh[8 + q]));
                    xl[q] = pack2(ya.x - lo.x, yb.x - lo.y);
                    xl[8 + q] = pack2(ya.y - hi.x, yb.y - hi.y);
                    if (!LITE) {
                        const float2 xa = __fmul2_rn(v[2 * q], xs2), xb = __fmul2_rn(v[2 * q + 1], xs2);
                        xf[q] = pack2(xa.x, xb.x);
                        xf[8 + q] = pack2(xa.y, xb.y);
                    }
                }
            }
            // ---- the previous chunk's state and inter MMAs have read their operands and
            // written S (its intra MMAs, which come last, only hold X)
            if (c > 0) {
                bad = !wait_or_abort(b_sdone, (uint32_t)(c - 1) & 1u, abort_flag) || bad;
                ptx::tc_fence_after();
            }
            ptx::tmem_st16u(tlane + TM_XH + 16 * half, xh);
            ptx::tmem_st16u(tlane + TM_XL + 16 * half, xl);
            const float rs = dec * pow2(so - sn);
#pragma unroll 1
            for (int j = 0; j < NH; j += 32) {
                float s[32];
                ptx::tmem_ld32(tlane + TM_S + NH * half + j, s);
                if (!LITE) {
                    uint32_t sh[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) sh[e] = pack2(s[2 * e], s[2 * e + 1]);
                    ptx::tmem_st16u(tlane + TM_SH + (NH * half + j) / 2, sh);
                }
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    const float2 d = __fmul2_rn(make_float2(s[x], s[x + 1]), make_float2(rs, rs));
                    s[x] = d.x;
                    s[x + 1] = d.y;
                }
                ptx::tmem_st32(tlane + TM_S + NH * half + j, s);
            }
            if (c > 0) {
                bad = !wait_or_abort(b_done, (uint32_t)(c - 1) & 1u, abort_flag) || bad;
                ptx::tc_fence_after();
            }
            if (!LITE) ptx::tmem_st16u(tlane + TM_XF + 16 * half, xf);
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            if (__any_sync(0xffffffffu, bad)) {
                *abort_flag = 1;                             // (the partner warp sees it at its next wait)
                bad = true;
            }
            if (lane == 0 && !bad) mbar_arrive(b_xready);
            so = sn;
            sbound = bound;
            lsum += lend;
        }
        // ---- end state
        const bool ok = nc > 0 && wait_or_abort(b_done, (uint32_t)(nc - 1) & 1u, abort_flag);
        ptx::tc_fence_after();
        if (ok && !*abort_flag && valid && (LITE || last_piece || piece == 0)) {
            float* out = last_piece ? g.S_out + ((size_t)seq * g.H + h) * state + p
                                    : a.local + (((size_t)seq * a.np + piece) * g.H + h) * state + p;
            const float f = pow2(so);
#pragma unroll 1
            for (int j = 0; j < NH; j += 32) {
                float s[32];
                ptx::tmem_ld32(tlane + TM_S + NH * half + j, s);
#pragma unroll
                for (int x = 0; x < 32; ++x) out[(size_t)(NH * half + j + x) * P] = s[x] * f;
            }
            if (LITE && half == 0 && p == 0) a.ltot[((size_t)seq * a.np + piece) * g.H + h] = lsum;
        }
    } else if (warp < 16) {
        // ================================ Y group ================================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_Y));
        if constexpr (!LITE) {
            const int yt = tid - NX, ch = 32 * quarter + lane;
            // a sequence without tokens: the unit's states as they are, bit by bit (X's scales would
            // lose values far from their row's largest)
            if (nc == 0) {
                const size_t at = ((size_t)seq * g.H + h0) * N * P;
                const uint4* src = g.S_in ? reinterpret_cast<const uint4*>(g.S_in + at) : nullptr;
                uint4* dst = reinterpret_cast<uint4*>(g.S_out + at);
#pragma unroll 1
                for (int x0 = yt; x0 < nh * N * P / 4; x0 += 8 * NY) {
                    uint4 v[8];                              // (in flight at once: dst may be src)
#pragma unroll
                    for (int x = 0; x < 8; ++x) v[x] = src && x0 + x * NY < nh * N * P / 4 ? src[x0 + x * NY] : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (x0 + x * NY < nh * N * P / 4) dst[x0 + x * NY] = v[x];
                }
            }
            const int rt = yt >> 3, rseg = yt & 7;           // row pass: rows rt and 32 + rt, values 32 q + 4 rseg ..
            const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(g.z);
            // this thread's rows of z and o, one chunk further each time; columns past the
            // unit's heads (a group's odd head of 64) are left out
            const int64_t zstep = CHUNK_T * g.z_stride;
            const __nv_bfloat16* zp = z + (bos + first * CHUNK_T + rt) * g.z_stride + c0 + 4 * rseg;
            __nv_bfloat16* op = static_cast<__nv_bfloat16*>(g.o) + (size_t)(bos + first * CHUNK_T + rt) * W + c0 + 4 * rseg;
            const int nq = nh * P / 32;                      // 32-column groups of this unit: 2 or 4
            const int64_t len_here = len_seq - first * CHUNK_T;
            uint2 zc[2][4];
            auto load_z = [&](int c, const __nv_bfloat16* src) {
                const int rem = (int)(len_here - (int64_t)c * CHUNK_T < CHUNK_T ? len_here - (int64_t)c * CHUNK_T : CHUNK_T);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (32 * hf + rt < rem && q < nq)
                            zc[hf][q] = __ldg(reinterpret_cast<const uint2*>(src + 32 * hf * g.z_stride + 32 * q));
            };
            float* ys = reinterpret_cast<float*>(sb + L::Y);
#pragma unroll 1
            for (int c = 0; c < nc; ++c) {
                if (z) load_z(c, zp);
                zp += zstep;
                const bool bad = !wait_or_abort(b_done, (uint32_t)c & 1u, abort_flag);
                if (ptx::bar_sync_or(BAR_Y, NY, bad)) break; // (and the rows of the chunk before are written)
                ptx::tc_fence_after();
                {
                    const int b3 = c % 3, th = half;
                    const float si = reinterpret_cast<const float*>(sb + L::SI)[b3 * 128 + ch];
                    const float sx = reinterpret_cast<const float*>(sb + L::SX)[b3 * 128 + ch];
                    const float2 si2 = make_float2(si, si), sx2 = make_float2(sx, sx);
                    const float4* el = reinterpret_cast<const float4*>(step_of(c, min(ch / P, nh - 1)) + ST_EL + 32 * th);
                    // (16 columns at a time: with 32 the thread's registers spill)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float di[16], dh[16];
                        ptx::tmem_ld16_nw(tlane + TM_DI + 32 * th + 16 * j, di);
                        ptx::tmem_ld16_nw(tlane + TM_D + 64 * (ch / P) + 32 * th + 16 * j, dh);
                        ptx::tmem_wait_ld(di, dh);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float4 e4 = el[4 * j + q];
                            float* yr = ys + (32 * th + 16 * j + 4 * q) * LDYS + ch;
#pragma unroll
                            for (int e = 0; e < 4; e += 2) {
                                const float2 ev = e ? make_float2(e4.z, e4.w) : make_float2(e4.x, e4.y);
                                const float2 y = __ffma2_rn(make_float2(di[4 * q + e], di[4 * q + e + 1]), __fmul2_rn(ev, si2),
                                                            __fmul2_rn(make_float2(dh[4 * q + e], dh[4 * q + e + 1]), sx2));
                                yr[e * LDYS] = y.x;
                                yr[(e + 1) * LDYS] = y.y;
                            }
                        }
                    }
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_dfree);     // D and this chunk's scales are read
                }
                ptx::bar_sync_or(BAR_Y, NY, false);
                const int rem = (int)(len_here - (int64_t)c * CHUNK_T < CHUNK_T ? len_here - (int64_t)c * CHUNK_T : CHUNK_T);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    float4 y[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        y[q] = *reinterpret_cast<const float4*>(ys + (32 * hf + rt) * LDYS + 32 * q + 4 * rseg);
                    if (z) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const __nv_bfloat162* zz = reinterpret_cast<const __nv_bfloat162*>(&zc[hf][q]);
                            const float2 a = __fmul2_rn(silu2(__bfloat1622float2(zz[0])), make_float2(y[q].x, y[q].y));
                            const float2 b = __fmul2_rn(silu2(__bfloat1622float2(zz[1])), make_float2(y[q].z, y[q].w));
                            y[q] = make_float4(a.x, a.y, b.x, b.y);
                        }
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const __nv_bfloat162 o0 = __floats2bfloat162_rn(y[q].x, y[q].y), o1 = __floats2bfloat162_rn(y[q].z, y[q].w);
                        if (32 * hf + rt < rem && q < nq)
                            *reinterpret_cast<uint2*>(op + (size_t)(32 * hf) * W + 32 * q) =
                                make_uint2(*reinterpret_cast<const uint32_t*>(&o0), *reinterpret_cast<const uint32_t*>(&o1));
                    }
                }
                op += (size_t)CHUNK_T * W;
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_ISSUE));
        if (warp > 16) {
            // ============================== M group ==============================
            if constexpr (!LITE) {
                const int mt = tid - NT + NM;
                // M tiles start zero: only pieces up to the diagonal are written below
                for (int i = mt; i < 2 * U * 512; i += NM) reinterpret_cast<uint4*>(sb + L::M)[i] = make_uint4(0, 0, 0, 0);
                ptx::bar_sync_or(BAR_M, NM, false);
                const float skip0 = g.skip ? g.skip[h0] : 0.f, skip1 = g.skip ? g.skip[h0 + nh - 1] : 0.f;
#pragma unroll 1
                for (int c = 0; c < nc; ++c) {
                    bool bad = !wait_or_abort(b_step + 8 * (c % NSTEP), (uint32_t)(c / NSTEP) & 1u, abort_flag);
                    bad = !wait_or_abort(b_rec + 8 * (c & 1), (uint32_t)(c >> 1) & 1u, abort_flag) || bad;
                    // the intra MMAs of chunk c - 2 have read this buffer
                    if (c > 1) bad = !wait_or_abort(b_mfree + 8 * (c & 1), (uint32_t)((c >> 1) - 1) & 1u, abort_flag) || bad;
                    const unsigned char* G = sb + L::REC + (c & 1) * Rec<N>::BYTES + Rec<N>::OFF_G;
                    const int2 ebc = scale_of(c);
                    // A piece is 8 columns s of block j of a row r.  On the diagonal (j = r / 8) every
                    // element takes its own 2^(lam_r - lam_s).  Left of it that splits at the block's
                    // last token e: 2^(lam_r - lam_e) of the piece times 2^(lam_e - lam_s) dt_s of the
                    // column, both <= 1 but for dt, so a piece costs one exponential and not eight.
                    unsigned char* Mt = sb + L::M + (c & 1) * U * 8192;
                    auto head = [&](int hd) { return min(hd, nh - 1); };
                    auto scale = [&](int hd, float& f, float& diag) {
                        const float skip = hd ? skip1 : skip0;
                        const int em = m_exponent(__float_as_int(step_of(c, head(hd))[ST_EDT]), ebc.x, ebc.y, skip);
                        f = pow2n(ebc.x + ebc.y - em + M_TOP - G_TOP);
                        diag = skip * pow2n(M_TOP - em);
                    };
#pragma unroll
                    for (int x = 0; x < (U * 64 + NM - 1) / NM; ++x) {
                        const int i = mt + x * NM, hd = i >> 6, r = i & 63, j = r >> 3;
                        if (i >= U * 64) break;
                        float f, diag;
                        scale(hd, f, diag);
                        const float* st = step_of(c, head(hd));
                        const uint32_t off = sw128_off(r, 8 * j, CHUNK_T);
                        const uint4 g4 = *reinterpret_cast<const uint4*>(G + off);
                        const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w};
                        const float lr = st[r];
                        float ls[8], dt[8];
                        lds8(st + 8 * j, ls);
                        lds8(st + ST_DT + 8 * j, dt);
                        float2 mv[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 d = __ffma2_rn(make_float2(ls[2 * e], ls[2 * e + 1]), make_float2(-1.f, -1.f), make_float2(lr, lr));
                            const float2 k2 = __fmul2_rn(__fmul2_rn(make_float2(dt[2 * e], dt[2 * e + 1]), make_float2(f, f)),
                                                         make_float2(ex2(d.x), ex2(d.y)));
                            mv[e] = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&gw[e])), k2);
                            // nothing past s = r, D on s = r
                            const int s = 8 * j + 2 * e;
                            mv[e].x = s > r ? 0.f : s == r ? mv[e].x + diag : mv[e].x;
                            mv[e].y = s + 1 > r ? 0.f : s + 1 == r ? mv[e].y + diag : mv[e].y;
                        }
                        *reinterpret_cast<uint4*>(Mt + hd * 8192 + off) = make_uint4(
                            pack2(mv[0].x, mv[0].y), pack2(mv[1].x, mv[1].y), pack2(mv[2].x, mv[2].y), pack2(mv[3].x, mv[3].y));
                    }
                    // the columns' factors take the place of dt, which nothing else reads
                    constexpr int MINE = (U * 64 + NM - 1) / NM;
                    float cf[MINE];
#pragma unroll
                    for (int x = 0; x < MINE; ++x) {
                        const int i = min(mt + x * NM, U * 64 - 1), hd = i >> 6, t = i & 63;
                        const float* st = step_of(c, head(hd));
                        float f, diag;
                        scale(hd, f, diag);
                        cf[x] = f * st[ST_DT + t] * ex2(st[t | 7] - st[t]);
                    }
                    ptx::bar_sync_or(BAR_M, NM, false);
#pragma unroll
                    for (int x = 0; x < MINE; ++x) {
                        const int i = mt + x * NM, hd = i >> 6;
                        if (i < U * 64 && hd < nh) const_cast<float*>(step_of(c, hd))[ST_DT + (i & 63)] = cf[x];
                    }
                    ptx::bar_sync_or(BAR_M, NM, false);
                    // left of the diagonal: blocks (b, j), j < b, 28 a head, rows 8 b and 8 (8 - b) paired
#pragma unroll
                    for (int x = 0; x < (U * 224 + NM - 1) / NM; ++x) {
                        const int i = mt + x * NM, hd = i >= 224, q = (i - 224 * hd) >> 3, p = q >> 3, t = q & 7;
                        if (i >= U * 224) break;
                        const int b = p == 3 ? 4 : t <= p ? p + 1 : 7 - p, j = p == 3 || t <= p ? t : t - p - 1, r = 8 * b + (i & 7);
                        const float* st = step_of(c, head(hd));
                        const uint32_t off = sw128_off(r, 8 * j, CHUNK_T);
                        const uint4 g4 = *reinterpret_cast<const uint4*>(G + off);
                        const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w};
                        const float rf = ex2(st[r] - st[8 * j + 7]);
                        float k[8];
                        lds8(st + ST_DT + 8 * j, k);
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 k2 = __fmul2_rn(make_float2(k[2 * e], k[2 * e + 1]), make_float2(rf, rf));
                            const float2 mv = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&gw[e])), k2);
                            o[e] = pack2(mv.x, mv.y);
                        }
                        *reinterpret_cast<uint4*>(Mt + hd * 8192 + off) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    ptx::fence_async_smem();
                    if (ptx::bar_sync_or(BAR_M, NM, bad)) break;
                    if (mt == 0) mbar_arrive(b_m + 8 * (c & 1));
                }
            }
        } else if (lane == 0) {
        // ============================ MMA issue (one thread) ======================
        // The loads are this thread's as well.  With chunk c's operands ready the X group has left
        // x tile c; the next load into it comes behind the chunk's MMAs, which the others wait
        // for (ahead of them it cost 5 % of the walk).
        for (int c = 0; c < nc && c < 2; ++c) load_x(c);
        // what the launch before this one wrote is read from here on; the start up to here, and
        // the X group's, may run beside its end
        cudaGridDependencySynchronize();
        for (int c = 0; c < nc && c < 2; ++c) {
            load_step(c);
            load_rec(c);
        }
        constexpr uint32_t ID64 = ptx::idesc_f16_f32(128, 64), IDN = ptx::idesc_f16_f32(128, N);
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
            const uint32_t rec = base + L::REC + (c & 1) * Rec<N>::BYTES;
            if (!wait_or_abort(b_rec + 8 * (c & 1), (uint32_t)(c >> 1) & 1u, abort_flag)) break;
            if (!LITE && c > 0) {
                // chunk c - 1 is read out, so its MMAs and M are done with their record; M waits for
                // the next one
                if (!wait_or_abort(b_dfree, (uint32_t)(c - 1) & 1u, abort_flag)) break;
                if (c + 1 < nc) load_rec(c + 1);
            }
            if (!wait_or_abort(b_xready, (uint32_t)c & 1u, abort_flag)) break;
            if (LITE && c > 0 && c + 1 < nc) load_rec(c + 1);
            ptx::tc_fence_after();
            // descriptors of a tile differ from its first one by their start address (in 16 bytes)
            if (!LITE) {
                const uint64_t dc = ptx::sdesc_sw128(rec + Rec<N>::OFF_C);
#pragma unroll
                for (int kk = 0; kk < N / 16; ++kk)
                    ptx::mma_f16_ta(tmem + TM_DI, tmem + TM_SH + 8 * kk, dc + (kk >> 2) * 512 + (kk & 3) * 2, ID64, kk > 0);
            }
            const uint64_t db = ptx::sdesc_sw128(rec);
#pragma unroll
            for (int term = 0; term < 3; ++term)             // hi hi, hi lo, lo hi
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    ptx::mma_f16_ta(tmem + TM_S, tmem + (term == 2 ? TM_XL : TM_XH) + 8 * kk,
                                    db + (term == 1 ? Rec<N>::OFF_LO / 16 : 0) + kk * 2, IDN, 1);
            ptx::mma_commit(b_sdone);
            if (!LITE) {
                // (an abort here leaves MMAs in flight: the drain below covers them)
                if (!wait_or_abort(b_m + 8 * (c & 1), (uint32_t)(c >> 1) & 1u, abort_flag)) break;
                ptx::tc_fence_after();
                const uint64_t dm = ptx::sdesc_sw128(base + L::M + (c & 1) * U * 8192);
#pragma unroll
                for (int hd = 0; hd < U; ++hd)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        if (hd < nh)
                            ptx::mma_f16_ta(tmem + TM_D + 64 * hd, tmem + TM_XF + 8 * kk, dm + hd * 512 + kk * 2, ID64, kk > 0);
                ptx::mma_commit(b_mfree + 8 * (c & 1));
            }
            ptx::mma_commit(b_done);
            if (c + 2 < nc) {
                ptx::fence_async_smem();
                load_x(c + 2);
                load_step(c + 2);
            }
        }
        // every MMA of this thread lands before its tensor memory is freed
        ptx::mma_commit(b_drain);
        ptx::mbar_wait(b_drain, 0, WAIT_LIMIT_NS);
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (*abort_flag && tid == 0) {
        atomicExch(a.status, ERR_TIMEOUT);
        // loads in flight land before the CTA leaves: the last one of each barrier
        for (int c = max(0, issued[0] - NSTEP); c < issued[0]; ++c) {
            if (c >= issued[0] - 2) ptx::mbar_wait(b_x + 8 * (c & 1), (uint32_t)(c >> 1) & 1u, WAIT_LIMIT_NS);
            ptx::mbar_wait(b_step + 8 * (c % NSTEP), (uint32_t)(c / NSTEP) & 1u, WAIT_LIMIT_NS);
        }
        for (int c = max(0, issued[1] - 2); c < issued[1]; ++c)
            ptx::mbar_wait(b_rec + 8 * (c & 1), (uint32_t)(c >> 1) & 1u, WAIT_LIMIT_NS);
    }
    __syncthreads();
    if (warp == 16) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, TMEM_COLS);
    }
}

// A call's pieces, in two launches where there is more than one: the first piece
// of each sequence in full beside the lite walks of the pieces up to the last
// but one (LEAD), then all pieces but the first (!LEAD).
template <int P, int N, bool LEAD>
__global__ void __launch_bounds__(NT, 1) chunk_kernel(const __grid_constant__ ChunkArgs a) {
    cudaTriggerProgrammaticLaunchCompletion();
    const int per = LEAD && a.np == 1 ? 1 : a.np - 1;    // pieces of a sequence in this launch
    const int unit = blockIdx.x % a.units, i = blockIdx.x / a.units;
    const int piece = (a.by_piece ? i / a.g.n_seqs : i % per) + (LEAD ? 0 : 1);
    const int seq = seq_at(a.g, a.by_piece ? i % a.g.n_seqs : i / per);
    if constexpr (LEAD)
        if (piece > 0) {
            walk<P, N, true>(a, unit, seq, piece);
            return;
        }
    walk<P, N, false>(a, unit, seq, piece);
}

template <int P, int N, bool LEAD>
cudaError_t launch(const ChunkArgs& a, bool after, cudaStream_t s) {
    const int64_t blocks = (int64_t)a.units * std::max(1, a.np - 1) * a.g.n_seqs;
    if (blocks > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
    constexpr int smem = (int)Map<P, N>::BYTES;
    auto k = chunk_kernel<P, N, LEAD>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k, a);
}

template <bool LEAD>
cudaError_t launch_pn(const ChunkArgs& a, bool after, cudaStream_t s) {
    if (a.g.P == 64) return a.g.N == 64 ? launch<64, 64, LEAD>(a, after, s) : launch<64, 128, LEAD>(a, after, s);
    return a.g.N == 64 ? launch<128, 64, LEAD>(a, after, s) : launch<128, 128, LEAD>(a, after, s);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

}  // namespace

bool encode_rows(CUtensorMap* m, const void* base, int es, int64_t T, int64_t W, int64_t stride, uint32_t rows, uint32_t cols) {
    static const EncodeTiled encode = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<EncodeTiled>(f) : nullptr;
    }();
    if (encode == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)W, (cuuint64_t)T}, strides[1] = {(cuuint64_t)stride * es};
    const cuuint32_t box[2] = {cols, rows}, ones[2] = {1, 1};
    return encode(m, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void*>(base), dims, strides, box, ones,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_chunks(const ChunkArgs& a, bool after, cudaStream_t s) {
    const cudaError_t e = launch_pn<true>(a, after, s);
    return e != cudaSuccess || a.np == 1 ? e : launch_pn<false>(a, true, s);
}

}  // namespace ssm
}  // namespace kda
