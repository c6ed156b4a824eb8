// Chunked prefill of the state space mixer: what its two kernels share.
#pragma once

#include <cuda.h>

#include "kda_chunk_layout.cuh"
#include "ssm_common.cuh"

namespace kda {
namespace ssm {

// Record of one (chunk, group): the operand tiles that do not depend on the
// head, as the byte image of the consumer's shared memory (fp16, K-major,
// 128-byte swizzle).  B and C are stored scaled by powers of two, the exponents of the
// tile's largest magnitude and how far up fp16's range that comes to lie:
//   B^T hi, B^T lo  [N rows][64 tok]   B' = hi + lo to 22 bits, below 2^(B_TOP + 1)
//   C               [64 tok rows][N]   below 2^(C_TOP + 1)
//   G = C B^T       [64 tok rows][64]  below 512 x 2^G_TOP; 8-column pieces up to the diagonal only
// The further up, the smaller a token's row may be beside the chunk's largest before it
// falls out of fp16's normal range and loses digits.  C has no other limit than that range;
// B shares the scale of the state that its product with X~ goes to (S' below 2^14), which
// leaves X~ less for every bit here; G lies as high as its sum of N products allows.
constexpr int B_TOP = 4, C_TOP = 14, G_TOP = 6;
template <int N> struct Rec {
    static constexpr uint32_t BT = N * 128;             // bytes of B^T hi (and of lo)
    static constexpr uint32_t OFF_LO = BT;
    static constexpr uint32_t OFF_C = 2 * BT;
    static constexpr uint32_t OFF_G = OFF_C + (N / 64) * 8192;
    static constexpr uint32_t BYTES = OFF_G + 8192;
};
inline size_t rec_bytes(int N) { return N == 64 ? Rec<64>::BYTES : Rec<128>::BYTES; }

// Step record of one (chunk, head), fp32, with l_s = the log2 decay of token s:
//   [0, 64)     lam_t: inclusive cumulative sum of max(l_s, -48), for differences
//               between two tokens of the chunk.  The clamp keeps |lam| below 2^12, so
//               that a difference of two is good to 2^-12; a decay of 2^-48 and one
//               of less both vanish in the fp16 operand they go to (below 2^16 before).
//   [64, 128)   dt
//   [128, 192)  2^(sum_{s > t} l_s) dt_t: the token's weight in the end state, from a
//               suffix sum (a difference of long prefix sums would cost the fp32
//               state its last digits); token t at w_at(t), next to token t + 16
//   [192, 256)  2^(sum_{s <= t} l_s)
//   [256]       2^(sum of all l_s), [257] exponent of the largest dt (int), [258] sum of l_s,
//               [259] sum of the tokens' weights (at least 2^-40): what bounds the chunk's
//               addition to the state
constexpr int STEP_FLOATS = 260;
constexpr int ST_DT = 64, ST_W = 128, ST_EL = 192, ST_DEC = 256, ST_EDT = 257, ST_LOG = 258, ST_WSUM = 259;
constexpr float LAM_MIN = -48.f;
// The X group takes tokens t and t + 16 of a 32-token half as one packed pair.
__host__ __device__ constexpr int w_at(int t) { return (t & 32) + 2 * (t & 15) + ((t >> 4) & 1); }

// Exponent e with 2^e <= x < 2^(e+1), clamped to +-40 (so that sums of a few
// exponents stay inside fp32's range; beyond it precision goes before range).
__device__ __forceinline__ int expo(float x) {
    const int e = (int)((__float_as_uint(x) >> 23) & 255u) - 127;
    return e < -40 ? -40 : e > 40 ? 40 : e;
}
// 2^e for an e within fp32's normal range.
__device__ __forceinline__ float pow2n(int e) { return __int_as_float((e + 127) << 23); }
// 2^e for any integer e, clamped to fp32's normal range.
__device__ __forceinline__ float pow2(int e) {
    e = e < -126 ? -126 : e > 127 ? 127 : e;
    return __uint_as_float((uint32_t)(e + 127) << 23);
}
struct ChunkArgs {
    CUtensorMap map67, map64;     // xbc rows: boxes of 67 and 64 rows x 128 channels
    PrefillArgs g;
    const ChunkDesc* chunks;      // [n_chunks]
    const int64_t* coff;          // [n_seqs + 1]
    unsigned char* rec;           // [n_chunks][G][Rec::BYTES]
    float* step;                  // [n_chunks][H][STEP_FLOATS]
    int4* scale;                  // [n_chunks][G] exponents of B and C
    int32_t* status;
    // Pieces run side by side, np per sequence at most: the first of lp0 chunks,
    // the others of lp; `local` and `ltot` take each piece's end state from its own
    // start (the first piece's: the sequence's) and its log2 decay.
    float* local;                 // [n_seqs][np][H][N][P]
    float* ltot;                  // [n_seqs][np][H]
    int32_t np, lp0, lp;
    int32_t by_piece;             // order of the walks: piece by piece, or sequence by sequence
    int32_t n_chunks, units, upg; // units of 128 channels, in all and per group
    int32_t prep_blocks;          // blocks of the preparation per chunk (set by launch_chunk_prep)
};

__device__ __forceinline__ int64_t first_chunk(const ChunkArgs& a, int n) { return a.g.meta.n ? a.g.meta.coff[n] : a.coff[n]; }
__device__ __forceinline__ ChunkDesc chunk_desc(const ChunkArgs& a, int chunk) {
    if (a.g.meta.n == 0) return a.chunks[chunk];
    int n = 0;
    for (int i = 1; i < INLINE_SEQS; ++i)
        if (i < a.g.meta.n && a.g.meta.coff[i] <= chunk) n = i;
    const int pos = (chunk - a.g.meta.coff[n]) * CHUNK_T, t0 = a.g.meta.cu[n] + pos, left = a.g.meta.cu[n + 1] - t0;
    return ChunkDesc{n, t0, left < CHUNK_T ? left : CHUNK_T, pos};
}

cudaError_t launch_chunk_prep(const ChunkArgs& a, cudaStream_t s);
// `after`: the first launch follows another of this call and may start beside its end.
cudaError_t launch_chunks(const ChunkArgs& a, bool after, cudaStream_t s);

}  // namespace ssm
}  // namespace kda
