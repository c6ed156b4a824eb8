// C ABI of the state space mixer: host-side checks, workspace layout and the
// launch sequence of each entry point.  As for the KDA entry points, every
// check happens before anything is enqueued.
#include <math.h>

#include <algorithm>
#include <new>
#include <numeric>
#include <vector>

#include "ssm_chunk.cuh"

namespace kda {
namespace ssm {
namespace {

constexpr size_t WS_ALIGN = 256;

size_t align_up(size_t x) { return (x + WS_ALIGN - 1) / WS_ALIGN * WS_ALIGN; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t channels(const kda_ssm_params* p) {
    return (int64_t)p->num_heads * p->head_dim + 2ll * p->num_groups * p->state_dim;
}
size_t esize(const kda_ssm_params* p) { return p->io_dtype == KDA_DTYPE_BF16 ? 2 : 4; }

kda_status check_params(const kda_ssm_params* p) {
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    if (p->num_heads < 1 || p->num_heads > (1 << 16)) return KDA_ERR_INVALID_ARG;
    if (p->num_groups < 1 || p->num_heads % p->num_groups != 0) return KDA_ERR_INVALID_ARG;
    if ((p->head_dim != 64 && p->head_dim != 128) || (p->state_dim != 64 && p->state_dim != 128) ||
        p->conv_kernel != CONV_K)
        return KDA_ERR_UNSUPPORTED;
    if (p->io_dtype != KDA_DTYPE_F32 && p->io_dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARG;
    if (p->algo != KDA_ALGO_AUTO && p->algo != KDA_ALGO_SCAN && p->algo != KDA_ALGO_CHUNKED)
        return p->algo == KDA_ALGO_CHUNKED_SEGMENTS ? KDA_ERR_UNSUPPORTED : KDA_ERR_INVALID_ARG;
    if (!p->conv_w || !p->A_log || !p->dt_bias) return KDA_ERR_INVALID_ARG;
    if (!aligned(p->conv_w, 16) || !aligned(p->conv_b, 16) || !aligned(p->A_log, 4) || !aligned(p->dt_bias, 4) ||
        !aligned(p->D, 4))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// KDA_ALGO_SCAN or KDA_ALGO_CHUNKED, for checked parameters.
kda_status resolve_algo(const kda_ssm_params* p, int* algo) {
    const bool bf16 = p->io_dtype == KDA_DTYPE_BF16;
    if (p->algo == KDA_ALGO_CHUNKED && !bf16) return KDA_ERR_UNSUPPORTED;
    *algo = p->algo == KDA_ALGO_AUTO ? (bf16 ? KDA_ALGO_CHUNKED : KDA_ALGO_SCAN) : p->algo;
    return KDA_OK;
}

// Row strides in elements: 0 is packed; otherwise at least the row's width and,
// for 16-byte rows, a multiple of 16 bytes.
bool row_stride(int64_t given, int64_t width, size_t es, bool rows16, int64_t* out) {
    *out = given == 0 ? width : given;
    if (*out < width || *out > (int64_t)INT32_MAX) return false;
    return !rows16 || (*out * (int64_t)es) % 16 == 0;
}

// The token tensors of a call (rows > 0), and their strides.
kda_status check_tokens(const kda_ssm_params* p, const void* xbc, int64_t* xbc_stride, const void* dt, int64_t* dt_stride,
                        const void* z, int64_t* z_stride, const void* o) {
    const size_t es = esize(p);
    if (!xbc || !dt || !o || !aligned(xbc, 16) || !aligned(dt, es) || !aligned(z, 16) || !aligned(o, 16))
        return KDA_ERR_INVALID_ARG;
    if (!row_stride(*xbc_stride, channels(p), es, true, xbc_stride) ||
        !row_stride(*dt_stride, p->num_heads, es, false, dt_stride) ||
        !row_stride(*z_stride, (int64_t)p->num_heads * p->head_dim, es, z != nullptr, z_stride))
        return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

constexpr int SMS_GB300 = 152;

// Units of 128 channels: two heads of 64 or one of 128, within a group.
int units_per_group(const kda_ssm_params* p) {
    return (int)(((int64_t)(p->num_heads / p->num_groups) * p->head_dim + 127) / 128);
}

// The most (sequence, piece) slots a call may cut its sequences into: enough
// for two CTAs per SM, or four pieces each where the sequences alone fill the
// SMs (a long one among short ones still is the last to end); none from eight
// sequence-units per SM on.
int64_t piece_slots(const kda_ssm_params* p, int64_t n_seqs) {
    const int64_t units = (int64_t)units_per_group(p) * p->num_groups;
    if (n_seqs * units >= 8 * SMS_GB300) return 0;
    return std::max<int64_t>(2 * SMS_GB300 / units, 4 * n_seqs);
}
// The most of any call of up to n_seqs sequences: a workspace for a full batch serves the
// smaller ones, whose sequences are the ones that are cut.
int64_t most_piece_slots(const kda_ssm_params* p, int64_t n_seqs) {
    const int64_t units = (int64_t)units_per_group(p) * p->num_groups;
    return piece_slots(p, std::min(n_seqs, (8 * SMS_GB300 - 1) / units));
}

// Workspace of a prefill: error word | cu_seqlens | first chunks | order, and
// for the chunked form chunk table | step records | scales | group records |
// piece end states and decays.
struct Layout {
    size_t cu = 0, coff = 0, order = 0, chunks = 0, step = 0, scale = 0, rec = 0, local = 0, ltot = 0, total = 0;
};
Layout layout(const kda_ssm_params* p, int algo, int64_t n_seqs, int64_t total_tokens, int64_t slots) {
    Layout L;
    size_t off = WS_ALIGN;
    auto take = [&](size_t bytes) { const size_t at = off; off = align_up(off + bytes); return at; };
    L.cu = take(sizeof(int64_t) * ((size_t)n_seqs + 1));
    L.coff = take(sizeof(int64_t) * ((size_t)n_seqs + 1));
    L.order = take(sizeof(int32_t) * (size_t)n_seqs);
    if (algo == KDA_ALGO_CHUNKED) {
        // every sequence may end in a partial chunk
        const size_t nck = (size_t)(total_tokens / CHUNK_T + std::min(n_seqs, total_tokens));
        const size_t H = p->num_heads, G = p->num_groups;
        L.chunks = take(sizeof(ChunkDesc) * nck);
        L.step = take(sizeof(float) * STEP_FLOATS * nck * H);
        L.scale = take(sizeof(int4) * nck * G);
        L.rec = take(rec_bytes(p->state_dim) * nck * G);
        L.local = take(sizeof(float) * (size_t)slots * H * p->state_dim * p->head_dim);
        L.ltot = take(sizeof(float) * (size_t)slots * H);
    }
    L.total = off;
    return L;
}

// One launch of chunk walks on the SMs, one CTA each, in launch order: every SM
// takes the next walk when it is free.  SMs that are free at the same time are
// kept as one entry.
class Schedule {
public:
    void add(int64_t walks, double time) {
        while (walks > 0) {
            const Entry e = free_[0];
            const int64_t each = walks / SMS_GB300;          // whole waves of a large equal lot
            if (n_ == 1 && each > 0) {
                free_[0].at += time * (double)each;
                walks -= each * SMS_GB300;
                continue;
            }
            const int m = (int)std::min<int64_t>(e.count, walks);
            if (m == e.count) {
                for (int i = 1; i < n_; ++i) free_[i - 1] = free_[i];
                --n_;
            } else {
                free_[0].count -= m;
            }
            int i = n_;                                      // after the entries of at <= e.at + time
            while (i > 0 && free_[i - 1].at > e.at + time) --i;
            if (i > 0 && free_[i - 1].at == e.at + time) {
                free_[i - 1].count += m;
            } else {
                for (int x = n_; x > i; --x) free_[x] = free_[x - 1];
                free_[i] = Entry{e.at + time, m};
                ++n_;
            }
            walks -= m;
        }
    }
    double end() const { return free_[n_ - 1].at; }

private:
    struct Entry {
        double at;
        int count;
    };
    Entry free_[SMS_GB300 + 1] = {{0.0, SMS_GB300}};
    int n_ = 1;
};

// Pieces of a sequence: the first of lp0 chunks, then up to np - 1 of lp.  The
// first launch walks the first pieces in full and, beside them, the pieces up to
// the last but one for their end state only; the second walks all but the first.
// A cut pays where the sequences' units leave SMs idle, all along or while the
// longest one ends.  Both launches are played through for a range of cuts, walks
// in the order sequence by sequence or piece by piece; the host does it while the
// preparation runs (3 to 40 us).  With equal pieces and the first ones cut short
// in the first launch too, 32768 tokens x 96 heads took 0.96 ms instead of 0.82, and
// 8 sequences of 6 to 388 chunks x 64 heads 1.08 instead of 0.95.
struct Pieces {
    int np = 1, lp0 = 1, lp = 1;
    bool by_piece = false;
};
Pieces plan_pieces(const kda_ssm_params* p, const int64_t* cu, const int32_t* order, int32_t n_seqs) {
    const int64_t units = (int64_t)units_per_group(p) * p->num_groups, slots = piece_slots(p, n_seqs);
    auto chunks = [&](int32_t i) { return (cu[order[i] + 1] - cu[order[i]] + CHUNK_T - 1) / CHUNK_T; };
    const int64_t longest = std::max<int64_t>(1, chunks(0));
    Pieces best;
    best.lp0 = (int)longest;
    constexpr int64_t MIN_CHUNKS = 4;                    // of the longest sequence, per piece
    if (2 * (int64_t)n_seqs > slots || longest < 2 * MIN_CHUNKS) return best;
    // in chunks of a full walk: a chunk of a walk for the end state, a walk's start (state,
    // first loads), and the end state of a piece before it that it reads
    constexpr double LITE = 0.65, START = 4, COMPOSE = 0.5;
    constexpr int LOTS = 16;                             // more sequences count as lots of neighbours in length
    int64_t lot[LOTS], lots = 0;
    const int64_t per = (n_seqs + LOTS - 1) / LOTS;
    for (int64_t i = 0; i < n_seqs; i += per) lot[lots++] = chunks((int32_t)i);
    const int64_t walks = units * per;                   // of one piece of a lot

    double best_t = 0;
    auto play = [&](int64_t np, int64_t lp0, int64_t lp, bool by_piece) {
        Schedule first, second;
        auto pieces = [&](int64_t i) { return (std::max<int64_t>(0, lot[i] - lp0) + lp - 1) / lp; };   // but the first
        auto lead = [&](int64_t i) { first.add(walks, START + (double)std::min(lot[i], lp0)); };
        auto lite = [&](int64_t n) { first.add(walks * n, START + LITE * (double)lp); };
        auto full = [&](int64_t i, int64_t q) {              // piece 1 + q of lot i
            second.add(walks, START + COMPOSE * (double)q + (double)std::min(lp, lot[i] - lp0 - q * lp));
        };
        if (by_piece) {
            for (int64_t i = 0; i < lots; ++i) lead(i);
            for (int64_t q = 0; q < np - 1; ++q)
                for (int64_t i = 0; i < lots && pieces(i) > q; ++i) {
                    if (pieces(i) > q + 1) lite(1);
                    full(i, q);
                }
        } else {
            for (int64_t i = 0; i < lots; ++i) {
                const int64_t k = pieces(i);
                lead(i);
                if (k == 0) continue;
                lite(k - 1);
                for (int64_t q = 0; q < k; ++q) full(i, q);
            }
        }
        const double t = first.end() + second.end();
        if (best_t == 0 || t < best_t) {
            best_t = t;
            best = Pieces{(int)np, (int)lp0, (int)lp, by_piece};
        }
    };
    play(1, longest, 1, false);
    // np in steps of a quarter, the first piece from as long as a lite walk of another to a
    // few of them
    for (int64_t np = 2; np * n_seqs <= slots && longest >= np * MIN_CHUNKS; np += std::max<int64_t>(1, np / 4))
        for (const double r : {LITE, 1.0, 1.6, 2.4, 3.6}) {
            const int64_t lp = (int64_t)ceil((double)longest / ((double)(np - 1) + r));
            const int64_t lp0 = std::max<int64_t>(1, longest - (np - 1) * lp);
            play(np, lp0, lp, false);
            if (lots > 1) play(np, lp0, lp, true);
        }
    return best;
}

}  // namespace
}  // namespace ssm
}  // namespace kda

using namespace kda;
using namespace kda::ssm;

extern "C" {

int32_t kda_ssm_prefill_algo(const kda_ssm_params* p) {
    int algo;
    if (ssm::check_params(p) != KDA_OK || ssm::resolve_algo(p, &algo) != KDA_OK) return -1;
    return algo;
}

size_t kda_ssm_prefill_workspace_bytes(const kda_ssm_params* p, int32_t n_seqs, int64_t total_tokens) {
    int algo;
    if (ssm::check_params(p) != KDA_OK || ssm::resolve_algo(p, &algo) != KDA_OK || n_seqs < 0 || total_tokens < 0)
        return 0;
    if (n_seqs == 0) return 0;
    return ssm::layout(p, algo, n_seqs, total_tokens, ssm::most_piece_slots(p, n_seqs)).total;
}

kda_status kda_ssm_prefill(const kda_ssm_params* p, const void* xbc, int64_t xbc_stride, const void* dt,
                           int64_t dt_stride, const void* z, int64_t z_stride, const int64_t* cu, int32_t n_seqs,
                           int64_t total_tokens, const float* S_in, float* S_out, const void* ring_in, void* ring_out,
                           void* o, void* workspace, size_t workspace_bytes, void* stream_) {
    int algo;
    kda_status st = ssm::check_params(p);
    if (st != KDA_OK || (st = ssm::resolve_algo(p, &algo)) != KDA_OK) return st;
    if (n_seqs < 0 || total_tokens < 0 || cu == nullptr || cu[0] != 0 || cu[n_seqs] != total_tokens)
        return KDA_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n_seqs; ++i)
        if (cu[i + 1] < cu[i]) return KDA_ERR_INVALID_ARG;
    if (total_tokens > (int64_t)INT32_MAX) return KDA_ERR_UNSUPPORTED;
    if (n_seqs == 0) return KDA_OK;
    if (total_tokens > 0 && (st = check_tokens(p, xbc, &xbc_stride, dt, &dt_stride, z, &z_stride, o)) != KDA_OK) return st;
    if (S_out == nullptr || !aligned(S_out, 16) || !aligned(S_in, 16) || !aligned(ring_in, 16) || !aligned(ring_out, 16))
        return KDA_ERR_INVALID_ARG;
    // CTAs of the largest launch: pieces of units, the preparation's blocks, column slices
    const int64_t chunks_most = total_tokens / CHUNK_T + std::min<int64_t>(n_seqs, total_tokens);
    if ((int64_t)n_seqs * p->num_heads * 8 > (int64_t)INT32_MAX ||
        chunks_most * (p->num_groups + p->num_heads / 32 + 1) > (int64_t)INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    if (workspace == nullptr || !aligned(workspace, WS_ALIGN) ||
        workspace_bytes < ssm::layout(p, algo, n_seqs, total_tokens, ssm::piece_slots(p, n_seqs)).total)
        return KDA_ERR_WORKSPACE;

    cudaStream_t s = static_cast<cudaStream_t>(stream_);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    const Layout L = ssm::layout(p, algo, n_seqs, total_tokens, ssm::piece_slots(p, n_seqs));
    // longest sequences first: their walks take longest
    std::vector<int32_t> order;
    try {
        order.resize(n_seqs);
        std::iota(order.begin(), order.end(), 0);
        std::stable_sort(order.begin(), order.end(),
                         [&](int32_t x, int32_t y) { return cu[x + 1] - cu[x] > cu[y + 1] - cu[y]; });
    } catch (const std::bad_alloc&) {
        return KDA_ERR_CUDA;
    }
    int64_t* d_cu = reinterpret_cast<int64_t*>(ws + L.cu);
    int32_t* d_order = reinterpret_cast<int32_t*>(ws + L.order);
    const bool chunked = algo == KDA_ALGO_CHUNKED;
    int64_t* d_coff = reinterpret_cast<int64_t*>(ws + L.coff);
    ChunkDesc* d_chunks = chunked ? reinterpret_cast<ChunkDesc*>(ws + L.chunks) : nullptr;
    int64_t n_chunks = 0;
    for (int32_t i = 0; i < n_seqs; ++i) n_chunks += (cu[i + 1] - cu[i] + CHUNK_T - 1) / CHUNK_T;
    const bool in_args = n_seqs <= INLINE_SEQS;
    // (the chunk preparation and the scan clear the error word themselves)
    if (chunked && n_chunks == 0 && cudaMemsetAsync(ws, 0, WS_ALIGN, s) != cudaSuccess) return KDA_ERR_CUDA;
    if (!in_args && build_meta(cu, order.data(), n_seqs, 0, d_cu, d_coff, d_order, d_chunks, s) != cudaSuccess)
        return KDA_ERR_CUDA;
    const int io_bf16 = p->io_dtype == KDA_DTYPE_BF16;
    ssm::PrefillArgs a{xbc, dt, z, xbc_stride, dt_stride, z_stride, p->conv_w, p->conv_b, p->A_log, p->dt_bias, p->D,
                       S_in, S_out, ring_in, ring_out, o, d_cu, d_order, n_seqs, p->num_heads, p->num_groups, p->head_dim,
                       p->state_dim, total_tokens, {}};
    if (in_args) {
        a.meta.n = n_seqs;
        for (int32_t i = 0; i <= n_seqs; ++i) {
            a.meta.cu[i] = (int32_t)cu[i];
            a.meta.coff[i] = i == 0 ? 0 : a.meta.coff[i - 1] + (int32_t)((cu[i] - cu[i - 1] + CHUNK_T - 1) / CHUNK_T);
            if (i < n_seqs) a.meta.order[i] = (uint8_t)order[i];
        }
    }
    if (chunked) {
        ChunkArgs c{};
        c.g = a;
        const int64_t Cx = channels(p);
        if (total_tokens > 0 && (!encode_rows(&c.map67, xbc, 2, total_tokens, Cx, xbc_stride, CHUNK_T + RING, 128) ||
                                 !encode_rows(&c.map64, xbc, 2, total_tokens, Cx, xbc_stride, CHUNK_T, 128)))
            return KDA_ERR_CUDA;
        c.chunks = d_chunks;
        c.coff = d_coff;
        c.rec = ws + L.rec;
        c.step = reinterpret_cast<float*>(ws + L.step);
        c.scale = reinterpret_cast<int4*>(ws + L.scale);
        c.status = reinterpret_cast<int32_t*>(ws);
        c.local = reinterpret_cast<float*>(ws + L.local);
        c.ltot = reinterpret_cast<float*>(ws + L.ltot);
        c.n_chunks = (int32_t)n_chunks;
        c.upg = units_per_group(p);
        c.units = c.upg * p->num_groups;
        if (ssm::launch_chunk_prep(c, s) != cudaSuccess) return KDA_ERR_CUDA;
        const Pieces pc = plan_pieces(p, cu, order.data(), n_seqs);
        c.np = pc.np;
        c.lp0 = pc.lp0;
        c.lp = pc.lp;
        c.by_piece = pc.by_piece;
        // the passes may start beside the preparation's end when all its blocks run at once
        // (2 us of a short call; behind a longer preparation they only take its SMs: 32768
        // tokens x 96 heads 1.02 ms, without 0.99)
        const bool beside = n_chunks > 0 && n_chunks * (p->num_groups + p->num_heads / 32 + 1) <= 2 * SMS_GB300;
        return launch_chunks(c, beside, s) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
    }
    if (ssm::launch_scan(a, io_bf16, reinterpret_cast<int32_t*>(ws), s) != cudaSuccess) return KDA_ERR_CUDA;
    if (ring_out && ssm::launch_ring(a, io_bf16, s) != cudaSuccess) return KDA_ERR_CUDA;
    return KDA_OK;
}

size_t kda_ssm_decode_workspace_bytes(const kda_ssm_params* p, int32_t n_sessions) {
    if (ssm::check_params(p) != KDA_OK || n_sessions <= 0) return 0;
    if (!ssm::decode_needs_workspace(n_sessions, p->num_heads, p->num_groups, p->head_dim, p->state_dim)) return 0;
    return ssm::align_up((size_t)n_sessions * ((size_t)channels(p) * sizeof(float) + (size_t)p->num_heads * sizeof(float2)));
}

kda_status kda_ssm_decode(const kda_ssm_params* p, int32_t n_sessions, const void* xbc, int64_t xbc_stride,
                          const void* dt, int64_t dt_stride, const void* z, int64_t z_stride, const int32_t* slots,
                          int32_t n_slots, float* S, void* ring, void* o, void* workspace, size_t workspace_bytes,
                          void* stream_) {
    kda_status st = ssm::check_params(p);
    if (st != KDA_OK) return st;
    if (n_sessions < 0 || n_slots < 0) return KDA_ERR_INVALID_ARG;
    if (n_sessions == 0) return KDA_OK;
    if (slots == nullptr ? n_slots < n_sessions : !aligned(slots, 4)) return KDA_ERR_INVALID_ARG;
    if ((st = check_tokens(p, xbc, &xbc_stride, dt, &dt_stride, z, &z_stride, o)) != KDA_OK) return st;
    if (!S || !ring || !aligned(S, 16) || !aligned(ring, 16)) return KDA_ERR_INVALID_ARG;
    if ((int64_t)n_sessions * channels(p) > (int64_t)INT32_MAX) return KDA_ERR_UNSUPPORTED;
    const size_t need = kda_ssm_decode_workspace_bytes(p, n_sessions);
    if (need > 0 && (workspace == nullptr || !aligned(workspace, WS_ALIGN) || workspace_bytes < need))
        return KDA_ERR_WORKSPACE;
    if ((int64_t)n_sessions * p->num_heads * 2 > (int64_t)INT32_MAX) return KDA_ERR_UNSUPPORTED;   // CTAs of the launch
    float* const u = need > 0 ? static_cast<float*>(workspace) : nullptr;
    float2* const step = u ? reinterpret_cast<float2*>(u + (size_t)n_sessions * channels(p)) : nullptr;   // (8-byte aligned)
    ssm::DecodeArgs a{xbc, dt, z, xbc_stride, dt_stride, z_stride, p->conv_w, p->conv_b, p->A_log, p->dt_bias, p->D,
                      slots, S, ring, o, u, step, n_sessions, n_slots, p->num_heads, p->num_groups, p->head_dim,
                      p->state_dim};
    return ssm::launch_decode(a, p->io_dtype == KDA_DTYPE_BF16, static_cast<cudaStream_t>(stream_)) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
