// C ABI of the gated linear recurrence: host-side checks, workspace layout and
// the launch sequence of each entry point.  Every check happens before anything
// is enqueued.
#include <new>
#include <vector>

#include "glr_common.cuh"

namespace kda {
namespace glr {
namespace {

constexpr size_t WS_ALIGN = 256;

size_t align_up(size_t x) { return (x + WS_ALIGN - 1) / WS_ALIGN * WS_ALIGN; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t esize(const kda_glr_params* p) { return p->io_dtype == KDA_DTYPE_BF16 ? 2 : 4; }

constexpr int32_t MAX_CHANNELS = 1 << 24;

kda_status check_params(const kda_glr_params* p) {
    if (p == nullptr) return KDA_ERR_INVALID_ARG;
    if (p->channels < 1 || p->channels > MAX_CHANNELS) return KDA_ERR_INVALID_ARG;
    if (p->io_dtype != KDA_DTYPE_F32 && p->io_dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARG;
    if (!p->A_log || !aligned(p->A_log, 4) || !aligned(p->r_bias, 4) || !aligned(p->i_bias, 4)) return KDA_ERR_INVALID_ARG;
    return KDA_OK;
}

// Row strides in elements: their bytes fit 32 bits.
constexpr int64_t MAX_STRIDE = (int64_t)1 << 30;

// A token tensor: element alignment, a row stride of 0 (packed) or at least C.
bool rows(const kda_glr_params* p, const void* base, bool needed, int64_t* stride) {
    if (*stride == 0) *stride = p->channels;
    if (base == nullptr) return !needed;
    return aligned(base, esize(p)) && *stride >= p->channels && *stride < MAX_STRIDE;
}

kda_status check_batch(const int64_t* cu, int32_t n_seqs, int64_t total_tokens) {
    if (n_seqs < 0 || total_tokens < 0 || cu == nullptr || cu[0] != 0 || cu[n_seqs] != total_tokens)
        return KDA_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n_seqs; ++i)
        if (cu[i + 1] < cu[i]) return KDA_ERR_INVALID_ARG;
    return total_tokens > (int64_t)INT32_MAX ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

// Workspace: error word | gates | ticket | the tiles' maps and values | token offsets and rows
// of the sequences | the tiles' borders | partial sums (backward pass).
struct Layout {
    size_t gates = 0, ticket = 0, map = 0, val = 0, cu = 0, id = 0, tile = 0, part = 0, total = 0;
    int64_t tiles_t = 0, tiles_c = 0;
};
Layout layout(const kda_glr_params* p, int32_t n_seqs, int64_t total_tokens, bool backward) {
    Layout L;
    L.tiles_t = (total_tokens + CHUNK - 1) / CHUNK;
    L.tiles_c = (p->channels + TILE_C - 1) / TILE_C;
    const size_t tiles = (size_t)L.tiles_t * L.tiles_c;
    size_t off = WS_ALIGN;
    auto take = [&](size_t bytes) { const size_t at = off; off = align_up(off + bytes); return at; };
    L.gates = take(sizeof(float) * 3 * TILE_C * (size_t)L.tiles_c);
    L.ticket = take(WS_ALIGN);
    L.map = take(sizeof(float) * 2 * TILE_C * tiles);
    L.val = take(sizeof(float) * TILE_C * tiles);
    L.cu = take(sizeof(int64_t) * ((size_t)n_seqs + 1));
    L.id = take(sizeof(int32_t) * (size_t)n_seqs);
    L.tile = take(sizeof(uint4) * (size_t)L.tiles_t);
    if (backward) L.part = take(sizeof(float) * 3 * (size_t)L.tiles_t * p->channels);
    L.total = off;
    return L;
}

// What the two walks share: the sequences with tokens, and the workspace's parts.
// (The walks set the workspace up themselves.)
cudaError_t prepare(const kda_glr_params* p, const int64_t* cu, int32_t n_seqs, unsigned char* ws, const Layout& L,
                    ScanArgs* a, cudaStream_t s) {
    a->status = reinterpret_cast<int32_t*>(ws);
    a->gates = reinterpret_cast<float2*>(ws + L.gates);
    a->ticket = reinterpret_cast<uint32_t*>(ws + L.ticket);
    a->borders = reinterpret_cast<uint4*>(ws + L.tile);
    a->map = reinterpret_cast<float*>(ws + L.map);
    a->val = reinterpret_cast<float*>(ws + L.val);
    a->part = reinterpret_cast<float*>(ws + L.part);
    a->tiles_t = (int32_t)L.tiles_t;
    a->tiles_c = (int32_t)L.tiles_c;
    if (L.tiles_t == 0) return cudaMemsetAsync(ws, 0, WS_ALIGN, s);
    Sequences& f = a->f;
    // one place along T waits for nothing: the ticket alone
    a->empty = (L.tiles_t > 1 ? L.val - L.ticket + sizeof(float) * TILE_C * (size_t)(L.tiles_t * L.tiles_c) : WS_ALIGN) / sizeof(uint4);
    f.d_cu = reinterpret_cast<int64_t*>(ws + L.cu);
    f.d_id = reinterpret_cast<int32_t*>(ws + L.id);
    f.n = 0;
    for (int32_t i = 0; i < n_seqs; ++i) f.n += cu[i + 1] > cu[i];
    if (f.n <= INLINE_SEQS) {
        int k = 0;
        for (int32_t i = 0; i < n_seqs; ++i)
            if (cu[i + 1] > cu[i]) {
                f.cu[k] = (int32_t)cu[i];
                f.id[k++] = i;
            }
        f.cu[k] = (int32_t)cu[n_seqs];
        return cudaSuccess;
    }
    std::vector<int64_t> start;
    std::vector<int32_t> id;
    try {
        start.reserve((size_t)f.n + 1);
        id.reserve((size_t)f.n);
        for (int32_t i = 0; i < n_seqs; ++i)
            if (cu[i + 1] > cu[i]) {
                start.push_back(cu[i]);
                id.push_back(i);
            }
        start.push_back(cu[n_seqs]);
    } catch (const std::bad_alloc&) {
        return cudaErrorMemoryAllocation;
    }
    return build_meta(start.data(), id.data(), f.n, 0, const_cast<int64_t*>(f.d_cu), nullptr, const_cast<int32_t*>(f.d_id),
                   nullptr, s);
}

// Copies the state of sequences without tokens, if there are any (all states: the walk then
// writes those of the others).
cudaError_t copy_states(const kda_glr_params* p, const int64_t* cu, int32_t n_seqs, const float* from, float* to,
                        cudaStream_t s) {
    bool any = false;
    for (int32_t i = 0; i < n_seqs; ++i) any |= cu[i + 1] == cu[i];
    if (!any || from == to) return cudaSuccess;
    const size_t bytes = sizeof(float) * (size_t)n_seqs * p->channels;
    return from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(to, 0, bytes, s);
}

}  // namespace
}  // namespace glr
}  // namespace kda

using namespace kda;
using namespace kda::glr;

extern "C" {

size_t kda_glr_prefill_workspace_bytes(const kda_glr_params* p, int32_t n_seqs, int64_t total_tokens) {
    if (glr::check_params(p) != KDA_OK || n_seqs <= 0 || total_tokens < 0 || total_tokens > (int64_t)INT32_MAX) return 0;
    return glr::layout(p, n_seqs, total_tokens, false).total;
}

size_t kda_glr_backward_workspace_bytes(const kda_glr_params* p, int32_t n_seqs, int64_t total_tokens) {
    if (glr::check_params(p) != KDA_OK || n_seqs <= 0 || total_tokens < 0 || total_tokens > (int64_t)INT32_MAX) return 0;
    return glr::layout(p, n_seqs, total_tokens, true).total;
}

kda_status kda_glr_prefill(const kda_glr_params* p, const void* x, int64_t x_stride, const void* r, int64_t r_stride,
                           const void* i, int64_t i_stride, const void* z, int64_t z_stride, const int64_t* cu,
                           int32_t n_seqs, int64_t total_tokens, const float* S_in, float* S_out, float* states, void* o,
                           void* workspace, size_t workspace_bytes, void* stream) {
    kda_status st = glr::check_params(p);
    if (st != KDA_OK || (st = check_batch(cu, n_seqs, total_tokens)) != KDA_OK) return st;
    if (n_seqs == 0) return KDA_OK;
    const bool any = total_tokens > 0;
    if (!glr::rows(p, x, any, &x_stride) || !glr::rows(p, r, any, &r_stride) || !glr::rows(p, i, any, &i_stride) ||
        !glr::rows(p, z, false, &z_stride) || (any && !o) || !aligned(o, esize(p)))
        return KDA_ERR_INVALID_ARG;
    if (!S_out || !aligned(S_out, 4) || !aligned(S_in, 4) || !aligned(states, 4)) return KDA_ERR_INVALID_ARG;
    const Layout L = glr::layout(p, n_seqs, total_tokens, false);
    if (L.tiles_t * L.tiles_c > (int64_t)INT32_MAX / 2) return KDA_ERR_UNSUPPORTED;
    if (workspace == nullptr || !aligned(workspace, WS_ALIGN) || workspace_bytes < L.total) return KDA_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    glr::ScanArgs a{};
    a.x = x; a.r = r; a.i = i; a.z = z;
    const uint32_t es = (uint32_t)esize(p);
    a.x_s = (uint32_t)x_stride * es; a.r_s = (uint32_t)r_stride * es;
    a.i_s = (uint32_t)i_stride * es; a.z_s = (uint32_t)z_stride * es;
    a.A_log = p->A_log; a.r_bias = p->r_bias; a.i_bias = p->i_bias;
    a.S_in = S_in; a.S_out = S_out; a.states = states; a.o = o; a.o_s = (uint32_t)p->channels * es;
    a.T = total_tokens; a.C = p->channels;
    if (copy_states(p, cu, n_seqs, S_in, S_out, s) != cudaSuccess || glr::prepare(p, cu, n_seqs, ws, L, &a, s) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (!any) return KDA_OK;
    return glr::launch_scan(a, p->io_dtype == KDA_DTYPE_BF16, s) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_glr_backward(const kda_glr_params* p, const void* x, int64_t x_stride, const void* r, int64_t r_stride,
                            const void* i, int64_t i_stride, const void* z, int64_t z_stride, const int64_t* cu,
                            int32_t n_seqs, int64_t total_tokens, const float* S_in, const float* states, const void* d_o,
                            int64_t do_stride, const float* dS_out, void* dx, int64_t dx_stride, void* dr,
                            int64_t dr_stride, void* di, int64_t di_stride, void* dz, int64_t dz_stride, float* dS_in,
                            float* dA_log, float* dr_bias, float* di_bias, void* workspace, size_t workspace_bytes,
                            void* stream) {
    kda_status st = glr::check_params(p);
    if (st != KDA_OK || (st = check_batch(cu, n_seqs, total_tokens)) != KDA_OK) return st;
    const bool any = total_tokens > 0;
    if (!glr::rows(p, x, any, &x_stride) || !glr::rows(p, r, any, &r_stride) || !glr::rows(p, i, any, &i_stride) ||
        !glr::rows(p, z, false, &z_stride) || !glr::rows(p, d_o, any, &do_stride) || !glr::rows(p, dx, any, &dx_stride) ||
        !glr::rows(p, dr, any, &dr_stride) || !glr::rows(p, di, any, &di_stride) ||
        !glr::rows(p, dz, any && z != nullptr, &dz_stride) || (dz != nullptr && z == nullptr) || (any && !states))
        return KDA_ERR_INVALID_ARG;
    if (dS_in != nullptr && dS_in == dS_out) return KDA_ERR_INVALID_ARG;   // (a tile may write the one before it reads the other)
    if (!dA_log || !aligned(S_in, 4) || !aligned(states, 4) || !aligned(dS_out, 4) || !aligned(dS_in, 4) ||
        !aligned(dA_log, 4) || !aligned(dr_bias, 4) || !aligned(di_bias, 4))
        return KDA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto empty_sums = [&]() {
        for (float* sum : {dA_log, dr_bias, di_bias})
            if (sum && cudaMemsetAsync(sum, 0, sizeof(float) * p->channels, s) != cudaSuccess) return KDA_ERR_CUDA;
        return KDA_OK;
    };
    if (n_seqs == 0) return empty_sums();
    const Layout L = glr::layout(p, n_seqs, total_tokens, true);
    if (L.tiles_t * L.tiles_c > (int64_t)INT32_MAX / 2) return KDA_ERR_UNSUPPORTED;
    if (workspace == nullptr || !aligned(workspace, WS_ALIGN) || workspace_bytes < L.total) return KDA_ERR_WORKSPACE;
    unsigned char* ws = static_cast<unsigned char*>(workspace);
    glr::ScanArgs a{};
    a.x = x; a.r = r; a.i = i; a.z = z;
    const uint32_t es = (uint32_t)esize(p);
    a.x_s = (uint32_t)x_stride * es; a.r_s = (uint32_t)r_stride * es;
    a.i_s = (uint32_t)i_stride * es; a.z_s = (uint32_t)z_stride * es;
    a.A_log = p->A_log; a.r_bias = p->r_bias; a.i_bias = p->i_bias;
    a.S_in = S_in; a.states = const_cast<float*>(states);
    a.d_o = d_o; a.do_s = (uint32_t)do_stride * es; a.dS_out = dS_out;
    a.dx = dx; a.dr = dr; a.di = di; a.dz = dz;
    a.dx_s = (uint32_t)dx_stride * es; a.dr_s = (uint32_t)dr_stride * es;
    a.di_s = (uint32_t)di_stride * es; a.dz_s = (uint32_t)dz_stride * es;
    a.dS_in = dS_in; a.dA_log = dA_log; a.dr_bias = dr_bias; a.di_bias = di_bias;
    a.T = total_tokens; a.C = p->channels;
    if ((dS_in && copy_states(p, cu, n_seqs, dS_out, dS_in, s) != cudaSuccess) ||
        glr::prepare(p, cu, n_seqs, ws, L, &a, s) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (!any) return empty_sums();
    return glr::launch_backward(a, p->io_dtype == KDA_DTYPE_BF16, s) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

static kda_status tokens_call(const kda_glr_params* p, int32_t n_sessions, int32_t n_tokens, const void* x, int64_t x_stride,
                              const void* r, int64_t r_stride, const void* i, int64_t i_stride, const void* z,
                              int64_t z_stride, const int32_t* path, const int32_t* path_len, int32_t max_len,
                              const int32_t* slots, int32_t n_slots, const float* S_in, float* S_out, void* o,
                              void* stream) {
    kda_status st = glr::check_params(p);
    if (st != KDA_OK) return st;
    if (n_sessions < 0 || n_slots < 0 || n_tokens < 1 || n_tokens > KDA_DECODE_MAX_TOKENS) return KDA_ERR_INVALID_ARG;
    if (n_sessions == 0) return KDA_OK;
    if (slots == nullptr ? n_slots < n_sessions : !aligned(slots, 4)) return KDA_ERR_INVALID_ARG;
    if (!glr::rows(p, x, true, &x_stride) || !glr::rows(p, r, true, &r_stride) || !glr::rows(p, i, true, &i_stride) ||
        !glr::rows(p, z, false, &z_stride) || !aligned(o, esize(p)) || !S_in || !aligned(S_in, 4) || !aligned(S_out, 4))
        return KDA_ERR_INVALID_ARG;
    if ((int64_t)n_sessions * ((p->channels + 127) / 128) > (int64_t)INT32_MAX) return KDA_ERR_UNSUPPORTED;
    const uint32_t es = (uint32_t)esize(p);
    glr::TokenArgs a{x, r, i, z, (uint32_t)x_stride * es, (uint32_t)r_stride * es, (uint32_t)i_stride * es,
                     (uint32_t)z_stride * es, p->A_log, p->r_bias, p->i_bias, path, path_len,
                     slots, S_in, S_out, o, n_sessions, n_tokens, max_len, n_slots, p->channels};
    return glr::launch_tokens(a, p->io_dtype == KDA_DTYPE_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_glr_decode(const kda_glr_params* p, int32_t n_sessions, int32_t n_tokens, const void* x, int64_t x_stride,
                          const void* r, int64_t r_stride, const void* i, int64_t i_stride, const void* z,
                          int64_t z_stride, const int32_t* slots, int32_t n_slots, const float* S_in, float* S_out,
                          void* o, void* stream) {
    if (n_sessions > 0 && !o) return KDA_ERR_INVALID_ARG;
    return tokens_call(p, n_sessions, n_tokens, x, x_stride, r, r_stride, i, i_stride, z, z_stride, nullptr, nullptr, 0,
                       slots, n_slots, S_in, S_out, o, stream);
}

kda_status kda_glr_commit(const kda_glr_params* p, int32_t n_sessions, int32_t n_nodes, const void* x, int64_t x_stride,
                          const void* r, int64_t r_stride, const void* i, int64_t i_stride, const int32_t* path,
                          const int32_t* path_len, int32_t max_len, const int32_t* slots, int32_t n_slots,
                          const float* S_in, float* S_out, void* stream) {
    if (max_len < 1 || max_len > KDA_TREE_MAX_NODES) return KDA_ERR_INVALID_ARG;
    if (n_sessions > 0 && (!S_out || !path || !path_len || !aligned(path, 4) || !aligned(path_len, 4)))
        return KDA_ERR_INVALID_ARG;
    return tokens_call(p, n_sessions, n_nodes, x, x_stride, r, r_stride, i, i_stride, nullptr, 0, path, path_len, max_len,
                       slots, n_slots, S_in, S_out, nullptr, stream);
}

}  // extern "C"
