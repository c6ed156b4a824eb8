// Verification of a round's drafted tokens: the accepted path through each
// session's nodes and the token that follows it.  One CTA per session: the walk
// goes through the nodes in the order of their index (parents come before their
// children, siblings in order), the sums over a row by all threads.
#include "draft_verify.cuh"

namespace kda {
namespace {

constexpr int NT = 256;

template <typename TP> __device__ __forceinline__ double prob(const TP* row, int64_t y) {
    const float v = to_f32(row[y]);
    return v > 0.f && v <= 3.402823466e38f ? (double)v : 0.0;
}

__device__ double block_sum(double v, double* sm) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) sm[threadIdx.x / 32] = v;
    __syncthreads();
    double s = 0.0;
    for (int k = 0; k < NT / 32; ++k) s += sm[k];
    return s;
}

template <typename TP>
__global__ void __launch_bounds__(NT) verify_kernel(const __grid_constant__ VerifyArgs g) {
    __shared__ double sm[NT / 32];
    __shared__ double base[NT];
    __shared__ int found, last;
    const int s = blockIdx.x, tid = threadIdx.x, R = g.R, V = g.V;
    const int32_t *tok = g.tokens + (size_t)s * R, *par = g.parents + (size_t)s * R;
    auto p_row = [&](int r) -> const TP* {
        if (r >= 0) return static_cast<const TP*>(g.p) + s * g.p_ss + r * g.p_rs;
        return g.p_last ? static_cast<const TP*>(g.p_last) + s * g.pl_s : nullptr;
    };
    auto q_row = [&](int r) -> const TP* {
        if (!g.q) return nullptr;
        if (r >= 0) return static_cast<const TP*>(g.q) + s * g.q_ss + r * g.q_rs;
        return g.q_last ? static_cast<const TP*>(g.q_last) + s * g.ql_s : nullptr;
    };
    uint64_t refused = 0;                             // siblings refused at the current node
    auto gone = [&](int y) {
        for (int r = 0; r < R; ++r)
            if ((refused >> r & 1) && tok[r] == y) return true;
        return false;
    };
    double c = 0.0, T = 1.0;
    int cur = -1, len = 0;
    auto W = [&](int y) -> double {
        const double pv = prob(p_row(cur), y);
        if (!g.q) return refused && gone(y) ? 0.0 : pv;
        return c == 0.0 ? pv : fmax(pv - c * prob(q_row(cur), y), 0.0);
    };
    for (int r = 0; r < R && len < g.max_len; ++r) {
        const int x = tok[r];
        if (par[r] != cur || x < 0 || x >= V) continue;
        bool yes = true;
        if (p_row(cur)) {
            const double w = W(x);
            yes = w > 0.0 && (double)g.u[(size_t)s * R + r] * T * (g.q ? prob(q_row(cur), x) : 1.0) < w;
            if (!yes && g.q) {
                c += T;
                double t = 0.0;
                for (int y = tid; y < V; y += NT) t += W(y);
                T = block_sum(t, sm);
            } else if (!yes) {
                T -= w;
                refused |= (uint64_t)1 << r;
            }
        }
        if (yes) {
            if (tid == 0) g.path[(size_t)s * g.max_len + len] = r;
            ++len;
            cur = r;
            c = 0.0;
            T = 1.0;
            refused = 0;
        }
    }
    for (int j = len + tid; j < g.max_len; j += NT) g.path[(size_t)s * g.max_len + j] = -1;
    if (tid == 0) g.path_len[s] = len;
    int next = -1;
    if (p_row(cur)) {
        const int per = (V + NT - 1) / NT, y0 = min(tid * per, V), y1 = min(y0 + per, V);
        for (int pass = 0; pass < 2; ++pass) {
            double t = 0.0;
            for (int y = y0; y < y1; ++y) t += W(y);
            __syncthreads();
            base[tid] = t;
            if (tid == 0) { found = INT32_MAX; last = -1; }
            __syncthreads();
            double before = 0.0, total = 0.0;
            for (int k = 0; k < NT; ++k) {
                if (k == tid) before = total;
                total += base[k];
            }
            if (total > 0.0) {
                const double goal = (double)g.u_next[s] * total;
                for (int y = y0; y < y1; ++y) {
                    const double w = W(y);
                    if (w <= 0.0) continue;
                    atomicMax(&last, y);
                    before += w;
                    if (before > goal) { atomicMin(&found, y); break; }
                }
                __syncthreads();
                next = found != INT32_MAX ? found : last;
                break;
            }
            c = 0.0;                                  // nothing is left: p itself
            refused = 0;
        }
    }
    if (tid == 0) g.next[s] = next;
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int io_bf16, cudaStream_t s) {
    if (io_bf16) verify_kernel<__nv_bfloat16><<<(unsigned)a.n, NT, 0, s>>>(a);
    else verify_kernel<float><<<(unsigned)a.n, NT, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace kda

using namespace kda;

extern "C" kda_status kda_draft_verify(int32_t dtype, int32_t n_sessions, int32_t n_nodes, int32_t vocab, const void* p,
                                       int64_t p_session_stride, int64_t p_row_stride, const void* p_last,
                                       int64_t p_last_stride, const void* q, int64_t q_session_stride,
                                       int64_t q_row_stride, const void* q_last, int64_t q_last_stride,
                                       const int32_t* tokens, const int32_t* parents, const float* u,
                                       const float* u_next, int32_t max_len, int32_t* path, int32_t* path_len,
                                       int32_t* next_token, void* stream) {
    if (dtype != KDA_DTYPE_F32 && dtype != KDA_DTYPE_BF16) return KDA_ERR_INVALID_ARG;
    if (n_sessions < 0 || n_nodes < 1 || n_nodes > KDA_TREE_MAX_NODES || vocab < 1 || max_len < 1 ||
        max_len > KDA_TREE_MAX_NODES)
        return KDA_ERR_INVALID_ARG;
    if (vocab > (1 << 30)) return KDA_ERR_UNSUPPORTED;
    if (n_sessions == 0) return KDA_OK;
    const uintptr_t es = dtype == KDA_DTYPE_BF16 ? 2 : 4;
    auto bad = [](const void* x, uintptr_t align) { return (reinterpret_cast<uintptr_t>(x) & (align - 1)) != 0; };
    if (!p || !tokens || !parents || !u || !u_next || !path || !path_len || !next_token) return KDA_ERR_INVALID_ARG;
    if (bad(p, es) || bad(p_last, es) || bad(q, es) || bad(q_last, es) || bad(tokens, 4) || bad(parents, 4) || bad(u, 4) ||
        bad(u_next, 4) || bad(path, 4) || bad(path_len, 4) || bad(next_token, 4))
        return KDA_ERR_INVALID_ARG;
    if ((q_last != nullptr) != (p_last != nullptr && q != nullptr)) return KDA_ERR_INVALID_ARG;
    // rows may share memory (one distribution for all), but not run backwards
    if (p_session_stride < 0 || p_row_stride < 0 || p_last_stride < 0 || q_session_stride < 0 || q_row_stride < 0 ||
        q_last_stride < 0)
        return KDA_ERR_INVALID_ARG;
    VerifyArgs a{p, p_last, q, q_last, p_session_stride, p_row_stride, p_last_stride, q_session_stride, q_row_stride,
                 q_last_stride, tokens, parents, u, u_next, path, path_len, next_token, n_sessions, n_nodes, vocab, max_len};
    return launch_verify(a, dtype == KDA_DTYPE_BF16, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
