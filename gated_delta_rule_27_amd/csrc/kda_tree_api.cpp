// kda_tree_api.cpp -- the C ABI of tree speculative decoding (declared in
// include/kda.h): argument checks on the host before any HIP call, as in
// kda_api.cpp, then one launcher call each.
#include "kda.h"

#include <stdint.h>

#include <limits>

#include "kda_check.h"
#include "kda_launch.h"
#include "kda_tree.h"

using namespace kda::check;

namespace {

// A launch holds fewer than 2^32 threads: workgroups of 256, of which a call
// has twice as many as (sequence, head) pairs at the most; kda_tree_accept's
// are of 1024, one per sequence.
constexpr uint64_t kMaxUnits = (((uint64_t)1 << 32) - 1) / 256 / 2;
constexpr int32_t kMaxAccept = (((int64_t)1 << 32) - 1) / 1024;

// B sequences of N nodes with H heads
bool tree_shape(int32_t B, int32_t N, int32_t H, int32_t most) {
    if (B < 0 || N < 1 || N > most || H < 1 || H > KDA_MAX_HEADS) return false;
    if ((uint64_t)B * (uint64_t)H > kMaxUnits) return false;
    return (uint64_t)B * (uint64_t)N * (uint64_t)H <= kMaxElems / kda::kHeadDim;
}

bool all_aligned(std::initializer_list<const void*> ps, uintptr_t a) {
    for (const void* p : ps)
        if (p && !aligned(p, a)) return false;
    return true;
}

Span counts(const int32_t* p, uint64_t n) { return span(p, n * 4); }

}  // namespace

extern "C" {

kda_status kda_tree_prologue(const void* xq, const void* xk, const void* xv, const void* a_raw,
                             const void* b_raw, const float* conv_w, const float* a_bias,
                             const int32_t* parent, const int32_t* n_node, int32_t B, int32_t N,
                             int32_t H, int32_t D, kda_dtype dt, const void* conv_state,
                             float l2_eps, void* q, void* k, void* v, void* log_alpha,
                             void* beta, hipStream_t stream) {
    if (!valid_dtype(dt)) return KDA_ERR_BAD_DTYPE;
    if (!tree_shape(B, N, H, KDA_MAX_TREE) || D != kda::kHeadDim) return KDA_ERR_BAD_SHAPE;
    if (!(l2_eps >= 0.f) || l2_eps > std::numeric_limits<float>::max()) return KDA_ERR_BAD_SHAPE;
    if (B > 0 && (!xq || !xk || !xv || !a_raw || !b_raw || !conv_w || !a_bias || !q || !k || !v ||
                  !log_alpha || !beta))
        return KDA_ERR_NULL_ARG;
    if (!all_aligned({xq, xk, xv, a_raw, conv_w, a_bias, conv_state, q, k, v, log_alpha}, 16) ||
        !all_aligned({b_raw, beta}, esize(dt)) || !all_aligned({parent, n_node}, 4))
        return KDA_ERR_MISALIGNED;

    const uint64_t es = esize(dt), row = (uint64_t)H * kda::kHeadDim;
    const uint64_t nNode = (uint64_t)B * N * row * es, nB = (uint64_t)B * N * H * es;
    const Span in[] = {span(xq, nNode), span(xk, nNode), span(xv, nNode), span(a_raw, nNode),
                       span(b_raw, nB), span(conv_w, B > 0 ? 3 * row * 16 : 0),
                       span(a_bias, B > 0 ? row * 4 : 0), counts(parent, (uint64_t)B * N),
                       counts(n_node, B), span(conv_state, (uint64_t)B * 9 * row * es)};
    const Span out[] = {span(q, nNode), span(k, nNode), span(v, nNode), span(log_alpha, nNode),
                        span(beta, nB)};
    for (int i = 0; i < 5; ++i) {
        for (const Span& s : in)
            if (overlaps(out[i], s)) return KDA_ERR_ALIAS;
        for (int j = i + 1; j < 5; ++j)
            if (overlaps(out[i], out[j])) return KDA_ERR_ALIAS;
    }
    if (B == 0) return KDA_OK;

    kda::TreePrologueArgs a;
    a.x[0] = xq;
    a.x[1] = xk;
    a.x[2] = xv;
    a.x[3] = a_raw;
    a.b_raw = b_raw;
    a.conv_w = conv_w;
    a.a_bias = a_bias;
    a.parent = parent;
    a.n_node = n_node;
    a.B = B;
    a.N = N;
    a.H = H;
    a.state = conv_state;
    a.l2_eps = l2_eps;
    a.out[0] = q;
    a.out[1] = k;
    a.out[2] = v;
    a.out[3] = log_alpha;
    a.beta = beta;
    if (kda::launch_tree_prologue(a, (int)dt, stream) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

kda_status kda_tree_decode(const void* q, const void* k, const void* v, const void* log_alpha,
                           const void* beta, const float* S, const int32_t* parent,
                           const int32_t* n_node, int32_t B, int32_t N, int32_t H, int32_t Dk,
                           int32_t Dv, kda_dtype dt, void* o, hipStream_t stream) {
    if (!valid_dtype(dt)) return KDA_ERR_BAD_DTYPE;
    if (!tree_shape(B, N, H, KDA_MAX_TREE) || Dk != kda::kHeadDim || Dv != kda::kHeadDim)
        return KDA_ERR_BAD_SHAPE;
    if (B > 0 && (!q || !k || !v || !log_alpha || !beta || !S || !o)) return KDA_ERR_NULL_ARG;
    if (!all_aligned({q, k, v, log_alpha, S, o}, 16) || !all_aligned({beta}, esize(dt)) ||
        !all_aligned({parent, n_node}, 4))
        return KDA_ERR_MISALIGNED;

    const uint64_t es = esize(dt), units = (uint64_t)B * H;
    const uint64_t nVec = units * N * kda::kHeadDim * es;
    if (overlaps_any(span(o, nVec),
                     {span(q, nVec), span(k, nVec), span(v, nVec), span(log_alpha, nVec),
                      span(beta, units * N * es), span(S, units * kda::kHeadDim * kda::kHeadDim * 4),
                      counts(parent, (uint64_t)B * N), counts(n_node, B)}))
        return KDA_ERR_ALIAS;
    if (B == 0) return KDA_OK;

    kda::TreeDecodeArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.log_alpha = log_alpha;
    a.beta = beta;
    a.S = S;
    a.parent = parent;
    a.n_node = n_node;
    a.B = B;
    a.N = N;
    a.H = H;
    a.o = o;
    if (kda::launch_tree_decode(a, (int)dt, stream) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

kda_status kda_tree_accept(const void* p, const void* q, const int32_t* tokens,
                           const int32_t* parent, const int32_t* n_node, const float* u,
                           int32_t B, int32_t N, int32_t V, kda_dtype dt, int32_t* path,
                           int32_t* n_path, int32_t* next_token, hipStream_t stream) {
    if (!valid_dtype(dt)) return KDA_ERR_BAD_DTYPE;
    if (B < 0 || B > kMaxAccept || N < 1 || N > KDA_MAX_TREE || V < 1 || V > KDA_MAX_VOCAB)
        return KDA_ERR_BAD_SHAPE;
    if (B > 0 && (!p || !tokens || !u || !path || !n_path || !next_token))
        return KDA_ERR_NULL_ARG;
    if (!all_aligned({p, q}, 16) ||
        !all_aligned({tokens, parent, n_node, u, path, n_path, next_token}, 4))
        return KDA_ERR_MISALIGNED;

    const uint64_t es = esize(dt), nodes = (uint64_t)B * N;
    const Span in[] = {span(p, nodes * V * es), span(q, (nodes - B) * V * es),
                       counts(tokens, nodes), counts(parent, nodes), counts(n_node, B),
                       span(u, nodes * 4)};
    const Span out[] = {counts(path, nodes), counts(n_path, B), counts(next_token, B)};
    for (int i = 0; i < 3; ++i) {
        for (const Span& s : in)
            if (overlaps(out[i], s)) return KDA_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(out[i], out[j])) return KDA_ERR_ALIAS;
    }
    if (B == 0) return KDA_OK;

    kda::TreeAcceptArgs a;
    a.p = p;
    a.q = N > 1 ? q : nullptr;   // (one node has no children)
    a.tokens = tokens;
    a.parent = parent;
    a.n_node = n_node;
    a.u = u;
    a.B = B;
    a.N = N;
    a.V = V;
    a.path = path;
    a.n_path = n_path;
    a.next_token = next_token;
    if (kda::launch_tree_accept(a, (int)dt, stream) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

kda_status kda_tree_commit(const void* k, const void* v, const void* log_alpha, const void* beta,
                           float* S, const int32_t* path, const int32_t* n_path, int32_t B,
                           int32_t N, int32_t P, int32_t H, int32_t Dk, int32_t Dv, kda_dtype dt,
                           const void* xq, const void* xk, const void* xv, void* conv_state,
                           hipStream_t stream) {
    if (!valid_dtype(dt)) return KDA_ERR_BAD_DTYPE;
    if (!tree_shape(B, N, H, std::numeric_limits<int32_t>::max()) || P < 1 ||
        P > KDA_MAX_PATH ||
        Dk != kda::kHeadDim || Dv != kda::kHeadDim)
        return KDA_ERR_BAD_SHAPE;
    if (B > 0 && (!k || !v || !log_alpha || !beta || !S || !path ||
                  (conv_state && (!xq || !xk || !xv))))
        return KDA_ERR_NULL_ARG;
    if (!conv_state) xq = xk = xv = nullptr;
    if (!all_aligned({k, v, log_alpha, S, xq, xk, xv, conv_state}, 16) ||
        !all_aligned({beta}, esize(dt)) || !all_aligned({path, n_path}, 4))
        return KDA_ERR_MISALIGNED;

    const uint64_t es = esize(dt), units = (uint64_t)B * H;
    const uint64_t nVec = units * N * kda::kHeadDim * es;
    const Span in[] = {span(k, nVec), span(v, nVec), span(log_alpha, nVec),
                       span(beta, units * N * es), counts(path, (uint64_t)B * P),
                       counts(n_path, B), span(xq, nVec), span(xk, nVec), span(xv, nVec)};
    const Span sS = span(S, units * kda::kHeadDim * kda::kHeadDim * 4),
               sst = span(conv_state, units * 9 * kda::kHeadDim * es);
    for (const Span& s : in)
        if (overlaps(sS, s) || overlaps(sst, s)) return KDA_ERR_ALIAS;
    if (overlaps(sS, sst)) return KDA_ERR_ALIAS;
    if (B == 0) return KDA_OK;

    kda::TreeCommitArgs a;
    a.k = k;
    a.v = v;
    a.log_alpha = log_alpha;
    a.beta = beta;
    a.S = S;
    a.path = path;
    a.n_path = n_path;
    a.B = B;
    a.N = N;
    a.P = P;
    a.H = H;
    a.x[0] = xq;
    a.x[1] = xk;
    a.x[2] = xv;
    a.state = conv_state;
    if (kda::launch_tree_commit(a, (int)dt, stream) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

}  // extern "C"
