// kda_cache_api.cpp -- the C ABI of the 8-bit state cache (declared in
// include/kda.h): argument checks on the host before any HIP call, as in
// kda_api.cpp, then one launcher call each.
#include "kda.h"

#include <stdint.h>

#include "kda_cache.h"
#include "kda_check.h"

using namespace kda::check;

namespace {

constexpr uint64_t kState = (uint64_t)kda::kHeadDim * kda::kHeadDim;
// A launch holds fewer than 2^32 threads: a workgroup of 256 a head at most.
constexpr uint64_t kMaxUnits = (((uint64_t)1 << 32) - 1) / 256;

bool cache_shape(int32_t B, int32_t P, int32_t H, int32_t Dk, int32_t Dv) {
    if (B < 0 || P < 0 || H < 1 || H > KDA_MAX_HEADS) return false;
    if (Dk != kda::kHeadDim || Dv != kda::kHeadDim) return false;
    return (uint64_t)B * (uint64_t)H <= kMaxUnits;
}
bool window_shape(int32_t W) { return W >= 1 && W <= KDA_MAX_WINDOW; }

bool all_aligned(std::initializer_list<const void*> ps, uintptr_t a) {
    for (const void* p : ps)
        if (p && !aligned(p, a)) return false;
    return true;
}

kda::CacheWindow window(const void* k, const void* la, const void* u, const int32_t* n, int32_t W) {
    kda::CacheWindow w;
    w.k = const_cast<void*>(k);
    w.log_alpha = const_cast<void*>(la);
    w.u = const_cast<void*>(u);
    w.n = n;
    w.W = W;
    return w;
}

}  // namespace

extern "C" {

kda_status kda_cache_store(const float* S, const int32_t* page, int32_t B, int32_t P, int32_t H,
                           int32_t Dk, int32_t Dv, int8_t* codes, float* scale,
                           hipStream_t stream) {
    if (!cache_shape(B, P, H, Dk, Dv) || (!page && B > P)) return KDA_ERR_BAD_SHAPE;
    if (B > 0 && P > 0 && (!S || !codes || !scale)) return KDA_ERR_NULL_ARG;
    if (!all_aligned({S, codes, scale}, 16) || !all_aligned({page}, 4)) return KDA_ERR_MISALIGNED;

    const uint64_t units = (uint64_t)B * H, held = (uint64_t)P * H;
    const Span in[] = {span(S, units * kState * 4), span(page, (uint64_t)B * 4)};
    const Span c = span(codes, held * kState), s = span(scale, held * kda::kHeadDim * 4);
    for (const Span& x : in)
        if (overlaps(c, x) || overlaps(s, x)) return KDA_ERR_ALIAS;
    if (overlaps(c, s)) return KDA_ERR_ALIAS;
    if (B == 0 || P == 0) return KDA_OK;

    kda::CacheMoveArgs a;
    a.S = const_cast<float*>(S);
    a.codes = codes;
    a.scale = scale;
    a.page = page;
    a.win = window(nullptr, nullptr, nullptr, nullptr, 0);
    a.B = B;
    a.P = P;
    a.H = H;
    if (kda::launch_cache_store(a, stream) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

kda_status kda_cache_load(const int8_t* codes, const float* scale, const int32_t* page,
                          const void* win_k, const void* win_log_alpha, const void* win_u,
                          const int32_t* n_win, int32_t B, int32_t P, int32_t H, int32_t W,
                          int32_t Dk, int32_t Dv, kda_dtype dt, float* S, hipStream_t stream) {
    const bool some = win_k || win_log_alpha || win_u;
    if (some && !valid_dtype(dt)) return KDA_ERR_BAD_DTYPE;
    if (!cache_shape(B, P, H, Dk, Dv) || (!page && B > P) || (some && !window_shape(W)))
        return KDA_ERR_BAD_SHAPE;
    if (B > 0 && P > 0 &&
        (!codes || !scale || !S || (some && (!win_k || !win_log_alpha || !win_u))))
        return KDA_ERR_NULL_ARG;
    if (!some) n_win = nullptr;
    if (!all_aligned({codes, scale, win_k, win_log_alpha, win_u, S}, 16) ||
        !all_aligned({page, n_win}, 4))
        return KDA_ERR_MISALIGNED;

    const uint64_t units = (uint64_t)B * H, held = (uint64_t)P * H;
    const uint64_t nWin = some ? held * W * kda::kHeadDim * esize(dt) : 0;
    if (overlaps_any(span(S, units * kState * 4),
                     {span(codes, held * kState), span(scale, held * kda::kHeadDim * 4),
                      span(page, (uint64_t)B * 4), span(n_win, (uint64_t)B * 4), span(win_k, nWin),
                      span(win_log_alpha, nWin), span(win_u, nWin)}))
        return KDA_ERR_ALIAS;
    if (B == 0 || P == 0) return KDA_OK;

    kda::CacheMoveArgs a;
    a.S = S;
    a.codes = const_cast<int8_t*>(codes);
    a.scale = const_cast<float*>(scale);
    a.page = page;
    a.win = window(win_k, win_log_alpha, win_u, n_win, W);
    a.B = B;
    a.P = P;
    a.H = H;
    if (kda::launch_cache_load(a, some ? (int)dt : 1, stream) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

kda_status kda_cache_decode(const void* q, const void* k, const void* v, const void* log_alpha,
                            const void* beta, const int8_t* codes, const float* scale,
                            void* win_k, void* win_log_alpha, void* win_u, const int32_t* n_win,
                            int32_t B, int32_t H, int32_t W, int32_t Dk, int32_t Dv, kda_dtype dt,
                            void* o, hipStream_t stream) {
    if (!valid_dtype(dt)) return KDA_ERR_BAD_DTYPE;
    if (!cache_shape(B, B, H, Dk, Dv) || !window_shape(W)) return KDA_ERR_BAD_SHAPE;
    if (B > 0 && (!q || !k || !v || !log_alpha || !beta || !codes || !scale || !win_k ||
                  !win_log_alpha || !win_u || !n_win || !o))
        return KDA_ERR_NULL_ARG;
    if (!all_aligned({q, k, v, log_alpha, codes, scale, win_k, win_log_alpha, win_u, o}, 16) ||
        !all_aligned({beta}, esize(dt)) || !all_aligned({n_win}, 4))
        return KDA_ERR_MISALIGNED;

    const uint64_t es = esize(dt), units = (uint64_t)B * H;
    const uint64_t nVec = units * kda::kHeadDim * es, nWin = nVec * W;
    const Span in[] = {span(q, nVec), span(k, nVec), span(v, nVec), span(log_alpha, nVec),
                       span(beta, units * es), span(codes, units * kState),
                       span(scale, units * kda::kHeadDim * 4), span(n_win, (uint64_t)B * 4)};
    const Span out[] = {span(o, nVec), span(win_k, nWin), span(win_log_alpha, nWin),
                        span(win_u, nWin)};
    for (int i = 0; i < 4; ++i) {
        for (const Span& s : in)
            if (overlaps(out[i], s)) return KDA_ERR_ALIAS;
        for (int j = i + 1; j < 4; ++j)
            if (overlaps(out[i], out[j])) return KDA_ERR_ALIAS;
    }
    if (B == 0) return KDA_OK;

    kda::CacheDecodeArgs a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.log_alpha = log_alpha;
    a.beta = beta;
    a.codes = codes;
    a.scale = scale;
    a.win = window(win_k, win_log_alpha, win_u, n_win, W);
    a.B = B;
    a.H = H;
    a.o = o;
    if (kda::launch_cache_decode(a, (int)dt, stream) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

kda_status kda_cache_fold(int8_t* codes, float* scale, const void* win_k,
                          const void* win_log_alpha, const void* win_u, const int32_t* n_win,
                          int32_t B, int32_t H, int32_t W, int32_t Dk, int32_t Dv, kda_dtype dt,
                          hipStream_t stream) {
    if (!valid_dtype(dt)) return KDA_ERR_BAD_DTYPE;
    if (!cache_shape(B, B, H, Dk, Dv) || !window_shape(W)) return KDA_ERR_BAD_SHAPE;
    if (B > 0 && (!codes || !scale || !win_k || !win_log_alpha || !win_u)) return KDA_ERR_NULL_ARG;
    if (!all_aligned({codes, scale, win_k, win_log_alpha, win_u}, 16) || !all_aligned({n_win}, 4))
        return KDA_ERR_MISALIGNED;

    const uint64_t units = (uint64_t)B * H, nWin = units * W * kda::kHeadDim * esize(dt);
    const Span in[] = {span(win_k, nWin), span(win_log_alpha, nWin), span(win_u, nWin),
                       span(n_win, (uint64_t)B * 4)};
    const Span c = span(codes, units * kState), s = span(scale, units * kda::kHeadDim * 4);
    for (const Span& x : in)
        if (overlaps(c, x) || overlaps(s, x)) return KDA_ERR_ALIAS;
    if (overlaps(c, s)) return KDA_ERR_ALIAS;
    if (B == 0) return KDA_OK;

    kda::CacheMoveArgs a;
    a.S = nullptr;
    a.codes = codes;
    a.scale = scale;
    a.page = nullptr;
    a.win = window(win_k, win_log_alpha, win_u, n_win, W);
    a.B = B;
    a.P = B;
    a.H = H;
    if (kda::launch_cache_fold(a, (int)dt, stream) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

}  // extern "C"
