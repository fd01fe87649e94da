// kda_sample_api.cpp -- the C ABI of sampling (declared in include/kda.h):
// argument checks on the host before any HIP call, as in kda_api.cpp, then one
// launcher call.
#include "kda.h"

#include <stdint.h>

#include "kda_check.h"
#include "kda_sample.h"

using namespace kda::check;

namespace {

// A launch holds fewer than 2^32 threads: a workgroup of 1024 a row, and
// workgroups of 256 for four tiles each.
constexpr int32_t kMaxRows = (((int64_t)1 << 32) - 1) / 1024;
constexpr int64_t kMaxGroups = (((int64_t)1 << 32) - 1) / 256;

bool sample_shape(int32_t R, int32_t V) {
    return R >= 0 && R <= kMaxRows && V >= 1 && V <= KDA_MAX_VOCAB && kda::sample_groups(R, V) <= kMaxGroups;
}

bool all_aligned(std::initializer_list<const void*> ps, uintptr_t a) {
    for (const void* p : ps)
        if (p && !aligned(p, a)) return false;
    return true;
}

}  // namespace

extern "C" {

size_t kda_sample_workspace_size(int32_t R, int32_t V) {
    return sample_shape(R, V) ? kda::sample_workspace(R, V) : 0;
}

kda_status kda_sample(const void* logits, const float* u, const float* temperature,
                      const int32_t* top_k, const float* top_p, const float* min_p, int32_t R,
                      int32_t V, kda_dtype dt, int32_t* token, void* probs, void* workspace,
                      size_t workspace_bytes, hipStream_t stream) {
    if (!valid_dtype(dt)) return KDA_ERR_BAD_DTYPE;
    if (!sample_shape(R, V)) return KDA_ERR_BAD_SHAPE;
    if (!u) token = nullptr;
    if (R > 0 && (!logits || (u && !token) || (!u && !probs))) return KDA_ERR_NULL_ARG;
    const uint64_t ws = kda::sample_workspace(R, V);
    if (R > 0 && !workspace) return KDA_ERR_NULL_ARG;
    if (!all_aligned({logits, probs, workspace}, 16) ||
        !all_aligned({u, temperature, top_k, top_p, min_p, token}, 4))
        return KDA_ERR_MISALIGNED;
    if (workspace_bytes < ws) return KDA_ERR_WORKSPACE;

    const uint64_t es = esize(dt), row = (uint64_t)R * 4, all = (uint64_t)R * V * es;
    const Span in[] = {span(logits, all), span(u, row), span(temperature, row),
                       span(top_k, row),  span(top_p, row), span(min_p, row)};
    const Span out[] = {span(token, row), span(probs, all), span(workspace, ws)};
    for (int i = 0; i < 3; ++i) {
        for (const Span& s : in)
            if (overlaps(out[i], s)) return KDA_ERR_ALIAS;
        for (int j = i + 1; j < 3; ++j)
            if (overlaps(out[i], out[j])) return KDA_ERR_ALIAS;
    }
    if (R == 0) return KDA_OK;

    kda::SampleArgs a;
    a.logits = logits;
    a.u = u;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.R = R;
    a.V = V;
    a.token = token;
    a.probs = probs;
    a.workspace = static_cast<char*>(workspace);
    if (kda::launch_sample(a, (int)dt, stream) != hipSuccess) return KDA_ERR_DEVICE;
    return KDA_OK;
}

}  // extern "C"
