// kda_sample.h -- internal interface between the C ABI of sampling
// (kda_sample_api.cpp) and its kernel launchers.  Arguments arrive here already
// validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_launch.h"

namespace kda {

constexpr int kSampleTile = 1024;   // tokens of a tile: 16 per lane of a wavefront

struct SampleArgs {
    const void* logits;         // [R, V]
    const float* u;             // [R] or null (no tokens)
    const float* temperature;   // [R] or null (1)
    const int32_t* top_k;       // [R] or null (off)
    const float* top_p;         // [R] or null (off)
    const float* min_p;         // [R] or null (off)
    int32_t R, V;
    int32_t* token;             // [R], with u
    void* probs;                // [R, V] or null
    char* workspace;
};

constexpr int kSampleGroups = 16;   // of a tile: 64 tokens each

// Workspace: per tile its largest logit, the largest of each of its groups, and
// the sum of its weights; then what the last pass needs of each row.
struct SampleRow {
    double scale;      // log2(e) / temperature
    double sum;        // log2 of the sum of the weights that are kept
    double least;      // smallest weight that is kept, where the cut is not all
    uint64_t cut;      // last place in the order that is kept
    float top;         // largest logit; -infinity: nothing is kept
    int32_t pad;
};
inline int64_t sample_tiles(int32_t V) { return ((int64_t)V + kSampleTile - 1) / kSampleTile; }
struct SampleSections {
    uint64_t tops, groups, sums, rows, end;   // bytes
};
__host__ __device__ inline SampleSections sample_sections(int32_t R, int64_t tiles) {
    const uint64_t n = (uint64_t)R * tiles;
    SampleSections s;
    s.tops = 0;
    s.groups = (n * 4 + 15) / 16 * 16;
    s.sums = s.groups + n * 4 * kSampleGroups;
    s.rows = s.sums + (n * 8 + 15) / 16 * 16;
    s.end = s.rows + (uint64_t)R * sizeof(SampleRow);
    return s;
}
inline size_t sample_workspace(int32_t R, int32_t V) { return (size_t)sample_sections(R, sample_tiles(V)).end; }
// workgroups of the first pass and of the last: four tiles each
inline int64_t sample_groups(int32_t R, int32_t V) { return R * ((sample_tiles(V) + 3) / 4); }

// dtype: 0 = fp32, 1 = bf16 (kda_dtype values)
hipError_t launch_sample(const SampleArgs& a, int dtype, hipStream_t stream);

}  // namespace kda
