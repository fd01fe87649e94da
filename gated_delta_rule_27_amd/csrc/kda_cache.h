// kda_cache.h -- internal interface between the C ABI of the 8-bit state
// cache (kda_cache_api.cpp) and its kernel launchers.  Arguments arrive here
// already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_launch.h"

namespace kda {

constexpr int kMaxWindow = 16;   // tokens of a window

struct CacheWindow {
    void* k;                   // [.., H, W, 128]
    void* log_alpha;
    void* u;
    const int32_t* n;          // tokens that count, or null (W)
    int32_t W;
};

// S <-> codes, scale for B states; page null: state b is page b
struct CacheMoveArgs {
    float* S;                  // [B, H, 128, 128]
    int8_t* codes;             // [P, H, 128 (value), 128 (key)]
    float* scale;              // [P, H, 128 (key)]
    const int32_t* page;       // [B] or null
    CacheWindow win;           // k null: none
    int32_t B, P, H;
};

struct CacheDecodeArgs {
    const void* q;             // [B, H, 128]
    const void* k;
    const void* v;
    const void* log_alpha;
    const void* beta;          // [B, H]
    const int8_t* codes;       // [B, H, 128, 128]
    const float* scale;        // [B, H, 128]
    CacheWindow win;
    int32_t B, H;
    void* o;
};

// dtype: 0 = fp32, 1 = bf16 (kda_dtype values), of the window and the vectors
hipError_t launch_cache_store(const CacheMoveArgs& a, hipStream_t stream);
hipError_t launch_cache_load(const CacheMoveArgs& a, int dtype, hipStream_t stream);
hipError_t launch_cache_fold(const CacheMoveArgs& a, int dtype, hipStream_t stream);
hipError_t launch_cache_decode(const CacheDecodeArgs& a, int dtype, hipStream_t stream);

}  // namespace kda
