// kda_cache_device.h -- device code shared by the kernels of the 8-bit state cache.
#pragma once

#include "kda_device.h"
#include "kda_tree_device.h"

namespace kda {

// A sum of log alpha, and e to it.  In one float sixteen strongly decaying tokens leave
// a rounding of 2^-18 each, up to 2e-5 of the decay; so whole multiples of 2^-17 are
// summed exactly (17 of them at the bound of -5 stay below 2^7) and what is left of each
// beside them.
struct LogDecay {
    float whole = 0.f, rest = 0.f;
    __device__ __forceinline__ void add(float la) {
        const float w = (la + 96.f) - 96.f;   // (a float from 64 to 128 is a multiple of 2^-17)
        whole += w;
        rest += w == la ? 0.f : la - w;       // (nothing is left of -infinity)
    }
    // (exp_f32 takes arguments that are finite)
    __device__ __forceinline__ float decay() const { return exp_f32(whole < -120.f ? -120.f : whole, rest); }
};

}  // namespace kda
