// kda_tree_device.h -- device code shared by the kernels of tree speculative
// decoding.
#pragma once

#include "kda_device.h"
#include "kda_tree.h"

namespace kda {

// e^(x + rest), and e^-(x + rest), to an ulp or two for |x| <= 87, |rest| <=
// 2^-13, from the hardware's 2^x: x log2 e as a product p and what its rounding
// leaves, with log2 e in two parts, the remainder r put back as the factor 1 +
// r ln 2 + rest.  (Arguments here are finite and <= 88; below -87 the result
// may be flushed to 0.)
__device__ __forceinline__ floatx2 exp_both_f32(float x, float rest) {
    constexpr float kL = 1.44269504088896340736f;                       // log2 e to 24 bits
    constexpr float kLlo = (float)(1.44269504088896340736 - (double)kL);
    const float p = x * kL;
    const float r = __builtin_fmaf(x, kLlo, __builtin_fmaf(x, kL, -p));
    const float t = __builtin_fmaf(r, 0.69314718055994530942f, rest);
    const float y = __builtin_amdgcn_exp2f(p), z = __builtin_amdgcn_exp2f(-p);
    return floatx2{__builtin_fmaf(y, t, y), __builtin_fmaf(z, -t, z)};
}
__device__ __forceinline__ float exp_f32(float x, float rest) { return exp_both_f32(x, rest)[0]; }

// (I + L)^{-1} of a strictly lower triangular tile in place; element (i, j)
// lies at lane 16 (j / 4) + i, j % 4.  One lane per column, row by row; rows
// at and past R are zeros of L (the inverse's are the identity's).
template <int R = 16>
__device__ __forceinline__ void invert(float* tile, int l16, int g) {
    if (g != 0) return;
    float x[16];
    x[0] = l16 == 0 ? 1.f : 0.f;
#pragma unroll
    for (int r = 1; r < 16; ++r) {
        float s = r == l16 ? 1.f : 0.f;
#pragma unroll
        for (int jq = 0; jq < (r < R ? (r + 3) / 4 : 0); ++jq) {
            const floatx4 c = *reinterpret_cast<const floatx4*>(tile + (16 * jq + r) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (4 * jq + e < r) s -= c[e] * x[4 * jq + e];
        }
        x[r] = s;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) tile[(16 * (l16 >> 2) + r) * 4 + (l16 & 3)] = x[r];
}

// parent of node i of sequence b, -1 for the cached state
__device__ __forceinline__ int tree_parent(const int32_t* parent, int64_t b, int N, int i) {
    const int p = parent ? parent[b * N + i] : i - 1;
    return p >= 0 && p < i ? p : -1;
}
// nodes of sequence b
__device__ __forceinline__ int tree_count(const int32_t* n_node, int64_t b, int N) {
    const int n = n_node ? n_node[b] : N;
    return n < 0 ? 0 : (n > N ? N : n);
}

}  // namespace kda
