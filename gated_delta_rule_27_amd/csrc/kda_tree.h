// kda_tree.h -- internal interface between the C ABI of tree speculative
// decoding (kda_tree_api.cpp) and its kernel launchers.  Arguments arrive
// here already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_launch.h"

namespace kda {

constexpr int kMaxTree = 64;   // nodes of a tree: one lane, one mask bit each

struct TreePrologueArgs {
    const void* x[4];          // x_q, x_k, x_v, decay logits a: [B, N, H, 128]
    const void* b_raw;         // [B, N, H]
    const float* conv_w;       // [3, H, 128, 4]
    const float* a_bias;       // [H, 128]
    const int32_t* parent;     // [B, N] or null (chain)
    const int32_t* n_node;     // [B] or null (N)
    int32_t B, N, H;
    const void* state;         // [B, 3, 3, H, 128] or null (zero history)
    float l2_eps;
    void* out[4];              // q, k, v, log_alpha
    void* beta;
};

struct TreeDecodeArgs {
    const void* q;             // [B, N, H, 128]
    const void* k;
    const void* v;
    const void* log_alpha;
    const void* beta;          // [B, N, H]
    const float* S;            // [B, H, 128, 128]
    const int32_t* parent;
    const int32_t* n_node;
    int32_t B, N, H;
    void* o;
};

struct TreeAcceptArgs {
    const void* p;             // [B, N, V]
    const void* q;             // [B, N - 1, V] or null (certain drafts)
    const int32_t* tokens;     // [B, N]
    const int32_t* parent;
    const int32_t* n_node;
    const float* u;            // [B, N]
    int32_t B, N, V;
    int32_t* path;             // [B, N]
    int32_t* n_path;           // [B]
    int32_t* next_token;       // [B]
};

struct TreeCommitArgs {
    const void* k;             // [B, N, H, 128]
    const void* v;
    const void* log_alpha;
    const void* beta;          // [B, N, H]
    float* S;                  // [B, H, 128, 128]
    const int32_t* path;       // [B, P]
    const int32_t* n_path;     // [B] or null (P)
    int32_t B, N, P, H;
    const void* x[3];          // x_q, x_k, x_v
    void* state;               // [B, 3, 3, H, 128] or null
};

// dtype: 0 = fp32, 1 = bf16 (kda_dtype values)
hipError_t launch_tree_prologue(const TreePrologueArgs& a, int dtype, hipStream_t stream);
hipError_t launch_tree_decode(const TreeDecodeArgs& a, int dtype, hipStream_t stream);
hipError_t launch_tree_accept(const TreeAcceptArgs& a, int dtype, hipStream_t stream);
hipError_t launch_tree_commit(const TreeCommitArgs& a, int dtype, hipStream_t stream);

// Workgroups of the tree prologue per group of sequences: q, k, v x two-head
// slices, then the gates' four-head slices.
inline int64_t tree_prologue_tasks(int32_t H) { return 3 * (((int64_t)H + 1) / 2) + ((int64_t)H + 3) / 4; }
// Sequences of a group: more than one once there are workgroups enough.  At 1,
// 2, 4, 8 (x 96 heads, us; * what the rule takes):
//   256 x 16 nodes  bf16 196 175 172* 175   fp32 313 317 306* 325
//   256 x  4 nodes  bf16  81  72  69*  70
//    64 x 64 nodes  bf16 172 172 186* 211   fp32 304 311 318* 360
//    64 x 16 nodes  bf16  43  45  49*  52
//    32 x 16 nodes  bf16  25  26*  28  38
//     8 x 64 nodes  bf16  30* 36  49   74
// many short trees gain up to 15%, a few long ones lose up to 12%.
inline int32_t tree_prologue_sequences(int32_t B, int32_t H) {
    const int64_t n = (int64_t)B * tree_prologue_tasks(H) / 2048;
    return n < 1 ? 1 : (n > 4 ? 4 : (int32_t)n);
}

}  // namespace kda
