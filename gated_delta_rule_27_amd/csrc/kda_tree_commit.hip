// kda_tree_commit.hip -- cached states and convolution histories moved along
// the accepted path of a tree of drafted tokens, in place.
//
// Mathematics: up to 16 path tokens at a time in the chunkwise form.  With
// G_t the running sum of log alpha over the block (per key channel, G_e at
// its end),
//   u = (I + L)^{-1} diag(beta) (V - X S),  X_t = k_t o e^{G_t},
//   L = diag(beta) strictly lower (X Y^T),  Y_t = k_t o e^{-G_t},
//   S <- Diag(e^{G_e}) S + sum_t (k_t o e^{G_e - G_t}) u_t^T.
// 16 tokens at the decay bound keep e^{-G} below e^80, finite in fp32.
// Everything is fp32 on fp32 MFMA: the state is fp32 and carries every
// rounding on to the tokens after it.  G in one float would be off by up to
// 2^-18 at |G| of 64 to 80, and e^{G_t} e^{-G_j} by that of its value (4e-6 to
// 7e-6 of the state where 12 tokens decay strongly and 4 hardly, token by token
// 1.5e-7; with two floats 1.7e-7).  So log alpha is summed as multiples of
// 2^-17, exactly (16 of them at the bound stay below 2^7), and the rests of
// at most 2^-18 beside them.
//
// Mapping.  One workgroup of four wavefronts per (sequence, head) (two heads
// of eight wavefronts stream whole 128 KB blocks but wait for each other:
// 543 us against 490 for 256 x 96 states).  Before the state is touched
// wavefront w owns key channels 32 w .. 32 w + 31 of the tokens, a lane 4
// channels of one token at a time: the running sums are DPP scans along the
// 16 lanes of a row, and the rows are at once the operands of X Y^T, whose
// parts are summed through LDS.  Then it owns value columns 32 w .. 32 w + 31
// over all 128 rows: the state stays in its registers from the one read to
// the one write, and a lane's rows 16 kb + 4 g + 0..3 of two columns are both
// the operand of X S and the accumulator of the update.
//
// What bounds it: reading and writing the states while paths are one block
// (256 x 96 bf16, paths of up to 8, one in nine empty: 480 us, 2.89 GB by the
// counters, 6.0 TB/s; a kernel that only copies the states' pattern reaches 5.9
// to 6.1); with paths of more blocks the blocks' chain, at three workgroups per
// compute unit (64 x 96: 32 tokens 217 us against 146 for 16).  One sequence
// of 8 tokens x 96 heads: 9 us, the latency of one workgroup; fetching path
// and count side by side and the first entries only once took off 0.15 us and
// was not kept.  The instance goes by the width P of the path array, which the
// host knows, not by the counts: 1 to 8 tokens in arrays of 64 instead of 8
// take 580 us against 580 for 256 x 96 states, 43 against 41 for 16 x 96, 10.7
// against 9.3 for one sequence.
#include "kda.h"
#include "kda_device.h"
#include "kda_tree_device.h"

namespace kda {

namespace {

constexpr int kTok = 16;              // path tokens of a block
constexpr int kXP = kHeadDim + 4;     // a token row in LDS
constexpr float kGrid = 96.f;         // added and taken off: a multiple of 2^-17, for |x| <= 32
constexpr int kStream = 2;            // states pass the caches by (the non-temporal policy)
typedef unsigned int uintx2_t __attribute__((ext_vector_type(2)));

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ floatx2 pair(const bf16* p) {
    const bf16x2 a = *reinterpret_cast<const bf16x2*>(p);
    return floatx2{(float)a[0], (float)a[1]};
}
__device__ __forceinline__ floatx2 pair(const float* p) { return *reinterpret_cast<const floatx2*>(p); }
__device__ __forceinline__ floatx4 four(const bf16* p) {
    const bf16x4 a = *reinterpret_cast<const bf16x4*>(p);
    return floatx4{(float)a[0], (float)a[1], (float)a[2], (float)a[3]};
}
__device__ __forceinline__ floatx4 four(const float* p) { return *reinterpret_cast<const floatx4*>(p); }

// Entries of the path that are applied: to the first one that is no node.
__device__ __forceinline__ int path_length(const TreeCommitArgs& a, int64_t b, int lane) {
    const int32_t* path = a.path + (size_t)b * a.P;
    const int most = tree_count(a.n_path, b, a.P);
    int m = 0;
    while (m < most) {
        const bool ok = m + lane < most && (unsigned)path[m + lane] < (unsigned)a.N;
        const uint64_t bad = ~__ballot(ok);
        if (bad) {
            m += __builtin_ctzll(bad);
            break;
        }
        m += 64;
    }
    return __builtin_amdgcn_readfirstlane(m);
}

// The last three inputs of (history, path inputs): a workgroup of its own
// per kHistHeads heads of a sequence, a thread 16 bytes of channels of one of
// q, k, v.  Each reads all it needs before it writes.
template <typename T>
struct History {
    static constexpr int M = Vec16<T>::N, kV = kHeadDim / M;      // threads per head and tensor
    static constexpr int kHeads = 256 / (3 * kV);
};
template <typename T>
__device__ __forceinline__ void commit_history(const TreeCommitArgs& a, int64_t wg) {
    typedef typename Vec16<T>::type vec;
    constexpr int kV = History<T>::kV, kHeads = History<T>::kHeads;
    const int groups = (a.H + kHeads - 1) / kHeads;
    const int64_t b = wg / groups;
    const int m = path_length(a, b, threadIdx.x & 63);
    const int hh = threadIdx.x / (3 * kV), rest = threadIdx.x % (3 * kV);
    const int h = (int)(wg % groups) * kHeads + hh;
    if (m == 0 || hh >= kHeads || h >= a.H) return;
    const int tensor = rest / kV, c = (rest % kV) * History<T>::M;
    const size_t HD = (size_t)a.H * kHeadDim, at = (size_t)h * kHeadDim + c;
    const T* x = static_cast<const T*>(tensor == 0 ? a.x[0] : (tensor == 1 ? a.x[1] : a.x[2])) +
                 (size_t)b * a.N * HD + at;
    T* hist = static_cast<T*>(a.state) + ((size_t)b * 3 + tensor) * 3 * HD + at;
    const int32_t* path = a.path + (size_t)b * a.P;
    vec row[3];
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        const int t = m - 3 + p;   // path position; before it the history's rows
        row[p] = *reinterpret_cast<const vec*>(t >= 0 ? x + path[t] * HD : hist + (3 + t) * HD);
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) *reinterpret_cast<vec*>(hist + p * HD) = row[p];
}

// LDS of one state
struct __attribute__((aligned(16))) CommitLds {
    float X[kTok * kXP];        // k o e^G
    float K[kTok * kXP];        // k o e^{G_e - G}
    float gam[kHeadDim];        // e^{G_e}
    floatx4 part[4][64];        // transposed X Y^T over a wavefront's channels
    float inv[4][kTok * kTok];  // (I + L)^{-1}, a copy per wavefront
};

// kLong: paths of more than one block.  (Where a path is one block at most
// there is no loop for the state's registers to be copied around.)
template <typename T, bool kLong>
__global__ __launch_bounds__(256, kLong ? 2 : 4) void tree_commit_kernel(TreeCommitArgs a, int32_t units) {
    __shared__ CommitLds lds;
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int H = a.H, N = a.N;
    if ((int)blockIdx.x >= units) {
        commit_history<T>(a, (int)blockIdx.x - units);
        return;
    }
    const int64_t b = blockIdx.x / (unsigned)H;
    const int h = blockIdx.x % (unsigned)H;
    const int32_t* path = a.path + (size_t)b * a.P;
    const int m = path_length(a, b, lane);
    if (m == 0) return;

    const size_t HD = (size_t)H * kHeadDim;
    const size_t base = ((size_t)b * N * H + h) * kHeadDim;   // node 0's row; nodes are HD apart
    const T* k = static_cast<const T*>(a.k) + base + 32 * w + 4 * g;
    const T* la = static_cast<const T*>(a.log_alpha) + base + 32 * w + 4 * g;
    const T* beta = static_cast<const T*>(a.beta) + (size_t)b * N * H + h;
    const int c0 = 32 * w + 2 * l16;
    const T* v = static_cast<const T*>(a.v) + base + c0;
    const rsrc_t S = make_rsrc_u32(a.S + ((size_t)b * H + h) * (kHeadDim * kHeadDim), kHeadDim * kHeadDim * 4);
    const int at_s = (4 * g * kHeadDim + c0) * 4;

    // a block's inputs; tokens past the path are zeros (and change nothing)
    floatx4 kr[2], lr[2];
    floatx2 vr[4];
    float bt[4];
    auto load_block = [&](int t0) {
        const int left = m - t0;
        const int node = path[t0 + min(l16, left - 1)];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            kr[t] = four(k + node * HD + 16 * t);
            lr[t] = four(la + node * HD + 16 * t);
            if (l16 >= left) kr[t] = lr[t] = zero4();
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = 4 * g + e;
            const int nd = __shfl(node, t, 64);   // (lanes 0..15 hold the block's nodes)
            vr[e] = pair(v + nd * HD);
            bt[e] = to_f32(beta[(size_t)nd * H]);
            if (t >= left) {
                vr[e] = floatx2{0.f, 0.f};
                bt[e] = 0.f;
            }
        }
    };
    load_block(0);
    floatx2 st[8][4];   // rows 16 kb + 4 g + e of columns c0, c0 + 1
#pragma unroll
    for (int kb = 0; kb < 8; ++kb)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            st[kb][e] = __builtin_bit_cast(
                floatx2, __builtin_amdgcn_raw_buffer_load_b64(S, at_s + e * kHeadDim * 4, kb * 16 * kHeadDim * 4,
                                                              kStream));
    __builtin_amdgcn_sched_barrier(0);
    auto store_rows = [&](int kb) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(uintx2_t, st[kb][e]), S,
                                                  at_s + e * kHeadDim * 4, kb * 16 * kHeadDim * 4, kStream);
    };

    for (int t0 = 0; t0 < (kLong ? m : 1); t0 += kTok) {
        if (t0 > 0) {
            load_block(t0);
            __syncthreads();   // the block before is no longer read
        }
        // ---- scaled rows; lane = token l16, channels 32 w + 16 t + 4 g + e ---
        floatx4 xt = zero4();
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int c = 32 * w + 16 * t + 4 * g;
            floatx4 x, y, kk, gm;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float whole = (lr[t][e] + kGrid) - kGrid;
                const float G = row_prefix_sum(whole), rest = row_prefix_sum(lr[t][e] - whole);
                const float ex = exp_f32(G, rest);
                x[e] = kr[t][e] * ex;
                y[e] = kr[t][e] * exp_f32(-G, -rest);
                kk[e] = kr[t][e] * exp_f32(row_bcast<15>(G) - G, row_bcast<15>(rest) - rest);
                gm[e] = row_bcast<15>(ex);
            }
            *reinterpret_cast<floatx4*>(lds.X + l16 * kXP + c) = x;
            *reinterpret_cast<floatx4*>(lds.K + l16 * kXP + c) = kk;
            if (l16 == 0) *reinterpret_cast<floatx4*>(lds.gam + c) = gm;
            xt = mma_f32_k16(y, x, xt);   // rows: token j = 4 g + e, column: token i = l16
            __builtin_amdgcn_sched_barrier(0);
        }
        lds.part[w][lane] = xt;
        __syncthreads();
        // ---- (I + L)^{-1}: every wavefront its own copy ----------------------
        {
            const floatx4* p = &lds.part[0][lane];
            floatx4 x = (p[0] + p[64]) + (p[128] + p[192]);
            // row i's beta: beta of token l16, held by group l16 / 4
            float bi = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float be = __shfl(bt[e], 16 * (l16 >> 2), 64);
                if ((l16 & 3) == e) bi = be;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = 4 * g + e < l16 ? bi * x[e] : 0.f;
            float* tile = lds.inv[w];   // element (i, j): lane 16 (j / 4) + i, j % 4
            *reinterpret_cast<floatx4*>(tile + lane * 4) = x;
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
            invert(tile, l16, g);
        }
        __builtin_amdgcn_sched_barrier(0);
        // ---- held = X S and the pseudo-values ---------------------------
        floatx4 u[2] = {zero4(), zero4()};
#pragma unroll
        for (int kb = 0; kb < 8; ++kb) {
            const floatx4 xa = frag_k16(lds.X + l16 * kXP, 16 * kb, g);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                u[t] = mma_f32_k16(xa, floatx4{st[kb][0][t], st[kb][1][t], st[kb][2][t], st[kb][3][t]}, u[t]);
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        const floatx4 ia = *reinterpret_cast<const floatx4*>(lds.inv[w] + lane * 4);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            floatx4 rhs;
#pragma unroll
            for (int e = 0; e < 4; ++e) rhs[e] = bt[e] * (vr[e][t] - u[t][e]);
            u[t] = mma_f32_k16(ia, rhs, zero4());
        }
        // ---- S <- Diag(e^{G_e}) S + (k o e^{G_e - G})^T u ----------------
#pragma unroll
        for (int kb = 0; kb < 8; ++kb) {
            const floatx4 gm = *reinterpret_cast<const floatx4*>(lds.gam + 16 * kb + 4 * g);
            floatx4 ka;   // channel 16 kb + l16 of tokens 4 g + e
#pragma unroll
            for (int e = 0; e < 4; ++e) ka[e] = lds.K[(4 * g + e) * kXP + 16 * kb + l16];
            floatx4 acc[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[t][e] = gm[e] * st[kb][e][t];
                acc[t] = mma_f32_k16(ka, u[t], acc[t]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) st[kb][e] = floatx2{acc[0][e], acc[1][e]};
            if (!kLong) store_rows(kb);
            __builtin_amdgcn_sched_barrier(0);   // (few rows in flight between the two layouts)
        }
    }
    if (kLong) {
#pragma unroll
        for (int kb = 0; kb < 8; ++kb) store_rows(kb);
    }
}

template <typename T>
hipError_t launch_t(const TreeCommitArgs& a, hipStream_t stream) {
    const int64_t units = (int64_t)a.B * a.H;
    const int64_t hist = a.state ? (int64_t)a.B * ((a.H + History<T>::kHeads - 1) / History<T>::kHeads) : 0;
    const dim3 grid((unsigned)(units + hist)), block(256);
    if (a.P > kTok) tree_commit_kernel<T, true><<<grid, block, 0, stream>>>(a, (int32_t)units);
    else tree_commit_kernel<T, false><<<grid, block, 0, stream>>>(a, (int32_t)units);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_tree_commit(const TreeCommitArgs& a, int dtype, hipStream_t stream) {
    return dtype == 0 ? launch_t<float>(a, stream) : launch_t<bf16>(a, stream);
}

}  // namespace kda
