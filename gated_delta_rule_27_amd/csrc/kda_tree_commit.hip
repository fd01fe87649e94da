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
// rounding on to the tokens after it.
//
// Mapping.  One workgroup of four wavefronts per (sequence, head); wavefront
// w owns value columns 32 w .. 32 w + 31 over all 128 rows.  The state stays
// in its registers from the one read to the one write; a lane's rows
// 16 kb + 4 g + 0..3 of two columns are at once the B operand of X S and the
// accumulator of the update.
#include "kda.h"
#include "kda_device.h"
#include "kda_tree.h"

namespace kda {

namespace {

constexpr int kTok = 16;              // path tokens of a block
constexpr int kXP = kHeadDim + 4;     // a token row in LDS
constexpr int kTP = kTok + 4;         // a channel row of tokens in LDS

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ floatx2 pair(const bf16* p) {
    const bf16x2 a = *reinterpret_cast<const bf16x2*>(p);
    return floatx2{(float)a[0], (float)a[1]};
}
__device__ __forceinline__ floatx2 pair(const float* p) { return *reinterpret_cast<const floatx2*>(p); }

// The last three inputs of (history, path inputs) for this head: a thread
// holds 16 bytes of channels of one of q, k, v.  Each reads all it needs
// before it writes.
template <typename T>
__device__ __forceinline__ void commit_history(const TreeCommitArgs& a, int64_t b, int h,
                                               const int32_t* path, int m, int tid) {
    constexpr int M = Vec16<T>::N, kV = kHeadDim / M;
    typedef typename Vec16<T>::type vec;
    if (tid >= 3 * kV) return;
    const int tensor = tid / kV, c = (tid % kV) * M;
    const size_t HD = (size_t)a.H * kHeadDim, at = (size_t)h * kHeadDim + c;
    const T* x = static_cast<const T*>(tensor == 0 ? a.x[0] : (tensor == 1 ? a.x[1] : a.x[2])) +
                 (size_t)b * a.N * HD + at;
    T* hist = static_cast<T*>(a.state) + ((size_t)b * 3 + tensor) * 3 * HD + at;
    vec row[3];
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        const int t = m - 3 + p;   // path position; before it the history's rows
        row[p] = *reinterpret_cast<const vec*>(t >= 0 ? x + path[t] * HD : hist + (3 + t) * HD);
    }
#pragma unroll
    for (int p = 0; p < 3; ++p) *reinterpret_cast<vec*>(hist + p * HD) = row[p];
}

template <typename T>
__global__ __launch_bounds__(256) void tree_commit_kernel(TreeCommitArgs a) {
    __shared__ __attribute__((aligned(16))) float X[kTok * kXP];
    __shared__ __attribute__((aligned(16))) float Y[kTok * kXP];
    __shared__ __attribute__((aligned(16))) float KT[kHeadDim * kTP];    // (k o e^{G_e - G})^T
    __shared__ __attribute__((aligned(16))) float gam[kHeadDim];         // e^{G_e}
    __shared__ __attribute__((aligned(16))) float part[4][kTok * kTP];   // X Y^T by channel quarter
    __shared__ __attribute__((aligned(16))) float Ls[kTok * kTP];
    __shared__ __attribute__((aligned(16))) float inv[4][kTok * kTP];    // a copy per wavefront
    __shared__ __attribute__((aligned(16))) float sbeta[kTok];
    __shared__ int32_t node[kTok];

    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int H = a.H, N = a.N;
    const int64_t b = blockIdx.x / (unsigned)H;
    const int h = blockIdx.x % (unsigned)H;
    const int32_t* path = a.path + (size_t)b * a.P;

    // the path's length: to the first entry that is no node
    const int most = tree_count(a.n_path, b, a.P);
    int m = 0;
    while (m < most) {
        const bool ok = m + lane < most && (unsigned)path[m + lane] < (unsigned)N;
        const uint64_t bad = ~__ballot(ok);
        if (bad) {
            m += __builtin_ctzll(bad);
            break;
        }
        m += 64;
    }
    m = __builtin_amdgcn_readfirstlane(m);
    if (m == 0) return;
    if (a.state) commit_history<T>(a, b, h, path, m, tid);

    const size_t HD = (size_t)H * kHeadDim;
    const size_t base = ((size_t)b * N * H + h) * kHeadDim;   // node 0's row; nodes are HD apart
    const T* k = static_cast<const T*>(a.k) + base;
    const T* v = static_cast<const T*>(a.v) + base;
    const T* la = static_cast<const T*>(a.log_alpha) + base;
    const T* beta = static_cast<const T*>(a.beta) + (size_t)b * N * H + h;
    const int c0 = 32 * w + 2 * l16;
    float* S = a.S + ((size_t)b * H + h) * (kHeadDim * kHeadDim) + (size_t)(4 * g) * kHeadDim + c0;

    floatx2 st[8][4];   // rows 16 kb + 4 g + e, columns c0, c0 + 1
#pragma unroll
    for (int kb = 0; kb < 8; ++kb)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            st[kb][e] = __builtin_nontemporal_load(
                reinterpret_cast<const floatx2*>(S + (16 * kb + e) * kHeadDim));

    for (int t0 = 0; t0 < m; t0 += kTok) {
        const int cnt = min(kTok, m - t0);
        __syncthreads();   // the block before is no longer read
        // ---- scaled rows: two threads per channel ---------------------------
        {
            const int c = tid & (kHeadDim - 1);
            float gs[kTok], kx[kTok];
#pragma unroll
            for (int t = 0; t < kTok; ++t) {
                const size_t row = t < cnt ? (size_t)path[t0 + t] * HD : 0;
                gs[t] = t < cnt ? to_f32(la[row + c]) : 0.f;
                kx[t] = t < cnt ? to_f32(k[row + c]) : 0.f;
            }
#pragma unroll
            for (int t = 1; t < kTok; ++t) gs[t] += gs[t - 1];
            if (tid < kHeadDim) {
#pragma unroll
                for (int t = 0; t < kTok; ++t) X[t * kXP + c] = kx[t] * expf(gs[t]);
                gam[c] = expf(gs[kTok - 1]);
            } else {
#pragma unroll
                for (int t = 0; t < kTok; ++t) {
                    Y[t * kXP + c] = kx[t] * expf(-gs[t]);
                    KT[c * kTP + t] = kx[t] * expf(gs[kTok - 1] - gs[t]);
                }
            }
            if (tid < kTok) {
                const int i = path[t0 + min(tid, cnt - 1)];
                node[tid] = i;
                sbeta[tid] = tid < cnt ? to_f32(beta[(size_t)i * H]) : 0.f;
            }
        }
        __syncthreads();
        // ---- X Y^T, a quarter of the channels per wavefront -----------------
        {
            floatx4 acc = zero4();
#pragma unroll
            for (int kb = 0; kb < 32; kb += 16)
                acc = mma_f32_k16(frag_k16(X + l16 * kXP, 32 * w + kb, g),
                                  frag_k16(Y + l16 * kXP, 32 * w + kb, g), acc);
#pragma unroll
            for (int e = 0; e < 4; ++e) part[w][(4 * g + e) * kTP + l16] = acc[e];
        }
        __syncthreads();
        {
            const int i = tid >> 4, j = tid & 15, x = i * kTP + j;
            Ls[x] = j < i ? sbeta[i] * ((part[0][x] + part[1][x]) + (part[2][x] + part[3][x])) : 0.f;
        }
        __syncthreads();
        // ---- (I + L)^{-1}: lane = column, the four groups of 16 alike -------
        {
            float x[kTok];
#pragma unroll
            for (int r = 0; r < kTok; ++r) {
                float s = r == l16 ? 1.f : 0.f;
#pragma unroll
                for (int j = 0; j < r; ++j) s -= Ls[r * kTP + j] * x[j];
                x[r] = s;
            }
            // (the four groups write the same values)
#pragma unroll
            for (int r = 0; r < kTok; ++r) inv[w][r * kTP + l16] = x[r];
        }
        // ---- held = X S and the pseudo-values -------------------------------
        floatx2 vv[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) vv[e] = pair(v + node[4 * g + e] * HD + c0);
        floatx4 u[2] = {zero4(), zero4()};
#pragma unroll
        for (int kb = 0; kb < 8; ++kb) {
            const floatx4 xa = frag_k16(X + l16 * kXP, 16 * kb, g);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                u[t] = mma_f32_k16(xa, floatx4{st[kb][0][t], st[kb][1][t], st[kb][2][t], st[kb][3][t]}, u[t]);
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        const floatx4 bt = *reinterpret_cast<const floatx4*>(sbeta + 4 * g);
        const floatx4 ia = frag_k16(inv[w] + l16 * kTP, 0, g);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            floatx4 rhs;
#pragma unroll
            for (int e = 0; e < 4; ++e) rhs[e] = bt[e] * (vv[e][t] - u[t][e]);
            u[t] = mma_f32_k16(ia, rhs, zero4());
        }
        // ---- S <- Diag(e^{G_e}) S + (k o e^{G_e - G})^T u --------------------
#pragma unroll
        for (int kb = 0; kb < 8; ++kb) {
            const floatx4 gm = *reinterpret_cast<const floatx4*>(gam + 16 * kb + 4 * g);
            const floatx4 ka = frag_k16(KT + (16 * kb + l16) * kTP, 0, g);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                floatx4 acc;
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[e] = gm[e] * st[kb][e][t];
                acc = mma_f32_k16(ka, u[t], acc);
#pragma unroll
                for (int e = 0; e < 4; ++e) st[kb][e][t] = acc[e];
            }
        }
    }
#pragma unroll
    for (int kb = 0; kb < 8; ++kb)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            __builtin_nontemporal_store(st[kb][e], reinterpret_cast<floatx2*>(S + (16 * kb + e) * kHeadDim));
}

}  // namespace

hipError_t launch_tree_commit(const TreeCommitArgs& a, int dtype, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.B * a.H)), block(256);
    if (dtype == 0) tree_commit_kernel<float><<<grid, block, 0, stream>>>(a);
    else tree_commit_kernel<bf16><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace kda
