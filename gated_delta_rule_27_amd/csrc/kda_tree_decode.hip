// kda_tree_decode.hip -- the KDA outputs of a tree of drafted tokens from one
// read of the cached state (speculative verification of a tree).
//
// Mathematics.  With A(i) the ancestors of node i and i itself and G_i = the
// sum of log alpha_j over A(i) (per key channel), the state of node i is
//   S_i = Diag(e^{G_i}) S + sum over j in A(i) of (k_j o e^{G_i - G_j}) u_j^T,
//   u_i = beta_i (v_i - S^T (k_i o e^{G_i}) - sum over j in A(i) \ {i} of
//                 <k_i o e^{G_i}, k_j o e^{-G_j}> u_j),
//   o_i = S^T (q_i o e^{G_i}) + sum over j in A(i) of
//                 <q_i o e^{G_i}, k_j o e^{-G_j}> u_j:
// the chunkwise form with "earlier token" replaced by "ancestor".  No node
// state is ever formed: all nodes share one product with the cached state,
// two N x N Gram tiles masked by ancestry, and a unit lower triangular solve
// (nodes are in topological order).  G itself is a product of the 0/1
// ancestor matrix with the nodes' log alpha.
//
// Range.  e^{-G_j} stays finite for at most 16 levels at the decay bound
// (log alpha >= -5).  Where some |G| of a (sequence, head) passes kMaxDecay,
// its Gram entries are summed pair by pair with e^{G_i - G_j} <= 1 instead.
//
// Masking.  Products with masked (zero) entries would spread a NaN or
// infinity of one node to its siblings.  Non-finite k, log alpha, beta (per
// node) and v (per column) are therefore taken as 0 and remembered as bits,
// and the outputs of the nodes that descend from them are set to NaN.
//
// Mapping.  One workgroup of four wavefronts per (sequence, head); wavefront
// w owns value columns 32 w .. 32 w + 31 (lane: columns 2 (l % 16), +1) over
// all 128 state rows, so everything after the Gram tiles (pseudo-values,
// solve, outputs) stays in its own accumulators.
#include "kda.h"
#include "kda_device.h"
#include "kda_tree.h"

namespace kda {

namespace {

constexpr float kMaxDecay = 64.f;   // |G| up to which e^{-G} is formed
constexpr int kFP = kHeadDim + 4;   // fp32 LDS row
constexpr int kBP = kHeadDim + 8;   // bf16 LDS row

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Rows of 128 channels as MFMA operands in LDS.  fp32 rows as they are;
// for bf16 inputs a scaled row is no longer a bf16 value, so it is held as
// the sum of two bf16 (hi and the rounding's remainder lo): the products
// hi hi + hi lo + lo hi leave a relative error of 2^-17, so that the one
// rounding that counts is the output's.
template <typename T>
struct Rows;
template <>
struct Rows<float> {
    static constexpr int kBytes = kFP * 4;   // of a row
    float* p;
    __device__ __forceinline__ Rows(unsigned char* base, int) : p(reinterpret_cast<float*>(base)) {}
    __device__ __forceinline__ void put8(int row, int c, const float (&x)[8]) const {
        float* d = p + row * kFP + c;
        *reinterpret_cast<floatx4*>(d) = floatx4{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<floatx4*>(d + 4) = floatx4{x[4], x[5], x[6], x[7]};
    }
};
template <>
struct Rows<bf16> {
    static constexpr int kBytes = 2 * kBP * 2;
    bf16* hi;
    bf16* lo;
    __device__ __forceinline__ Rows(unsigned char* base, int rows)
        : hi(reinterpret_cast<bf16*>(base)), lo(hi + rows * kBP) {}
    __device__ __forceinline__ void put8(int row, int c, const float (&x)[8]) const {
        bf16x8 h, l;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[e] = (bf16)x[e];
            l[e] = (bf16)(x[e] - (float)h[e]);
        }
        *reinterpret_cast<bf16x8*>(hi + row * kBP + c) = h;
        *reinterpret_cast<bf16x8*>(lo + row * kBP + c) = l;
    }
};

// acc += (rows a0 .. a0 + 15 of A) (rows b0 .. b0 + 15 of B)^T over 128 channels
__device__ __forceinline__ floatx4 gram(const Rows<float>& A, int a0, const Rows<float>& B, int b0,
                                        int l16, int g) {
    floatx4 acc = zero4();
#pragma unroll
    for (int kb = 0; kb < kHeadDim; kb += 16)
        acc = mma_f32_k16(frag_k16(A.p + (a0 + l16) * kFP, kb, g), frag_k16(B.p + (b0 + l16) * kFP, kb, g),
                          acc);
    return acc;
}
__device__ __forceinline__ floatx4 gram(const Rows<bf16>& A, int a0, const Rows<bf16>& B, int b0,
                                        int l16, int g) {
    floatx4 acc = zero4();
#pragma unroll
    for (int kb = 0; kb < kHeadDim; kb += 32) {
        const bf16x8 ah = frag_k32(A.hi + (a0 + l16) * kBP, kb, g), al = frag_k32(A.lo + (a0 + l16) * kBP, kb, g);
        const bf16x8 bh = frag_k32(B.hi + (b0 + l16) * kBP, kb, g), bl = frag_k32(B.lo + (b0 + l16) * kBP, kb, g);
        acc = mma_bf16_k32(al, bh, acc);
        acc = mma_bf16_k32(ah, bl, acc);
        acc = mma_bf16_k32(ah, bh, acc);
    }
    return acc;
}

// Row tiles of X times 32 rows kb .. kb + 31 of this wavefront's state
// columns (s[8 rows][2 columns]: rows kb + 4 g + 0..3 and kb + 16 + 4 g + 0..3)
template <int RT>
__device__ __forceinline__ void state_product(const Rows<float>& X, int kb, const floatx2 (&s)[8],
                                              floatx4 (&acc)[RT][2], int nrt, int l16, int g) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        floatx4 b[2];
#pragma unroll
        for (int t = 0; t < 2; ++t)
            b[t] = floatx4{s[4 * half][t], s[4 * half + 1][t], s[4 * half + 2][t], s[4 * half + 3][t]};
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            if (r < nrt) {
                const floatx4 a = frag_k16(X.p + (16 * r + l16) * kFP, kb + 16 * half, g);
#pragma unroll
                for (int t = 0; t < 2; ++t) acc[r][t] = mma_f32_k16(a, b[t], acc[r][t]);
            }
        }
    }
}
template <int RT>
__device__ __forceinline__ void state_product(const Rows<bf16>& X, int kb, const floatx2 (&s)[8],
                                              floatx4 (&acc)[RT][2], int nrt, int l16, int g) {
    bf16x8 bh[2], bl[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            bh[t][e] = (bf16)s[e][t];
            bl[t][e] = (bf16)(s[e][t] - (float)bh[t][e]);
        }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        if (r < nrt) {
            const bf16x8 ah = frag_k32(X.hi + (16 * r + l16) * kBP, kb, g);
            const bf16x8 al = frag_k32(X.lo + (16 * r + l16) * kBP, kb, g);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                acc[r][t] = mma_bf16_k32(al, bh[t], acc[r][t]);
                acc[r][t] = mma_bf16_k32(ah, bl[t], acc[r][t]);
                acc[r][t] = mma_bf16_k32(ah, bh[t], acc[r][t]);
            }
        }
    }
}

__device__ __forceinline__ void row8(const bf16* p, float (&x)[8]) {
    const bf16x8 a = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = (float)a[e];
}
__device__ __forceinline__ void row8(const float* p, float (&x)[8]) {
    const floatx4 a = *reinterpret_cast<const floatx4*>(p), b = *reinterpret_cast<const floatx4*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        x[e] = a[e];
        x[4 + e] = b[e];
    }
}
__device__ __forceinline__ floatx2 pair(const bf16* p) {
    const bf16x2 a = *reinterpret_cast<const bf16x2*>(p);
    return floatx2{(float)a[0], (float)a[1]};
}
__device__ __forceinline__ floatx2 pair(const float* p) { return *reinterpret_cast<const floatx2*>(p); }
__device__ __forceinline__ void put_pair(bf16* p, float x, float y) {
    *reinterpret_cast<bf16x2*>(p) = bf16x2{(bf16)x, (bf16)y};   // RNE
}
__device__ __forceinline__ void put_pair(float* p, float x, float y) {
    *reinterpret_cast<floatx2*>(p) = floatx2{x, y};
}

__device__ __forceinline__ float finite_or_0(float x) { return x - x == 0.f ? x : 0.f; }
// non-finite elements become 0; whether there was one
__device__ __forceinline__ bool drop_nonfinite(float (&x)[8]) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fmaf(x[e], 0.f, s);   // 0, or NaN
    if (s == 0.f) return false;
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = finite_or_0(x[e]);
    return true;
}
// whether any of this lane's row of 16 lanes says so
__device__ __forceinline__ bool any_of_row(bool x, int lane) {
    return ((__ballot(x) >> (lane & 48)) & 0xffff) != 0;
}

// LDS of a workgroup for up to 16 NT nodes
template <typename T, int NT>
struct TreeLds {
    static constexpr int kN = 16 * NT;
    static constexpr int kLP = kN + 4;                        // a row of a Gram matrix
    static constexpr int kRowsB = kN * Rows<T>::kBytes;       // an operand array
    static constexpr int kGramB = 2 * kN * kLP * 4;           // both Gram matrices
    static constexpr int kGB = kN * kFP * 4;                  // G
    static constexpr int kXk = 0, kXq = kRowsB;
    static constexpr int kY = 2 * kRowsB;                     // log alpha, then Y or the Gram matrices
    static constexpr int kG = kY + (kRowsB > kGramB ? kRowsB : kGramB);   // G, then the Gram matrices
    static constexpr int kInv = kG + (kGramB > kGB ? kGramB : kGB);
    static constexpr int kBeta = kInv + NT * 16 * 20 * 4;
    static constexpr int kAnc = kBeta + kN * 4;
    static constexpr int kBad = kAnc + kN * 8;                // non-finite log alpha, k, beta of a node
    static constexpr int kFlag = kBad + 3 * kN * 4;
    static constexpr int kBytes = kFlag + 16;
};

template <typename T, int NT>
__global__ __launch_bounds__(256) void tree_decode_kernel(TreeDecodeArgs a) {
    using L = TreeLds<T, NT>;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int H = a.H, N = a.N;
    const int64_t b = blockIdx.x / (unsigned)H;
    const int h = blockIdx.x % (unsigned)H;
    const int n = __builtin_amdgcn_readfirstlane(tree_count(a.n_node, b, N));
    if (n == 0) return;
    const int nt = (n + 15) / 16;
    const size_t HD = (size_t)H * kHeadDim;
    const size_t base = ((size_t)b * N * H + h) * kHeadDim;   // node 0's row; nodes are HD apart
    const T* k = static_cast<const T*>(a.k) + base;
    const T* q = static_cast<const T*>(a.q) + base;
    const T* v = static_cast<const T*>(a.v) + base;
    const T* la = static_cast<const T*>(a.log_alpha) + base;
    const T* beta = static_cast<const T*>(a.beta) + (size_t)b * N * H + h;
    T* o = static_cast<T*>(a.o) + base;
    const int c0 = 32 * w + 2 * l16;                          // this lane's first column
    const float* S = a.S + ((size_t)b * H + h) * (kHeadDim * kHeadDim) + (size_t)(4 * g) * kHeadDim + c0;

    const Rows<T> Xk(lds + L::kXk, L::kN), Xq(lds + L::kXq, L::kN), Y(lds + L::kY, L::kN);
    float* stage = reinterpret_cast<float*>(lds + L::kY);     // log alpha, then Y
    float* G = reinterpret_cast<float*>(lds + L::kG);
    float* inv = reinterpret_cast<float*>(lds + L::kInv);
    float* sbeta = reinterpret_cast<float*>(lds + L::kBeta);
    uint64_t* anc = reinterpret_cast<uint64_t*>(lds + L::kAnc);
    int* bad = reinterpret_cast<int*>(lds + L::kBad);
    int* flag = reinterpret_cast<int*>(lds + L::kFlag);

    // ---- node rows: thread = (row, 8 channels), 16 rows a pass --------------
    const int r16 = tid >> 4, c8 = 8 * (tid & 15);
#pragma unroll
    for (int I = 0; I < NT; ++I) {
        if (I >= nt) break;
        const int i = 16 * I + r16;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (i < n) row8(la + i * HD + c8, x);
        const bool unsound = drop_nonfinite(x);
        const bool any = any_of_row(unsound, lane);
        if (l16 == 0) bad[i] = any;
        float* d = stage + i * kFP + c8;
        *reinterpret_cast<floatx4*>(d) = floatx4{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<floatx4*>(d + 4) = floatx4{x[4], x[5], x[6], x[7]};
    }
    if (w == 0) {
        // ancestor masks by doubling: a lane joins the mask of the node it points at, then points where
        // that node points
        int p = lane < n ? tree_parent(a.parent, b, N, lane) : -1;
        uint64_t m = (uint64_t)1 << lane;
        while (__ballot(p >= 0)) {
            const uint64_t pm = __shfl(m, p < 0 ? lane : p, 64);
            const int pp = __shfl(p, p < 0 ? lane : p, 64);
            if (p >= 0) {
                m |= pm;
                p = pp;
            }
        }
        if (lane < L::kN) {
            const float bt = lane < n ? to_f32(beta[(size_t)lane * H]) : 0.f;
            const bool sound = bt - bt == 0.f;
            anc[lane] = m;
            sbeta[lane] = sound ? bt : 0.f;
            bad[2 * L::kN + lane] = !sound;
        }
    }
    __syncthreads();

    // ---- G = (ancestor matrix) (log alpha): this wavefront's 32 channels ----
    bool deep = false;
#pragma unroll
    for (int I = 0; I < NT; ++I) {
        if (I >= nt) break;
        const uint64_t m = anc[16 * I + l16];
        floatx4 acc[2] = {zero4(), zero4()};
#pragma unroll
        for (int J = 0; J <= I; ++J) {
            const uint32_t bits = (uint32_t)(m >> (16 * J + 4 * g));
            const floatx4 am = {(bits & 1) ? 1.f : 0.f, (bits & 2) ? 1.f : 0.f, (bits & 4) ? 1.f : 0.f,
                                (bits & 8) ? 1.f : 0.f};
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float* src = stage + (16 * J + 4 * g) * kFP + 32 * w + 16 * t + l16;
                acc[t] = mma_f32_k16(am, floatx4{src[0], src[kFP], src[2 * kFP], src[3 * kFP]}, acc[t]);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                G[(16 * I + 4 * g + e) * kFP + 32 * w + 16 * t + l16] = acc[t][e];
                deep |= !(acc[t][e] >= -kMaxDecay);
            }
    }
    const bool any_deep = __any(deep);
    if (lane == 0) flag[w] = any_deep ? 1 : 0;
    __syncthreads();
    deep = (flag[0] | flag[1] | flag[2] | flag[3]) != 0;

    // ---- scaled rows --------------------------------------------------------
#pragma unroll
    for (int I = 0; I < NT; ++I) {
        if (I >= nt) break;
        const int i = 16 * I + r16;
        float kx[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, qx[8], x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) qx[e] = 0.f;
        if (i < n) {
            row8(k + i * HD + c8, kx);
            row8(q + i * HD + c8, qx);
        }
        const bool unsound = drop_nonfinite(kx);
        const bool any = any_of_row(unsound, lane);
        if (l16 == 0) bad[L::kN + i] = any;
        float gv[8];
        row8(G + i * kFP + c8, gv);
        float ex[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) ex[e] = expf(gv[e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = kx[e] * ex[e];
        Xk.put8(i, c8, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = qx[e] * ex[e];
        Xq.put8(i, c8, x);
        if (!deep) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = kx[e] * expf(-gv[e]);
            Y.put8(i, c8, x);
        }
    }
    __syncthreads();

    // ---- Gram matrices, masked by ancestry ----------------------------------
    // (pair by pair they are written while G is read: to the unused Y)
    float* gkk = reinterpret_cast<float*>(lds + (deep ? L::kY : L::kG));
    float* gqk = gkk + L::kN * L::kLP;
    if (!deep) {
        int tile = 0;
#pragma unroll
        for (int I = 0; I < NT; ++I) {
            if (I >= nt) break;
#pragma unroll
            for (int J = 0; J <= I; ++J) {
#pragma unroll
                for (int s = 0; s < 2; ++s, ++tile) {
                    if ((tile & 3) != w) continue;
                    const floatx4 acc = gram(s ? Xq : Xk, 16 * I, Y, 16 * J, l16, g);
                    const int j = 16 * J + l16;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = 16 * I + 4 * g + e;
                        const bool on = ((anc[i] >> j) & 1) && (s || j != i);
                        (s ? gqk : gkk)[i * L::kLP + j] = on ? (s ? acc[e] : sbeta[i] * acc[e]) : 0.f;
                    }
                }
            }
        }
    } else {
        for (int pr = tid; pr < 256 * nt * nt; pr += 256) {
            const int i = pr / (16 * nt), j = pr % (16 * nt);
            float skk = 0.f, sqk = 0.f;
            if (i < n && ((anc[i] >> j) & 1)) {
                for (int c = 0; c < kHeadDim; ++c) {
                    const float kd = finite_or_0(to_f32(k[j * HD + c])) * expf(G[i * kFP + c] - G[j * kFP + c]);
                    skk += finite_or_0(to_f32(k[i * HD + c])) * kd;
                    sqk += to_f32(q[i * HD + c]) * kd;
                }
            }
            gkk[i * L::kLP + j] = i == j ? 0.f : sbeta[i] * skk;
            gqk[i * L::kLP + j] = sqk;
        }
    }
    __syncthreads();

    // ---- inverses of the unit lower triangular diagonal blocks I + L --------
    if (w == 0 && g < nt) {   // lane = (block g, column l16)
        const float* Lg = gkk + 16 * g * L::kLP + 16 * g;
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float s = r == l16 ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < r; ++j) s -= Lg[r * L::kLP + j] * x[j];
            x[r] = s;
            inv[(16 * g + r) * 20 + l16] = s;
        }
    }

    // ---- held and read: X S, this wavefront's columns -----------------------
    floatx4 held[NT][2], read[NT][2];
#pragma unroll
    for (int r = 0; r < NT; ++r) held[r][0] = held[r][1] = read[r][0] = read[r][1] = zero4();
#pragma unroll
    for (int kb = 0; kb < kHeadDim; kb += 32) {
        floatx2 s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s[e] = __builtin_nontemporal_load(
                reinterpret_cast<const floatx2*>(S + (kb + 16 * (e >> 2) + (e & 3)) * kHeadDim));
        state_product<NT>(Xk, kb, s, held, nt, l16, g);
        state_product<NT>(Xq, kb, s, read, nt, l16, g);
    }
    __syncthreads();

    // ---- pseudo-values and outputs, block by block --------------------------
    const uint64_t bad_node = __ballot(lane < n && (bad[lane] | bad[L::kN + lane] | bad[2 * L::kN + lane]));
    uint64_t bad_col[2] = {bad_node, bad_node};   // bit j: node j taints this lane's column t
    floatx2 vv[NT][4];
#pragma unroll
    for (int I = 0; I < NT; ++I) {
        if (I >= nt) break;
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 16 * I + 4 * g + e;
            vv[I][e] = i < n ? pair(v + i * HD + c0) : floatx2{0.f, 0.f};
            s = __builtin_fmaf(vv[I][e][0], 0.f, __builtin_fmaf(vv[I][e][1], 0.f, s));
        }
        if (__any(s != 0.f)) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t m = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = vv[I][e][t];
                    vv[I][e][t] = finite_or_0(x);
                    m |= (x - x == 0.f ? 0u : 1u) << (4 * g + e);
                }
                m |= __shfl_xor(m, 16, 64);
                m |= __shfl_xor(m, 32, 64);
                bad_col[t] |= (uint64_t)m << (16 * I);
            }
        }
    }
    const bool tainted = __any((bad_col[0] | bad_col[1]) != 0);
#pragma unroll
    for (int I = 0; I < NT; ++I) {
        if (I >= nt) break;
        const floatx4 bt = *reinterpret_cast<const floatx4*>(sbeta + 16 * I + 4 * g);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            floatx4 rhs;
#pragma unroll
            for (int e = 0; e < 4; ++e) rhs[e] = bt[e] * (vv[I][e][t] - held[I][t][e]);
            floatx4 prev = zero4();
#pragma unroll
            for (int J = 0; J < I; ++J)
                prev = mma_f32_k16(frag_k16(gkk + (16 * I + l16) * L::kLP, 16 * J, g), held[J][t], prev);
            rhs -= prev;
            held[I][t] = mma_f32_k16(frag_k16(inv + (16 * I + l16) * 20, 0, g), rhs, zero4());
        }
        floatx4 out[2] = {zero4(), zero4()};
#pragma unroll
        for (int J = 0; J <= I; ++J) {
            const floatx4 am = frag_k16(gqk + (16 * I + l16) * L::kLP, 16 * J, g);
#pragma unroll
            for (int t = 0; t < 2; ++t) out[t] = mma_f32_k16(am, held[J][t], out[t]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) out[t] += read[I][t];
        if (tainted) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t m = anc[16 * I + 4 * g + e];
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (m & bad_col[t]) out[t][e] = __builtin_nanf("");
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = 16 * I + 4 * g + e;
            if (i < n) put_pair(o + i * HD + c0, out[0][e], out[1][e]);
        }
    }
}

template <typename T, int NT>
hipError_t launch_nt(const TreeDecodeArgs& a, hipStream_t stream) {
    static std::atomic<uint64_t> done{0};
    constexpr int bytes = TreeLds<T, NT>::kBytes;
    const auto kern = tree_decode_kernel<T, NT>;
    if (bytes > 64 * 1024) {
        const hipError_t e = raise_lds_limit_once(reinterpret_cast<const void*>(kern), bytes, done);
        if (e != hipSuccess) return e;
    }
    kern<<<dim3((unsigned)((int64_t)a.B * a.H)), dim3(256), bytes, stream>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const TreeDecodeArgs& a, hipStream_t stream) {
    if (a.N <= 16) return launch_nt<T, 1>(a, stream);
    if (a.N <= 32) return launch_nt<T, 2>(a, stream);
    return launch_nt<T, 4>(a, stream);
}

}  // namespace

hipError_t launch_tree_decode(const TreeDecodeArgs& a, int dtype, hipStream_t stream) {
    return dtype == 0 ? launch_t<float>(a, stream) : launch_t<bf16>(a, stream);
}

}  // namespace kda
