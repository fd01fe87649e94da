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
// Mapping.  One workgroup of four wavefronts per (sequence, head).  Before
// the product with the state wavefront w owns key channels 32 w .. 32 w + 31
// of all nodes: G^T comes out of its MFMA with a lane holding 4 channels of
// one node, the layout in which k and q are loaded and the scaled rows leave
// for LDS, so none of it needs another wavefront.  From the state product on
// it owns value columns 32 w .. 32 w + 31 (lane: columns 2 (l % 16), +1) over
// all 128 state rows, and pseudo-values, solve and outputs stay in its own
// accumulators.  All loads, the state's included, are issued at the start.
#include <type_traits>

#include "kda.h"
#include "kda_device.h"
#include "kda_tree.h"

namespace kda {

namespace {

constexpr float kMaxDecay = 64.f;   // |G| up to which e^{-G} is formed
constexpr int kFP = kHeadDim + 4;   // fp32 LDS row
constexpr int kBP = kHeadDim + 8;   // bf16 LDS row

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// x, y as bf16 (hi) and the bf16 of what that leaves out (lo)
__device__ __forceinline__ void split2(float x, float y, bf16x2& hi, bf16x2& lo) {
    hi = __builtin_convertvector((floatx2{x, y}), bf16x2);
    const uint32_t u = __builtin_bit_cast(uint32_t, hi);
    lo = __builtin_convertvector((floatx2{x - __builtin_bit_cast(float, u << 16),
                                          y - __builtin_bit_cast(float, u & 0xffff0000u)}), bf16x2);
}
__device__ __forceinline__ bf16x4 join(bf16x2 a, bf16x2 b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3); }
__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

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
    __device__ __forceinline__ void put4(int row, int c, floatx4 x) const {
        *reinterpret_cast<floatx4*>(p + row * kFP + c) = x;
    }
    __device__ __forceinline__ float get(int row, int c) const { return p[row * kFP + c]; }
    // fp32 values kept whole in the place of a row's elements
    __device__ __forceinline__ void put4_f32(int row, int c, floatx4 x) const { put4(row, c, x); }
    __device__ __forceinline__ float get_f32(int row, int c) const { return get(row, c); }
};
template <>
struct Rows<bf16> {
    static constexpr int kBytes = 2 * kBP * 2;
    bf16* hi;
    bf16* lo;
    __device__ __forceinline__ Rows(unsigned char* base, int rows)
        : hi(reinterpret_cast<bf16*>(base)), lo(hi + rows * kBP) {}
    __device__ __forceinline__ void put4(int row, int c, floatx4 x) const {
        bf16x2 h[2], l[2];
        split2(x[0], x[1], h[0], l[0]);
        split2(x[2], x[3], h[1], l[1]);
        *reinterpret_cast<bf16x4*>(hi + row * kBP + c) = join(h[0], h[1]);
        *reinterpret_cast<bf16x4*>(lo + row * kBP + c) = join(l[0], l[1]);
    }
    __device__ __forceinline__ float get(int row, int c) const {
        return (float)hi[row * kBP + c] + (float)lo[row * kBP + c];
    }
    // fp32 values kept whole in the place of a row's elements: upper half in hi, lower half in lo
    __device__ __forceinline__ void put4_f32(int row, int c, floatx4 x) const {
        shortx4 h, l;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t u = __builtin_bit_cast(uint32_t, (float)x[e]);
            h[e] = (short)(u >> 16);
            l[e] = (short)u;
        }
        *reinterpret_cast<shortx4*>(hi + row * kBP + c) = h;
        *reinterpret_cast<shortx4*>(lo + row * kBP + c) = l;
    }
    __device__ __forceinline__ float get_f32(int row, int c) const {
        const uint32_t h = *reinterpret_cast<const uint16_t*>(hi + row * kBP + c);
        const uint32_t l = *reinterpret_cast<const uint16_t*>(lo + row * kBP + c);
        return __builtin_bit_cast(float, h << 16 | l);
    }
};

// (rows a0 .. a0 + 15 of A) (rows b0 .. b0 + 15 of B)^T over channels c0 .. c1 - 1
__device__ __forceinline__ floatx4 gram(const Rows<float>& A, int a0, const Rows<float>& B, int b0,
                                        int c0, int c1, int l16, int g) {
    floatx4 acc = zero4();
#pragma unroll
    for (int kb = c0; kb < c1; kb += 16)
        acc = mma_f32_k16(frag_k16(A.p + (a0 + l16) * kFP, kb, g), frag_k16(B.p + (b0 + l16) * kFP, kb, g),
                          acc);
    return acc;
}
__device__ __forceinline__ floatx4 gram(const Rows<bf16>& A, int a0, const Rows<bf16>& B, int b0,
                                        int c0, int c1, int l16, int g) {
    floatx4 acc = zero4();
#pragma unroll
    for (int kb = c0; kb < c1; kb += 32) {
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
        bf16x2 h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(s[2 * e][t], s[2 * e + 1][t], h[e], l[e]);
        bh[t] = join(join(h[0], h[1]), join(h[2], h[3]));
        bl[t] = join(join(l[0], l[1]), join(l[2], l[3]));
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

// Elements through a buffer resource of the sequence's nodes: 32-bit
// offsets, and rows past the nodes read 0 and drop their stores.
template <typename T>
struct Elems;
template <>
struct Elems<bf16> {
    typedef bf16x2 two;    // as loaded
    typedef bf16x4 four;
    static __device__ __forceinline__ bf16 load1(rsrc_t r, uint32_t off) { return buf_load_bf16(r, off); }
    static __device__ __forceinline__ two load2(rsrc_t r, uint32_t off) {
        return __builtin_bit_cast(bf16x2, __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
    }
    static __device__ __forceinline__ four load4(rsrc_t r, uint32_t off) { return buf_load_bf16x4(r, off); }
    static __device__ __forceinline__ void store2(rsrc_t r, uint32_t off, float x, float y) {   // RNE
        __builtin_amdgcn_raw_buffer_store_b32(
            __builtin_bit_cast(int, __builtin_convertvector((floatx2{x, y}), bf16x2)), r, (int)off, 0, 0);
    }
};
typedef unsigned int uintx2_t __attribute__((ext_vector_type(2)));
template <>
struct Elems<float> {
    typedef floatx2 two;
    typedef floatx4 four;
    static __device__ __forceinline__ float load1(rsrc_t r, uint32_t off) {
        return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0));
    }
    static __device__ __forceinline__ two load2(rsrc_t r, uint32_t off) {
        return __builtin_bit_cast(floatx2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, 0));
    }
    static __device__ __forceinline__ four load4(rsrc_t r, uint32_t off) {
        return __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
    }
    static __device__ __forceinline__ void store2(rsrc_t r, uint32_t off, float x, float y) {
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(uintx2_t, floatx2{x, y}), r, (int)off, 0, 0);
    }
};
__device__ __forceinline__ floatx4 widen(bf16x4 x) {
    return floatx4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
}
__device__ __forceinline__ floatx4 widen(floatx4 x) { return x; }

// s, or NaN where an element is not finite
__device__ __forceinline__ float probe(float s, floatx2 x) {
    return __builtin_fmaf(x[0], 0.f, __builtin_fmaf(x[1], 0.f, s));
}
__device__ __forceinline__ float probe(float s, bf16x2 x) {
    return probe(s, floatx2{(float)x[0], (float)x[1]});
}
template <typename V>
__device__ __forceinline__ float probe4(float s, V x) {
    return probe(probe(s, __builtin_shufflevector(x, x, 0, 1)), __builtin_shufflevector(x, x, 2, 3));
}

// bits 0..3 as four bf16, 1 or 0
__device__ __forceinline__ bf16x4 bits4(uint32_t b) {
    typedef uint32_t u2 __attribute__((ext_vector_type(2)));
    // two bits to the low bits of two halves, times the bf16 one
    const uint32_t lo = ((b & 3u) * 0x8001u) & 0x10001u, hi = (((b >> 2) & 3u) * 0x8001u) & 0x10001u;
    return __builtin_bit_cast(bf16x4, u2{lo * 0x3f80u, hi * 0x3f80u});
}

// G^T of 16 nodes (columns) and 16 channels: log alpha^T (a: channel l16,
// nodes 16 J + 4 g + 0..3) times the ancestor bits of node l16
template <int NT, typename M>
__device__ __forceinline__ floatx4 gather_decay(const floatx4 (&a)[NT], M m, int I, int g) {
    floatx4 acc = zero4();
#pragma unroll
    for (int J = 0; J < NT; ++J) {
        if (J > I) break;
        const uint32_t bits = (uint32_t)(m >> (16 * J + 4 * g));
        acc = mma_f32_k16(a[J], floatx4{(bits & 1) ? 1.f : 0.f, (bits & 2) ? 1.f : 0.f,
                                        (bits & 4) ? 1.f : 0.f, (bits & 8) ? 1.f : 0.f}, acc);
    }
    return acc;
}
// (bf16 log alpha times 0 or 1 is exact)
template <int NT, typename M>
__device__ __forceinline__ floatx4 gather_decay(const bf16x4 (&a)[NT], M m, int I, int g) {
    floatx4 acc = zero4();
#pragma unroll
    for (int J = 0; J < NT; J += 2) {
        if (J > I) break;
        const bf16 z = (bf16)0.f;
        const bf16x4 zero = {z, z, z, z};
        const bool two = J + 1 < NT;
        acc = mma_bf16_k32(join(a[J], two ? a[two ? J + 1 : J] : zero),
                           join(bits4((uint32_t)(m >> (16 * J + 4 * g))),
                                two ? bits4((uint32_t)(m >> (two ? 16 * J + 16 + 4 * g : 0))) : zero),
                           acc);
    }
    return acc;
}

// e^x: for bf16 results the hardware's 2^x (x log2 e rounds to |x| 2^-24, at
// |x| <= 64 some 2^-18 of the result), for fp32 the library's
template <typename T>
__device__ __forceinline__ float exp_t(float x) { return __expf(x); }
template <>
__device__ __forceinline__ float exp_t<float>(float x) { return expf(x); }

__device__ __forceinline__ float finite_or_0(float x) { return x - x == 0.f ? x : 0.f; }
// LDS of a workgroup for up to 16 NT nodes
template <typename T, int NT>
struct TreeLds {
    static constexpr int kN = 16 * NT;
    static constexpr int kLP = kN + 4;                        // a row of a Gram matrix
    static constexpr int kRowsB = kN * Rows<T>::kBytes;       // an operand array
    static constexpr int kXk = 0, kXq = kRowsB;
    static constexpr int kY = 2 * kRowsB;                     // Y; for channels out of range G itself
    static constexpr int kGram = 3 * kRowsB;                  // both Gram matrices
    static constexpr int kDiag = kGram + 2 * kN * kLP * 4;    // diagonal blocks of the first, transposed
    static constexpr int kInv = kDiag + NT * 16 * 20 * 4;     // their inverses (of I + block)
    // NT = 1: the wavefronts' parts of both Gram tiles
    static constexpr int kPart = kInv + NT * 16 * 20 * 4;
    static constexpr int kBeta = kPart + (NT == 1 ? 4 * 2 * 16 * 20 * 4 : 0);
    static constexpr int kAnc = kBeta + kN * 4;               // (8 bytes a node)
    static constexpr int kBad = kAnc + kN * 8;                // per wavefront: nodes with non-finite inputs
    static constexpr int kFlag = kBad + 4 * 8;                // per wavefront: channels out of range
    static constexpr int kBytes = kFlag + 16;
};

template <typename T, int NT>
__global__ __launch_bounds__(256, NT == 1 ? 3 : (NT == 2 ? 2 : 1)) void tree_decode_kernel(TreeDecodeArgs a) {
    using L = TreeLds<T, NT>;
    using E = Elems<T>;
    using Mask = typename std::conditional<NT <= 2, uint32_t, uint64_t>::type;   // a bit per node
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int H = a.H, N = a.N;
    const int64_t b = blockIdx.x / (unsigned)H;
    const int h = blockIdx.x % (unsigned)H;
    const int n = __builtin_amdgcn_readfirstlane(tree_count(a.n_node, b, N));
    if (n == 0) return;
    const int nt = (n + 15) / 16;
    constexpr uint32_t es = sizeof(T);
    const uint32_t row_b = (uint32_t)H * kHeadDim * es;       // from node to node (64 rows: < 2^32 bytes)
    const size_t base = ((size_t)b * N * H + h) * kHeadDim;   // node 0's row
    const uint32_t rows_b = (uint32_t)(n - 1) * row_b + kHeadDim * es;
    auto rows = [&](const void* p) { return make_rsrc_u32(static_cast<const T*>(p) + base, rows_b); };
    const rsrc_t kr_ = rows(a.k), qr_ = rows(a.q), vr_ = rows(a.v), lr_ = rows(a.log_alpha), or_ = rows(a.o);
    const int c0 = 32 * w + 2 * l16;                          // this lane's first value column

    const Rows<T> Xk(lds + L::kXk, L::kN), Xq(lds + L::kXq, L::kN), Y(lds + L::kY, L::kN);
    float* gkk = reinterpret_cast<float*>(lds + L::kGram);
    float* gqk = gkk + L::kN * L::kLP;
    float* diag = reinterpret_cast<float*>(lds + L::kDiag);
    float* inv = reinterpret_cast<float*>(lds + L::kInv);
    float* part = reinterpret_cast<float*>(lds + L::kPart);
    float* sbeta = reinterpret_cast<float*>(lds + L::kBeta);
    Mask* anc = reinterpret_cast<Mask*>(lds + L::kAnc);
    Mask* bad = reinterpret_cast<Mask*>(lds + L::kBad);
    int* flag = reinterpret_cast<int*>(lds + L::kFlag);

    // ---- everything this workgroup reads, in the order it is needed ---------
    int par = lane < n ? tree_parent(a.parent, b, N, lane) : -1;
    typename E::four lar[2][NT], kr[NT][2], qr[NT][2];
    const uint32_t at_g = 4 * g * row_b, at_l = l16 * row_b;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int J = 0; J < NT; ++J)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                lar[t][J][e] = E::load1(lr_, at_g + (32 * w + l16) * es + (16 * J + e) * row_b + 16 * t * es);
#pragma unroll
    for (int I = 0; I < NT; ++I)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t off = at_l + (32 * w + 4 * g) * es + 16 * I * row_b + 16 * t * es;
            kr[I][t] = E::load4(kr_, off);
            qr[I][t] = E::load4(qr_, off);
        }
    float bt = to_f32(E::load1(make_rsrc_u32(static_cast<const T*>(a.beta) + (size_t)b * N * H + h,
                                             ((uint32_t)(n - 1) * H + 1) * es),
                               (uint32_t)lane * H * es));
    typename E::two vv[NT][4];
#pragma unroll
    for (int I = 0; I < NT; ++I)
#pragma unroll
        for (int e = 0; e < 4; ++e) vv[I][e] = E::load2(vr_, at_g + c0 * es + (16 * I + e) * row_b);
    floatx2 st[4][8];
    {
        const rsrc_t sr = make_rsrc_u32(a.S + ((size_t)b * H + h) * (kHeadDim * kHeadDim),
                                        kHeadDim * kHeadDim * 4);
        const int at = (4 * g * kHeadDim + c0) * 4;
#pragma unroll
        for (int kb = 0; kb < 4; ++kb)
#pragma unroll
            for (int e = 0; e < 8; ++e)   // read once: streamed past the caches
                st[kb][e] = __builtin_bit_cast(
                    floatx2, __builtin_amdgcn_raw_buffer_load_b64(
                                 sr, at + (e & 3) * kHeadDim * 4, (32 * kb + 16 * (e >> 2)) * kHeadDim * 4, 2));
    }
    __builtin_amdgcn_sched_barrier(0);

    // ---- ancestor masks, lane = node, by doubling: a lane joins the mask of the node it points at, then
    // points where that node points
    Mask mask = lane < L::kN ? (Mask)1 << (lane & (L::kN - 1)) : 0;
    while (__ballot(par >= 0)) {
        const Mask pm = __shfl(mask, par < 0 ? lane : par, 64);
        const int pp = __shfl(par, par < 0 ? lane : par, 64);
        if (par >= 0) {
            mask |= pm;
            par = pp;
        }
    }
    if (w == 0 && lane < L::kN) {
        anc[lane] = mask;
        sbeta[lane] = finite_or_0(bt);
    }

    // ---- G^T, scaled rows: this wavefront's 32 channels ----------------------
    Mask bad_node = (Mask)__ballot(!(bt - bt == 0.f));   // non-finite beta, log alpha, k
    {
        float s = 0.f;
#pragma unroll
        for (int J = 0; J < NT; ++J)
#pragma unroll
            for (int t = 0; t < 2; ++t) s = probe4(probe4(s, lar[t][J]), kr[J][t]);
        if (__any(s != 0.f)) {
#pragma unroll
            for (int J = 0; J < NT; ++J)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = (float)lar[t][J][e];   // node 16 J + 4 g + e
                        uint64_t off = __ballot(!(x - x == 0.f));
#pragma unroll
                        for (int gg = 0; gg < 4; ++gg)
                            if ((off >> (16 * gg)) & 0xffff) bad_node |= (Mask)1 << (16 * J + 4 * gg + e);
                        lar[t][J][e] = (T)finite_or_0(x);
                        x = (float)kr[J][t][e];          // node 16 J + l16
                        off = __ballot(!(x - x == 0.f));
                        off |= off >> 32;
                        off |= off >> 16;
                        bad_node |= (Mask)(off & 0xffff) << (16 * J);
                        kr[J][t][e] = (T)finite_or_0(x);
                    }
        }
    }
    floatx4 GT[NT][2];
    float least = 0.f;
#pragma unroll
    for (int I = 0; I < NT; ++I) {
        if (I >= nt) break;
        const Mask m = __shfl(mask, 16 * I + l16, 64);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            GT[I][t] = gather_decay<NT>(lar[t], m, I, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) least = fminf(least, GT[I][t][e]);
        }
    }
    const bool deep = __any(least < -kMaxDecay);
#pragma unroll
    for (int I = 0; I < NT; ++I) {
        if (I >= nt) break;
        const int i = 16 * I + l16;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int c = 32 * w + 16 * t + 4 * g;
            const floatx4 kx = widen(kr[I][t]), qx = widen(qr[I][t]);
            floatx4 ex;
#pragma unroll
            for (int e = 0; e < 4; ++e) ex[e] = exp_t<T>(GT[I][t][e]);
            Xk.put4(i, c, kx * ex);
            Xq.put4(i, c, qx * ex);
            if (!deep) {
#pragma unroll
                for (int e = 0; e < 4; ++e) ex[e] = exp_t<T>(-GT[I][t][e]);
                Y.put4(i, c, kx * ex);
            } else {
                Y.put4_f32(i, c, GT[I][t]);
            }
        }
    }
    if (lane == 0) {
        bad[w] = bad_node;
        flag[w] = deep ? 1 : 0;
    }
    if (NT == 1) {
        // both Gram tiles over this wavefront's channels, which it alone has written
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const floatx4 acc = gram(s ? Xq : Xk, 0, Y, 0, 32 * w, 32 * w + 32, l16, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) part[((s * 4 + w) * 16 + 4 * g + e) * 20 + l16] = acc[e];
        }
    }
    __syncthreads();

    // ---- Gram matrices, masked by ancestry ----------------------------------
    const int deep_waves = flag[0] | flag[1] << 1 | flag[2] << 2 | flag[3] << 3;
    if (deep_waves == 0 && NT == 1) {
        const int i = tid >> 4, j = tid & 15, x = i * 20 + j;
        const bool on = (anc[i] >> j) & 1;
        float s[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const float* pm = part + m * 4 * 320 + x;
            s[m] = (pm[0] + pm[320]) + (pm[640] + pm[960]);
        }
        diag[j * 20 + i] = on && i != j ? sbeta[i] * s[0] : 0.f;
        gqk[i * L::kLP + j] = on ? s[1] : 0.f;
    } else if (deep_waves == 0) {
        int tile = 0;
#pragma unroll
        for (int I = 0; I < NT; ++I) {
            if (I >= nt) break;
#pragma unroll
            for (int J = 0; J <= I; ++J) {
#pragma unroll
                for (int s = 0; s < 2; ++s, ++tile) {
                    if ((tile & 3) != w) continue;
                    const floatx4 acc = gram(s ? Xq : Xk, 16 * I, Y, 16 * J, 0, kHeadDim, l16, g);
                    const int j = 16 * J + l16;
                    floatx4 x;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int i = 16 * I + 4 * g + e;
                        const bool on = ((anc[i] >> j) & 1) && (s || j != i);
                        x[e] = on ? (s ? acc[e] : sbeta[i] * acc[e]) : 0.f;
                        if (s || J < I) (s ? gqk : gkk)[i * L::kLP + j] = x[e];
                    }
                    if (!s && J == I) *reinterpret_cast<floatx4*>(diag + j * 20 + 4 * g) = x;
                }
            }
        }
    } else {
        // pair by pair: e^{G_i - G_j} for the channels out of range
        for (int pr = tid; pr < 256 * nt * nt; pr += 256) {
            const int i = pr / (16 * nt), j = pr % (16 * nt);
            float skk = 0.f, sqk = 0.f;
            if (i < n && ((anc[i] >> j) & 1)) {
                for (int c = 0; c < kHeadDim; ++c) {
                    if ((deep_waves >> (c >> 5)) & 1) {
                        const uint32_t at_i = i * row_b + c * es, at_j = j * row_b + c * es;
                        const float kd = finite_or_0(to_f32(E::load1(kr_, at_j))) *
                                         exp_t<T>(Y.get_f32(i, c) - Y.get_f32(j, c));
                        skk += finite_or_0(to_f32(E::load1(kr_, at_i))) * kd;
                        sqk += to_f32(E::load1(qr_, at_i)) * kd;
                    } else {
                        const float y = Y.get(j, c);
                        skk += Xk.get(i, c) * y;
                        sqk += Xq.get(i, c) * y;
                    }
                }
            }
            skk = i == j ? 0.f : sbeta[i] * skk;
            gkk[i * L::kLP + j] = skk;
            if ((i ^ j) < 16) diag[j * 20 + (i & 15)] = skk;
            gqk[i * L::kLP + j] = sqk;
        }
    }

    // ---- held and read: X S, this wavefront's columns -----------------------
    floatx4 held[NT][2], read[NT][2];
#pragma unroll
    for (int r = 0; r < NT; ++r) held[r][0] = held[r][1] = read[r][0] = read[r][1] = zero4();
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
        state_product<NT>(Xk, 32 * kb, st[kb], held, nt, l16, g);
        state_product<NT>(Xq, 32 * kb, st[kb], read, nt, l16, g);
    }
    __syncthreads();

    // ---- inverses of the unit lower triangular diagonal blocks I + L: wavefront w that of block w, lane =
    // column, column by column (once x[j] is final it leaves all later rows)
    if (w < nt && g == 0) {
        const float* Lw = diag + 16 * w * 20;   // [column][row]
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) x[r] = r == l16 ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            inv[(16 * w + j) * 20 + l16] = x[j];
#pragma unroll
            for (int r4 = (j + 1) / 4; r4 < 4; ++r4) {
                const floatx4 c = *reinterpret_cast<const floatx4*>(Lw + j * 20 + 4 * r4);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * r4 + e > j) x[4 * r4 + e] -= c[e] * x[j];
            }
        }
    }
    __syncthreads();

    // ---- pseudo-values and outputs, block by block --------------------------
    bad_node = bad[0] | bad[1] | bad[2] | bad[3];
    Mask bad_col[2] = {bad_node, bad_node};   // bit j: node j taints this lane's column t
    {
        float s = 0.f;
#pragma unroll
        for (int I = 0; I < NT; ++I)
#pragma unroll
            for (int e = 0; e < 4; ++e) s = probe(s, vv[I][e]);
        if (__any(s != 0.f)) {
#pragma unroll
            for (int I = 0; I < NT; ++I)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t m = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x = (float)vv[I][e][t];
                        vv[I][e][t] = (T)finite_or_0(x);
                        m |= (x - x == 0.f ? 0u : 1u) << (4 * g + e);
                    }
                    m |= __shfl_xor(m, 16, 64);
                    m |= __shfl_xor(m, 32, 64);
                    bad_col[t] |= (Mask)m << (16 * I);
                }
        }
    }
    const bool tainted = __any((bad_col[0] | bad_col[1]) != 0);
#pragma unroll
    for (int I = 0; I < NT; ++I) {
        if (I >= nt) break;
        const floatx4 bt4 = *reinterpret_cast<const floatx4*>(sbeta + 16 * I + 4 * g);
        const floatx4 ia = frag_k16(inv + (16 * I + l16) * 20, 0, g);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            floatx4 rhs;
#pragma unroll
            for (int e = 0; e < 4; ++e) rhs[e] = bt4[e] * ((float)vv[I][e][t] - held[I][t][e]);
            if (I > 0) {
                floatx4 prev = zero4();
#pragma unroll
                for (int J = 0; J < I; ++J)
                    prev = mma_f32_k16(frag_k16(gkk + (16 * I + l16) * L::kLP, 16 * J, g), held[J][t], prev);
                rhs -= prev;
            }
            held[I][t] = mma_f32_k16(ia, rhs, zero4());
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
                const Mask m = anc[16 * I + 4 * g + e];
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (m & bad_col[t]) out[t][e] = __builtin_nanf("");
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            E::store2(or_, at_g + c0 * es + (16 * I + e) * row_b, out[0][e], out[1][e]);
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
