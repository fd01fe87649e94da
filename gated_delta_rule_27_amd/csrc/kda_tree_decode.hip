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
// ancestor matrix with the nodes' log alpha.  In one float it would be off by
// 2^-18 at |G| of 64 and by 2^-16 at 320, and every coupling of the node by
// that of its value (outputs of nodes that keep their state below a strongly
// decayed one: 2e-5 to 3e-5 off; now at most 2e-6, where 1e-6 comes with
// any factors e^{G_i}, e^{-G_j} of 24 bits).  So it is summed in two parts, the
// first exactly, and held as a whole number of 2^-22.
//
// Range.  e^{-G_j} stays finite for at most 16 levels at the decay bound
// (log alpha >= -5).  Where some |G| of a wavefront's channels passes 64, a
// Gram tile is the sum of products over levels of G_j, 64 wide, from the
// greatest G_j of its tile of ancestors down: in a level the factors are
// e^{r - G_j} <= e^64 and, for descendants, e^{G_i - r} <= 1, r the level's
// upper end, per channel.  What underflows there is below e^{-23} of the
// level's largest entries.  (64 x 96 bf16 states, chains of 64: 495 us where
// log alpha is -0.7 on average and some |G| pass 64, 586 at -2.5, 362 where
// none does; pair by pair, with e^{G_i - G_j}, the first two took 1330 and 2540.)
//
// Masking.  Products with masked (zero) entries would spread a NaN or
// infinity of one node to its siblings.  Non-finite k, log alpha, beta (per
// node) and v (per column) are therefore taken as 0 and remembered as bits,
// and the outputs of the nodes that descend from them are set to NaN.
//
// Mapping.  One workgroup of four wavefronts per (sequence, head); all loads,
// the state's included, are issued at the start.
// Before the product with the state wavefront w owns key channels 32 w ..
// 32 w + 31 of all nodes.  G^T comes out of its MFMA with a lane holding 4
// channels of one node: the layout k and q are loaded in, and at once the
// operand layout of the Gram tiles, so these take their operands from
// registers, each wavefront over its own channels, and only the partial
// tiles are summed over the wavefronts through LDS.  The tiles are formed
// transposed (ancestor x node): a lane then holds what it has to hold of the
// tile as an operand of the solve, and keeps and reads it as 16 bytes.
// From the state product on wavefront w owns value columns 32 w .. 32 w + 31
// (lane: columns 2 (l % 16), +1) over all 128 state rows, and pseudo-values,
// solve and outputs stay in its own accumulators.  The scaled rows are all
// that every wavefront needs of the others' work; beyond 32 nodes (16 for bf16
// inputs) k's and q's rows take turns in LDS, so that two (three) workgroups
// share a compute unit.
//
// Bits.  Whatever the inputs' type, everything between them and the one
// rounding of the outputs is held in 24 bits or more: fp32 MFMA for the Gram
// tiles, the solve and the outputs, and for the product with the state fp32
// MFMA or bf16 MFMA on both operands in three bf16 parts.  (In two parts, 16
// bits, a read of neighbouring state rows with opposite signs lost what
// differs between them, as kda_decode_multi does not; 64 x 96 states of 64
// nodes took 254 us in two parts, 359 now, 32 nodes 128 against 171, 256 x 96
// of 8 nodes 304 against 308.)
//
// What bounds it, measured on bf16 inputs: the states' read up to 16 nodes,
// while four workgroups share a compute unit (256 x 96 states, 8 nodes: 308
// us, 6.0 TB/s of everything read and written, 16 nodes 418 us, 5.1 TB/s);
// from then on MFMA (fp32 for Gram tiles and solve) and the chain of load,
// Gram rounds, solve and outputs of a workgroup (64 x 96: 32 nodes 171 us, 3.8
// TB/s, 64 nodes 359 us, 2.5 TB/s and 72 TFLOP/s).  fp32 inputs: fp32 MFMA from
// 17 nodes on (64 x 96: 16 nodes 117 us, 32 nodes 221 us, 64 nodes 444 us).
// One sequence of 8 nodes x 96 heads: 6.9 us, the latency of one workgroup.
#include <type_traits>
#include <utility>

#include "kda.h"
#include "kda_device.h"
#include "kda_tree_device.h"

namespace kda {

namespace {

constexpr float kGrid = 768.f;      // added and taken off: a multiple of 2^-14, for |x| <= 256
constexpr int kLevels = 8;          // steps of it below a tile's greatest G (64 nodes of log alpha >= -5: five)
constexpr int kFP = kHeadDim + 4;   // fp32 LDS row
constexpr int kBP = kHeadDim + 8;   // bf16 LDS row

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// x, y as bf16 and, in their place, what that leaves out
__device__ __forceinline__ bf16x2 take(float& x, float& y) {
    const bf16x2 h = __builtin_convertvector((floatx2{x, y}), bf16x2);
    const uint32_t u = __builtin_bit_cast(uint32_t, h);
    x -= __builtin_bit_cast(float, u << 16);
    y -= __builtin_bit_cast(float, u & 0xffff0000u);
    return h;
}
__device__ __forceinline__ bf16x4 take4(floatx4& v) {
    float x[4] = {v[0], v[1], v[2], v[3]};
    const bf16x2 a = take(x[0], x[1]), b = take(x[2], x[3]);
    v = floatx4{x[0], x[1], x[2], x[3]};
    return __builtin_shufflevector(a, b, 0, 1, 2, 3);
}
__device__ __forceinline__ bf16x8 join(bf16x4 a, bf16x4 b) {
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// acc += a b over 32 k, fp32
__device__ __forceinline__ floatx4 mma(floatx4 a0, floatx4 a1, floatx4 b0, floatx4 b1, floatx4 acc) {
    return mma_f32_k16(a1, b1, mma_f32_k16(a0, b0, acc));
}

// Rows of 128 channels in LDS, as A operands of the state product: fp32, or
// for bf16 inputs the same value as three bf16 (24 bits, exact).
template <typename T>
struct Rows;
template <>
struct Rows<float> {
    static constexpr int kBytes = kFP * 4;   // of a row
    float* p;
    __device__ __forceinline__ Rows(unsigned char* base, int) : p(reinterpret_cast<float*>(base)) {}
    __device__ __forceinline__ void put(int row, int c, floatx4 x) const {
        *reinterpret_cast<floatx4*>(p + row * kFP + c) = x;
    }
};
template <>
struct Rows<bf16> {
    static constexpr int kBytes = 3 * kBP * 2;
    bf16* p;
    int part;   // from part to part
    __device__ __forceinline__ Rows(unsigned char* base, int rows)
        : p(reinterpret_cast<bf16*>(base)), part(rows * kBP) {}
    __device__ __forceinline__ void put(int row, int c, floatx4 x) const {
#pragma unroll
        for (int i = 0; i < 3; ++i) *reinterpret_cast<bf16x4*>(p + i * part + row * kBP + c) = take4(x);
    }
};

// 32 rows kb .. kb + 31 of one state column as the other operand: rows
// kb + 4 g + 0..3 and kb + 16 + 4 g + 0..3
template <typename T>
struct StateOp;
template <>
struct StateOp<float> {
    floatx4 half[2];
    static __device__ __forceinline__ StateOp of(const floatx2 (&s)[8], int t) {
        return StateOp{{floatx4{s[0][t], s[1][t], s[2][t], s[3][t]}, floatx4{s[4][t], s[5][t], s[6][t], s[7][t]}}};
    }
};
template <>
struct StateOp<bf16> {
    bf16x8 part[3];
    static __device__ __forceinline__ StateOp of(const floatx2 (&s)[8], int t) {
        floatx4 a = {s[0][t], s[1][t], s[2][t], s[3][t]}, b = {s[4][t], s[5][t], s[6][t], s[7][t]};
        StateOp o;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const bf16x4 x = take4(a), y = take4(b);
            o.part[i] = join(x, y);
        }
        return o;
    }
};
// acc += row tiles of X times them
template <int RT>
__device__ __forceinline__ void state_product(const Rows<float>& X, int kb, const StateOp<float> (&s)[2],
                                              floatx4 (&acc)[RT][2], int l16, int g) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const floatx4 a = frag_k16(X.p + (16 * r + l16) * kFP, kb + 16 * half, g);
#pragma unroll
            for (int t = 0; t < 2; ++t) acc[r][t] = mma_f32_k16(a, s[t].half[half], acc[r][t]);
        }
}
template <int RT>
__device__ __forceinline__ void state_product(const Rows<bf16>& X, int kb, const StateOp<bf16> (&s)[2],
                                              floatx4 (&acc)[RT][2], int l16, int g) {
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        bf16x8 a[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const bf16* row = X.p + i * X.part + (16 * r + l16) * kBP;
            a[i] = join(frag_k16(row, kb, g), frag_k16(row, kb + 16, g));
        }
        // the parts' products down to 2^-18 of the value; the three left out are below 2^-25
#pragma unroll
        for (int i = 2; i >= 0; --i)
#pragma unroll
            for (int j = 2 - i; j >= 0; --j)
#pragma unroll
                for (int t = 0; t < 2; ++t) acc[r][t] = mma_bf16_k32(a[i], s[t].part[j], acc[r][t]);
    }
}

typedef unsigned int uintx2_t __attribute__((ext_vector_type(2)));

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
    // the one of two that is not 0
    static __device__ __forceinline__ four either(four a, four b) {
        return __builtin_bit_cast(four, __builtin_bit_cast(uintx2_t, a) | __builtin_bit_cast(uintx2_t, b));
    }
    static __device__ __forceinline__ void store2(rsrc_t r, uint32_t off, float x, float y) {   // RNE
        __builtin_amdgcn_raw_buffer_store_b32(
            __builtin_bit_cast(int, __builtin_convertvector((floatx2{x, y}), bf16x2)), r, (int)off, 0, 0);
    }
};
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
    static __device__ __forceinline__ four either(four a, four b) {
        typedef unsigned int uintx4_t __attribute__((ext_vector_type(4)));
        return __builtin_bit_cast(four, __builtin_bit_cast(uintx4_t, a) | __builtin_bit_cast(uintx4_t, b));
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

typedef int intx4 __attribute__((ext_vector_type(4)));

// G as a whole number of 2^-22, down to -511
constexpr int kOne = 1 << 22;
constexpr int kLevelBits = 28;
constexpr int kDecay = 1 << kLevelBits;   // |G| of 64: up to it e^{-G} is formed
constexpr int kNothing = 90 * kOne;       // e^ of minus which is 0 in fp32
// e^G, and e^{-G}: the exponent in two parts, the first exact in fp32
__device__ __forceinline__ floatx2 exp_both(int G) {
    return exp_both_f32((float)(G >> 8) * 0x1p-14f, (float)(G & 255) * 0x1p-22f);
}
__device__ __forceinline__ float exp_whole(int G) { return exp_both(G)[0]; }

// log alpha^T of 16 channels as operands: multiples of 2^-14, of which sums
// down to -320 are exact in fp32, and the rests of at most 2^-15 (their sums
// are off by 2^-33); a fp32 value takes two bf16 for each (17 bits hold the
// first where log alpha >= -5), a bf16 value one
template <typename T, int NT>
struct Decays {
    static constexpr int kParts = sizeof(T) == 4 ? 2 : 1, kPairs = (NT + 1) / 2;
    bf16x8 whole[kParts][kPairs], rest[kParts][kPairs];   // of nodes 32 J + 4 g + 0..3, 32 J + 16 + 4 g + 0..3

    template <typename V>
    __device__ __forceinline__ void split(const V (&a)[NT]) {
#pragma unroll
        for (int J = 0; J < kPairs; ++J) {
            floatx4 w[2], r[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                floatx4 x = 2 * J + h < NT ? widen(a[2 * J + h < NT ? 2 * J + h : 0]) : zero4();
                // (the bounds are far outside the contract; past the greatest bf16 the parts would be infinite)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = __builtin_amdgcn_fmed3f(x[e], -120.f, 120.f);
                w[h] = (x + kGrid) - kGrid;
                r[h] = x - w[h];
            }
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                const bf16x4 w0 = take4(w[0]), w1 = take4(w[1]);
                whole[p][J] = join(w0, w1);
            }
            r[0] += w[0];   // (0 within the bound)
            r[1] += w[1];
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                const bf16x4 r0 = take4(r[0]), r1 = take4(r[1]);
                rest[p][J] = join(r0, r1);
            }
        }
    }
    // G^T of 16 nodes (columns) and the 16 channels: times the ancestor bits
    // of node l16
    template <typename M>
    __device__ __forceinline__ intx4 gather(M m, int I, int g) const {
        floatx4 x = zero4(), r = zero4();
#pragma unroll
        for (int J = 0; J < kPairs; ++J) {
            if (2 * J > I) break;
            const bool two = 2 * J + 1 < NT;
            const bf16x4 b0 = bits4((uint32_t)(m >> (32 * J + 4 * g)));
            const bf16x4 b1 = bits4(two ? (uint32_t)(m >> (two ? 32 * J + 16 + 4 * g : 0)) : 0u);
            const bf16x8 b = join(b0, b1);
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                x = mma_bf16_k32(whole[p][J], b, x);
                r = mma_bf16_k32(rest[p][J], b, r);
            }
        }
        intx4 G;
#pragma unroll
        for (int e = 0; e < 4; ++e)   // (the bounds are met outside the contract of log alpha only)
            G[e] = (int)(__builtin_amdgcn_fmed3f(x[e], -510.f, 510.f) * kOne) +
                   (int)__builtin_rintf(__builtin_amdgcn_fmed3f(r[e], -1.f, 1.f) * kOne);
        return G;
    }
};

__device__ __forceinline__ float finite_or_0(float x) { return x - x == 0.f ? x : 0.f; }
// f(0), ..., f(N - 1) with the index a constant expression
template <typename F, int... I>
__device__ __forceinline__ void each(std::integer_sequence<int, I...>, F&& f) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
    each(std::make_integer_sequence<int, N>{}, f);
}

// A (sequence, head)'s state columns c0, c0 + 1, rows 32 kb + 4 g + 0..3 and
// 32 kb + 16 + 4 g + 0..3: read once, streamed past the caches
__device__ __forceinline__ void load_state(const float* S, floatx2 (&st)[4][8], int g, int c0) {
    const rsrc_t sr = make_rsrc_u32(S, kHeadDim * kHeadDim * 4);
    const int at = (4 * g * kHeadDim + c0) * 4;
#pragma unroll
    for (int kb = 0; kb < 4; ++kb)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            st[kb][e] = __builtin_bit_cast(
                floatx2, __builtin_amdgcn_raw_buffer_load_b64(
                             sr, at + (e & 3) * kHeadDim * 4, (32 * kb + 16 * (e >> 2)) * kHeadDim * 4, 2));
}

// Ancestor masks, lane = node, by doubling: a lane joins the mask of the node
// it points at, then points where that node points.
template <typename Mask>
__device__ __forceinline__ Mask ancestors(int par, int lane, int nodes) {
    Mask mask = lane < nodes ? (Mask)1 << (lane & (8 * (int)sizeof(Mask) - 1)) : 0;
    while (__ballot(par >= 0)) {
        const Mask pm = __shfl(mask, par < 0 ? lane : par, 64);
        const int pp = __shfl(par, par < 0 ? lane : par, 64);
        if (par >= 0) {
            mask |= pm;
            par = pp;
        }
    }
    return mask;
}

// The Gram tiles (I, J <= I) of both matrices, in the order in which they
// are formed: diagonal tiles of k k first (wavefront I sums and inverts that
// of block I), then k k, then q k.
template <int NT>
struct Tiles {
    static constexpr int kHalf = NT * (NT + 1) / 2, kAll = 2 * kHalf;
    static constexpr int kRound = kAll < 8 ? kAll : 8;   // summed at a time
    static constexpr bool q(int t) { return t >= kHalf; }
    static constexpr int row(int t) {
        if (t < NT) return t;
        int i = q(t) ? 0 : 1, left = q(t) ? t - kHalf : t - NT;
        for (; left >= (q(t) ? i + 1 : i); ++i) left -= q(t) ? i + 1 : i;
        return i;
    }
    static constexpr int col(int t) {
        if (t < NT) return t;
        int i = q(t) ? 0 : 1, left = q(t) ? t - kHalf : t - NT;
        for (; left >= (q(t) ? i + 1 : i); ++i) left -= q(t) ? i + 1 : i;
        return left;
    }
    // both for every tile, 2 bits each, to look up by a tile that is not a constant
    static constexpr uint64_t packed(bool rows) {
        uint64_t p = 0;
        for (int t = 0; t < kAll; ++t) p |= (uint64_t)(rows ? row(t) : col(t)) << (2 * t);
        return p;
    }
    // place of a finished tile
    static constexpr __host__ __device__ int place(bool q, int I, int J) {
        return (q ? kHalf : 0) + I * (I + 1) / 2 + J;
    }
};

// greatest x of a row of 16 lanes, in all of them (rotations by 8, 4, 2, 1)
template <int kBy>
__device__ __forceinline__ int row_turned(int x) {
    return __builtin_amdgcn_update_dpp(0, x, 0x120 + kBy, 0xf, 0xf, false);
}
__device__ __forceinline__ int row_max(int x) {
    x = max(x, row_turned<8>(x));
    x = max(x, row_turned<4>(x));
    x = max(x, row_turned<2>(x));
    return max(x, row_turned<1>(x));
}

// Rows of the state product: fp32 up to 16 nodes, where fp32 MFMA hides behind
// the states' read (256 x 96 bf16 states of 16 nodes: 406 us, in three bf16
// 460); beyond, for bf16 inputs, three bf16, six products of them in less than
// half the time of one in fp32 (64 x 96, 64 nodes: 365 us against 418 then).
template <typename T, int NT>
using RowType = typename std::conditional<NT == 1, float, T>::type;

// LDS of a workgroup for up to 16 NT nodes
template <typename T, int NT>
struct TreeLds {
    using R = RowType<T, NT>;
    static constexpr int kN = 16 * NT;
    static constexpr int kRowsB = kN * Rows<R>::kBytes;       // an operand array
    static constexpr bool kTurns = NT > (sizeof(R) == 2 ? 1 : 2);   // k's and q's rows in the same place
    static constexpr int kPartB = Tiles<NT>::kRound * 4 * 1024;
    static constexpr int kXk = 0, kXq = kTurns ? 0 : kRowsB;
    static constexpr int kRowsEnd = (kTurns ? 1 : 2) * kRowsB;
    static constexpr int kPart = 0;                           // partial tiles in the place of the rows
    static constexpr int kGram = kRowsEnd > kPartB ? kRowsEnd : kPartB;
    static constexpr int kBeta = kGram + Tiles<NT>::kAll * 1024;
    static constexpr int kAnc = kBeta + kN * 4;               // (8 bytes a node)
    static constexpr int kBad = kAnc + kN * 8;                // per wavefront: nodes with non-finite inputs
    static constexpr int kBytes = kBad + 4 * 8;
};

// One sequence of n <= 16 NT nodes and one head.
template <typename T, int NT>
__device__ __forceinline__ void tree_decode(const TreeDecodeArgs& a, unsigned char* lds, int64_t b, int h, int n) {
    using L = TreeLds<T, NT>;
    using E = Elems<T>;
    using R = typename L::R;
    using TT = Tiles<NT>;
    using Mask = typename std::conditional<NT <= 2, uint32_t, uint64_t>::type;   // a bit per node
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int H = a.H, N = a.N;
    constexpr uint32_t es = sizeof(T);
    const uint32_t row_b = (uint32_t)H * kHeadDim * es;       // from node to node (64 rows: < 2^32 bytes)
    const size_t base = ((size_t)b * N * H + h) * kHeadDim;   // node 0's row
    const uint32_t rows_b = (uint32_t)(n - 1) * row_b + kHeadDim * es;
    auto rows = [&](const void* p) { return make_rsrc_u32(static_cast<const T*>(p) + base, rows_b); };
    const rsrc_t kr_ = rows(a.k), qr_ = rows(a.q), vr_ = rows(a.v), lr_ = rows(a.log_alpha), or_ = rows(a.o);
    const int c0 = 32 * w + 2 * l16;                          // this lane's first value column

    const Rows<R> Xk(lds + L::kXk, L::kN), Xq(lds + L::kXq, L::kN);
    floatx4* part = reinterpret_cast<floatx4*>(lds + L::kPart);   // [wavefront][tile of the round][lane]
    floatx4* gram = reinterpret_cast<floatx4*>(lds + L::kGram);   // [tile][lane]
    float* sbeta = reinterpret_cast<float*>(lds + L::kBeta);
    Mask* anc = reinterpret_cast<Mask*>(lds + L::kAnc);
    Mask* bad = reinterpret_cast<Mask*>(lds + L::kBad);

    // ---- everything this workgroup reads, in the order it is needed ---------
    const int par = lane < n ? tree_parent(a.parent, b, N, lane) : -1;
    typename E::four lar[2][NT], kr[NT][2], qr[NT][2];
    const uint32_t at_g = 4 * g * row_b;
    const uint32_t at_kq = l16 * row_b + (32 * w + 4 * g) * es;
    auto load_rows = [&](typename E::four (&x)[NT][2], rsrc_t r) {
#pragma unroll
        for (int I = 0; I < NT; ++I)
#pragma unroll
            for (int t = 0; t < 2; ++t) x[I][t] = E::load4(r, at_kq + 16 * I * row_b + 16 * t * es);
    };
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int J = 0; J < NT; ++J)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                lar[t][J][e] = E::load1(lr_, at_g + (32 * w + l16) * es + (16 * J + e) * row_b + 16 * t * es);
    load_rows(kr, kr_);
    load_rows(qr, qr_);
    float bt = to_f32(E::load1(make_rsrc_u32(static_cast<const T*>(a.beta) + (size_t)b * N * H + h,
                                             ((uint32_t)(n - 1) * H + 1) * es),
                               (uint32_t)lane * H * es));
    typename E::two vv[NT][4];
    auto load_v = [&]() {
#pragma unroll
        for (int I = 0; I < NT; ++I)
#pragma unroll
            for (int e = 0; e < 4; ++e) vv[I][e] = E::load2(vr_, at_g + c0 * es + (16 * I + e) * row_b);
    };
    floatx2 st[4][8];
    load_state(a.S + ((size_t)b * H + h) * (kHeadDim * kHeadDim), st, g, c0);
    __builtin_amdgcn_sched_barrier(0);

    const Mask mask = ancestors<Mask>(par, lane, L::kN);

    // ---- G^T, scaled rows: this wavefront's 32 channels ----------------------
    Mask bad_node = (Mask)__ballot(!(bt - bt == 0.f));   // non-finite beta, log alpha, k
    bt = finite_or_0(bt);
    if (w == 0 && lane < L::kN) {
        anc[lane] = mask;
        sbeta[lane] = bt;
    }
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
    if (lane == 0) bad[w] = bad_node;
    intx4 GT[NT][2];
    int least = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        Decays<T, NT> d;
        d.split(lar[t]);
#pragma unroll
        for (int I = 0; I < NT; ++I) {
            GT[I][t] = d.gather(__shfl(mask, 16 * I + l16, 64), I, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) least = min(least, GT[I][t][e]);
        }
    }
    const bool deep = __any(least < -kDecay);   // (of this wavefront's channels)
    floatx4 xk[NT][2], xq[NT][2], y[NT][2];
#pragma unroll
    for (int I = 0; I < NT; ++I)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const floatx4 kx = widen(kr[I][t]), qx = widen(qr[I][t]);
            floatx4 ex, over;
            if (!deep) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const floatx2 both = exp_both(GT[I][t][e]);
                    ex[e] = both[0];
                    over[e] = both[1];
                }
                xk[I][t] = kx * ex;
                xq[I][t] = qx * ex;
            } else {   // (scaled once the Gram tiles are formed)
                xk[I][t] = kx;
                xq[I][t] = qx;
            }
            y[I][t] = deep ? __builtin_bit_cast(floatx4, GT[I][t]) : kx * over;
            // (one tile's conversions at a time: the registers are full)
            __builtin_amdgcn_sched_barrier(0);
        }
    auto put_rows = [&](const Rows<R>& X, const floatx4 (&x)[NT][2]) {
#pragma unroll
        for (int I = 0; I < NT; ++I)
#pragma unroll
            for (int t = 0; t < 2; ++t) X.put(16 * I + l16, 32 * w + 16 * t + 4 * g, x[I][t]);
    };

    // ---- Gram tiles, transposed: ancestors x nodes --------------------------
    each<(TT::kAll + TT::kRound - 1) / TT::kRound>([&](auto round) {
        constexpr int t0 = round() * TT::kRound;
        constexpr int count = TT::kAll - t0 < TT::kRound ? TT::kAll - t0 : TT::kRound;
        if (t0 > 0) __syncthreads();   // (the round before has been summed)
        if (!deep) {
            each<count>([&](auto u) {
                constexpr int t = t0 + u();
                constexpr int I = TT::row(t), J = TT::col(t);
                const floatx4(&x)[2] = TT::q(t) ? xq[I] : xk[I];
                part[(w * TT::kRound + u()) * 64 + lane] = mma(y[J][0], y[J][1], x[0], x[1], zero4());
            });
        } else {
            // level by level down from the tile's greatest G_j: those of 64 at a time, referred to the
            // greatest that they may have
            each<count>([&](auto u) {
                constexpr int t = t0 + u();
                constexpr int I = TT::row(t), J = TT::col(t);
                floatx4 acc = zero4();
#pragma unroll
                for (int c = 0; c < 2; ++c) {   // (16 channels at a time: the registers are full)
                    __builtin_amdgcn_sched_barrier(0);
                    const floatx4 xi = (TT::q(t) ? xq : xk)[I][c], kj = xk[J][c];
                    const intx4 Gi = __builtin_bit_cast(intx4, y[I][c]), Gj = __builtin_bit_cast(intx4, y[J][c]);
                    intx4 below;   // of G_j under the tile's greatest, per channel
                    intx4 under;   // of G_i
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int top = row_max(Gj[e]);
                        below[e] = top - Gj[e];
                        under[e] = top - Gi[e];
                    }
#pragma unroll 1
                    for (int m = 0; m < kLevels; ++m) {
                        const int down = kDecay * m;
                        // (formed from these each time, not kept over the loop)
                        if (NT == 1) asm volatile("" : "+v"(below), "+v"(under));
                        bool some = false, felt = false, further = false;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            some |= (below[e] >> kLevelBits) == m;
                            further |= (below[e] >> kLevelBits) > m;
                            felt |= under[e] - down < kNothing;
                        }
                        const bool more = __any(further);
                        if (!__any(some) || !__any(felt)) {
                            if (!more) break;
                            continue;
                        }
                        floatx4 ks, z;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            ks[e] = (below[e] >> kLevelBits) == m ? kj[e] * exp_whole(below[e] - down) : 0.f;
                        __builtin_amdgcn_sched_barrier(0);
                        // (a descendant's G is no greater than G_j but for its rounding: only masked entries
                        // meet the bound)
#pragma unroll
                        for (int e = 0; e < 4; ++e) z[e] = xi[e] * exp_whole(min(down - under[e], kOne));
                        acc = mma_f32_k16(ks, z, acc);
                        if (!more) break;
                    }
                }
                part[(w * TT::kRound + u()) * 64 + lane] = acc;
            });
        }
        __syncthreads();
        // tile t is summed by wavefront t % 4 and masked by ancestry, rows of k k scaled by beta
#pragma unroll
        for (int j = 0; j < (count + 3) / 4; ++j) {
            const int u = 4 * j + ((w - t0) & 3), t = t0 + u;
            if (u >= count) break;
            constexpr uint64_t kRowOf = TT::packed(true), kColOf = TT::packed(false);
            const int I = (kRowOf >> (2 * t)) & 3, J = (kColOf >> (2 * t)) & 3;
            const bool isq = t >= TT::kHalf;
            const floatx4* p = part + u * 64 + lane;
            constexpr int kW = TT::kRound * 64;   // from wavefront to wavefront
            floatx4 x = (p[0] + p[kW]) + (p[2 * kW] + p[3 * kW]);
            const Mask m = __shfl(mask, 16 * I + l16, 64) >> (16 * J + 4 * g);   // node i = 16 I + l16
            const float scale = isq ? 1.f : __shfl(bt, 16 * I + l16, 64);
            const int diag = !isq && I == J ? l16 : 64;   // (no node is its own ancestor in k k)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = ((m >> e) & 1) && 4 * g + e != diag ? scale * x[e] : 0.f;
            gram[TT::place(isq, I, J) * 64 + lane] = x;
        }
    });

    if (deep) {
#pragma unroll
        for (int I = 0; I < NT; ++I)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                floatx4 ex;
#pragma unroll
                for (int e = 0; e < 4; ++e) ex[e] = exp_whole(__builtin_bit_cast(intx4, y[I][t])[e]);
                xk[I][t] *= ex;
                xq[I][t] *= ex;
                __builtin_amdgcn_sched_barrier(0);
            }
    }

    // ---- held and read: X S, this wavefront's columns -----------------------
    floatx4 held[NT][2], read[NT][2];
#pragma unroll
    for (int r = 0; r < NT; ++r) held[r][0] = held[r][1] = read[r][0] = read[r][1] = zero4();
    __syncthreads();   // the last round has been summed
    put_rows(Xk, xk);
    if (!L::kTurns) put_rows(Xq, xq);
    if (w < NT) invert(reinterpret_cast<float*>(gram + TT::place(false, w, w) * 64), l16, g);
    __syncthreads();
    load_v();   // (registers are free only now)
    StateOp<R> so[4][2];
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
#pragma unroll
        for (int t = 0; t < 2; ++t) so[kb][t] = StateOp<R>::of(st[kb], t);
        state_product<NT>(Xk, 32 * kb, so[kb], held, l16, g);
        if (!L::kTurns) state_product<NT>(Xq, 32 * kb, so[kb], read, l16, g);
    }
    if (L::kTurns) {
        __syncthreads();
        put_rows(Xq, xq);
        __syncthreads();
#pragma unroll
        for (int kb = 0; kb < 4; ++kb) state_product<NT>(Xq, 32 * kb, so[kb], read, l16, g);
    }

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
    uint32_t at_o = at_g + c0 * es;
    asm volatile("" : "+v"(at_o));   // (store offsets are formed here, not kept since v's loads)
    floatx4 uo[NT][2];   // pseudo-values as operands
#pragma unroll
    for (int I = 0; I < NT; ++I) {
        const floatx4 bt4 = *reinterpret_cast<const floatx4*>(sbeta + 16 * I + 4 * g);
        const floatx4 ia = gram[TT::place(false, I, I) * 64 + lane];
        floatx4 prev[2] = {zero4(), zero4()};
        auto tile = [&](bool q, int J) { return gram[TT::place(q, I, J) * 64 + lane]; };
#pragma unroll
        for (int J = 0; J + 1 < I; J += 2) {
            const floatx4 a0 = tile(false, J), a1 = tile(false, J + 1);
#pragma unroll
            for (int t = 0; t < 2; ++t) prev[t] = mma(a0, a1, uo[J][t], uo[J + 1][t], prev[t]);
        }
        if (I & 1) {
            const floatx4 a0 = tile(false, I - 1);
#pragma unroll
            for (int t = 0; t < 2; ++t) prev[t] = mma_f32_k16(a0, uo[I - 1][t], prev[t]);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            floatx4 rhs;
#pragma unroll
            for (int e = 0; e < 4; ++e) rhs[e] = bt4[e] * ((float)vv[I][e][t] - held[I][t][e]);
            if (I > 0) rhs -= prev[t];
            uo[I][t] = mma_f32_k16(ia, rhs, zero4());
        }
        floatx4 out[2] = {zero4(), zero4()};
#pragma unroll
        for (int J = 0; J < I; J += 2) {
            const floatx4 a0 = tile(true, J), a1 = tile(true, J + 1);
#pragma unroll
            for (int t = 0; t < 2; ++t) out[t] = mma(a0, a1, uo[J][t], uo[J + 1][t], out[t]);
        }
        if (!(I & 1)) {
            const floatx4 a0 = tile(true, I);
#pragma unroll
            for (int t = 0; t < 2; ++t) out[t] = mma_f32_k16(a0, uo[I][t], out[t]);
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
            E::store2(or_, at_o + (16 * I + e) * row_b, out[0][e], out[1][e]);
    }
}

// (workgroups per CU: as many as fit without spills; 23 x 31 fp32 states of
// 21 nodes take 29.7 us at two, 26.3 at three.)  A sequence with fewer nodes
// than the batch's N allows runs the code of one tile (N <= 32) or two where
// that holds it; the code of a size has no branches on the number of tiles
// (64 x 96 bf16 states of 64 nodes, operands in two bf16 parts: 280 us with
// them, 266 without).
constexpr int smaller(int NT) { return NT > 2 ? 2 : 1; }
template <typename T, int NT>
constexpr int launch_lds() {
    constexpr int less = TreeLds<T, smaller(NT)>::kBytes, own = TreeLds<T, NT>::kBytes;
    return less > own ? less : own;
}
template <typename T, int NT>
__global__ __launch_bounds__(256, NT == 1 ? 4 : (NT == 2 ? 3 : 2))
void tree_decode_kernel(TreeDecodeArgs a) {
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const int64_t b = blockIdx.x / (unsigned)a.H;
    const int h = blockIdx.x % (unsigned)a.H;
    const int n = __builtin_amdgcn_readfirstlane(tree_count(a.n_node, b, a.N));
    if (n == 0) return;
    constexpr int kLess = smaller(NT);
    if (kLess < NT && n <= 16 * kLess) tree_decode<T, kLess>(a, lds, b, h, n);
    else tree_decode<T, NT>(a, lds, b, h, n);
}

// Up to 8 nodes: k's rows and q's share one tile of 16, rows 0..7 and 8..15
// (lane l16: node l16 % 8).  One product with the state gives what is held
// (accumulator rows 0..7) and what is read (8..15), one Gram tile the
// couplings of both, and the outputs accumulate onto the read rows: half the
// operands, exponentials and matrix instructions of the general kernel.
constexpr int kSmall = 8;

template <typename T>
struct __attribute__((aligned(16))) SmallLds {
    unsigned char rows[16 * Rows<float>::kBytes];
    floatx4 part[4][64];      // the wavefronts' parts of the Gram tile
    floatx4 gram[64];         // rows 0..7 strictly lower k k, 8..15 lower q k
    float inv[256];           // (I + L)^{-1}
    float beta[16];
    uint32_t anc[kSmall];
    uint32_t bad[4];
};

template <typename T>
__global__ __launch_bounds__(256, 4) void tree_decode_small_kernel(TreeDecodeArgs a) {
    using E = Elems<T>;
    __shared__ SmallLds<T> lds;
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, g = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int H = a.H, N = a.N;
    const int64_t b = blockIdx.x / (unsigned)H;
    const int h = blockIdx.x % (unsigned)H;
    const int n = __builtin_amdgcn_readfirstlane(tree_count(a.n_node, b, N));
    if (n == 0) return;
    constexpr uint32_t es = sizeof(T);
    constexpr uint32_t kOut = 0xffffff00u;                    // an offset past every resource
    const uint32_t row_b = (uint32_t)H * kHeadDim * es;       // from node to node
    const size_t base = ((size_t)b * N * H + h) * kHeadDim;   // node 0's row
    const uint32_t rows_b = (uint32_t)(n - 1) * row_b + kHeadDim * es;
    auto rows = [&](const void* p) { return make_rsrc_u32(static_cast<const T*>(p) + base, rows_b); };
    const int c0 = 32 * w + 2 * l16;                          // this lane's first value column
    const Rows<float> X(lds.rows, 16);
    const bool isq = l16 >= kSmall;
    const int i = l16 & (kSmall - 1);

    // ---- everything this workgroup reads -------------------------------------
    const int par = lane < n ? tree_parent(a.parent, b, N, lane) : -1;
    typename E::four lar[2][1], x[2];
    {
        const rsrc_t lr = rows(a.log_alpha), kr = rows(a.k), qr = rows(a.q);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                lar[t][0][e] = E::load1(lr, (4 * g + e) * row_b + (32 * w + 16 * t + l16) * es);
        // lanes of k and of q read 0 from the other's tensor
        const uint32_t off = i * row_b + (32 * w + 4 * g) * es;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const typename E::four kx = E::load4(kr, (isq ? kOut : off) + 16 * t * es);
            const typename E::four qx = E::load4(qr, (isq ? off : kOut) + 16 * t * es);
            x[t] = E::either(kx, qx);
        }
    }
    float bt = to_f32(E::load1(make_rsrc_u32(static_cast<const T*>(a.beta) + (size_t)b * N * H + h,
                                             ((uint32_t)(n - 1) * H + 1) * es),
                               (uint32_t)lane * H * es));
    typename E::two vv[4];
    {
        const rsrc_t vr = rows(a.v);
#pragma unroll
        for (int e = 0; e < 4; ++e) vv[e] = E::load2(vr, (4 * g + e) * row_b + c0 * es);
    }
    floatx2 st[4][8];
    load_state(a.S + ((size_t)b * H + h) * (kHeadDim * kHeadDim), st, g, c0);
    __builtin_amdgcn_sched_barrier(0);

    const uint32_t mask = ancestors<uint32_t>(par, lane, kSmall);
    uint32_t bad_node = (uint32_t)__ballot(!(bt - bt == 0.f));   // non-finite beta, log alpha, k
    bt = finite_or_0(bt);
    if (w == 0 && lane < 16) {
        lds.beta[lane] = bt;   // (0 past the nodes)
        if (lane < kSmall) lds.anc[lane] = mask;
    }
    {
        float s = 0.f;
#pragma unroll
        for (int t = 0; t < 2; ++t) s = probe4(probe4(s, lar[t][0]), x[t]);
        if (__any(s != 0.f)) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float z = (float)lar[t][0][e];   // node 4 g + e
                    uint64_t off = __ballot(!(z - z == 0.f));
#pragma unroll
                    for (int gg = 0; gg < 2; ++gg)
                        if ((off >> (16 * gg)) & 0xffff) bad_node |= 1u << (4 * gg + e);
                    lar[t][0][e] = (T)finite_or_0(z);
                    z = (float)x[t][e];              // k of node l16; q's rows keep theirs to themselves
                    off = __ballot(!isq && !(z - z == 0.f));
                    off |= off >> 32;
                    off |= off >> 16;
                    bad_node |= (uint32_t)(off & 0xff);
                    if (!isq) x[t][e] = (T)finite_or_0(z);
                }
        }
    }
    if (lane == 0) lds.bad[w] = bad_node;

    // ---- G^T, scaled rows, this wavefront's part of the Gram tile -------------
    const uint32_t m = __shfl(mask, i, 64);
    floatx4 xo[2], y[2];
    // (8 levels at the decay bound: |G| <= 40 where the inputs keep their contract)
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        Decays<T, 1> d;
        d.split(lar[t]);
        const intx4 G = d.gather(m, 0, g);
        const floatx4 z = widen(x[t]);
        floatx4 ex, over;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const floatx2 both = exp_both(G[e]);
            ex[e] = both[0];
            over[e] = both[1];
        }
        xo[t] = z * ex;
        y[t] = z * over;
        X.put(l16, 32 * w + 16 * t + 4 * g, xo[t]);
    }
    lds.part[w][lane] = mma(y[0], y[1], xo[0], xo[1], zero4());
    __syncthreads();

    if (w == 0) {   // summed, masked, and the solve's inverse
        const floatx4* p = &lds.part[0][lane];
        floatx4 z = (p[0] + p[64]) + (p[128] + p[192]);
        const float scale = isq ? 1.f : __shfl(bt, i, 64);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = 4 * g + e;
            const bool on = ((m >> j) & 1) && (isq || j != i);
            z[e] = on ? scale * z[e] : 0.f;
        }
        lds.gram[lane] = z;
        *reinterpret_cast<floatx4*>(lds.inv + 4 * lane) = isq ? zero4() : z;
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
        invert<kSmall>(lds.inv, l16, g);
    }

    // ---- held and read, this wavefront's columns ------------------------------
    floatx4 acc[1][2] = {{zero4(), zero4()}};
#pragma unroll
    for (int kb = 0; kb < 4; ++kb) {
        const StateOp<float> so[2] = {StateOp<float>::of(st[kb], 0), StateOp<float>::of(st[kb], 1)};
        state_product<1>(X, 32 * kb, so, acc, l16, g);
    }
    __syncthreads();

    // ---- pseudo-values and outputs --------------------------------------------
    bad_node = lds.bad[0] | lds.bad[1] | lds.bad[2] | lds.bad[3];
    uint32_t bad_col[2] = {bad_node, bad_node};
    {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) s = probe(s, vv[e]);
        if (__any(s != 0.f)) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t z = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float u = (float)vv[e][t];
                    vv[e][t] = (T)finite_or_0(u);
                    z |= (u - u == 0.f ? 0u : 1u) << (4 * g + e);
                }
                z |= __shfl_xor(z, 16, 64);
                z |= __shfl_xor(z, 32, 64);
                bad_col[t] |= z;
            }
        }
    }
    const floatx4 bt4 = *reinterpret_cast<const floatx4*>(lds.beta + 4 * g);
    const floatx4 ia = *reinterpret_cast<const floatx4*>(lds.inv + 4 * lane);
    const floatx4 gm = lds.gram[lane];
    floatx4 out[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        floatx4 rhs;   // (rows 8..15: beta is 0)
#pragma unroll
        for (int e = 0; e < 4; ++e) rhs[e] = g < 2 ? bt4[e] * ((float)vv[e][t] - acc[0][t][e]) : 0.f;
        out[t] = mma_f32_k16(gm, mma_f32_k16(ia, rhs, zero4()), acc[0][t]);
    }
    // rows 8..15 are the outputs of nodes 0..7
    if (__any((bad_col[0] | bad_col[1]) != 0)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t z = lds.anc[(4 * g + e) & (kSmall - 1)];
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (z & bad_col[t]) out[t][e] = __builtin_nanf("");
        }
    }
    const rsrc_t orr = rows(a.o);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        E::store2(orr, g < 2 ? kOut : (4 * g + e - kSmall) * row_b + c0 * es, out[0][e], out[1][e]);
}

template <typename T, int NT>
hipError_t launch_nt(const TreeDecodeArgs& a, hipStream_t stream) {
    static std::atomic<uint64_t> done{0};
    constexpr int bytes = launch_lds<T, NT>();
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
    if (a.N <= kSmall) {
        tree_decode_small_kernel<T><<<dim3((unsigned)((int64_t)a.B * a.H)), dim3(256), 0, stream>>>(a);
        return hipGetLastError();
    }
    if (a.N <= 16) return launch_nt<T, 1>(a, stream);
    if (a.N <= 32) return launch_nt<T, 2>(a, stream);
    if (a.N <= 48) return launch_nt<T, 3>(a, stream);
    return launch_nt<T, 4>(a, stream);
}

}  // namespace

hipError_t launch_tree_decode(const TreeDecodeArgs& a, int dtype, hipStream_t stream) {
    return dtype == 0 ? launch_t<float>(a, stream) : launch_t<bf16>(a, stream);
}

}  // namespace kda
