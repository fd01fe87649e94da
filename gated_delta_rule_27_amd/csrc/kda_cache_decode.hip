// kda_cache_decode.hip -- one token per sequence from the 8-bit cache: the
// output from one read of the codes and the window, the token's update
// appended to the window.
//
// One wavefront per head.  The two reads of the state, S^T k for the update
// and S^T q for the output, are two vectors against 128 x 128 codes, taken as
// whole numbers: each vector (times decay and scale, per key channel) becomes
// a 62-bit fixed-point number under a power of two of its own, split into two
// halves of four signed 8-bit digits, and the sixteen digits are the rows of the
// 8-bit matrix instruction, whose other operand is the codes as they lie in memory.
// So no code is converted or multiplied by the vector unit, and the sums are exact;
// what is rounded is each half's result, to 24 bits.  Entries of less than 2^-38 of
// their vector's largest have bits beyond the 62 and a second round takes them (rarely:
// the products alone are done again), so that an output that the largest channels'
// codes leave alone has all its bits, as fp32 products would give it.
// Bounded by memory: 256 x 96 states with windows of 4 tokens take 105 us for 0.53 GB,
// 5.1 TB/s (reads alone, laid out as the codes are, reach 6.1); a step of fp32 states
// moves 3.2 GB.  The window's three new rows, 19 MB in lines of their own, cost 13 us of
// it.  One sequence: 5.6 us, a launch and the chain of loads, digits and products.
// 23 x 31 states with 6 fp32 tokens on average: 11.0 us, the window's tokens one after
// the other in a wavefront.
#include "kda.h"
#include "kda_cache.h"
#include "kda_cache_device.h"

namespace kda {

namespace {

constexpr int kD = kHeadDim;
constexpr int kDigitLd = 144;   // bytes of a digit row in LDS (16 more: other banks)

typedef int intx4 __attribute__((ext_vector_type(4)));

// two elements of a row
template <typename T>
struct Pair;
template <>
struct Pair<float> {
    typedef floatx2 type;
};
template <>
struct Pair<bf16> {
    typedef bf16 type __attribute__((ext_vector_type(2)));
};
template <typename T>
__device__ __forceinline__ floatx2 widen(typename Pair<T>::type x) {
    return floatx2{(float)x[0], (float)x[1]};
}

template <int kCtrl>
__device__ __forceinline__ uint32_t max_with(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kCtrl, 0xf, 0xf, true));
}
// largest of the wavefront's magnitudes' bits (a NaN is larger than anything)
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
    x = max_with<0x128>(x);
    x = max_with<0x124>(x);
    x = max_with<0x122>(x);
    x = max_with<0x121>(x);
    const int a = __builtin_amdgcn_readlane((int)x, 0), b = __builtin_amdgcn_readlane((int)x, 16);
    const int c = __builtin_amdgcn_readlane((int)x, 32), d = __builtin_amdgcn_readlane((int)x, 48);
    return max(max((uint32_t)a, (uint32_t)b), max((uint32_t)c, (uint32_t)d));
}
__device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint32_t, x); }

template <int kCtrl>
__device__ __forceinline__ float add_with(float x) {
    return x + __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), kCtrl, 0xf, 0xf, true));
}
// sum over the wavefront, in every lane
__device__ __forceinline__ float sum64(float x) {
    x = add_with<0x128>(x);
    x = add_with<0x124>(x);
    x = add_with<0x122>(x);
    x = add_with<0x121>(x);
    const float a = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 0));
    const float b = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 16));
    const float c = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 32));
    const float d = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 48));
    return (a + b) + (c + d);
}

struct WaveLds {
    uint8_t digit[16 * kDigitLd];  // four rows of digits, lowest first, of the key's upper half, its lower, the query's two
    float read[4][kD];             // what they read
};

__device__ __forceinline__ void fence() { __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront"); }

// x as multiples of its vector's unit, of which its largest has 2^29 to 2^30; the exponent
// of the unit.  A vector that is not finite makes NaN of `read`, what its result is added to.
__device__ __forceinline__ int to_units(floatx2& x, floatx2& read) {
    const uint32_t top = wave_max(max(bits(x[0]) & 0x7fffffffu, bits(x[1]) & 0x7fffffffu));
    const int up = 29 + 127 - (int)(top >> 23);
    if (top >= 0x7f800000u) read = floatx2{__builtin_nanf(""), __builtin_nanf("")};
#pragma unroll
    for (int e = 0; e < 2; ++e) x[e] = top >= 0x7f800000u ? 0.f : __builtin_amdgcn_ldexpf(x[e], up);
    return -up;
}
// the whole parts of the lane's two entries, |x| <= 2^30, as digits into LDS; x
// becomes what is left, in units of 2^-31 (exact, as the difference is)
__device__ __forceinline__ void to_digits(floatx2& x, uint8_t* row0, int lane) {
    uint32_t d[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const float v = __builtin_rintf(x[e]);
        d[e] = ((uint32_t)(int)v + 0x00808080u) ^ 0x00808080u;   // signed digits of 8 bits
        x[e] = (x[e] - v) * 2147483648.f;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        *reinterpret_cast<uint16_t*>(row0 + r * kDigitLd + 2 * lane) =
            (uint16_t)__builtin_amdgcn_perm(d[1], d[0], 0x0c0c0400u + 0x0101u * r);
}

template <typename T>
__global__ __launch_bounds__(256, 4) void cache_decode_kernel(CacheDecodeArgs a) {
    __shared__ __align__(16) WaveLds all[4];
    typedef typename Pair<T>::type pair;
    constexpr int kRound = 16 / sizeof(T);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t unit = blockIdx.x * 4 + wave;
    if (unit >= (uint32_t)a.B * (uint32_t)a.H) return;
    const int n = a.win.n[unit / (uint32_t)a.H], W = a.win.W;
    if (n < 0 || n >= W) return;   // (an idle place of the batch)
    WaveLds& lds = all[wave];

    const size_t vec = (size_t)unit * kD + 2 * lane, row0 = (size_t)unit * W * kD + 2 * lane;
    auto load = [](const void* p, size_t at) { return *reinterpret_cast<const pair*>(static_cast<const T*>(p) + at); };
    // (256 x 96 states, windows of 8: 111 us with ordinary stores, 106 with streaming ones)
    auto store = [](void* p, size_t at, pair x) {
        __builtin_nontemporal_store(x, reinterpret_cast<pair*>(static_cast<T*>(p) + at));
    };

    const int l16 = lane & 15, g = lane >> 4;
    intx4 c[8][2];
    const int8_t* codes = a.codes + (size_t)unit * kD * kD + l16 * kD + 16 * g;
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int s = 0; s < 2; ++s)
            c[t][s] = __builtin_nontemporal_load(reinterpret_cast<const intx4*>(codes + 16 * t * kD + 64 * s));
    const pair k0 = load(a.k, vec), la0 = load(a.log_alpha, vec);
    const floatx2 q = widen<T>(load(a.q, vec)), k = widen<T>(k0), la = widen<T>(la0), v = widen<T>(load(a.v, vec));
    const float beta = to_f32(static_cast<const T*>(a.beta)[unit]);
    const floatx2 scale = *reinterpret_cast<const floatx2*>(a.scale + vec);

    // the window, newest first, kRound tokens at a time: what its updates add to
    // the two reads
    floatx2 by_k{0.f, 0.f}, by_q{0.f, 0.f};
    LogDecay gone[2];
    gone[0].add(la[0]);
    gone[1].add(la[1]);
#pragma unroll 1
    for (int t0 = (n - 1) / kRound * kRound; n > 0 && t0 >= 0; t0 -= kRound) {
        pair kw[kRound], lw[kRound], uw[kRound];
#pragma unroll
        for (int t = 0; t < kRound; ++t) {
            if (t0 + t < n) {
                kw[t] = load(a.win.k, row0 + (t0 + t) * kD);
                lw[t] = load(a.win.log_alpha, row0 + (t0 + t) * kD);
                uw[t] = load(a.win.u, row0 + (t0 + t) * kD);
            }
        }
#pragma unroll
        for (int t = kRound - 1; t >= 0; --t) {
            if (t0 + t < n) {
                const floatx2 kt = widen<T>(kw[t]), lt = widen<T>(lw[t]), ut = widen<T>(uw[t]);
                const float x0 = kt[0] * gone[0].decay(), x1 = kt[1] * gone[1].decay();
                by_k += sum64(x0 * k[0] + x1 * k[1]) * ut;
                by_q += sum64(x0 * q[0] + x1 * q[1]) * ut;
                gone[0].add(lt[0]);
                gone[1].add(lt[1]);
            }
        }
    }
    const floatx2 held{scale[0] * gone[0].decay(), scale[1] * gone[1].decay()};
    floatx2 xk = k * held, xq = q * held, sk{0.f, 0.f}, sq{0.f, 0.f};
    const int ek = to_units(xk, by_k), eq = to_units(xq, by_q);
    float step = 1.f;
    // (the first round on its own: 256 x 96 states 106.2 us, 107.4 by a loop around it)
    auto round = [&]() {
        to_digits(xk, lds.digit, lane);
        to_digits(xk, lds.digit + 4 * kDigitLd, lane);
        to_digits(xq, lds.digit + 8 * kDigitLd, lane);
        to_digits(xq, lds.digit + 12 * kDigitLd, lane);
        fence();
        intx4 d[2];
#pragma unroll
        for (int s = 0; s < 2; ++s)
            d[s] = *reinterpret_cast<const intx4*>(lds.digit + l16 * kDigitLd + 16 * g + 64 * s);
#pragma unroll
        for (int t = 0; t < 8; ++t) {
            intx4 x{0, 0, 0, 0};
            x = __builtin_amdgcn_mfma_i32_16x16x64_i8(d[0], c[t][0], x, 0, 0, 0);
            x = __builtin_amdgcn_mfma_i32_16x16x64_i8(d[1], c[t][1], x, 0, 0, 0);
            // lanes of group g: the four digits of half g at column l16
            const float y = __builtin_fmaf((float)(x[3] * 256 + x[2]), 65536.f, (float)(x[1] * 256 + x[0]));
            lds.read[g][16 * t + l16] = y;
        }
        fence();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            sk[e] += step * __builtin_fmaf(lds.read[1][2 * lane + e], 0x1p-31f, lds.read[0][2 * lane + e]);
            sq[e] += step * __builtin_fmaf(lds.read[3][2 * lane + e], 0x1p-31f, lds.read[2][2 * lane + e]);
        }
        fence();
        step *= 0x1p-62f;
        // (what is left loses 62 bits a round, and fp32 ends at 2^-149)
        return __ballot(xk[0] != 0.f || xk[1] != 0.f || xq[0] != 0.f || xq[1] != 0.f) != 0;
    };
    bool more = round();
#pragma unroll 1
    while (__builtin_expect(more, 0)) more = round();
    const float kq = sum64(k[0] * q[0] + k[1] * q[1]);
    pair u, o;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        u[e] = from_f32<T>(beta * (v[e] - (__builtin_amdgcn_ldexpf(sk[e], ek) + by_k[e])));
        // (the update as it is held: what the tokens to come will read)
        o[e] = from_f32<T>(__builtin_amdgcn_ldexpf(sq[e], eq) + by_q[e] + kq * to_f32((T)u[e]));
    }
    store(a.o, vec, o);
    store(a.win.k, row0 + (size_t)n * kD, k0);
    store(a.win.log_alpha, row0 + (size_t)n * kD, la0);
    store(a.win.u, row0 + (size_t)n * kD, u);
}

template <typename T>
hipError_t launch_cache_decode_t(const CacheDecodeArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)a.B * a.H + 3) / 4)), block(256);
    cache_decode_kernel<T><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_decode(const CacheDecodeArgs& a, int dtype, hipStream_t stream) {
    return dtype == 0 ? launch_cache_decode_t<float>(a, stream) : launch_cache_decode_t<bf16>(a, stream);
}

}  // namespace kda
