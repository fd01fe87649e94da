// kda_cache.hip -- fp32 states into the 8-bit cache, back, and a window's
// updates taken into the 8-bit state in place.
//
// A state S [key i][value j] is scale[i] * codes[j][i], scale[i] = max_j |S[i][j]| / 127.
// With G the sum of log alpha over a window's n tokens and G_t that up to token t, it
// is read back as S[i][j] = scale[i] e^G[i] codes[j][i] + sum_t e^(G - G_t)[i] k_t[i] u_t[j]:
// decay belongs to the key channel, as the scale does, so that it costs the codes
// nothing, and the n updates are a product of 128 x n by n x 128.
// All three move memory: a workgroup of 256 threads holds one state in registers (64
// values a thread) and passes the codes, which lie the other way round, through LDS;
// every global access is whole lines.  256 x 96 states: stored in 364 us (2.03 GB,
// 5.6 TB/s), folded with 8 bf16 tokens in 178 us (0.98 GB, 5.5 TB/s; 4 tokens 145 us,
// 6.3 TB/s); 192 x 96 loaded in 268 us (1.52 GB, 5.7 TB/s).  A large device copy
// reaches 4.7 TB/s.  One state each of 96 heads: 4.6 us to store, a launch and one trip
// through the workgroup.
#include "kda.h"
#include "kda_cache.h"
#include "kda_cache_device.h"

namespace kda {

namespace {

constexpr int kD = kHeadDim;
constexpr int kLd = 36;   // dwords of a value channel's 128 codes in LDS, with padding

typedef uint32_t uintx4 __attribute__((ext_vector_type(4)));

// In a store and a load the workgroup's four wavefronts hold a state as blocks of four rows and
// four columns a lane: block t of wavefront w, lane (half, l) covers rows
// 32 w + 8 t + 4 half + 0..3 and columns 4 l + 0..3, so that a row's loads and
// stores are whole lines and four rows' codes of a column are one dword.
struct Place {
    int l, half, wave;
    __device__ Place() : l(threadIdx.x & 31), half((threadIdx.x >> 5) & 1), wave(threadIdx.x >> 6) {}
    __device__ __forceinline__ int row(int t) const { return 32 * wave + 8 * t + 4 * half; }
};
typedef floatx4 State[4][4];   // [block][row], four columns

__device__ __forceinline__ uint32_t magnitude(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }
// largest of 16, of 32 lanes (the magnitudes' bits: a NaN is larger than anything)
template <int kCtrl>
__device__ __forceinline__ uint32_t max_with(uint32_t x) {
    return max(x, (uint32_t)__builtin_amdgcn_mov_dpp((int)x, kCtrl, 0xf, 0xf, true));
}
__device__ __forceinline__ uint32_t max16(uint32_t x) {
    x = max_with<0x128>(x);   // rotations of a row of 16 by 8, 4, 2, 1
    x = max_with<0x124>(x);
    x = max_with<0x122>(x);
    return max_with<0x121>(x);
}
__device__ __forceinline__ uint32_t max32(uint32_t x) {
    x = max16(x);
    return max(x, (uint32_t)__builtin_amdgcn_ds_swizzle((int)x, 0x401f));   // the other row
}

// the code of x, in the low byte: adding 1.5 * 2^23 to the exact product rounds to
// a whole number, ties to even, and leaves it in the low bits
__device__ __forceinline__ uint32_t code(float x, float inverse) {
    return __builtin_bit_cast(uint32_t, __builtin_fmaf(x, inverse, 12582912.f));
}
// four rows' codes of a column
__device__ __forceinline__ uint32_t codes_of(floatx4 x, floatx4 inverse) {
    const uint32_t lo = __builtin_amdgcn_perm(code(x[1], inverse[1]), code(x[0], inverse[0]), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(code(x[3], inverse[3]), code(x[2], inverse[2]), 0x04000c0cu);
    return lo | hi;
}
// four rows of a column back
__device__ __forceinline__ floatx4 values_of(uint32_t codes, floatx4 m) {
    floatx4 x;
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = (float)(int8_t)(codes >> (8 * r)) * m[r];
    return x;
}

// Scales and codes of a state out, through an LDS tile of [value][key] codes.
struct QuantiseLds {
    uint32_t tile[kD * kLd];
    uint32_t top[kD];      // largest magnitude of each row
    float inverse[kD];
};
// top -> inverse and scale; all threads, a barrier before and after
__device__ __forceinline__ void scales(QuantiseLds& lds, float* scale) {
    __syncthreads();
    if (threadIdx.x < kD) {
        const uint32_t m = lds.top[threadIdx.x];
        const float top = __builtin_bit_cast(float, m);
        const bool held = m >= 0x0d800000u;   // 2^-100
        lds.inverse[threadIdx.x] = held ? 127.f / top : 0.f;
        // (a row with a NaN or an infinity reads back as NaN)
        scale[threadIdx.x] = !held ? 0.f : m >= 0x7f800000u ? __builtin_nanf("") : top / 127.f;
    }
    __syncthreads();
}
__device__ __forceinline__ void codes_out(const QuantiseLds& lds, int8_t* codes) {
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int piece = threadIdx.x + 256 * s;   // 16 bytes: eight of a value channel
        const uintx4 x = *reinterpret_cast<const uintx4*>(lds.tile + (piece >> 3) * kLd + 4 * (piece & 7));
        __builtin_nontemporal_store(x, reinterpret_cast<uintx4*>(codes) + piece);
    }
}

// LDS of a state read back: codes, and what each key channel's codes are multiplied
// by; the window as it is in memory (rows of zeros up to a multiple of four tokens),
// and its keys as far as they are decayed after the last token.  kMost: the longest
// window of an instance.
struct ReadLds {
    uint32_t tile[kD * kLd];
    float row[kD];
};
constexpr int kWinLd = kD + 16;   // (16 elements more: other banks)
template <typename T, int kMost>
struct WindowLds {
    T raw[3][kMost][kWinLd];   // k, log alpha, u
    float wide[sizeof(T) == 4 ? 1 : kMost][kWinLd];
    // (of fp32 keys the decayed ones take the place)
    __device__ __forceinline__ float* k(int t) { return sizeof(T) == 4 ? reinterpret_cast<float*>(raw[0][t]) : wide[t]; }
};

// codes, window and scales into LDS; all threads, a barrier at the end
template <typename T, int kMost, bool kStream>
__device__ __forceinline__ void stage(ReadLds& lds, WindowLds<T, kMost>& wl, const int8_t* codes, const float* scale,
                                      const CacheWindow& w, size_t at, int n) {
    constexpr int kRow = kD * sizeof(T) / 16;                     // pieces of 16 bytes of a row
    constexpr int kPieces = (3 * kMost * kRow + 255) / 256;       // that a thread takes
    const int most = (n + 3) & ~3, i = threadIdx.x & (kD - 1);
    uintx4 x[4], y[kPieces];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const uintx4* p = reinterpret_cast<const uintx4*>(codes) + threadIdx.x + 256 * s;
        x[s] = kStream ? __builtin_nontemporal_load(p) : *p;
    }
    const float sc = scale[i];
    // (token by token, its three rows one after the other)
    auto piece = [&](int s, int& t, int& array, int& q) {
        const int p = (int)threadIdx.x + 256 * s;
        t = p / (3 * kRow);
        array = p / kRow % 3;
        q = p % kRow;
    };
#pragma unroll
    for (int s = 0; s < kPieces; ++s) {
        int t, array, q;
        piece(s, t, array, q);
        y[s] = uintx4{0, 0, 0, 0};
        if (t < n) {
            const void* p = array == 0 ? w.k : array == 1 ? w.log_alpha : w.u;
            y[s] = reinterpret_cast<const uintx4*>(p)[(at * w.W + t) * kRow + q];
        }
    }
#pragma unroll
    for (int s = 0; s < kPieces; ++s) {
        int t, array, q;
        piece(s, t, array, q);
        if (t < most) *reinterpret_cast<uintx4*>(&wl.raw[array][t][q * (16 / sizeof(T))]) = y[s];
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        const int q = threadIdx.x + 256 * s;
        *reinterpret_cast<uintx4*>(lds.tile + (q >> 3) * kLd + 4 * (q & 7)) = x[s];
    }
    __syncthreads();
    // a key channel's later tokens in one thread, its earlier ones in another
    const int half = most / 2;
    LogDecay g;
    if (threadIdx.x < kD) {
#pragma unroll 2
        for (int t = most - 1; t >= half; --t) {
            wl.k(t)[i] = to_f32(wl.raw[0][t][i]) * g.decay();
            g.add(to_f32(wl.raw[1][t][i]));
        }
    } else {
#pragma unroll 2
        for (int t = most - 1; t >= half; --t) g.add(to_f32(wl.raw[1][t][i]));
#pragma unroll 2
        for (int t = half - 1; t >= 0; --t) {
            wl.k(t)[i] = to_f32(wl.raw[0][t][i]) * g.decay();
            g.add(to_f32(wl.raw[1][t][i]));
        }
        lds.row[i] = sc * g.decay();
    }
    __syncthreads();
}

__device__ __forceinline__ int window_count(const CacheWindow& w, int64_t b) {
    if (!w.k) return 0;
    const int n = w.n ? w.n[b] : w.W;
    return n < 0 ? 0 : (n > w.W ? w.W : n);
}

__global__ __launch_bounds__(256) void cache_store_kernel(CacheMoveArgs a) {
    __shared__ __align__(16) QuantiseLds lds;
    const uint32_t unit = blockIdx.x;
    const int b = (int)(unit / (uint32_t)a.H), h = (int)(unit % (uint32_t)a.H);
    const int page = a.page ? a.page[b] : b;
    if (page < 0 || page >= a.P) return;
    const Place p;
    State v;
    const float* S = a.S + (size_t)unit * kD * kD + 4 * p.l;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            v[t][r] = __builtin_nontemporal_load(reinterpret_cast<const floatx4*>(S + (p.row(t) + r) * kD));
    if (a.page) {
        // of several states for one page the last one counts
        int later = 0;
        for (int j = b + 1 + (int)threadIdx.x; j < a.B; j += 256) later |= a.page[j] == page;
        if (__syncthreads_or(later)) return;
    }
    const size_t at = (size_t)page * a.H + h;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        uint32_t m[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            m[r] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) m[r] = max(m[r], magnitude(v[t][r][e]));
            m[r] = max32(m[r]);
        }
        if (p.l == 0) *reinterpret_cast<uintx4*>(lds.top + p.row(t)) = uintx4{m[0], m[1], m[2], m[3]};
    }
    scales(lds, a.scale + at * kD);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const floatx4 inverse = *reinterpret_cast<const floatx4*>(lds.inverse + p.row(t));
#pragma unroll
        for (int e = 0; e < 4; ++e)
            lds.tile[(4 * p.l + e) * kLd + (p.row(t) >> 2)] = codes_of(floatx4{v[t][0][e], v[t][1][e], v[t][2][e], v[t][3][e]}, inverse);
    }
    codes_out(lds, a.codes + at * kD * kD);
}

// (Codes by streaming loads beside a window only: 192 x 96 states with windows of 4 of 8
// and 8 of 16 tokens, bf16, take 286 and 296 us so and 288 and 307 by ordinary ones, fp32
// 283, 345 and 299, 357; without windows 290 and 270, four requests a page 256 and 222.)
template <typename T, bool kWindow>
__global__ __launch_bounds__(256, kWindow ? 3 : 5) void cache_load_kernel(CacheMoveArgs a) {
    constexpr int kMost = kWindow ? kMaxWindow : 4;   // (an instance for short ones gains nothing)
    __shared__ __align__(16) ReadLds lds;
    __shared__ __align__(16) WindowLds<T, kMost> wl;
    const uint32_t unit = blockIdx.x;
    const int b = (int)(unit / (uint32_t)a.H), h = (int)(unit % (uint32_t)a.H);
    const int page = a.page ? a.page[b] : b;
    if (page < 0 || page >= a.P) return;
    const Place p;
    State v;
    const size_t at = (size_t)page * a.H + h;
    const int n = window_count(a.win, b);
    stage<T, kMost, kWindow>(lds, wl, a.codes + at * kD * kD, a.scale + at * kD, a.win, at, n);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const floatx4 m = *reinterpret_cast<const floatx4*>(lds.row + p.row(t));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const floatx4 x = values_of(lds.tile[(4 * p.l + e) * kLd + (p.row(t) >> 2)], m);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[t][r][e] = x[r];
        }
    }
    for (int t = 0; t < n; ++t) {
        floatx4 u;
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = to_f32(wl.raw[2][t][4 * p.l + e]);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const floatx4 k = *reinterpret_cast<const floatx4*>(wl.k(t) + p.row(b));
#pragma unroll
            for (int r = 0; r < 4; ++r) v[b][r] += k[r] * u;
        }
    }
    float* S = a.S + (size_t)unit * kD * kD + 4 * p.l;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            __builtin_nontemporal_store(v[t][r], reinterpret_cast<floatx4*>(S + (p.row(t) + r) * kD));
}

// A fold holds its state as matrix tiles: wavefront w rows 32 w + 16 R + 4 g + 0..3
// of column 16 T + l, so that the window's updates are products of 16 x 4 and 4 x 16
// (exact fp32 factors), a row's largest magnitude lies in 16 lanes, and four rows'
// codes of a column are one dword here, too.  (With rank-one updates by the vector unit
// 256 x 96 states and 8 tokens took 311 us, not 178.)  Two instances by the longest
// window: the LDS of a short one lets more workgroups in (192 x 96 states, windows of 8,
// bf16 and fp32: 164 and 150 us, by the instance for 16 189 and 216); the registers are
// bounded to match it (fp32, 16: 271 us at three workgroups a CU, 351 at two).
template <typename T, int kMost>
__global__ __launch_bounds__(256, sizeof(T) * kMost <= 16 ? 5 : kMost <= 8 ? 4 : 3) void cache_fold_kernel(CacheMoveArgs a) {
    __shared__ __align__(16) union {
        ReadLds in;
        QuantiseLds out;
    } lds;
    __shared__ __align__(16) WindowLds<T, kMost> wl;
    const uint32_t unit = blockIdx.x;
    const int n = window_count(a.win, (int)(unit / (uint32_t)a.H));
    if (n == 0) return;
    int8_t* codes = a.codes + (size_t)unit * kD * kD;
    float* scale = a.scale + (size_t)unit * kD;
    stage<T, kMost, true>(lds.in, wl, codes, scale, a.win, unit, n);
    const int l = threadIdx.x & 15, g = threadIdx.x >> 4 & 3, row = threadIdx.x >> 6 << 5;
    floatx4 v[2][8];
#pragma unroll
    for (int R = 0; R < 2; ++R) {
        const floatx4 m = *reinterpret_cast<const floatx4*>(lds.in.row + row + 16 * R + 4 * g);
#pragma unroll
        for (int c = 0; c < 8; ++c) v[R][c] = values_of(lds.in.tile[(16 * c + l) * kLd + (row >> 2) + 4 * R + g], m);
    }
#pragma unroll 1
    for (int t = 0; t < n; t += 4) {
        const float k0 = wl.k(t + g)[row + l], k1 = wl.k(t + g)[row + 16 + l];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float u = to_f32(wl.raw[2][t + g][16 * c + l]);
            v[0][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(k0, u, v[0][c], 0, 0, 0);
            v[1][c] = __builtin_amdgcn_mfma_f32_16x16x4f32(k1, u, v[1][c], 0, 0, 0);
        }
    }
    __syncthreads();   // (what is read is read)
#pragma unroll
    for (int R = 0; R < 2; ++R) {
        uint32_t m[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            m[r] = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c) m[r] = max(m[r], magnitude(v[R][c][r]));
            m[r] = max16(m[r]);
        }
        if (l == 0) *reinterpret_cast<uintx4*>(lds.out.top + row + 16 * R + 4 * g) = uintx4{m[0], m[1], m[2], m[3]};
    }
    scales(lds.out, scale);
#pragma unroll
    for (int R = 0; R < 2; ++R) {
        const floatx4 inverse = *reinterpret_cast<const floatx4*>(lds.out.inverse + row + 16 * R + 4 * g);
#pragma unroll
        for (int c = 0; c < 8; ++c) lds.out.tile[(16 * c + l) * kLd + (row >> 2) + 4 * R + g] = codes_of(v[R][c], inverse);
    }
    // (the largest instance: a thread's four addresses anew, or they stay in registers all along, which spills; the
    // others are 3% faster without)
    if (sizeof(T) * kMost > 32) asm volatile("" : "+s"(codes));
    codes_out(lds.out, codes);
}

}  // namespace

hipError_t launch_cache_store(const CacheMoveArgs& a, hipStream_t stream) {
    cache_store_kernel<<<dim3((unsigned)((int64_t)a.B * a.H)), dim3(256), 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_cache_load(const CacheMoveArgs& a, int dtype, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.B * a.H)), block(256);
    if (!a.win.k) cache_load_kernel<bf16, false><<<grid, block, 0, stream>>>(a);
    else if (dtype == 0) cache_load_kernel<float, true><<<grid, block, 0, stream>>>(a);
    else cache_load_kernel<bf16, true><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_cache_fold(const CacheMoveArgs& a, int dtype, hipStream_t stream) {
    const dim3 grid((unsigned)((int64_t)a.B * a.H)), block(256);
    if (dtype == 0) {
        if (a.win.W <= 8) cache_fold_kernel<float, 8><<<grid, block, 0, stream>>>(a);
        else cache_fold_kernel<float, kMaxWindow><<<grid, block, 0, stream>>>(a);
    } else {
        if (a.win.W <= 8) cache_fold_kernel<bf16, 8><<<grid, block, 0, stream>>>(a);
        else cache_fold_kernel<bf16, kMaxWindow><<<grid, block, 0, stream>>>(a);
    }
    return hipGetLastError();
}

}  // namespace kda
