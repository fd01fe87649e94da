// kda_sample.hip -- the next token from a row of logits, by temperature, top-k,
// top-p, min-p and a given random number, and the probabilities that are left.
//
// The order of a row is by logit, largest first, equal ones by index: a token's
// place in it is one 54-bit number, the logit's bits made monotone above the
// index counted down, so that no two are equal and every filter keeps the
// tokens from some place on.  Three passes, each a launch:
//   tiles   the largest logit of every 1024-token tile, and of each of its 16
//           groups, and the sum of its weights e^((l - largest) / T): the row
//           read once at full width
//   rows    one workgroup a row finds the last place that is kept and draws
//   probs   the probabilities, tiles without a kept token unread
// The second pass rarely reads the row again as a whole.  A group's maximum says
// whether anything of it can be large enough: the k-th largest of them bounds the
// k-th largest logit from below, and some hundred of the largest groups hold most
// nuclei.  Their tokens over such a bound go to a list in LDS, and everything is
// decided there: a short one by counting, for each token, those before it; a
// longer one by histograms of 1024 bins, each level inside one bin of the last.
// Where the list overflows, or turns out not to hold the nucleus, some or all of the
// row's tiles are read to count their tokens in bins, from which follows where the
// last kept one lies, within some bins; and all of them once more to collect those
// bins and to sum each tile's weight above them, which shows that it does.
// Weights are taken in 64 bits and added up as whole numbers of 2^-F: their sums
// are the same in any order, and the drawn token is a whole number, too, which a
// rounding of a running sum must not move.
// What bounds it, 256 x 160,000 fp32 (0.16 GB): the first pass HBM, 35 us (4.6 TB/s;
// 30 without weights); the second the slowest row, which one CU reads: 10 us without a
// filter, 10 to 30 us where the list holds all that is kept, 55 to 115 us where a nucleus has
// thousands of tokens (0.64 MB through one CU, some 25 fp64 and integer instructions a
// logit), 205 where in one of many rows the cut is not where some tiles said it was.  The third pass, 192 x 50,021 bf16: 10 us (19 MB written, as much read where
// something is kept).  One row of 32,000: 18.5 us, three launches' trips to memory and
// the second one's instructions, fetched as they run.
#include "kda.h"
#include "kda_device.h"
#include "kda_sample.h"
#include "kda_scan.h"

namespace kda {

namespace {

constexpr int kTile = kSampleTile;
constexpr int kPer = kTile / 64;
constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = kThreads;
constexpr uint32_t kCap = 2048;        // tokens of the list
// of them, that are counted pair by pair (one row of 32,000 with top-k some hundred and top-p: 18 us, 21 by histograms;
// top-k 300 the other way round: 27 by histograms, 50 by pairs)
constexpr uint32_t kFew = 192;
constexpr uint32_t kDense = 96;        // tokens of a piece's 256 (512) from which on they are weighed in place
constexpr uint32_t kRing = 256;        // 63 and a piece's fewer ones fit
static_assert(63 + kDense <= kRing, "the ring's length");
constexpr int kGroupTiles = 512;       // most tiles whose groups' maxima are kept (32 KB)
constexpr int kIndexBits = 22;         // KDA_MAX_VOCAB
constexpr uint64_t kIndexMask = (1u << kIndexBits) - 1;
static_assert(KDA_MAX_VOCAB == 1 << kIndexBits, "an index fits its bits");

__device__ __forceinline__ float minus_inf() { return -__builtin_inff(); }

// ---- places ------------------------------------------------------------------

// a logit's bits, larger for larger ones (both zeros the same)
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
    return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
// the next smaller logit (of zero, whichever: the smallest negative number)
__device__ __forceinline__ float under(float x) {
    const uint32_t k = key_of(x);
    return of_key(k - (k == 0x80000000u ? 2 : 1));
}
// a token's place; larger ones come first
__device__ __forceinline__ uint64_t place(float x, int v) {
    return (uint64_t)key_of(x) << kIndexBits | (kIndexMask - (uint32_t)v);
}
__device__ __forceinline__ int index_of(uint64_t place) { return (int)(kIndexMask - (place & kIndexMask)); }
__device__ __forceinline__ float logit_of(uint64_t place) { return of_key((uint32_t)(place >> kIndexBits)); }

// ---- weights -----------------------------------------------------------------

// 2^y for -1020 <= y <= 0, relative error 4e-14, 1 at 0: 2^n 2^f, |f| <= 1/2, and
// 2^f = 1 + f q(f), q of degree 8 through (2^f - 1) / f at the Chebyshev points
__device__ __forceinline__ double exp2_neg(double y) {
    const double round = 6755399441055744.0;   // 1.5 * 2^52: a whole number in the low bits
    const double t = y + round;
    const double f = y - (t - round);
    double q = 1.0203121071468306e-07;
    q = __builtin_fma(q, f, 1.3255224879377917e-06);
    q = __builtin_fma(q, f, 1.52526868462088e-05);
    q = __builtin_fma(q, f, 0.000154034558524499);
    q = __builtin_fma(q, f, 0.001333355817904325);
    q = __builtin_fma(q, f, 0.009618129159402565);
    q = __builtin_fma(q, f, 0.055504108664760424);
    q = __builtin_fma(q, f, 0.2402265069581299);
    q = __builtin_fma(q, f, 0.6931471805599453);
    const uint64_t p = __builtin_bit_cast(uint64_t, __builtin_fma(q, f, 1.0));
    const uint32_t n = (uint32_t)__builtin_bit_cast(uint64_t, t);
    return __builtin_bit_cast(double, p + ((uint64_t)(n << 20) << 32));
}
// e^((x - top) / T), scale = log2(e) / T, 0 below 2^-1020; top may be infinite
// (then what equals it weighs 1)
__device__ __forceinline__ double weight(float x, float top, double scale) {
    const double y = x == top ? 0.0 : ((double)x - (double)top) * scale;
    const double w = exp2_neg(__builtin_fmax(y, -1020.0));
    return y > -1020.0 ? w : 0.0;
}

// 2^y for y <= 0 in fp32, of a y in 64 bits: its whole part is exact, and 2^f, |f| <=
// 1/2, the hardware's (an ulp off at most)
__device__ __forceinline__ float exp2_f32(double y) {
    const double round = 6755399441055744.0;
    y = __builtin_fmax(y, -1020.0);
    const double t = y + round;
    return __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f((float)(y - (t - round))), (int)__builtin_bit_cast(uint64_t, t));
}

// the same in every lane, into scalar registers
template <typename V>
__device__ __forceinline__ V uniform(V x) {
    uint32_t w[sizeof(V) / 4];
    __builtin_memcpy(w, &x, sizeof(V));
#pragma unroll
    for (uint32_t& y : w) y = (uint32_t)__builtin_amdgcn_readfirstlane((int)y);
    __builtin_memcpy(&x, w, sizeof(V));
    return x;
}

// what a row is asked for
struct Ask {
    double scale, p, least;
    int k;
    bool greedy, by_k, by_p, by_m;
    __device__ __forceinline__ Ask(const SampleArgs& a, int64_t row) {
        const float T = a.temperature ? a.temperature[row] : 1.f;
        const float P = a.top_p ? a.top_p[row] : 1.f, m = a.min_p ? a.min_p[row] : 0.f;
        k = a.top_k ? a.top_k[row] : 0;
        greedy = !(T > 0.f);
        scale = uniform(1.44269504088896340736 / (greedy ? 1.0 : (double)T));
        by_k = k >= 1 && k < a.V;
        by_p = P < 1.f;
        by_m = m > 0.f;
        p = uniform(P > 0.f ? (double)P : 0.0);
        least = uniform(by_m ? (m < 1.f ? (double)m : 1.0) : 0.0);
    }
    // whether the sum of all weights takes part
    __device__ __forceinline__ bool sums() const { return !greedy && !by_k && (by_p || !by_m); }
    // whether the maxima of the tiles' groups do
    __device__ __forceinline__ bool groups(int tiles) const { return !greedy && (by_k || by_p || by_m) && tiles <= kGroupTiles; }
};

// ---- tiles -------------------------------------------------------------------

// a tile's logits, the lane's (j, e) being token (j * 64 + lane) * M + e of it
template <typename T>
struct Tile {
    static constexpr int M = Vec16<T>::N, J = kPer / M;
    typename Vec16<T>::type v[J];
    __device__ __forceinline__ void load(const T* from, int t, int V, int lane) {
        typedef const T __attribute__((address_space(1))) * global;   // (also where the compiler cannot see it)
        const global row = (global)from;
        const int at = t * kTile + lane * M;
        if ((t + 1) * kTile <= V) {
#pragma unroll
            for (int j = 0; j < J; ++j) __builtin_memcpy(&v[j], row + at + j * 64 * M, 16);
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < M; ++e) {
                    const int i = at + j * 64 * M + e;
                    const T x = row[min(i, V - 1)];
                    v[j][e] = i < V ? x : (T)minus_inf();
                }
        }
    }
    // f(logit, token); past the row's end -infinity
    template <typename F>
    __device__ __forceinline__ void each(int t, int lane, F&& f) const {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < M; ++e) f(to_f32((T)v[j][e]), t * kTile + (j * 64 + lane) * M + e);
    }
    // waits for the loads (or a loop over the pieces waits for those of the next tile, too)
    __device__ __forceinline__ void arrived() {
#pragma unroll
        for (int j = 0; j < J; ++j) asm volatile("" : "+v"(v[j]));
    }
    // the same piece by piece, f(logits, first token), in a loop: a quarter (a half) of the code;
    // the tile is gone afterwards
    template <typename F>
    __device__ __forceinline__ void pieces(int t, int lane, F&& f) {
#pragma unroll 1
        for (int j = 0; j < J; ++j) {
            float l[M];
#pragma unroll
            for (int e = 0; e < M; ++e) l[e] = to_f32((T)v[0][e]);
            f(l, t * kTile + (j * 64 + lane) * M);
#pragma unroll
            for (int q = 0; q + 1 < J; ++q) v[q] = v[q + 1];
        }
    }
    template <typename F>
    __device__ __forceinline__ void each_in_turn(int t, int lane, F&& f) {
        pieces(t, lane, [&](const float* l, int i) {
#pragma unroll
            for (int e = 0; e < M; ++e) f(l[e], i + e);
        });
    }
};

template <int kCtrl>
__device__ __forceinline__ float top_with(float x) {
    return __builtin_fmaxf(x, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), kCtrl, 0xf, 0xf, true)));
}
// largest of each four lanes, of the wavefront
__device__ __forceinline__ float quad_top(float x) { return top_with<0x4e>(top_with<0xb1>(x)); }
__device__ __forceinline__ float wave_top_of_quads(float x) {
    x = top_with<0x128>(top_with<0x124>(x));   // rotations of a row of 16 by 4 and 8
    float m = minus_inf();
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = __builtin_fmaxf(m, __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 16 * i)));
    return m;
}
__device__ __forceinline__ float wave_top(float x) { return wave_top_of_quads(quad_top(x)); }

// (One tile a wavefront: two to eight, one after the other with the next one's
// loads in flight, took 256 x 160,000 fp32 from 35 to 41 us with sums and not from
// 33 without.)
template <typename T>
__global__ __launch_bounds__(256) void sample_tiles_kernel(SampleArgs a) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = (a.V + kTile - 1) / kTile;
    const uint32_t per_row = (uint32_t)(tiles + 3) / 4;
    const uint32_t row = blockIdx.x / per_row;
    const int t = (int)(blockIdx.x % per_row) * 4 + wave;
    if (t >= tiles) return;
    Tile<T> x;
    x.load(static_cast<const T*>(a.logits) + (size_t)row * a.V, t, a.V, lane);
    const Ask ask(a, row);
    const SampleSections at = sample_sections(a.R, tiles);
    const size_t i = (size_t)row * tiles + t;
    float top = minus_inf();
    x.each(t, lane, [&](float l, int) { top = __builtin_fmaxf(top, l); });
    top = quad_top(top);
    if (ask.groups(tiles) && (lane & 3) == 0)
        reinterpret_cast<float*>(a.workspace + at.groups)[i * kSampleGroups + (lane >> 2)] = top;
    top = wave_top_of_quads(top);
    if (lane == 0) reinterpret_cast<float*>(a.workspace + at.tops)[i] = top;
    if (!ask.sums()) return;
    double sum = 0.0;
    if (top == __builtin_inff()) {
        x.each(t, lane, [&](float l, int) { sum += l == top ? 1.0 : 0.0; });
    } else if (top > minus_inf()) {
        // (2^-1020 for what weighs less than that: nothing beside the tile's largest)
        const double d = (double)top;
        x.each(t, lane, [&](float l, int) { sum += exp2_neg(__builtin_fmax(((double)l - d) * ask.scale, -1020.0)); });
    }
    sum = wave_sum(sum);
    if (lane == 0) reinterpret_cast<double*>(a.workspace + at.sums)[i] = sum;
}

// ---- rows --------------------------------------------------------------------

struct Entry {
    uint64_t place, w;
};
// One workgroup a row.  Its state lies in LDS, where the functions below, which
// are called and not inlined (their code is read once by every workgroup, from
// far away: a short one is a fast one), find it.  They call nothing themselves, and so
// need no stack.
struct RowLds {
    Entry list[kCap];
    uint64_t bin_w[kBins];
    uint32_t bin_n[kBins];
    uint64_t part_w[kWaves];
    uint32_t part_n[kWaves];
    float part_f[3][kWaves];
    Entry few[64];
    float ring[kWaves][kRing];   // logits to be weighed, on their way
    // the row
    const void* logits;
    double scale, unit;
    float top;
    int V;
    // what one thread tells the others
    uint64_t total_w, before_w, key, key_w, kept_w, above_w;
    uint32_t total_n, before_n, here_n, n, key_n;
    int bin, token;
};
constexpr int kRowBytes = (sizeof(RowLds) + 15) / 16 * 16;
extern __shared__ __align__(16) char row_memory[];
#define KDA_ROW_LDS RowLds& l = *reinterpret_cast<RowLds*>(row_memory)

__device__ __forceinline__ void add(uint64_t* to, uint64_t w) {
    atomicAdd(reinterpret_cast<unsigned long long*>(to), (unsigned long long)w);
}
__device__ __forceinline__ void clear_bins(RowLds& l) {
    l.bin_n[threadIdx.x] = 0;
    l.bin_w[threadIdx.x] = 0;
    __syncthreads();
}
__device__ __forceinline__ void count(RowLds& l, int bin, uint64_t w) {
    atomicAdd(&l.bin_n[bin], 1u);
    add(&l.bin_w[bin], w);
}

// Where sums over the bins, first to last, reach `target`: counts or weights.
// All threads; the histogram is complete.  Returns the bin, -1 if none; the
// sums before it, what it counts, and all sums are in LDS.
template <bool kWeights>   // false: counts alone, in bin_n
__device__ __forceinline__ int cross(bool by_count, uint64_t target) {
    KDA_ROW_LDS;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t n = l.bin_n[threadIdx.x];
    const uint64_t w = kWeights ? l.bin_w[threadIdx.x] : 0;
    uint32_t sn = wave_scan_whole(n);
    uint64_t sw = kWeights ? wave_scan_whole(w) : 0;
    if (lane == 63) {
        l.part_n[wave] = sn;
        if (kWeights) l.part_w[wave] = sw;
    }
    if (threadIdx.x == 0) l.bin = -1;
    __syncthreads();
    const uint32_t pn = wave_scan_whole(lane < kWaves ? l.part_n[lane] : 0u);
    const uint64_t pw = kWeights ? wave_scan_whole(lane < kWaves ? l.part_w[lane] : (uint64_t)0) : 0;
    if (wave > 0) {
        sn += lane_value(pn, wave - 1);
        if (kWeights) sw += lane_value(pw, wave - 1);
    }
    const uint64_t now = by_count ? (uint64_t)sn : sw, own = by_count ? (uint64_t)n : w;
    if (now >= target && now - own < target) {
        l.bin = (int)threadIdx.x;
        l.before_n = sn - n;
        l.before_w = sw - w;
        l.here_n = n;
    }
    if (threadIdx.x == kBins - 1) {
        l.total_n = sn;
        l.total_w = sw;
    }
    __syncthreads();
    return l.bin;
}

// Of n entries, in descending order of their keys (distinct), keys between lo and
// hi: the first at which the number of them, or their weights, reach `target` (not
// 0).  All threads.  False if none; else its key in l.key, and what has been
// reached in l.key_n and l.key_w.
enum Keys { kByPlace, kByIndex };   // the list's entries; those with weight, first index first
__device__ __noinline__ bool find(Keys keys, uint32_t n, uint64_t lo, uint64_t hi, bool by_count, uint64_t target) {
    KDA_ROW_LDS;
    uint32_t base_n = 0;
    uint64_t base_w = 0;
    auto entry = [&](uint32_t i) {
        const Entry x = l.list[i];
        return keys == kByPlace ? x : Entry{x.w ? (x.place & kIndexMask) + 1 : 0, x.w};
    };
    for (;;) {
        // (after the shift at most 1024 bins; the last level's hold one key each)
        const int bits = 64 - __builtin_clzll((hi - lo) | 1);
        const int shift = bits > 10 ? bits - 10 : 0;
        clear_bins(l);
        for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
            const Entry x = entry(i);
            if (x.place && x.place >= lo && x.place <= hi) count(l, (int)((hi - x.place) >> shift), x.w);
        }
        __syncthreads();
        const int bin = cross<true>(by_count, target - (by_count ? (uint64_t)base_n : base_w));
        if (bin < 0) return false;
        base_n += l.before_n;
        base_w += l.before_w;
        const uint32_t here = l.here_n;
        hi -= (uint64_t)bin << shift;
        const uint64_t width = ((uint64_t)1 << shift) - 1;
        lo = hi - lo > width ? hi - width : lo;
        if (threadIdx.x == 0) l.n = 0;
        __syncthreads();
        if (here > 64) continue;
        for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
            const Entry x = entry(i);
            if (x.place && x.place >= lo && x.place <= hi) l.few[atomicAdd(&l.n, 1u)] = x;
        }
        __syncthreads();
        if (threadIdx.x < 64) {
            const Entry mine = threadIdx.x < here ? l.few[threadIdx.x] : Entry{0, 0};
            uint64_t sw = base_w;
            uint32_t sn = base_n;
            for (uint32_t j = 0; j < here; ++j) {
                const Entry x = l.few[j];
                if (x.place >= mine.place) {
                    sw += x.w;
                    ++sn;
                }
            }
            const uint64_t now = by_count ? (uint64_t)sn : sw, before = by_count ? now - 1 : now - mine.w;
            if (mine.place && now >= target && before < target) {
                l.key = mine.place;
                l.key_n = sn;
                l.key_w = sw;
            }
        }
        __syncthreads();
        return true;
    }
}

// For each of n <= kFew entries, over the entries at or before it (by place, or by
// index): their number in l.bin_n and weights in l.bin_w.  All threads.
__device__ __noinline__ void count_pairs(uint32_t n, bool by_index) {
    KDA_ROW_LDS;
    clear_bins(l);
    const uint64_t mask = by_index ? kIndexMask : ~(uint64_t)0;
    const int shared = n <= 64 ? 6 : 32 - __builtin_clz(n - 1);   // 2^shared threads take an entry each
    const uint32_t e = threadIdx.x & ((1u << shared) - 1), part = threadIdx.x >> shared, parts = kThreads >> shared;
    const uint32_t per = (n + parts - 1) / parts, j0 = part * per, j1 = min(n, j0 + per);
    if (e < n && j0 < j1) {
        const uint64_t mine = l.list[e].place & mask;
        uint32_t sn = 0;
        uint64_t sw = 0;
#pragma unroll 4
        for (uint32_t j = j0; j < j1; ++j) {
            const Entry x = l.list[j];
            const bool yes = (x.place & mask) >= mine;
            sn += yes;
            sw += yes ? x.w : 0;
        }
        atomicAdd(&l.bin_n[e], sn);
        add(&l.bin_w[e], sw);
    }
    __syncthreads();
}

// Bins of equal width in the logit, from 2^high of the largest weight down to 2^low
// (any function that never rises with the logit will do).
struct Bins {
    float top, slope, start;
    __device__ __forceinline__ Bins(float top, double scale, double high, double low) : top(top) {
        const double steps = (kBins - 1) / (high - low);
        slope = (float)__builtin_fmin(__builtin_fmax(steps * scale, 1e-30), 1e30);
        start = (float)(high * steps);
    }
    __device__ __forceinline__ int operator()(float x) const {
        const float d = x == top ? 0.f : x - top;
        return (int)__builtin_fminf(__builtin_fmaxf(__builtin_fmaf(-d, slope, start), 0.f), kBins - 1.f);
    }
    // about the logit at which bin b begins
    __device__ __forceinline__ float edge(float b) const { return top - (b - start) / slope; }
};

// What those of `count` maxima weigh that are > below.
__device__ __noinline__ uint64_t weigh_maxima(const __attribute__((address_space(3))) float* maxima, uint32_t count, float below) {
    KDA_ROW_LDS;
    if (threadIdx.x == 0) l.above_w = 0;
    __syncthreads();
    float w = 0.f;
    for (uint32_t i = threadIdx.x; i < count; i += kThreads) {
        const float m = maxima[i];
        if (m > below) w += __builtin_amdgcn_exp2f((m - l.top) * (float)l.scale);
    }
    const double all = wave_sum((double)w);
    if ((threadIdx.x & 63) == 0 && all > 0.0) add(&l.above_w, (uint64_t)(all * l.unit));
    __syncthreads();
    const uint64_t sum = l.above_w;
    __syncthreads();
    return sum;
}

// The nth largest of `count` maxima, of which the largest is `top` and nth ones or
// more, as a rule, are not below `low`.  All threads; -infinity if there are not as many.
__device__ __noinline__ float nth_maximum(const __attribute__((address_space(3))) float* maxima, uint32_t count, uint32_t nth,
                                          float top, float low) {
    KDA_ROW_LDS;
    const Bins bin_of(top, 1.0, 0.0, low < top ? (double)low - (double)top : -1.0);
    uint64_t lo = 1, hi = ~(uint64_t)0 >> (32 - kIndexBits);
    uint32_t before = 0, here = 65;
    int bin = -1;
    while (here > 64) {   // (once, but for many equal maxima, or far ones)
        l.bin_n[threadIdx.x] = 0;
        __syncthreads();
        const int bits = 64 - __builtin_clzll((hi - lo) | 1), shift = bits > 10 ? bits - 10 : 0;
        uint32_t rest = 0;   // of the last bin: most of them, as a rule
        for (uint32_t i = threadIdx.x; i < count; i += kThreads) {
            const float m = maxima[i];
            if (!(m > minus_inf())) continue;
            const uint64_t k = place(m, i);
            const int at = bin < 0 ? bin_of(m) : bin_of(m) == bin && k >= lo && k <= hi ? (int)((hi - k) >> shift) : kBins;
            if (at < kBins - 1) atomicAdd(&l.bin_n[at], 1u);
            else rest += at == kBins - 1;
        }
        rest = wave_scan_whole(rest);
        if ((threadIdx.x & 63) == 63 && rest) atomicAdd(&l.bin_n[kBins - 1], rest);
        __syncthreads();
        const int b = cross<false>(true, nth - before);
        if (b < 0) return minus_inf();
        before += l.before_n;
        here = l.here_n;
        if (bin < 0) {
            bin = b;
        } else {
            hi -= (uint64_t)b << shift;
            const uint64_t width = ((uint64_t)1 << shift) - 1;
            lo = hi - lo > width ? hi - width : lo;
        }
        if (threadIdx.x == 0) l.n = 0;
        __syncthreads();
    }
    for (uint32_t i = threadIdx.x; i < count; i += kThreads) {
        const float m = maxima[i];
        const uint64_t k = place(m, i);
        if (m > minus_inf() && bin_of(m) == bin && k >= lo && k <= hi) l.few[atomicAdd(&l.n, 1u)].place = k;
    }
    __syncthreads();
    if (threadIdx.x < here) {
        const uint64_t mine = l.few[threadIdx.x].place;
        uint32_t n = before;
        for (uint32_t j = 0; j < here; ++j) n += l.few[j].place >= mine;
        if (n == nth) l.key = mine;
    }
    __syncthreads();
    return logit_of(l.key);
}

// About how many tokens of logit > below there are: of G groups with n such tokens
// spread over them, G (1 - e^(-n / G)) have one at least.
__device__ __noinline__ float expected(const __attribute__((address_space(3))) float* maxima, uint32_t count, float below) {
    KDA_ROW_LDS;
    if (threadIdx.x == 0) l.n = 0;
    __syncthreads();
    uint32_t over = 0;
    for (uint32_t i = threadIdx.x; i < count; i += kThreads) over += maxima[i] > below;
    over = wave_scan_whole(over);
    if ((threadIdx.x & 63) == 63) atomicAdd(&l.n, over);
    __syncthreads();
    const float share = (float)l.n / (float)count;
    __syncthreads();
    return -(float)count * __logf(__builtin_fmaxf(1.f - share, 1.f / (float)(4 * count)));
}

enum Found { kNot, kMissed, kFound };   // kNot: in a bin of too many
struct Near {
    Found found;
    float from, border;   // logit > from, and not > border
};
struct Far {
    uint32_t n;           // of the list; 0: nowhere
    uint64_t lo, hi;      // places
    uint64_t before_n, before_w;
};
constexpr int kSome = 4;   // tiles that one stands for

template <typename T>
struct Row {
    const T* logits;
    int V, tiles;
    float top;
    double scale;
    double unit;         // 2^F, F <= 50: what sums are counted in is 2^-F
    int lane, wave;

    // the row of this workgroup, from LDS
    static __device__ __forceinline__ Row here() {
        KDA_ROW_LDS;
        Row r;
        r.logits = static_cast<const T*>(uniform(l.logits));
        r.V = uniform(l.V);
        r.tiles = (r.V + kTile - 1) / kTile;
        r.top = uniform(l.top);
        r.scale = uniform(l.scale);
        r.unit = uniform(l.unit);
        r.lane = threadIdx.x & 63;
        r.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        return r;
    }

    __device__ __forceinline__ uint64_t* sums() const {    // [tiles], weights of what is kept
        return reinterpret_cast<uint64_t*>(row_memory + kRowBytes);
    }
    __device__ __forceinline__ float* tops() const { return reinterpret_cast<float*>(sums() + tiles); }   // [tiles]
    __device__ __forceinline__ float* groups() const { return tops() + tiles; }   // [tiles * 16], if they are kept
    __device__ __forceinline__ float logit(int i) const {
        return to_f32(((const T __attribute__((address_space(1)))*)logits)[i]);
    }
    // w <= 1 as a whole number: beside 2^(52 - F) its last bit is 2^-F
    __device__ __forceinline__ uint64_t whole(double w) const {
        const double c = 4503599627370496.0 / unit;
        return __builtin_bit_cast(uint64_t, w + c) - __builtin_bit_cast(uint64_t, c);
    }
    __device__ __forceinline__ double weight_of(float x) const { return weight(x, top, scale); }
    // whether tile t is one that stands for `step`, a power of two: each step-th of a
    // wavefront's, others than its neighbours'
    static __device__ __forceinline__ bool taken(int t, int step) { return ((t / kWaves + t) & (step - 1)) == 0; }
    // f(tile, its number) for the tiles with a logit > below (with a `step`, those that
    // stand for it), the next one's loads in flight
    template <typename F>
    __device__ __forceinline__ void tiles_over(float below, int step, F&& f) const {
        auto next = [&](int t) {
            for (; t < tiles; t += kWaves) {
                if (!taken(t, step)) continue;
                const float m = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, tops()[t])));
                if (m > below) break;
            }
            return t;
        };
        int t = next(wave);
        if (t >= tiles) return;
        Tile<T> x;
        x.load(logits, t, V, lane);
        for (;;) {
            const int then = next(t + kWaves);
            Tile<T> y;
            x.arrived();
            if (then < tiles) y.load(logits, then, V, lane);
            f(x, t);
            if (then >= tiles) return;
            x = y;
            t = then;
        }
    }
    // lanes of `those` before this one
    static __device__ __forceinline__ uint32_t rank_in(uint64_t those) {
        return __builtin_amdgcn_mbcnt_hi((uint32_t)(those >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)those, 0));
    }
    // the tokens of a tile that the lanes' bits name, the first one's the highest, to the
    // list (past kCap they are only counted)
    __device__ __forceinline__ void append(int t, uint32_t bits) const {
        KDA_ROW_LDS;
        constexpr int M = Tile<T>::M;
        if (__ballot(bits != 0) == 0) return;
        const uint32_t mine = (uint32_t)__builtin_popcount(bits), upto = wave_scan_whole(mine);
        uint32_t at = 0;
        if (lane == 63) at = atomicAdd(&l.n, upto);
        at = (uint32_t)__builtin_amdgcn_readlane((int)at, 63) + upto - mine;
        for (; bits; bits &= bits - 1, ++at) {
            const int slot = kPer - 1 - __builtin_ctz(bits);
            if (at < kCap) l.list[at].w = (uint64_t)(t * kTile + (slot / M * 64 + lane) * M + slot % M);   // (its place follows)
        }
    }
    __device__ __forceinline__ void start_list() const {
        KDA_ROW_LDS;
        __syncthreads();
        if (threadIdx.x == 0) l.n = 0;
        __syncthreads();
    }
    // after that, the list's weights, and its places from indices where they are not
    // there yet; how many were named
    __device__ __forceinline__ uint32_t listed(bool placed = false) const {
        KDA_ROW_LDS;
        __syncthreads();
        const uint32_t n = l.n;
        for (uint32_t i = threadIdx.x; i < min(n, kCap); i += kThreads) {
            uint64_t at = l.list[i].place;
            if (!placed) at = place(logit((int)l.list[i].w), (int)l.list[i].w);
            l.list[i] = Entry{at, whole(weight_of(logit_of(at)))};
        }
        __syncthreads();
        return n;
    }
    // every token of logit > below to the list
    __device__ __forceinline__ uint32_t gather(float below, bool by_group) const {
        KDA_ROW_LDS;
        constexpr int M = Tile<T>::M;
        start_list();
        if (!by_group) {
            tiles_over(below, 1, [&](Tile<T>& x, int t) {
                uint32_t bits = 0;
                x.each_in_turn(t, lane, [&](float v, int) { bits = 2 * bits + (v > below); });
                append(t, bits);
            });
            return listed();
        }
        // a group's 64 tokens, one a lane, eight groups in flight
        constexpr int kAhead = 8;
        const int count = tiles * kSampleGroups, mine = lane / (4 * M) * 64 * M + lane % (4 * M);
        for (int g0 = wave * 64; g0 < count; g0 += kThreads) {
            uint64_t todo = __ballot(g0 + lane < count && groups()[min(g0 + lane, count - 1)] > below);
            while (todo) {
                float x[kAhead];
                int i[kAhead];
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    const int g = g0 + (todo ? __builtin_ctzll(todo) : 0);
                    i[q] = todo ? g / kSampleGroups * kTile + g % kSampleGroups * 4 * M + mine : V;
                    todo &= todo - (todo != 0);
                    x[q] = logit(min(i[q], V - 1));
                }
                uint64_t those[kAhead];
                uint32_t named = 0;
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    those[q] = __ballot(i[q] < V && x[q] > below);
                    named += (uint32_t)__builtin_popcountll(those[q]);
                }
                uint32_t at = 0;
                if (lane == 0) at = atomicAdd(&l.n, named);
                at = (uint32_t)__builtin_amdgcn_readfirstlane((int)at);
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    const uint32_t to = at + rank_in(those[q]);
                    if ((those[q] >> lane & 1) && to < kCap) l.list[to].place = place(x[q], i[q]);
                    at += (uint32_t)__builtin_popcountll(those[q]);
                }
            }
        }
        return listed(true);
    }

    // Sums over a tile of the weights of its tokens over `border`: `all`, the lane's part,
    // and `kept`, of those that weigh `least`, in lane 63.  Their number is added to
    // `passed`; those over `from` and not over `border` go to the list.  A piece with many
    // of them is weighed in place, few are packed by a ring first (256 x 160,000 fp32, normal
    // logits: by min-p 1e-4 110 us with the ring alone, 90 so; by top-p 0.99 121 and 124).
    __device__ __forceinline__ void weigh(Tile<T>& x, int t, float from, float border, double least, uint64_t& all,
                                          uint64_t& kept, uint32_t& passed) const {
        constexpr int M = Tile<T>::M;
        const double c = 4503599627370496.0 / unit;   // (as in whole())
        const bool infinite = top == __builtin_inff();
        KDA_ROW_LDS;
        float* ring = l.ring[wave];
        uint32_t bits = 0, summed = 0, head = 0, held = 0;   // of all lanes
        all = kept = 0;
        auto take = [&](float v, bool counts) {
            const double y = __builtin_fmax(((double)v - (double)top) * scale, -1020.0);
            double w = exp2_neg(y);
            if (infinite) w = v == top ? 1.0 : 0.0;
            w = counts && (infinite || y > -1020.0) ? w : 0.0;
            all += __builtin_bit_cast(uint64_t, w + c);
            if (least > 0.0) kept += __builtin_bit_cast(uint64_t, (w >= least ? w : 0.0) + c);
            ++summed;
        };
        auto flush = [&](uint32_t n) {
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
            take(ring[(head + lane) % kRing], (uint32_t)lane < n);
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
            head += n;
            held -= n;
        };
        x.pieces(t, lane, [&](const float* v, int) {
            uint64_t those[M];
            uint32_t n = 0;
#pragma unroll
            for (int e = 0; e < M; ++e) {
                those[e] = __ballot(v[e] > border);
                n += (uint32_t)__builtin_popcountll(those[e]);
                bits = 2 * bits + (v[e] > from && !(v[e] > border));
            }
            if (n == 0) return;
            passed += n;
            if (n >= kDense) {
#pragma unroll
                for (int e = 0; e < M; ++e) take(v[e], v[e] > border);
                return;
            }
#pragma unroll
            for (int e = 0; e < M; ++e) {
                if (v[e] > border) ring[(head + held + rank_in(those[e])) % kRing] = v[e];
                held += (uint32_t)__builtin_popcountll(those[e]);
            }
            while (held >= 64) flush(64);
        });
        if (held) flush(held);
        all -= summed * __builtin_bit_cast(uint64_t, c);
        kept = wave_scan_whole(least > 0.0 ? kept - summed * __builtin_bit_cast(uint64_t, c) : all);
        append(t, bits);
    }

    // what the tokens of this thread's bin weigh, taken at its middle
    __device__ __forceinline__ double about(double high, double low) const {
        KDA_ROW_LDS;
        const float y = (float)high - ((float)threadIdx.x + 0.5f) * ((float)(high - low) * (1.f / (kBins - 1)));
        return (double)((float)l.bin_n[threadIdx.x] * __builtin_amdgcn_exp2f(__builtin_fminf(y, 0.f))) * unit;
    }
    // Between which logits, of a number that fits the list, the row's tokens reach
    // `target`, as find() has it, as far as can be told from a histogram of them: `below` <
    // logit < `above`, which weigh 2^high at most and, where weights are to reach it, 2^low at
    // least (what weighs less cannot be where they do).  `off` is what those from `above`
    // on weigh.  `all`, not 0: what all tokens weigh, of which those behind `target` are to
    // be told from some tiles.
    __device__ __forceinline__ Near near(bool by_count, uint64_t target, float above, uint64_t off, float below, double high,
                                         double low, uint64_t all) const {
        KDA_ROW_LDS;
        const Bins bin_of(top, scale, high, low);
        const int exact = !by_count && off == 0 ? kBins / 4 : 0;
        if (threadIdx.x == 0) {
            l.above_w = 0;
            l.before_n = 0;
        }
        clear_bins(l);
        uint32_t rest = 0;
        uint64_t aim = target - off;
        if (all) {
            // what the tokens behind weigh
            uint32_t tokens = 0;   // of the tiles taken
            if ((int)threadIdx.x < tiles && taken((int)threadIdx.x, kSome)) tokens = (uint32_t)min(kTile, V - (int)threadIdx.x * kTile);
            float beyond = 0.f;   // (what weighs less than 2^low)
            tiles_over(minus_inf(), kSome, [&](Tile<T>& x, int t) {
                x.each_in_turn(t, lane, [&](float v, int) {
                    if (!(v < above)) return;
                    const int b = bin_of(v);
                    if (b < kBins - 1) {
                        atomicAdd(&l.bin_n[b], 1u);
                    } else {
                        rest += v > minus_inf();
                        beyond += __builtin_amdgcn_exp2f((v - top) * (float)scale);
                    }
                });
            });
            tokens = wave_scan_whole(tokens);
            rest = wave_scan_whole(rest);
            const double beyond_w = wave_sum((double)beyond);
            if (lane == 63) {
                atomicAdd(&l.before_n, tokens);
                atomicAdd(&l.bin_n[kBins - 1], rest);
                add(&l.above_w, (uint64_t)(beyond_w * unit));
            }
            __syncthreads();
            const double each = (double)V / (double)max(l.before_n, 1u);
            const double w = threadIdx.x == kBins - 1 ? (double)l.above_w : about(high, low);
            const uint64_t here_w = (uint64_t)(w * each);
            l.bin_w[threadIdx.x] = here_w;
            l.bin_n[threadIdx.x] = (uint32_t)(l.bin_n[threadIdx.x] * each);
            __syncthreads();
            if (threadIdx.x == 0) l.above_w = 0;
            __syncthreads();
            const uint64_t sum = wave_scan_whole(here_w);
            if (lane == 63) add(&l.above_w, sum);
            __syncthreads();
            const uint64_t found = uniform(l.above_w), behind = all - target;
            aim = found > behind ? found - behind : 1;
        } else {
            // (where there are many tiles, every other one stands for two: thousands of tokens are off by a fraction of a
            // bin, and several are collected.  Not so for weights, of which a few tokens may be most.)
            const int step = by_count && tiles >= 64 ? 2 : 1;
            tiles_over(below, step, [&](Tile<T>& x, int t) {
                x.each_in_turn(t, lane, [&](float v, int) {
                    if (v > below && v < above) {
                        const int b = bin_of(v);
                        if (b < kBins - 1) atomicAdd(&l.bin_n[b], (uint32_t)step);
                        else rest += step;
                        if (b < exact) add(&l.bin_w[b], whole(weight_of(v)));
                    }
                });
            });
            rest = wave_scan_whole(rest);
            if (lane == 63) atomicAdd(&l.bin_n[kBins - 1], rest);
            __syncthreads();
            // (what a bin weighs: about its middle, but for the first ones, whose few tokens may be most of it)
            if (!by_count && (int)threadIdx.x >= exact) {
                l.bin_w[threadIdx.x] = (uint64_t)about(high, low);
            }
        }
        const int bin = cross<true>(by_count, aim);
        if (bin < 0) return Near{kMissed, 0.f, 0.f};
        // that bin and as many beside it as fit the list, up to eight: edges and estimated weights are not exact; 64
        // where some tiles stand for all
        const uint32_t here = l.here_n;
        const int left = bin - 1 - lane, right = bin + 1 + lane;
        const uint32_t more = (left >= 0 ? l.bin_n[left] : 0) + (right < kBins ? l.bin_n[right] : 0);
        const bool fit = here + wave_scan_whole(more) <= kCap - 256 && (all || lane < 8);
        const int beside = __builtin_popcountll(__ballot(fit));
        const int j0 = max(bin - beside, 0), j1 = min(bin + beside, kBins - 1);
        if (here > kCap) return Near{kNot, 0.f, 0.f};
        const float over = j0 > 0 ? bin_of.edge((float)j0) : __builtin_inff(), from = j1 < kBins - 1 ? __builtin_fmaxf(bin_of.edge(j1 + 1.f), below) : below;
        // (what is from `above` on is over, wherever bin 0 begins)
        return Near{from < over ? kFound : kNot, from, __builtin_fminf(over, under(above))};
    }
    // Those tokens to the list (returned: their number), each tile's weight of those over
    // them that weigh `least` to sums, of all over them to l.above_w, and their number to
    // l.before_n.
    __device__ __forceinline__ uint32_t collect(bool by_count, float from, float border, double least) const {
        KDA_ROW_LDS;
        if (threadIdx.x == 0) {
            l.above_w = 0;
            l.before_n = 0;
        }
        for (int t = threadIdx.x; t < tiles; t += kThreads) sums()[t] = 0;
        start_list();
        uint64_t over_w = 0;
        uint32_t passed = 0;   // of all lanes
        tiles_over(from, 1, [&](Tile<T>& x, int t) {
            uint64_t w, kept;
            weigh(x, t, from, border, least, w, kept, passed);
            over_w += w;
            if (lane == 63) sums()[t] = kept;
        });
        over_w = wave_scan_whole(over_w);
        if (lane == 63) {
            add(&l.above_w, over_w);
            if (by_count) atomicAdd(&l.before_n, passed);
        }
        return uniform(listed());
    }
    // What of the list is kept to sums: from place `cut` on, and of weight `least`.
    __device__ __forceinline__ void keep(uint32_t n, uint64_t cut, double least) const {
        KDA_ROW_LDS;
        for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
            const Entry x = l.list[i];
            if (x.place >= cut && weight_of(logit_of(x.place)) >= least) add(&sums()[index_of(x.place) / kTile], x.w);
        }
        __syncthreads();
    }
    // The same as near() and collect() wherever it lies, without the sums: a histogram of
    // the weights themselves, and as many levels inside one bin as it takes (thousands of
    // equal logits, a distribution that fits no bins).
    __device__ __forceinline__ Far far(bool by_count, uint64_t target) const {
        KDA_ROW_LDS;
        uint32_t base_n = 0, here = kCap + 1;
        uint64_t base_w = 0, lo = 1, hi = place(top, 0);
        while (here > kCap) {
            const int bits = 64 - __builtin_clzll((hi - lo) | 1);
            const int shift = bits > 10 ? bits - 10 : 0;
            __syncthreads();
            clear_bins(l);
            tiles_over(minus_inf(), 1, [&](Tile<T>& x, int t) {
                x.each_in_turn(t, lane, [&](float v, int i) {
                    if (v > minus_inf()) {
                        const uint64_t k = place(v, i);
                        if (k >= lo && k <= hi) count(l, (int)((hi - k) >> shift), whole(weight_of(v)));
                    }
                });
            });
            __syncthreads();
            const int b = cross<true>(by_count, target - (by_count ? (uint64_t)base_n : base_w));
            if (b < 0) return Far{0, 0, 0, 0, 0};
            base_n += uniform(l.before_n);
            base_w += uniform(l.before_w);
            here = uniform(l.here_n);
            hi -= (uint64_t)b << shift;
            const uint64_t width = ((uint64_t)1 << shift) - 1;
            lo = hi - lo > width ? hi - width : lo;
        }
        start_list();
        tiles_over(minus_inf(), 1, [&](Tile<T>& x, int t) {
            x.each_in_turn(t, lane, [&](float v, int i) {
                if (v > minus_inf()) {
                    const uint64_t k = place(v, i);
                    if (k >= lo && k <= hi) {
                        const uint32_t at = atomicAdd(&l.n, 1u);
                        if (at < kCap) l.list[at].w = (uint64_t)i;
                    }
                }
            });
        });
        return Far{min(listed(), kCap), lo, hi, base_n, base_w};
    }
    // each tile's weight of what is kept
    __device__ __forceinline__ void sum_kept(uint64_t cut, double least) const {
        for (int t = threadIdx.x; t < tiles; t += kThreads) sums()[t] = 0;
        __syncthreads();
        const float from = cut > 1 ? logit_of(cut) : minus_inf(), below = cut > 1 ? under(from) : from;
        const int border = index_of(cut);
        tiles_over(below, 1, [&](Tile<T>& x, int t) {
            uint64_t all, kept;
            uint32_t passed = 0;
            if (cut > 1)   // (of logits equal to the cut's, those up to its index)
#pragma unroll
                for (int j = 0; j < Tile<T>::J; ++j)
#pragma unroll
                    for (int e = 0; e < Tile<T>::M; ++e)
                        if (to_f32((T)x.v[j][e]) == from && t * kTile + (j * 64 + lane) * Tile<T>::M + e > border) x.v[j][e] = (T)minus_inf();
            weigh(x, t, below, below, least, all, kept, passed);
            if (lane == 63) sums()[t] = kept;
        });
        __syncthreads();
    }
    // Sum of the tiles' sums; the same in every thread.
    __device__ __forceinline__ uint64_t total() const {
        uint64_t s = 0;
        for (int t0 = 0; t0 < tiles; t0 += 64) s += wave_scan_whole(t0 + lane < tiles ? sums()[t0 + lane] : (uint64_t)0);
        return lane_value(s, 63);
    }
    // The first token at which the running sum of the kept weights reaches `target` of
    // `sum`, from the tiles' sums.  Inside the tile weights are counted in 2^-50 of its own
    // largest and share the tile's sum in proportion: it may be made up of tokens that
    // weigh less than half of 2^-F each, and so be nothing one by one (a row of one token
    // and a tail 34 nats under it).  A tile with a sum has a kept token, its largest, so one
    // that is kept is drawn whatever u is.  All threads; the result is l.token's afterwards.
    __device__ __forceinline__ void draw(uint64_t target, uint64_t sum, uint64_t cut, double least) const {
        KDA_ROW_LDS;
        int tile = -1;
        uint64_t base = 0, run = 0, own = 0;
        for (int t0 = 0; t0 < tiles && tile < 0; t0 += 64) {
            const uint64_t mine = t0 + lane < tiles ? sums()[t0 + lane] : (uint64_t)0;
            const uint64_t incl = run + wave_scan_whole(mine);
            const uint64_t hit = __ballot(incl >= target);
            if (hit) {
                const int i = __builtin_ctzll(hit);
                tile = t0 + i;
                own = lane_value(mine, i);
                base = lane_value(incl, i) - own;
            }
            run = lane_value(incl, 63);
        }
        tile = max(tile, 0);
        const int i = tile * kTile + (int)threadIdx.x;
        const float largest = tops()[tile];
        uint64_t w = 0;
        if (i < V) {
            const float x = logit(i);
            if (x > minus_inf() && place(x, i) >= cut && weight_of(x) >= least)
                w = __builtin_bit_cast(uint64_t, weight(x, largest, scale) + 4.0) - __builtin_bit_cast(uint64_t, 4.0);
        }
        uint64_t upto = wave_scan_whole(w);
        if (lane == 63) l.part_w[wave] = upto;
        if (threadIdx.x == 0) l.token = V;
        __syncthreads();
        const uint64_t parts = wave_scan_whole(lane < kWaves ? l.part_w[lane] : (uint64_t)0);
        if (wave > 0) upto += lane_value(parts, wave - 1);
        const uint64_t whole_tile = lane_value(parts, kWaves - 1), before = target - 1 - base;
        // upto / whole_tile > before / own, in 128 bits; u = 1: the last one
        const uint64_t a = __umul64hi(upto, own), b = __umul64hi(before, whole_tile);
        const bool there = target >= sum ? upto == whole_tile : a > b || (a == b && upto * own > before * whole_tile);
        const uint64_t hit = __ballot(w != 0 && there);
        if (hit && lane == 0) atomicMin(&l.token, i + __builtin_ctzll(hit));
        __syncthreads();
    }
};

template <typename T>
__device__ __noinline__ uint32_t gather(float below, bool by_group) { return Row<T>::here().gather(below, by_group); }
// The same as find(), over the row's tokens, by near() and collect().  If it is found, sums
// holds each tile's weight of what is kept if it ends there and weighs `least`, and
// l.key_w the weights up to there.  kNot, kMissed: it may be there all the same.
template <typename T>
__device__ __forceinline__ Found find_near(const Row<T>& r, bool by_count, uint64_t target, float above, uint64_t off, float below,
                                           double high, double low, double least, uint64_t all) {
    KDA_ROW_LDS;
    const Near at = r.near(by_count, target, above, off, below, high, low, all);
    if (at.found != kFound) return at.found;
    const uint32_t n = r.collect(by_count, at.from, at.border, least);
    const uint64_t base = uniform(by_count ? (uint64_t)l.before_n : l.above_w);
    const uint64_t first = at.border < r.top ? place(at.border, 0) : place(r.top, 0), last = at.from > minus_inf() ? place(at.from, 0) : 1;
    __syncthreads();
    if (n > kCap || base >= target || !find(kByPlace, n, last, first, by_count, target - base)) return kMissed;
    const uint64_t cut = l.key;
    __syncthreads();
    if (threadIdx.x == 0) l.key_w += l.above_w;
    r.keep(n, cut, least);
    return kFound;
}
// The same by far(), without the sums.
template <typename T>
__device__ __forceinline__ bool find_far(const Row<T>& r, bool by_count, uint64_t target) {
    KDA_ROW_LDS;
    const Far at = r.far(by_count, target);
    if (at.n == 0 || !find(kByPlace, at.n, at.lo, at.hi, by_count, target - (by_count ? at.before_n : at.before_w))) return false;
    if (threadIdx.x == 0) l.key_w += at.before_w;
    __syncthreads();
    return true;
}

// the weight that top-p asks for, of that of what it is taken from
__device__ __forceinline__ uint64_t share_of(double p, uint64_t w) {
    const double x = __builtin_ceil(p * (double)w);
    return x < 1.0 ? (uint64_t)1 : (uint64_t)x;
}

// What is kept where no list holds it, from the row's tiles: the last place, and the
// sum, with each tile's in sums.  `all`: the weights of all tokens; `listed_w`, not 0:
// of those of logit > listed_over, which are less than top-p asks for.
struct Kept {
    uint64_t cut, sum;
};
template <typename T>
__device__ __forceinline__ Kept over_row(int k, bool by_p, double p, double least, uint64_t all, float listed_over, uint64_t listed_w) {
    KDA_ROW_LDS;
    const Row<T> r = Row<T>::here();
    __syncthreads();
    uint64_t cut = 1, sum = all;
    bool summed = false;
    // the first k; the share, from some tiles; from all of them (a loop: each function stands here once)
#pragma unroll 1
    for (int step = k ? 0 : 1; step < 3; ++step) {
        // (from a quarter of the tiles the place of the cut is off by some hundred tokens, of over a thousand that are
        // collected; beyond 256 tiles by too many.  256 x 160,000 fp32 by top-p 0.5, 0.9, 0.99: 115, 129, 146 us from all
        // tiles, 97, 111, 124 from a quarter, 92, 106, 198 from an eighth.  Fewer than 32 take no longer than the rest.  Of
        // logits of deviation 1 by 0.9 some of 256 rows miss, 245 us where all tiles at once take 178; by 0.5 and 0.99 none
        // does, 149 and 152 where they take 147 and 198.)
        if (step > 0 && !by_p) break;
        if (step == 1 && (k || r.tiles < 32 || r.tiles > 256)) continue;
        const bool by_count = step == 0;
        uint64_t target = (uint64_t)k, off = 0;
        float above = __builtin_inff(), from = minus_inf();
        double high = 0.0, bottom = -66.4;
        if (!by_count) {
            // the last one kept weighs at least (what lies behind it) / V; where the list did not reach the share, it
            // lies below
            target = share_of(p, sum);
            const double behind = ((double)sum - (double)target) / ((double)r.V * r.unit);
            if (behind > 0.0) bottom = (double)__builtin_fmaxf(__builtin_amdgcn_logf((float)behind) - 0.01f, -66.4f);   // (to base 2)
            if (listed_w && listed_w < target) {
                off = listed_w;
                above = of_key(key_of(listed_over) + 1);
                high = ((double)above - (double)r.top) * r.scale;
            }
            if (!(high < 0.0)) high = 0.0;
            if (bottom > high - 0.01) bottom = high - 0.01;
            const double low_x = (double)r.top + bottom / r.scale;
            from = !(low_x > -3e38) || r.top == __builtin_inff() ? minus_inf() : under(under(under((float)low_x)));
        }
        const Found found = find_near<T>(r, by_count, target, above, off, from, high, bottom, least, step == 1 ? sum : 0);
        if (step == 1 && found == kMissed) {
            __syncthreads();
            continue;
        }
        summed = found == kFound;
        const bool ok = summed || find_far<T>(r, by_count, target);
        if (ok) cut = max(cut, uniform(l.key));
        if (by_count) {
            sum = uniform(ok ? l.key_w : l.total_w);
            summed = summed && !by_p;
        }
        __syncthreads();
        if (!by_count) break;
    }
    if (!summed) r.sum_kept(cut, least);
    return Kept{cut, r.total()};
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_rows_kernel(SampleArgs a) {
    KDA_ROW_LDS;
    const int64_t row = blockIdx.x;
    const int V = a.V, tiles = (V + kTile - 1) / kTile;
    const SampleSections at = sample_sections(a.R, tiles);
    SampleRow* to = reinterpret_cast<SampleRow*>(a.workspace + at.rows) + row;
    Row<T> r;
    r.logits = static_cast<const T*>(a.logits) + (size_t)row * V;
    r.V = V;
    r.tiles = tiles;
    r.lane = threadIdx.x & 63;
    r.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Ask ask(a, row);
    const float u0 = a.u ? a.u[row] : 0.f;
    const double u = uniform(u0 > 0.f ? (u0 < 1.f ? (double)u0 : 1.0) : 0.0);

    float top = minus_inf(), low = __builtin_inff();   // largest; smallest of full tiles that are not empty,
    float least_top = __builtin_inff();                // of groups that are not
    const int full = V / kTile;
    for (int t = threadIdx.x; t < tiles; t += kThreads) {
        const float m = reinterpret_cast<const float*>(a.workspace + at.tops)[row * tiles + t];
        r.tops()[t] = m;
        top = __builtin_fmaxf(top, m);
        if (t < full && m > minus_inf()) low = __builtin_fminf(low, m);
    }
    if (ask.groups(tiles)) {
        const float* from = reinterpret_cast<const float*>(a.workspace + at.groups) + row * tiles * kSampleGroups;
        for (int i = threadIdx.x; i < tiles * kSampleGroups; i += kThreads) {
            const float m = from[i];
            r.groups()[i] = m;
            if (m > minus_inf()) least_top = __builtin_fminf(least_top, m);
        }
    }
    top = wave_top(top);
    low = -wave_top(-low);
    least_top = -wave_top(-least_top);
    if (r.lane == 0) {
        l.part_f[0][r.wave] = top;
        l.part_f[1][r.wave] = low;
        l.part_f[2][r.wave] = least_top;
    }
    if (threadIdx.x == 0) l.token = V;
    __syncthreads();
    top = uniform(wave_top(r.lane < kWaves ? l.part_f[0][r.lane] : minus_inf()));
    low = -wave_top(r.lane < kWaves ? -l.part_f[1][r.lane] : minus_inf());
    least_top = -wave_top(r.lane < kWaves ? -l.part_f[2][r.lane] : minus_inf());
    r.top = top;
    r.scale = ask.scale;
    const int bits = 32 - __builtin_clz((uint32_t)V);   // V < 2^bits
    r.unit = __builtin_ldexp(1.0, min(62 - bits, 50));
    if (threadIdx.x == 0) {
        l.logits = r.logits;
        l.scale = r.scale;
        l.unit = r.unit;
        l.top = top;
        l.V = V;
    }
    __syncthreads();

    SampleRow out;
    out.scale = ask.scale;
    out.sum = 0.0;
    out.least = 0.0;
    out.cut = 1;
    out.top = top;
    out.pad = 0;
    if (top == minus_inf()) {   // nothing to draw from
        if (threadIdx.x == 0) {
            if (a.u) a.token[row] = -1;
            *to = out;
        }
        return;
    }
    if (ask.greedy) {
        r.tiles_over(under(top), 1, [&](Tile<T>& x, int t) {
            int first = V;
            x.each(t, r.lane, [&](float v, int i) {
                if (v == top) first = min(first, i);
            });
            if (first < V) atomicMin(&l.token, first);
        });
        __syncthreads();
        if (threadIdx.x == 0) {
            if (a.u) a.token[row] = l.token;
            out.cut = place(top, l.token);
            *to = out;
        }
        return;
    }

    // the sum of all weights, where it takes part
    uint64_t all = 0;
    if (ask.sums()) {
        for (int t = threadIdx.x; t < tiles; t += kThreads) {
            const float m = r.tops()[t];
            r.sums()[t] = m > minus_inf()
                ? (uint64_t)(reinterpret_cast<const double*>(a.workspace + at.sums)[row * tiles + t] * r.weight_of(m) * r.unit + 0.5) : 0;
        }
        __syncthreads();
        all = r.total();
    }
    uint64_t sum = all, cut = 1;
    bool drawn = false;
    if (ask.by_k || ask.by_p || ask.by_m) {
        // no lower than min-p can keep, less a little for its rounding (not where the sum of the first k counts)
        float floor = minus_inf();
        if (ask.by_m && !(ask.by_k && ask.by_p)) {
            const double x = (double)top + (log2(ask.least) - 1e-6) / ask.scale;
            if (x > -3e38) floor = top == __builtin_inff() ? under(top) : under(under((float)x));
        }
        const bool by_group = ask.groups(tiles);
        const auto* maxima = (const __attribute__((address_space(3))) float*)(by_group ? r.groups() : r.tops());
        const uint32_t count = by_group ? tiles * kSampleGroups : tiles;
        // The list is to hold every token of logit > below.  Sure: then it holds all that can be kept (and summed for
        // top-p).  By top-p alone, the 64 largest maxima first, then 256, then as many as 1500 tokens or so
        // exceed (128 and 1500: 57 instead of 53 us for peaked rows, 256 x 160,000 by top-p 0.9; one row by top-p 0.5, 56
        // instead of 34).
        float below = minus_inf(), listed_over = top;
        bool sure = false, done = false;
        uint32_t n = kCap + 1;
        uint64_t listed_w = 0, about_w = 0;
        auto share = [&](uint64_t w) { return share_of(ask.p, w); };
        for (int attempt = 0;; ++attempt) {
            if (attempt == 1 && count <= 128) attempt = 2;   // (the same list again)
            below = top;   // (none)
            sure = V <= (int)kCap;
            if (sure) {
                below = minus_inf();
            } else if (ask.by_k ? (uint32_t)ask.k <= count : ask.by_p && attempt < 3) {
                const uint32_t few = min(attempt == 0 ? 64u : 256u, (count + 1) / 2), many = (uint32_t)(count * (1.f - __expf(-1500.f / (float)count)));
                const uint32_t nth = ask.by_k ? (uint32_t)ask.k : attempt < 2 ? few : many;
                const float bound = attempt == 2 && many <= few ? minus_inf() : nth_maximum(maxima, count, nth, top, nth <= (uint32_t)full ? low : __builtin_fminf(low, least_top));
                if (bound > minus_inf()) {
                    below = under(bound);
                    sure = ask.by_k;
                }
            }
            // (min-p's bound where it comes first, or leaves a list that fits: one row of 160,000, normal logits, by top-p 0.9
            // and min-p 0.01 42 us, without 46, up to half of the list 45; up to 1.2 of it as fast)
            if (floor > minus_inf() && (floor >= below || !(below < top) || (attempt == 0 && !sure && expected(maxima, count, floor) < 0.9f * kCap))) {
                below = floor;
                sure = true;
            }
            // (hardly one that will do, if much of what the last one left out is asked for: then as far as min-p goes.  By
            // top-p 0.5 of normal logits 256 x 32,000 take 45 us at 0.3, 60 at 0.1 and 49 at 0.5; of logits of deviation 1
            // 64 x 160,000 92, 92 and 144; by 0.9, without it, 256 x 160,000 128 -> 159)
            const double less = (double)max(listed_w, about_w);
            if (attempt > 0 && !sure && (double)share(sum) - less > 0.3 * ((double)sum - less)) {
                below = floor > minus_inf() ? floor : top;
                sure = true;
            }
            if (!(below < top)) break;
            // (hardly a token over the first bound that is not its group's largest: not listed if those do not make it, or by
            // less than a fifth.  256 x 160,000 peaked by top-p 0.99 61 us, 119 without the fifth, 256 x 32,000 29, 38 with a
            // tenth; one row of 32,000, normal, by 0.5 28.6, 30.5 with 1.6; listed in any case: 5 to 20% more for most wide nuclei)
            if (attempt < 2 && !sure && !ask.by_k) {
                about_w = weigh_maxima(maxima, count, below);
                if ((double)about_w * 1.25 < (double)share(sum)) continue;
            }
            // (not even tried if so many are expected that the longest of many rows' lists overflows: 64 x 160,000, normal, by
            // min-p 0.01 72 us at 0.8 of the list, 98 at 1.2; 256 x 160,000 by 0.02 69 us, 85 at 0.65)
            if (below == floor && V > (int)kCap && expected(maxima, count, below) > 0.8f * kCap) {
                n = kCap + 1;
                done = false;
                break;
            }
            n = gather<T>(below, by_group);
            listed_over = below;
            done = n <= kCap;
            cut = 1;
            if (!done) break;
            if (n <= kFew) {
                count_pairs(n, false);
                // entry e's number and running weight in the order
                const uint32_t e = threadIdx.x;
                const Entry mine = e < n ? l.list[e] : Entry{0, 0};
                const uint32_t rank = e < n ? l.bin_n[e] : 0;
                const uint64_t run = e < n ? l.bin_w[e] : 0;
                if (threadIdx.x == 0) {
                    l.key = 0;
                    l.key_w = 0;
                    l.kept_w = 0;
                    l.above_w = ~(uint64_t)0;   // the last place that is kept
                }
                __syncthreads();
                if (e < n && rank == (ask.by_k ? min(n, (uint32_t)ask.k) : n)) {
                    l.total_w = run;
                    if (ask.by_k && n >= (uint32_t)ask.k) l.key = mine.place;
                }
                __syncthreads();
                listed_w = l.total_w;
                if (ask.by_k) {
                    sum = listed_w;
                    cut = max(cut, l.key);
                    done = l.key != 0 || sure;
                }
                if (done && ask.by_p) {
                    const uint64_t target = share(sum);
                    if (e < n && run >= target && run - mine.w < target) l.key_w = mine.place;
                    __syncthreads();
                    cut = max(cut, l.key_w);
                    done = l.key_w != 0 || sure;
                }
                if (done) {
                    const bool kept = e < n && mine.place >= cut && (!ask.by_m || r.weight_of(logit_of(mine.place)) >= ask.least);
                    if (e < n && !kept) l.list[e].w = 0;
                    if (kept) {
                        atomicMax(reinterpret_cast<unsigned long long*>(&l.kept_w), (unsigned long long)run);
                        if (ask.by_m) atomicMin(reinterpret_cast<unsigned long long*>(&l.above_w), (unsigned long long)mine.place);
                    }
                    if (a.u) {
                        count_pairs(n, true);   // (its first barrier is one for what is above, too)
                        sum = l.kept_w;
                        const uint64_t target = min((uint64_t)(u * (double)sum) + 1, sum);
                        if (kept && l.bin_w[e] >= target && l.bin_w[e] - mine.w < target) l.token = index_of(mine.place);
                    }
                    __syncthreads();
                    sum = l.kept_w;
                    if (ask.by_m) cut = l.above_w;
                    drawn = true;
                }
            } else {
                const uint64_t first = place(top, 0), last = below > minus_inf() ? place(below, 0) : 1;
                if (ask.by_k) {
                    const bool ok = find(kByPlace, n, last, first, true, ask.k);
                    if (ok) cut = l.key;
                    sum = ok ? l.key_w : l.total_w;
                    done = ok || sure;
                    __syncthreads();
                }
                if (done && ask.by_p) {
                    const bool ok = find(kByPlace, n, last, first, false, share(sum));
                    if (ok) cut = max(cut, l.key);
                    done = ok || sure;
                    listed_w = l.total_w;
                    __syncthreads();
                }
                if (done) {
                    uint64_t s = 0, end = ~(uint64_t)0;   // the last place that is kept
                    if (threadIdx.x == 0) l.above_w = end;
                    __syncthreads();
                    for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
                        const Entry x = l.list[i];
                        if (x.place < cut || (ask.by_m && r.weight_of(logit_of(x.place)) < ask.least)) {
                            l.list[i].w = 0;
                        } else {
                            s += x.w;
                            end = min(end, x.place);
                        }
                    }
                    if (ask.by_m) atomicMin(reinterpret_cast<unsigned long long*>(&l.above_w), (unsigned long long)end);
                    s = wave_scan_whole(s);
                    if (r.lane == 63) l.part_w[r.wave] = s;
                    __syncthreads();
                    sum = lane_value(wave_scan_whole(r.lane < kWaves ? l.part_w[r.lane] : (uint64_t)0), kWaves - 1);
                    if (ask.by_m) cut = l.above_w;
                    __syncthreads();
                    if (a.u) {
                        find(kByIndex, n, kIndexMask + 2 - V, kIndexMask + 1, false, min((uint64_t)(u * (double)sum) + 1, sum));
                        if (threadIdx.x == 0) l.token = index_of(l.key - 1);
                    }
                    drawn = true;
                }
            }
            __syncthreads();
            if (done) break;
        }
        if (!done) {
            const Kept found = over_row<T>(ask.by_k ? ask.k : 0, ask.by_p, ask.p, ask.least, all, listed_over,
                                           n <= kCap && !ask.by_k ? listed_w : 0);
            cut = found.cut;
            sum = found.sum;
        }
        out.cut = cut;
        if (!drawn) out.least = ask.least;   // (else the cut has it)
    }
    if (a.u && !drawn) r.draw(min((uint64_t)(u * (double)sum) + 1, sum), sum, out.cut, out.least);
    if (threadIdx.x == 0) {
        if (a.u) a.token[row] = l.token;
        if (a.probs) out.sum = log2((double)sum / r.unit);
        *to = out;
    }
}

// ---- probabilities -----------------------------------------------------------

// (Rows of an odd vocabulary are read and written at the tokens' own places: in pieces
// that begin at a multiple of 16 bytes 256 x 160,001 fp32 took 64 us here, not 58.)
template <typename T>
__global__ __launch_bounds__(256) void sample_probs_kernel(SampleArgs a) {
    constexpr int M = Tile<T>::M, J = Tile<T>::J;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = (a.V + kTile - 1) / kTile;
    const uint32_t per_row = (uint32_t)(tiles + 3) / 4;
    const uint32_t row = blockIdx.x / per_row;
    const int t = (int)(blockIdx.x % per_row) * 4 + wave;
    if (t >= tiles) return;
    const SampleSections at = sample_sections(a.R, tiles);
    const SampleRow r = reinterpret_cast<const SampleRow*>(a.workspace + at.rows)[row];
    const float m = reinterpret_cast<const float*>(a.workspace + at.tops)[(size_t)row * tiles + t];
    const size_t begin = (size_t)row * a.V;
    const bool some = m > minus_inf() && ((uint64_t)key_of(m) << kIndexBits | kIndexMask) >= r.cut && weight(m, r.top, r.scale) >= r.least;
    Tile<T> x;
    if (some) x.load(static_cast<const T*>(a.logits) + begin, t, a.V, lane);
    T* probs = static_cast<T*>(a.probs) + begin;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int v = t * kTile + (j * 64 + lane) * M;
        typename Vec16<T>::type y;
#pragma unroll
        for (int e = 0; e < M; ++e) {
            y[e] = (T)0.f;
            if (some) {
                const float l = to_f32((T)x.v[j][e]);
                bool kept = l > minus_inf() && place(l, v + e) >= r.cut;
                if (r.least > 0.0) kept = kept && weight(l, r.top, r.scale) >= r.least;
                // (one power of two for the weight over the sum)
                const double y0 = l == r.top ? 0.0 : ((double)l - (double)r.top) * r.scale;
                y[e] = from_f32<T>(kept ? exp2_f32(y0 - r.sum) : 0.f);
            }
        }
        if ((t + 1) * kTile <= a.V) {
            __builtin_memcpy(probs + v, &y, 16);
        } else {
#pragma unroll
            for (int e = 0; e < M; ++e)
                if (v + e < a.V) probs[v + e] = y[e];
        }
    }
}

template <typename T>
hipError_t launch_sample_t(const SampleArgs& a, hipStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const int64_t tiles = sample_tiles(a.V);
    // (and the maxima of the groups of kGroupTiles tiles, which are fewer bytes than those of the most tiles)
    static_assert(kGroupTiles * (12 + 4 * kSampleGroups) <= KDA_MAX_VOCAB / kTile * 12, "the larger of the two");
    const int most = kRowBytes + (int)sample_tiles(KDA_MAX_VOCAB) * 12;
    const hipError_t e = raise_lds_limit_once(reinterpret_cast<const void*>(sample_rows_kernel<T>), most, done);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)(a.R * ((tiles + 3) / 4))), block(256);
    sample_tiles_kernel<T><<<grid, block, 0, stream>>>(a);
    sample_rows_kernel<T><<<dim3((unsigned)a.R), dim3(kThreads), kRowBytes + (size_t)tiles * (tiles <= kGroupTiles ? 12 + 4 * kSampleGroups : 12), stream>>>(a);
    if (a.probs)
        sample_probs_kernel<T><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int dtype, hipStream_t stream) {
    return dtype == 0 ? launch_sample_t<float>(a, stream) : launch_sample_t<bf16>(a, stream);
}

}  // namespace kda
