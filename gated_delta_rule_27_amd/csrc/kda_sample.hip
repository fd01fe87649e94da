// kda_sample.hip -- the next token from a row of logits, by temperature, top-k,
// top-p, min-p and a given random number, and the probabilities that are left.
//
// The order of a row is by logit, largest first, equal ones by index: a token's
// place in it is one 54-bit number, the logit's bits made monotone above the
// index counted down, so that no two are equal and every filter keeps the
// tokens from some place on.  Three passes, each a launch:
//   tiles   the largest logit of every 1024-token tile and the sum of its
//           weights e^((l - largest) / T), the row read once at full width
//   rows    one workgroup a row finds the last place that is kept and draws
//   probs   the probabilities, tiles without a kept token unread
// The second pass rarely reads the row again as a whole.  The k-th largest tile
// maximum bounds the k-th largest logit from below, and the smallest tile
// maximum lies low enough for most of a nucleus: what is at least that large (a
// few tokens a tile) goes to a list in LDS, and places are found there by
// histograms of 1024 bins, each level inside one bin of the last.  Where the
// list overflows, or turns out not to hold the nucleus, the first levels read
// the row's tiles instead.
// Weights are taken in 64 bits, the histograms' as whole numbers of 2^-F, whose
// sums are the same in any order: the drawn token is a whole number, too, which
// a rounding of a running sum must not move.
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
// a token's place; larger ones come first
__device__ __forceinline__ uint64_t place(float x, int v) {
    return (uint64_t)key_of(x) << kIndexBits | (kIndexMask - (uint32_t)v);
}
__device__ __forceinline__ float logit_of(uint64_t place) { return of_key((uint32_t)(place >> kIndexBits)); }

// ---- weights -----------------------------------------------------------------

// 2^y for y <= 0, to an ulp or two (0 below 2^-1020), 1 at 0: 2^n e^r, |r| <= ln 2 / 2, the
// series to r^12 (the next term: 2^-52)
__device__ __forceinline__ double exp2_neg(double y) {
    const double n = __builtin_rint(y);
    const double r = (y - n) * 0.693147180559945309417;
    double p = 1.0 / 479001600;
    p = __builtin_fma(p, r, 1.0 / 39916800);
    p = __builtin_fma(p, r, 1.0 / 3628800);
    p = __builtin_fma(p, r, 1.0 / 362880);
    p = __builtin_fma(p, r, 1.0 / 40320);
    p = __builtin_fma(p, r, 1.0 / 5040);
    p = __builtin_fma(p, r, 1.0 / 720);
    p = __builtin_fma(p, r, 1.0 / 120);
    p = __builtin_fma(p, r, 1.0 / 24);
    p = __builtin_fma(p, r, 1.0 / 6);
    p = __builtin_fma(p, r, 0.5);
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    if (!(y > -1020.0)) return 0.0;
    const uint64_t b = __builtin_bit_cast(uint64_t, p) + ((uint64_t)(int64_t)(int32_t)n << 52);
    return __builtin_bit_cast(double, b);
}
// e^((x - top) / T), scale = log2(e) / T; top may be infinite (then what equals it weighs 1)
__device__ __forceinline__ double weight(float x, float top, double scale) {
    return x == top ? 1.0 : exp2_neg(((double)x - (double)top) * scale);
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
        scale = 1.44269504088896340736 / (greedy ? 1.0 : (double)T);
        by_k = k >= 1 && k < a.V;
        by_p = P < 1.f;
        by_m = m > 0.f;
        p = P > 0.f ? (double)P : 0.0;
        least = by_m ? (m < 1.f ? (double)m : 1.0) : 0.0;
    }
    // whether the sum of all weights takes part
    __device__ __forceinline__ bool sums() const { return !greedy && !by_k && (by_p || !by_m); }
};

// ---- tiles -------------------------------------------------------------------

// a tile's logits, the lane's (j, e) being token (j * 64 + lane) * M + e of it;
// past the row's end, and for NaN, -infinity
template <typename T>
struct Tile {
    static constexpr int M = Vec16<T>::N, J = kPer / M;
    float x[J][M];
    __device__ __forceinline__ void load(const T* row, int t, int V, int lane) {
        typename Vec16<T>::type v[J];
        const int at = t * kTile + lane * M;
        if ((t + 1) * kTile <= V) {
#pragma unroll
            for (int j = 0; j < J; ++j) v[j] = load16(row + at + j * 64 * M);
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < M; ++e) x[j][e] = __builtin_fmaxf(to_f32((T)v[j][e]), minus_inf());
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < M; ++e) v[j][e] = row[min(at + j * 64 * M + e, V - 1)];
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < M; ++e)
                    x[j][e] = at + j * 64 * M + e < V ? __builtin_fmaxf(to_f32((T)v[j][e]), minus_inf()) : minus_inf();
        }
    }
    // f(logit, token)
    template <typename F>
    __device__ __forceinline__ void each(int t, int lane, F&& f) const {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < M; ++e) f(x[j][e], t * kTile + (j * 64 + lane) * M + e);
    }
};

__device__ __forceinline__ float wave_top(float x) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) x = __builtin_fmaxf(x, __shfl_xor(x, off, 64));
    return x;
}

struct Sections {
    float* tops;        // [R, tiles]
    double* sums;       // [R, tiles]
    SampleRow* rows;    // [R]
};
__device__ __forceinline__ Sections sections(const SampleArgs& a, int64_t tiles) {
    Sections s;
    const uint64_t n = (uint64_t)a.R * tiles;
    s.tops = reinterpret_cast<float*>(a.workspace);
    s.sums = reinterpret_cast<double*>(a.workspace + (n * 4 + 15) / 16 * 16);
    s.rows = reinterpret_cast<SampleRow*>(a.workspace + (n * 4 + 15) / 16 * 16 + (n * 8 + 15) / 16 * 16);
    return s;
}

template <typename T>
__global__ __launch_bounds__(256) void sample_tiles_kernel(SampleArgs a) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = (a.V + kTile - 1) / kTile;
    const uint32_t groups = (uint32_t)(tiles + 3) / 4;
    const uint32_t row = blockIdx.x / groups;
    const int t = (int)(blockIdx.x % groups) * 4 + wave;
    if (t >= tiles) return;
    Tile<T> x;
    x.load(static_cast<const T*>(a.logits) + (size_t)row * a.V, t, a.V, lane);
    const Ask ask(a, row);
    float top = minus_inf();
    x.each(t, lane, [&](float l, int) { top = __builtin_fmaxf(top, l); });
    top = wave_top(top);
    const Sections s = sections(a, tiles);
    const size_t at = (size_t)row * tiles + t;
    if (lane == 0) s.tops[at] = top;
    if (!ask.sums()) return;
    double sum = 0.0;
    if (top > minus_inf()) x.each(t, lane, [&](float l, int) { sum += weight(l, top, ask.scale); });
    sum = wave_sum(sum);
    if (lane == 0) s.sums[at] = sum;
}

// ---- rows --------------------------------------------------------------------

struct RowLds {
    uint64_t list[kCap];      // places
    uint64_t w[kCap];         // their weights
    uint64_t bin_w[kBins];
    uint32_t bin_n[kBins];
    uint64_t part_w[kWaves];
    uint32_t part_n[kWaves];
    double part_d[kWaves];
    float part_f[kWaves];
    uint64_t few[64], few_w[64];
    // what one thread tells the others
    uint64_t total_w, before_w, key, key_w;
    uint32_t total_n, before_n, here_n, n, key_n;
    int bin, token;
};

// Where sums over the bins, first to last, reach `target`: counts or weights.
// All threads; the histogram is complete.  Returns the bin, -1 if none; the
// sums before it, what it counts, and all sums are in `l`.
__device__ int cross(RowLds& l, bool by_count, uint64_t target) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t n = l.bin_n[threadIdx.x];
    const uint64_t w = l.bin_w[threadIdx.x];
    uint32_t sn = wave_scan_whole(n);
    uint64_t sw = wave_scan_whole(w);
    if (lane == 63) {
        l.part_n[wave] = sn;
        l.part_w[wave] = sw;
    }
    if (threadIdx.x == 0) l.bin = -1;
    __syncthreads();
    uint32_t bn = 0;
    uint64_t bw = 0;
    for (int i = 0; i < wave; ++i) {
        bn += l.part_n[i];
        bw += l.part_w[i];
    }
    sn += bn;
    sw += bw;
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
__device__ __forceinline__ void clear_bins(RowLds& l) {
    l.bin_n[threadIdx.x] = 0;
    l.bin_w[threadIdx.x] = 0;
    __syncthreads();
}
__device__ __forceinline__ void count(RowLds& l, int bin, uint64_t w) {
    atomicAdd(&l.bin_n[bin], 1u);
    atomicAdd(reinterpret_cast<unsigned long long*>(&l.bin_w[bin]), (unsigned long long)w);
}

// Of the n entries of the list, in descending order of key(i) (distinct; 0: not
// one of them), keys at most `hi`: the first at which the number of them, or
// their weights, reach `target` (not 0).  All threads.  False if none; else its
// key in l.key, and what has been reached in l.key_n and l.key_w.
template <typename K>
__device__ bool find(RowLds& l, uint32_t n, K key, uint64_t lo, uint64_t hi, bool by_count, uint64_t target) {
    uint32_t base_n = 0;
    uint64_t base_w = 0;
    for (;;) {
        // (after the shift at most 1024 bins; the last level's hold one key each)
        const int bits = 64 - __builtin_clzll((hi - lo) | 1);
        const int shift = bits > 10 ? bits - 10 : 0;
        clear_bins(l);
        for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
            const uint64_t k = key(i);
            if (k && k >= lo && k <= hi) count(l, (int)((hi - k) >> shift), l.w[i]);
        }
        __syncthreads();
        const uint64_t base = by_count ? base_n : base_w;
        const int bin = cross(l, by_count, target - base);
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
            const uint64_t k = key(i);
            if (k && k >= lo && k <= hi) {
                const uint32_t at = atomicAdd(&l.n, 1u);
                l.few[at] = k;
                l.few_w[at] = l.w[i];
            }
        }
        __syncthreads();
        if (threadIdx.x < 64) {
            const int lane = threadIdx.x;
            const uint64_t k = lane < (int)here ? l.few[lane] : 0, w = lane < (int)here ? l.few_w[lane] : 0;
            uint64_t sw = base_w;
            uint32_t sn = base_n;
            for (uint32_t j = 0; j < here; ++j) {
                const uint64_t kj = lane_value(k, j), wj = lane_value(w, j);
                if (kj >= k) {
                    sw += wj;
                    ++sn;
                }
            }
            const uint64_t now = by_count ? (uint64_t)sn : sw, before = by_count ? now - 1 : now - w;
            if (k && now >= target && before < target) {
                l.key = k;
                l.key_n = sn;
                l.key_w = sw;
            }
        }
        __syncthreads();
        return true;
    }
}

// one workgroup a row
template <typename T>
struct Row {
    RowLds& l;
    float* tops;         // LDS: [tiles]
    double* sums;        // LDS: [tiles]
    const T* logits;
    int V, tiles;
    int lane, wave;
    float top;
    double scale, unit;  // unit: 2^F

    __device__ __forceinline__ uint64_t whole(double w) const { return (uint64_t)(w * unit + 0.5); }
    __device__ __forceinline__ double weight_of(float x) const { return weight(x, top, scale); }
    template <typename F>
    __device__ __forceinline__ void tiles_from(float least, F&& f) const {
        for (int t = wave; t < tiles; t += kWaves) {
            const float m = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, tops[t])));
            if (!(m >= least) || m == minus_inf()) continue;
            Tile<T> x;
            x.load(logits, t, V, lane);
            f(x, t);
        }
    }
    // tokens of logit >= least that `keep` names, and their weights, to the list;
    // how many there are (more than kCap: those past it are left out)
    template <typename F>
    __device__ uint32_t gather(float least, F&& keep) {
        if (threadIdx.x == 0) l.n = 0;
        __syncthreads();
        tiles_from(least, [&](const Tile<T>& x, int t) {
            uint32_t mine = 0;
            x.each(t, lane, [&](float v, int i) { mine += v >= least && v > minus_inf() && keep(v, i); });
            const uint32_t incl = wave_scan_whole(mine), all = lane_value(incl, 63);
            if (all == 0) return;
            uint32_t at = 0;
            if (lane == 0) at = atomicAdd(&l.n, all);
            at = lane_value(at, 0) + incl - mine;
            if (mine)
                x.each(t, lane, [&](float v, int i) {
                    if (v >= least && v > minus_inf() && keep(v, i)) {
                        if (at < kCap) l.list[at] = place(v, i);
                        ++at;
                    }
                });
        });
        __syncthreads();
        const uint32_t n = l.n;
        for (uint32_t i = threadIdx.x; i < min(n, kCap); i += kThreads) l.w[i] = whole(weight_of(logit_of(l.list[i])));
        __syncthreads();
        return n;
    }
    // linear bins of 46 T below the largest logit (less than e^-46 of its weight: in the last)
    __device__ __forceinline__ int bin_of(float x) const {
        if (x == top) return 0;
        return (int)__builtin_fmin(((double)top - (double)x) * scale * (kBins / 66.4), kBins - 1.0);
    }
    // the same as find(), over the row
    __device__ bool find_row(bool by_count, uint64_t target) {
        clear_bins(l);
        tiles_from(minus_inf(), [&](const Tile<T>& x, int t) {
            x.each(t, lane, [&](float v, int) {
                if (v > minus_inf()) count(l, bin_of(v), whole(weight_of(v)));
            });
        });
        __syncthreads();
        const int bin = cross(l, by_count, target);
        if (bin < 0) return false;
        uint32_t base_n = l.before_n, here = l.here_n;
        uint64_t base_w = l.before_w, lo = 1, hi = ~(uint64_t)0 >> (32 - kIndexBits);
        while (here > kCap) {
            // (many equal logits: by their places)
            const int bits = 64 - __builtin_clzll((hi - lo) | 1);
            const int shift = bits > 10 ? bits - 10 : 0;
            __syncthreads();
            clear_bins(l);
            tiles_from(minus_inf(), [&](const Tile<T>& x, int t) {
                x.each(t, lane, [&](float v, int i) {
                    if (v > minus_inf() && bin_of(v) == bin) {
                        const uint64_t k = place(v, i);
                        if (k >= lo && k <= hi) count(l, (int)((hi - k) >> shift), whole(weight_of(v)));
                    }
                });
            });
            __syncthreads();
            const int b = cross(l, by_count, target - (by_count ? (uint64_t)base_n : base_w));
            if (b < 0) return false;
            base_n += l.before_n;
            base_w += l.before_w;
            here = l.here_n;
            hi -= (uint64_t)b << shift;
            const uint64_t width = ((uint64_t)1 << shift) - 1;
            lo = hi - lo > width ? hi - width : lo;
        }
        __syncthreads();
        const uint32_t n = gather(minus_inf(), [&](float v, int i) {
            const uint64_t k = place(v, i);
            return bin_of(v) == bin && k >= lo && k <= hi;
        });
        const bool ok = find(l, n, [&](uint32_t i) { return l.list[i]; }, lo, hi, by_count,
                             target - (by_count ? (uint64_t)base_n : base_w));
        if (ok && threadIdx.x == 0) {
            l.key_n += base_n;
            l.key_w += base_w;
        }
        __syncthreads();
        return ok;
    }
    // sum of the tiles' sums; the same in every thread
    __device__ double total() {
        double s = 0.0;
        for (int t0 = 0; t0 < tiles; t0 += 64) s += wave_sum(t0 + lane < tiles ? sums[t0 + lane] : 0.0);
        return s;
    }
    // the first token at which the running sum of weights passes `target`, from
    // the tiles' sums (in the first wavefront)
    __device__ int draw(double target, uint64_t cut, double least) {
        int tile = -1, filled = -1;
        double base = 0.0, run = 0.0;
        for (int t0 = 0; t0 < tiles && tile < 0; t0 += 64) {
            const double s = t0 + lane < tiles ? sums[t0 + lane] : 0.0;
            const double incl = run + wave_scan(s);
            const uint64_t hit = __ballot(s > 0.0 && incl > target), any = __ballot(s > 0.0);
            if (any) filled = t0 + 63 - __builtin_clzll(any);
            if (hit) {
                const int i = __builtin_ctzll(hit);
                tile = t0 + i;
                base = i ? lane_value(incl, i - 1) : run;
            }
            run = lane_value(incl, 63);
        }
        if (tile < 0) {   // (the target rounded past the end: the last token with weight)
            tile = max(filled, 0);
            base = -1e300;
        }
        const int v0 = tile * kTile + lane * kPer;   // a lane's tokens are consecutive
        double w[kPer], s = 0.0;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const float x = v0 + e < V ? __builtin_fmaxf(to_f32(logits[min(v0 + e, V - 1)]), minus_inf()) : minus_inf();
            w[e] = x > minus_inf() && place(x, min(v0 + e, V - 1)) >= cut ? weight_of(x) : 0.0;
            if (w[e] < least) w[e] = 0.0;
            s += w[e];
        }
        const double incl = base + wave_scan(s);
        double sum = __shfl_up(incl, 1, 64);
        if (lane == 0) sum = base;
        int first = -1, last = -1;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            sum += w[e];
            if (w[e] > 0.0) {
                last = v0 + e;
                if (first < 0 && sum > target) first = v0 + e;
            }
        }
        const uint64_t hit = __ballot(first >= 0), any = __ballot(last >= 0);
        if (hit) return __builtin_amdgcn_readlane(first, __builtin_ctzll(hit));
        if (any) return __builtin_amdgcn_readlane(last, 63 - __builtin_clzll(any));
        return min(tile * kTile, V - 1);
    }
};

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_rows_kernel(SampleArgs a) {
    extern __shared__ __align__(16) char dynamic[];
    RowLds& l = *reinterpret_cast<RowLds*>(dynamic);
    const int64_t row = blockIdx.x;
    const int V = a.V, tiles = (V + kTile - 1) / kTile;
    const Sections sec = sections(a, tiles);
    Row<T> r{l};
    r.sums = reinterpret_cast<double*>(dynamic + (sizeof(RowLds) + 15) / 16 * 16);
    r.tops = reinterpret_cast<float*>(r.sums + tiles);
    r.logits = static_cast<const T*>(a.logits) + (size_t)row * V;
    r.V = V;
    r.tiles = tiles;
    r.lane = threadIdx.x & 63;
    r.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Ask ask(a, row);
    const float u0 = a.u ? a.u[row] : 0.f;
    const double u = u0 > 0.f ? (u0 < 1.f ? (double)u0 : 1.0) : 0.0;

    float top = minus_inf(), low = __builtin_inff();   // largest; smallest of full tiles that are not empty
    const int full = V / kTile;
    for (int t = threadIdx.x; t < tiles; t += kThreads) {
        const float m = sec.tops[row * tiles + t];
        r.tops[t] = m;
        top = __builtin_fmaxf(top, m);
        if (t < full && m > minus_inf()) low = __builtin_fminf(low, m);
    }
    top = wave_top(top);
    low = -wave_top(-low);
    if (r.lane == 0) {
        l.part_f[r.wave] = top;
        l.part_d[r.wave] = (double)low;
    }
    if (threadIdx.x == 0) l.token = V;
    __syncthreads();
    for (int i = 0; i < kWaves; ++i) {
        top = __builtin_fmaxf(top, l.part_f[i]);
        low = __builtin_fminf(low, (float)l.part_d[i]);
    }
    r.top = top;
    r.scale = ask.scale;
    const int bits = 32 - __builtin_clz((uint32_t)V);   // V < 2^bits
    r.unit = __builtin_ldexp(1.0, 62 - bits);

    SampleRow out;
    out.scale = ask.scale;
    out.per = 1.0;
    out.least = 0.0;
    out.cut = 1;
    out.top = top;
    out.pad = 0;
    if (top == minus_inf()) {   // nothing to draw from
        if (threadIdx.x == 0) {
            if (a.u) a.token[row] = -1;
            sec.rows[row] = out;
        }
        return;
    }
    if (ask.greedy) {
        r.tiles_from(top, [&](const Tile<T>& x, int t) {
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
            sec.rows[row] = out;
        }
        return;
    }

    // the sum of all weights, where it takes part
    double Z = 0.0;
    if (ask.sums()) {
        for (int t = threadIdx.x; t < tiles; t += kThreads) {
            const float m = r.tops[t];
            r.sums[t] = m > minus_inf() ? sec.sums[row * tiles + t] * r.weight_of(m) : 0.0;
        }
        __syncthreads();
        Z = r.total();
    }
    if (ask.by_k || ask.by_p || ask.by_m) {
        // what the list holds: everything from `least` on
        float least = minus_inf();
        bool listed = true, holds_all = true;   // holds_all: every token that can be kept (and summed for top-p)
        if (ask.by_k && ask.k <= full && full <= (int)kCap) {
            for (int t = threadIdx.x; t < full; t += kThreads) {
                l.list[t] = r.tops[t] > minus_inf() ? place(r.tops[t], t) : 0;
                l.w[t] = 0;
            }
            __syncthreads();
            if (find(l, full, [&](uint32_t i) { return l.list[i]; }, place(low, V - 1), place(top, 0), true, ask.k))
                least = logit_of(l.key);
            __syncthreads();
        } else if (V > (int)kCap) {
            holds_all = false;
            least = low;
            listed = full <= 320;   // (on the average n (ln n + 0.6) tokens lie above the smallest of n tile maxima)
        }
        if (ask.by_m && !(ask.by_k && ask.by_p)) {
            // (and no lower than min-p can keep, less a little for its rounding)
            const double x = (double)top + (log2(ask.least) - 1e-6) / ask.scale;
            const float m = !(x > -3e38) ? minus_inf() : top == __builtin_inff() ? top : of_key(key_of((float)x) - 1);
            if (holds_all) {
                least = __builtin_fmaxf(least, m);
            } else if (m >= least || !listed || !ask.by_p) {
                holds_all = listed = true;
                least = m;
            }
        }
        uint32_t n = listed ? r.gather(least, [](float, int) { return true; }) : kCap + 1;
        bool done = n <= kCap;
        uint64_t cut = 1;
        auto entry = [&](uint32_t i) { return l.list[i]; };
        const uint64_t first = place(top, 0), last = least > minus_inf() ? place(least, V - 1) : 1;
        auto share = [&](double w) {   // the weight that top-p asks for
            const double x = __builtin_ceil(ask.p * w);
            return x < 1.0 ? (uint64_t)1 : (uint64_t)x;
        };
        if (done) {
            uint64_t sum = 0;
            if (ask.by_k) {
                const bool ok = find(l, n, entry, last, first, true, ask.k);
                if (ok) {
                    cut = l.key;
                    sum = l.key_w;
                } else {
                    sum = l.total_w;
                }
                done = ok || holds_all;
                __syncthreads();
            }
            if (done && ask.by_p) {
                const bool ok = find(l, n, entry, last, first, false, share(ask.by_k ? (double)sum : Z * r.unit));
                if (ok) cut = max(cut, l.key);
                done = ok || holds_all;
                __syncthreads();
            }
        }
        if (done) {
            // draw from the list, by index
            uint64_t sum = 0;
            for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
                if (l.list[i] < cut || r.weight_of(logit_of(l.list[i])) < ask.least) l.w[i] = 0;
                sum += l.w[i];
            }
            sum = wave_scan_whole(sum);
            if (r.lane == 63) l.part_w[r.wave] = sum;
            __syncthreads();
            sum = 0;
            for (int i = 0; i < kWaves; ++i) sum += l.part_w[i];
            if (a.u) {
                const double x = u * (double)sum;
                const uint64_t target = min((uint64_t)x + 1, sum);
                __syncthreads();
                find(l, n, [&](uint32_t i) { return l.w[i] ? (l.list[i] & kIndexMask) + 1 : 0; }, kIndexMask + 2 - V, kIndexMask + 1,
                     false, target);
                if (threadIdx.x == 0) a.token[row] = (int)(kIndexMask + 1 - l.key);
            }
            if (threadIdx.x == 0) {
                out.per = r.unit / (double)sum;
                out.cut = cut;
                out.least = ask.least;
                sec.rows[row] = out;
            }
            return;
        }
        // over the row
        cut = 1;
        uint64_t sum = 0;
        if (ask.by_k) {
            const bool ok = r.find_row(true, ask.k);
            if (ok) cut = l.key;
            sum = ok ? l.key_w : l.total_w;
            __syncthreads();
        }
        if (ask.by_p) {
            if (r.find_row(false, share(ask.by_k ? (double)sum : Z * r.unit))) cut = max(cut, l.key);
            __syncthreads();
        }
        for (int t = threadIdx.x; t < tiles; t += kThreads) r.sums[t] = 0.0;
        __syncthreads();
        r.tiles_from(cut > 1 ? logit_of(cut) : minus_inf(), [&](const Tile<T>& x, int t) {
            double s = 0.0;
            x.each(t, r.lane, [&](float v, int i) {
                if (v > minus_inf() && place(v, i) >= cut) {
                    const double w = r.weight_of(v);
                    if (w >= ask.least) s += w;
                }
            });
            s = wave_sum(s);
            if (r.lane == 0) r.sums[t] = s;
        });
        __syncthreads();
        Z = r.total();
        out.cut = cut;
        out.least = ask.least;
    }
    if (threadIdx.x < 64) {
        const int token = a.u ? r.draw(u * Z, out.cut, out.least) : 0;
        if (threadIdx.x == 0) {
            if (a.u) a.token[row] = token;
            out.per = 1.0 / Z;
            sec.rows[row] = out;
        }
    }
}

// ---- probabilities -----------------------------------------------------------

template <typename T>
__global__ __launch_bounds__(256) void sample_probs_kernel(SampleArgs a) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = (a.V + kTile - 1) / kTile;
    const uint32_t groups = (uint32_t)(tiles + 3) / 4;
    const uint32_t row = blockIdx.x / groups;
    const int t = (int)(blockIdx.x % groups) * 4 + wave;
    if (t >= tiles) return;
    const Sections s = sections(a, tiles);
    const SampleRow r = s.rows[row];
    const float m = s.tops[(size_t)row * tiles + t];
    T* probs = static_cast<T*>(a.probs) + (size_t)row * a.V;
    Tile<T> x;
    if (m > minus_inf() && ((uint64_t)key_of(m) << kIndexBits | kIndexMask) >= r.cut && weight(m, r.top, r.scale) >= r.least) {
        x.load(static_cast<const T*>(a.logits) + (size_t)row * a.V, t, a.V, lane);
#pragma unroll
        for (int j = 0; j < Tile<T>::J; ++j)
#pragma unroll
            for (int e = 0; e < Tile<T>::M; ++e) {
                const float l = x.x[j][e];
                const int v = t * kTile + (j * 64 + lane) * Tile<T>::M + e;
                const double w = l > minus_inf() && place(l, min(v, a.V - 1)) >= r.cut ? weight(l, r.top, r.scale) : 0.0;
                x.x[j][e] = w >= r.least ? (float)(w * r.per) : 0.f;
            }
    } else {
#pragma unroll
        for (int j = 0; j < Tile<T>::J; ++j)
#pragma unroll
            for (int e = 0; e < Tile<T>::M; ++e) x.x[j][e] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < Tile<T>::J; ++j) {
        const int v = t * kTile + (j * 64 + lane) * Tile<T>::M;
        typename Vec16<T>::type y;
#pragma unroll
        for (int e = 0; e < Tile<T>::M; ++e) y[e] = from_f32<T>(x.x[j][e]);
        if (v + Tile<T>::M <= a.V) {
            __builtin_memcpy(probs + v, &y, 16);
        } else {
#pragma unroll
            for (int e = 0; e < Tile<T>::M; ++e)
                if (v + e < a.V) probs[v + e] = y[e];
        }
    }
}

template <typename T>
hipError_t launch_sample_t(const SampleArgs& a, hipStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const int64_t tiles = sample_tiles(a.V);
    const int fixed = (int)((sizeof(RowLds) + 15) / 16 * 16);
    const int most = fixed + (int)sample_tiles(KDA_MAX_VOCAB) * 12;
    const hipError_t e = raise_lds_limit_once(reinterpret_cast<const void*>(sample_rows_kernel<T>), most, done);
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)sample_groups(a.R, a.V)), block(256);
    sample_tiles_kernel<T><<<grid, block, 0, stream>>>(a);
    sample_rows_kernel<T><<<dim3((unsigned)a.R), dim3(kThreads), fixed + (size_t)tiles * 12, stream>>>(a);
    if (a.probs) sample_probs_kernel<T><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int dtype, hipStream_t stream) {
    return dtype == 0 ? launch_sample_t<float>(a, stream) : launch_sample_t<bf16>(a, stream);
}

}  // namespace kda
