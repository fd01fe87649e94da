// kda_tree_accept.hip -- verification of a tree of drafted tokens: the
// accepted path and the next token of every sequence, from the target's and
// the drafts' probabilities and given random numbers.
//
// Node r's residual after some refused children is max(p - c q, 0): with
// r_0 = p of mass Z_0 = 1 and r_{j+1} = max(r_j - Z_j q, 0) (a refusal takes
// the draft distribution out of what is left, normalised), nested maxima
// collapse as q >= 0, so c = Z_0 + ... + Z_j and one sum over the vocabulary
// per refusal gives the next Z.  It is only formed when another child of r
// is left to try; a chain never needs it.  Certain drafts (no q) need no sum
// at all: a refusal takes p(t) out.
//
// The walk is a few dozen scalar decisions: lane i of every wavefront holds
// node i's parent, token, random number and the two probabilities its test
// reads (all fetched at once), and the wavefronts take the same decisions
// side by side, so nothing is broadcast.  The bytes are in the last step:
// the row that the next token is drawn from, read once for the sum of every
// 1024-token tile (kept in LDS), and the one tile that holds the drawn
// position again.  Sums are fp64: the drawn index is a whole number that a
// rounding of the running sum must not move.
//
// What bounds it: 256 sequences over 160,000 fp32 tokens, chains with q: the
// two rows' bytes, 52 us, 6.3 TB/s.  A few sequences: one workgroup's latency
// (32,000 tokens 7.1 us) and then its fp64 arithmetic, five instructions per
// token with q and two without (160,000 tokens, one sequence: 15 and 12 us).
// Sharing a row out over workgroups in a second launch (sums, then the last
// one to arrive draws) took 17 us there and far more for more sequences, for
// the device-wide fences of every arrival.
#include "kda.h"
#include "kda_device.h"
#include "kda_tree_device.h"

namespace kda {

namespace {

constexpr int kTile = 1024;          // tokens of a tile: 16 per lane of a wavefront
constexpr int kPer = kTile / 64;
constexpr int kMaxTiles = KDA_MAX_VOCAB / kTile;
constexpr int kAcceptWaves = 16;

__device__ __forceinline__ double lane_value(double x, int lane) {
    union { double d; int w[2]; } v;
    v.d = x;
    v.w[0] = __builtin_amdgcn_readlane(v.w[0], lane);
    v.w[1] = __builtin_amdgcn_readlane(v.w[1], lane);
    return v.d;
}
// x of the lane that the data-parallel move `kCtrl` names, 0 where it names
// none or the lane's row of 16 is not in kRows
template <int kCtrl, int kRows>
__device__ __forceinline__ double moved(double x) {
    union { double d; int w[2]; } v;
    v.d = x;
    v.w[0] = __builtin_amdgcn_update_dpp(0, v.w[0], kCtrl, kRows, 0xf, false);
    v.w[1] = __builtin_amdgcn_update_dpp(0, v.w[1], kCtrl, kRows, 0xf, false);
    return v.d;
}
// inclusive prefix sum over the lanes: along the rows of 16 (shifts by 1, 2,
// 4, 8), then lane 15 of rows 0 and 2 to the row after, lane 31 to the upper half
__device__ __forceinline__ double wave_scan(double x) {
    x += moved<0x111, 0xf>(x);
    x += moved<0x112, 0xf>(x);
    x += moved<0x114, 0xf>(x);
    x += moved<0x118, 0xf>(x);
    x += moved<0x142, 0xa>(x);
    x += moved<0x143, 0xc>(x);
    return x;
}
__device__ __forceinline__ double wave_sum(double x) { return lane_value(wave_scan(x), 63); }

// 16 bytes of probabilities from an address that only its elements align
// (rows of an odd vocabulary)
template <typename T>
__device__ __forceinline__ typename Vec16<T>::type load16(const T* p) {
    typename Vec16<T>::type x;
    __builtin_memcpy(&x, p, 16);
    return x;
}

// What is left at a node: max(p - c q, 0), or p without the refused tokens
// (lanes of `gone`).
template <typename T, bool kQ>
struct Residual {
    const T* p;
    const T* q;       // kQ; read only where c > 0
    double c;
    uint64_t gone;    // !kQ
    int tok;          // this lane's token
    int V;

    __device__ __forceinline__ double weight(double pv, double qv) const {
        return __builtin_fmax(kQ ? pv - c * qv : pv, 0.0);   // (a NaN counts as 0)
    }
    // nodes whose tokens are refused and lie in `tile`
    __device__ __forceinline__ uint64_t gone_of(int tile) const {
        return kQ ? 0 : gone & __ballot(tok / kTile == tile);
    }
    static constexpr int M = Vec16<T>::N;   // tokens of 16 bytes
    typedef typename Vec16<T>::type vec;
    // tokens v0 .. v0 + M - 1 of a row (past the last one, that one again: loads
    // without branches are in flight together)
    template <bool kFull>
    __device__ __forceinline__ vec tokens(const T* row, int v0) const {
        if (kFull) return load16(row + v0);
        vec x;
#pragma unroll
        for (int e = 0; e < M; ++e) x[e] = row[min(v0 + e, V - 1)];
        return x;
    }
    // their weights (0 at and past V).  kAll: all of them lie in [0, V) and are
    // no refused tokens
    template <bool kAll, bool kWithQ>
    __device__ __forceinline__ void weights(int v0, vec pv, vec qv, uint64_t here, double (&w)[M]) const {
#pragma unroll
        for (int e = 0; e < M; ++e) {
            const float x = to_f32((T)pv[e]);
            w[e] = kWithQ ? weight((double)x, (double)to_f32((T)qv[e])) : (double)__builtin_fmaxf(x, 0.f);
            if (!kAll && v0 + e >= V) w[e] = 0.0;
        }
        if (!kQ && !kAll) {
            for (uint64_t g = here; g; g &= g - 1) {
                const int t = __builtin_amdgcn_readlane(tok, __builtin_ctzll(g));
#pragma unroll
                for (int e = 0; e < M; ++e)
                    if (v0 + e == t) w[e] = 0.0;
            }
        }
    }
    // f(tile, sum) for this wavefront's tiles, several in flight
    template <bool kWithQ, typename F>
    __device__ __forceinline__ void sums(int wave, int lane, F&& f) const {
        // (128 bytes of a lane; 256: the same to 5% slower)
        constexpr int kU = 128 / (kPer * (int)sizeof(T) * (kWithQ ? 2 : 1)), W = kAcceptWaves;
        auto at = [&](int t, int j) { return t * kTile + (j * 64 + lane) * M; };
        auto one = [&](int t) {   // with a refused token, or the vocabulary's end, in it
            const uint64_t here = gone_of(t);
            double x = 0.0;
#pragma unroll 1
            for (int j = 0; j < kPer / M; ++j) {
                const int v0 = at(t, j);
                const vec pv = tokens<false>(p, v0), qv = kWithQ ? tokens<false>(q, v0) : pv;
                double w[M];
                weights<false, kWithQ>(v0, pv, qv, here, w);
#pragma unroll
                for (int e = 0; e < M; ++e) x += w[e];
            }
            f(t, wave_sum(x));
        };
        const int full = V / kTile;
        for (int t0 = wave; t0 < full; t0 += kU * W) {
            const int count = min(kU, (full - t0 + W - 1) / W);
            vec pv[kU][kPer / M], qv[kU][kPer / M];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (u >= count) break;
#pragma unroll
                for (int j = 0; j < kPer / M; ++j) {
                    pv[u][j] = load16(p + at(t0 + u * W, j));
                    if (kWithQ) qv[u][j] = load16(q + at(t0 + u * W, j));
                }
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (u >= count) break;
                if (!kQ && gone && gone_of(t0 + u * W)) {
                    one(t0 + u * W);
                    continue;
                }
                double x = 0.0;
#pragma unroll
                for (int j = 0; j < kPer / M; ++j) {
                    double w[M];
                    weights<true, kWithQ>(0, pv[u][j], qv[u][j], 0, w);
#pragma unroll
                    for (int e = 0; e < M; ++e) x += w[e];
                }
                f(t0 + u * W, wave_sum(x));
            }
        }
        if (full * kTile < V && full % W == wave) one(full);
    }
    template <typename F>
    __device__ __forceinline__ void tile_sums(int wave, int lane, F&& f) const {
        if (kQ && c > 0.0) sums<kQ>(wave, lane, f);
        else sums<false>(wave, lane, f);
    }
    // the first token of `tile` at which `base` plus the tile's running sum
    // passes `target`; where rounding leaves none, its last one with weight
    __device__ __forceinline__ int find(int tile, double base, double target, int lane) const {
        const uint64_t here = gone_of(tile);
        const bool with_q = kQ && c > 0.0;
        const int v0 = tile * kTile + lane * kPer;   // a lane's tokens are consecutive
        vec pv[kPer / M], qv[kPer / M];
        if ((tile + 1) * kTile <= V) {
#pragma unroll
            for (int j = 0; j < kPer / M; ++j) {
                pv[j] = tokens<true>(p, v0 + j * M);
                if (with_q) qv[j] = tokens<true>(q, v0 + j * M);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPer / M; ++j) {
                pv[j] = tokens<false>(p, v0 + j * M);
                if (with_q) qv[j] = tokens<false>(q, v0 + j * M);
            }
        }
        double w[kPer], s = 0.0;
#pragma unroll
        for (int j = 0; j < kPer / M; ++j) {
            double x[M];
            if (with_q) weights<false, kQ>(v0 + j * M, pv[j], qv[j], here, x);
            else weights<false, false>(v0 + j * M, pv[j], qv[j], here, x);
#pragma unroll
            for (int e = 0; e < M; ++e) {
                w[j * M + e] = x[e];
                s += x[e];
            }
        }
        const double incl = base + wave_scan(s);
        double run = __shfl_up(incl, 1, 64);
        if (lane == 0) run = base;
        int first = -1, last = -1;
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            run += w[e];
            if (w[e] > 0.0) {
                last = v0 + e;
                if (first < 0 && run > target) first = v0 + e;
            }
        }
        const uint64_t hit = __ballot(first >= 0), any = __ballot(last >= 0);
        if (hit) return __builtin_amdgcn_readlane(first, __builtin_ctzll(hit));
        if (any) return __builtin_amdgcn_readlane(last, 63 - __builtin_clzll(any));
        return min(tile * kTile, V - 1);
    }
};

template <typename T, bool kQ>
__global__ __launch_bounds__(64 * kAcceptWaves) void tree_accept_kernel(TreeAcceptArgs a) {
    __shared__ double tiles[kMaxTiles];
    __shared__ double part[kAcceptWaves];
    const int64_t b = blockIdx.x;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int N = a.N, V = a.V, ntile = (V + kTile - 1) / kTile;
    const int n = tree_count(a.n_node, b, N);
    int32_t* path = a.path + b * N;
    if (n == 0) {
        if (wave == 0) {
            if (lane < N) path[lane] = -1;
            if (lane == 0) {
                a.n_path[b] = 0;
                a.next_token[b] = -1;
            }
        }
        return;
    }

    // node i in lane i
    const bool node = lane >= 1 && lane < n;
    const int par = node ? tree_parent(a.parent, b, N, lane) : -1;
    const int tok = node ? a.tokens[b * N + lane] : -1;
    const double u = lane < n ? (double)a.u[b * N + lane] : 0.0;
    const bool sound = par >= 0 && tok >= 0 && tok < V;
    const T* P = static_cast<const T*>(a.p) + (size_t)b * N * V;
    const T* Q = kQ ? static_cast<const T*>(a.q) + (size_t)b * (N - 1) * V : nullptr;
    const double pt = sound ? (double)to_f32(P[(size_t)par * V + tok]) : 0.0;
    const double qt = kQ && sound ? (double)to_f32(Q[(size_t)par * V + tok]) : 0.0;
    const uint64_t sound_mask = __ballot(sound);

    Residual<T, kQ> res;
    res.V = V;
    res.tok = tok;
    res.c = 0.0;
    res.gone = 0;
    auto at_node = [&](int r) {
        res.p = P + (size_t)r * V;
        res.q = kQ ? Q + (size_t)min(r, N - 2) * V : nullptr;
    };
    at_node(0);
    int at = 0, m = 1, mine = lane == 0 ? 0 : -1;   // lane j: path[j]
    double Z = 1.0;
    uint64_t todo = __ballot(par == 0);
    while (todo) {
        const int i = __builtin_ctzll(todo);
        todo &= todo - 1;
        if (!((sound_mask >> i) & 1)) continue;
        const double ui = lane_value(u, i), pi = lane_value(pt, i);
        bool ok;
        if (kQ) {
            const double qi = lane_value(qt, i);
            ok = ui * qi * Z < res.weight(pi, qi);
            if (!ok) {
                res.c += Z;
                if (todo) {
                    double s = 0.0;
                    res.template sums<kQ>(wave, lane, [&](int, double x) { s += x; });
                    __syncthreads();   // (part of the sum before is read)
                    if (lane == 0) part[wave] = s;
                    __syncthreads();
                    Z = 0.0;
#pragma unroll
                    for (int w = 0; w < kAcceptWaves; ++w) Z += part[w];
                }
            }
        } else {
            const int ti = __builtin_amdgcn_readlane(tok, i);
            const bool again = (__ballot(tok == ti) & res.gone) != 0;
            const double w = again ? 0.0 : res.weight(pi, 0.0);
            ok = ui * Z < w;
            if (!ok) {
                res.gone |= (uint64_t)1 << i;
                Z -= w;
            }
        }
        if (ok) {
            at = i;
            if (lane == m) mine = i;
            ++m;
            at_node(at);
            res.c = 0.0;
            res.gone = 0;
            Z = 1.0;
            todo = __ballot(par == at);
        }
    }
    if (wave == 0) {
        if (lane < N) path[lane] = mine;
        if (lane == 0) a.n_path[b] = m;
    }

    // the next token: from the residual, or from p where nothing is left
    for (int again = 0; again < 2; ++again) {
        res.tile_sums(wave, lane, [&](int t, double x) {
            if (lane == 0) tiles[t] = x;
        });
        __syncthreads();
        // every wavefront: the running sum over the tiles
        double total = 0.0;
        for (int t0 = 0; t0 < ntile; t0 += 64)
            total += wave_sum(t0 + lane < ntile ? tiles[t0 + lane] : 0.0);
        if (total > 0.0 || again) {
            if (wave == 0) {
                const double target = lane_value(u, 0) * total;
                int tile = -1, filled = -1;   // the tile that passes the target; the last with weight
                double base = 0.0, run = 0.0;
                for (int t0 = 0; t0 < ntile && tile < 0; t0 += 64) {
                    const double s = t0 + lane < ntile ? tiles[t0 + lane] : 0.0;
                    const double incl = run + wave_scan(s);
                    const uint64_t hit = __ballot(s > 0.0 && incl > target), any = __ballot(s > 0.0);
                    if (any) filled = t0 + 63 - __builtin_clzll(any);
                    if (hit) {
                        const int l = __builtin_ctzll(hit);
                        tile = t0 + l;
                        base = l ? lane_value(incl, l - 1) : run;
                    }
                    run = lane_value(incl, 63);
                }
                if (tile < 0) {   // (the target rounded past the end: the last token with weight)
                    tile = max(filled, 0);
                    base = -1e300;
                }
                const int next = res.find(tile, base, target, lane);
                if (lane == 0) a.next_token[b] = next;
            }
            break;
        }
        __syncthreads();
        res.c = 0.0;
        res.gone = 0;
    }
}

template <typename T>
hipError_t launch_tree_accept_t(const TreeAcceptArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)a.B), block(64 * kAcceptWaves);
    if (a.q) tree_accept_kernel<T, true><<<grid, block, 0, stream>>>(a);
    else tree_accept_kernel<T, false><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_tree_accept(const TreeAcceptArgs& a, int dtype, hipStream_t stream) {
    return dtype == 0 ? launch_tree_accept_t<float>(a, stream) : launch_tree_accept_t<bf16>(a, stream);
}

}  // namespace kda
