// prefill_plan.cuh -- the work of a prefill call cut into ranges, one a block, from lengths
// in device memory.
//
// The rows of a request and key head are its tokens' query heads, token after token: row
// m is token m / G, head m % G of the key head.  A tile is TM rows; a step is KT key
// positions (aligned in the request) against a tile.  A tile's cost is taken as the
// positions that its last row sees, and a constant for its queries and outputs: a formula
// whose sums over tiles are one too, so that a thread sums up a request, and a block finds
// the borders of its range in a few steps, whatever the lengths.  The costs of all tiles,
// request after request, key head after key head, are cut into equal ranges, the border
// inside a tile set back to a whole step.  A tile that a border cuts leaves partial sums, which
// a second kernel joins in the order of the ranges.  So all blocks have the same work but for a
// step, and a captured call follows the lengths.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "la_common.cuh"
#include "la_launch.h"

namespace la {
namespace prefill {

struct Args {
    PrefillShape s;
    int G, tile_tokens;       // query heads a key head; tokens from a tile of rows to the next, 1 at least
    unsigned g_mul, g_shift;  // m / G = m g_mul >> g_shift for m < 2^31 (set_group)
    const int *table, *lens, *starts;
    float* lse;
    int fill;
    float* part;   // [blocks][2][TM][D] output sums of cut tiles
    float2* ml;    // [blocks][2][TM] their maxima (to base 2) and sums
    int4* desc;    // [blocks][2] the cut tile whose first step is in the block's range: {request, key head, first row, rows}, {ranges, -, -, -}
    unsigned* status;
};

// Rounding 2^s / G up with s = 31 + ceil(log2 G) is off by less than 2^(s - 31) / 2^s of a
// quotient below 2^31, so the product's floor is the quotient's.
inline void set_group(Args& p, int G, int tile_rows) {
    int log = 0;
    p.tile_tokens = tile_rows / G > 1 ? tile_rows / G : 1;
    while ((1 << log) < G) ++log;  // G < 2^30
    p.G = G;
    p.g_shift = 31 + log;
    p.g_mul = static_cast<unsigned>((1ull << p.g_shift) / G + 1);
}
__device__ __forceinline__ int token_of(const Args& p, int m) {  // of row m
    return static_cast<int>(static_cast<uint64_t>(static_cast<unsigned>(m)) * p.g_mul >> p.g_shift);
}

// A request's rows and positions made valid.
struct Request {
    int first, n, cached;  // its first row of T, its tokens, positions before them
    int end;               // positions that its table has room for
    bool bad, pad;
    __device__ __forceinline__ Request(const Args& p, int r) {
        const int a = p.starts[r], b = p.starts[r + 1], len = p.lens[r];
        first = min(max(a, 0), p.s.T);
        n = min(max(b, first), p.s.T) - first;
        pad = len < 0;
        cached = max(len, 0);
        end = p.s.max_pages << p.s.log2p;  // below 2^30
        bad = a != first || b != first + n || (!pad && n > 0 && (cached > end || n > end - cached));
        cached = min(cached, end);
    }
    __device__ __forceinline__ int rows(const Args& p) const { return pad ? 0 : n * p.G; }
};

// The keys that rows [m0, m1) of a request see: positions [lo, hi) in tiles [k0, k1) of KT.
template <int KT>
struct Keys {
    int first, last;  // positions of the first and the last row
    int lo, hi, k0, k1;
    __device__ __forceinline__ Keys(const Args& p, const Request& q, int m0, int m1) {
        first = q.cached + token_of(p, m0);
        last = q.cached + token_of(p, m1 - 1);
        lo = p.s.window ? max(first - p.s.window + 1, 0) : 0;
        hi = min(last + 1, q.end);
        k0 = min(lo, hi) / KT;
        k1 = max((hi + KT - 1) / KT, k0 + 1);
    }
};

template <int TM>
__device__ __forceinline__ int tile_count(int rows) { return (rows + TM - 1) / TM; }

// A part of a block's range in one tile: steps [a, b) of the tile's `steps`.
struct Segment {
    int r, kh, m0, rows;  // request, key head, first row, rows of the request
    int a, b, steps;
    __device__ __forceinline__ bool whole() const { return a == 0 && b == steps; }
};

// A border of a range: step a of tile mt of a request and key head.
struct Place {
    int r, kh, mt, a;
};
struct Range {
    Place from, to;     // to.r = R: the end of all
    int ranges;         // that tile `to` touches, from this block on
    int any;
};

// Walks over a range; every role of the block has its own.
template <int TM, int KT>
struct Walk {
    Place at, to;
    Request q;
    __device__ __forceinline__ Walk(const Args& p, const Range& g) : at(g.from), to(g.to), q(p, g.from.r) {}
    // The next segment with a step; false at the range's end.
    __device__ __forceinline__ bool next(const Args& p, Segment& g) {
        while (at.r < p.s.R) {
            const int rows = q.rows(p), m0 = at.mt * TM;
            const bool last = at.r == to.r && at.kh == to.kh && at.mt == to.mt;
            const Keys<KT> k(p, q, m0, min(m0 + TM, rows));
            g = {at.r, at.kh, m0, rows, at.a, last ? to.a : k.k1 - k.k0, k.k1 - k.k0};
            if (last) {
                at.r = p.s.R;
            } else {  // on to the next tile
                at.a = 0;
                if ((++at.mt) * static_cast<int64_t>(TM) >= rows) {
                    at.mt = 0;
                    if (++at.kh == p.s.Hkv) {
                        at.kh = 0;
                        while (++at.r < p.s.R) {
                            q = Request(p, at.r);
                            if (q.rows(p)) break;
                        }
                    }
                }
            }
            if (g.b > g.a) return true;
        }
        return false;
    }
};

__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {  // of numbers that mostly have 32 bits
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The cost of a request's tiles: cost(mt) of the tiles before mt.
template <int TM, int KT>
struct Cost {
    // Of a tile's queries, outputs and of the step that its border cuts: as much as 1.5 steps.
    static constexpr int kTile = KT + KT / 2;
    // A tile of few steps is not cut, and the others by four steps at least: joining costs more than
    // they would take.  And a range is at least about a small tile, so that it has one.
    static constexpr int kWhole = 12, kCut = 4, kLeast = KT * 5 / 2;
    int tiles, each;      // positions from a tile to the next
    int64_t base, limit;  // cost of tile i: min(base + each i, limit)
    int grow;             // tiles whose cost grows
    __device__ __forceinline__ Cost(const Args& p, const Request& q) {
        tiles = tile_count<TM>(q.rows(p));
        each = p.tile_tokens;
        base = static_cast<int64_t>(q.cached) + each + kTile;
        limit = p.s.window ? static_cast<int64_t>(p.s.window) + each + kTile : INT64_MAX;
        grow = p.s.window == 0 ? tiles : limit <= base ? 0 : static_cast<int>(min(divide(limit - base, each) + 1, static_cast<int64_t>(tiles)));
    }
    __device__ __forceinline__ int64_t operator()(int mt) const {
        const int64_t g = min(mt, grow);
        return g * base + g * (g - 1) / 2 * each + (mt > grow ? (mt - grow) * limit : 0);
    }
};

// Finds a block's range, by all its NT threads.
template <int TM, int KT, int NT>
struct Planner {
    int64_t sums[NT];     // inclusive sums of costs over chunks of requests
    int64_t warps[NT / 32];
    Range range;
    int64_t tile_end;     // cost up to the end of tile range.to

    // The border at cost u < total, by a warp; `end` gets the cost up to its tile's end.
    __device__ __forceinline__ Place locate(const Args& p, int64_t u, int64_t& end) const {
        const int lane = threadIdx.x & 31, each = (p.s.R + NT - 1) / NT;
        int c = __popc(__ballot_sync(0xffffffffu, lane < NT / 32 && sums[min(lane, NT / 32 - 1) * 32 + 31] <= u));
        c = min(c, NT / 32 - 1);
        c = 32 * c + min(__popc(__ballot_sync(0xffffffffu, sums[32 * c + lane] <= u)), 31);
        int64_t before = c ? sums[c - 1] : 0, total = 0;
        int r = c * each;
        for (;; r += 32) {  // 32 requests at once
            int64_t x = 0;
            if (r + lane < min((c + 1) * each, p.s.R)) {
                const Cost<TM, KT> cost(p, Request(p, r + lane));
                x = cost(cost.tiles) * p.s.Hkv;
            }
            int64_t s = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += y;
            }
            const int n = __popc(__ballot_sync(0xffffffffu, before + s <= u));
            if (n == 32 && r + 32 < (c + 1) * each) {
                before += __shfl_sync(0xffffffffu, s, 31);
                continue;
            }
            const int i = min(n, 31);
            total = __shfl_sync(0xffffffffu, x, i);
            before += __shfl_sync(0xffffffffu, s, i) - total;
            r = min(r + i, p.s.R - 1);
            break;
        }
        const Request q(p, r);
        const Cost<TM, KT> cost(p, q);
        const int64_t one = max(cost(cost.tiles), static_cast<int64_t>(1));
        const int64_t kh = min(divide(u - before, one), static_cast<int64_t>(p.s.Hkv - 1));
        const int64_t x = u - before - kh * one;
        int lo = 0, hi = max(cost.tiles, 1);  // cost(lo) <= x < cost(hi)
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32;
            const int n = __popc(__ballot_sync(0xffffffffu, lo + (lane + 1) * static_cast<int64_t>(step) < hi && cost(lo + (lane + 1) * step) <= x));
            lo += n * step;
            hi = min(hi, lo + step);
        }
        const int rows = q.rows(p);
        const Keys<KT> k(p, q, lo * TM, min(lo * TM + TM, rows));
        const int64_t c0 = cost(lo), c1 = cost(lo + 1);
        end = before + kh * one + c1;
        int a = 0;
        if (k.k1 - k.k0 >= Cost<TM, KT>::kWhole)
            a = static_cast<int>(divide((x - c0) * (k.k1 - k.k0), max(c1 - c0, static_cast<int64_t>(1)))) / Cost<TM, KT>::kCut * Cost<TM, KT>::kCut;
        return {r, static_cast<int>(kh), lo, a};
    }

    __device__ __forceinline__ void run(const Args& p) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, each = (p.s.R + NT - 1) / NT;
        int64_t x = 0;
        bool bad = false;
        for (int i = 0; i < each; ++i) {
            const int r = tid * each + i;
            if (r >= p.s.R) break;
            const Request q(p, r);
            bad |= q.bad;
            const Cost<TM, KT> cost(p, q);
            x += cost(cost.tiles);
        }
        x *= p.s.Hkv;
        if (bad && blockIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warps[warp] = x;
        __syncthreads();
        int64_t before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) {
            const int64_t y = warps[w];
            before += w < warp ? y : 0;
            total += y;
        }
        sums[tid] = x + before;
        __syncthreads();
        if (warp < 2) {  // one finds the first border, one the last
            const int64_t per = max(divide(total + gridDim.x - 1, gridDim.x), static_cast<int64_t>(Cost<TM, KT>::kLeast));
            const int64_t u = per * (blockIdx.x + warp);
            Place at = {p.s.R, 0, 0, 0};
            int64_t end = 0;
            if (u < total) at = locate(p, u, end);
            if (lane == 0) {
                if (warp == 0) {
                    range.from = at;
                    range.any = u < total;
                } else {
                    range.to = at;
                    range.ranges = u < total ? static_cast<int>(divide(end - 1, per)) - static_cast<int>(blockIdx.x) + 1 : 0;
                }
            }
        }
        __syncthreads();
    }
};

}  // namespace prefill
}  // namespace la
