// prefill_plan.cuh -- the work of a prefill call cut into equal ranges, one a block, from
// lengths in device memory.
//
// The rows of a request and key head are its tokens' query heads, token after token: row
// m is token m / G, head m % G of the key head.  A tile is TM rows; a step is KT key
// positions (aligned in the request) against a tile.  The steps of all tiles, request after
// request, key head after key head, tile after tile, with `over` units in front of each
// tile for its queries and outputs, are cut into equal ranges; a tile that a range's
// border cuts leaves partial sums, which a second kernel joins in the order of the ranges.
// So every block has the same work, whatever the lengths, and a captured call follows them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "la_common.cuh"
#include "la_launch.h"

namespace la {
namespace prefill {

struct Args {
    PrefillShape s;
    int G, least;  // least: units of a range at least
    const int *table, *lens, *starts;
    float* lse;
    int fill;
    float* part;   // [blocks][2][TM][D] output sums of cut tiles
    float2* ml;    // [blocks][2][TM] their maxima (to base 2) and sums
    int4* desc;    // [blocks][2] a cut tile that starts in the block's range: {request, key head, tile, 0}, {ranges, -, -, -}
    unsigned* status;
};

// A request's rows and positions made valid.
struct Request {
    int first, n, cached;  // its first row of T, its tokens (0: none to do), positions before them
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
        first = q.cached + m0 / p.G;
        last = q.cached + (m1 - 1) / p.G;
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

// Walks over a range; every role of the block has its own.
template <int TM, int KT, int OVER>
struct Walk {
    int r, kh, mt, off;   // the place: units into tile mt
    int64_t left;         // units still to do
    Request q;
    __device__ __forceinline__ Walk(const Args& p, int r_, int kh_, int mt_, int off_, int64_t left_)
        : r(r_), kh(kh_), mt(mt_), off(off_), left(left_), q(p, r_) {}
    // The next segment with a step; false at the range's end.
    __device__ __forceinline__ bool next(const Args& p, Segment& g) {
        while (left > 0) {
            const int rows = q.rows(p), m0 = mt * TM;
            const Keys<KT> k(p, q, m0, min(m0 + TM, rows));
            const int units = k.k1 - k.k0 + OVER;
            const int take = static_cast<int>(min(static_cast<int64_t>(units - off), left));
            g = {r, kh, m0, rows, max(off - OVER, 0), off + take - OVER, k.k1 - k.k0};
            left -= take;
            off += take;
            if (off == units && left > 0) {  // on to the next tile
                off = 0;
                if (++mt == tile_count<TM>(rows)) {
                    mt = 0;
                    if (++kh == p.s.Hkv) {
                        kh = 0;
                        do {
                            ++r;
                            if (r >= p.s.R) return g.b > g.a ? (left = 0, true) : false;
                            q = Request(p, r);
                        } while (q.rows(p) == 0);
                    }
                }
            }
            if (g.b > g.a) return true;
        }
        return false;
    }
};

// Block-wide inclusive sums over threads (s holds NT words).
template <int NT>
__device__ __forceinline__ void block_sums(int64_t x, int64_t* s) {
    const int tid = threadIdx.x, lane = tid & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    s[tid] = x;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < tid / 32; ++w) before += s[w * 32 + 31];
    __syncthreads();
    s[tid] = x + before;
    __syncthreads();
}

// Number of entries of s[0 .. NT) that are <= x; s does not decrease.
template <int NT>
__device__ __forceinline__ int count_to(const int64_t* s, int64_t x) {
    int lo = 0, hi = NT;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s[mid] <= x) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// Where a block's range starts, found by all its threads from the lengths.
struct Start {
    int r, kh, mt, off;
    int64_t left, per;   // units of the range; of every range but the last
    bool any;
};

template <int TM, int KT, int OVER, int NT>
struct Planner {
    int64_t tiles[NT], units[NT];  // inclusive sums: of tiles over chunks of requests, of units over chunks of tiles
    Start start;

    __device__ __forceinline__ static int chunk(int n) { return (n + NT - 1) / NT; }

    // Request and tile of tile number i (below the number of tiles).
    __device__ __forceinline__ void tile_at(const Args& p, int64_t i, int& r, int& mt) const {
        const int c = count_to<NT>(tiles, i);
        int64_t rest = i - (c ? tiles[c - 1] : 0);
        for (r = min(c * chunk(p.s.R), p.s.R - 1); r < p.s.R - 1; ++r) {
            const int n = tile_count<TM>(Request(p, r).rows(p));
            if (rest < n) break;
            rest -= n;
        }
        mt = static_cast<int>(rest);
    }
    __device__ __forceinline__ static int units_of(const Args& p, const Request& q, int mt) {
        const int rows = q.rows(p);
        const Keys<KT> k(p, q, mt * TM, min(mt * TM + TM, rows));
        return k.k1 - k.k0 + OVER;
    }
    // Units of the tiles before number i, by a warp.
    __device__ __forceinline__ int64_t before(const Args& p, int64_t i, int64_t per) const {
        const int64_t c = i / per;
        int64_t x = 0;
        for (int64_t j = c * per + (threadIdx.x & 31); j < i; j += 32) {
            int r, mt;
            tile_at(p, j, r, mt);
            x += units_of(p, Request(p, r), mt);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        return x + (c ? units[c - 1] : 0);
    }
    // The tile with unit x of the sums over tiles, and the units before it, by a warp.
    __device__ __forceinline__ int64_t find(const Args& p, int64_t x, int64_t count, int64_t per, int64_t& base) const {
        const int c = count_to<NT>(units, x), lane = threadIdx.x & 31;
        base = c ? units[c - 1] : 0;
        for (int64_t i = c * per;; i += 32) {
            int64_t u = 0;
            if (i + lane < count) {
                int r, mt;
                tile_at(p, i + lane, r, mt);
                u = units_of(p, Request(p, r), mt);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, u, o);
                if (lane >= o) u += y;
            }
            const int n = __popc(__ballot_sync(0xffffffffu, base + u <= x));
            const int64_t skip = __shfl_sync(0xffffffffu, u, n ? n - 1 : 0);
            if (n) base += skip;
            if (n < 32 || i + 32 >= count) return min(i + n, count - 1);
        }
    }

    // Fills `start`, by all threads.
    __device__ __forceinline__ void run(const Args& p) {
        const int tid = threadIdx.x;
        const int each = chunk(p.s.R);
        int64_t mine = 0;
        bool bad = false;
        for (int i = 0; i < each; ++i) {
            const int r = tid * each + i;
            if (r >= p.s.R) break;
            const Request q(p, r);
            bad |= q.bad;
            mine += tile_count<TM>(q.rows(p));
        }
        if (bad && blockIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
        block_sums<NT>(mine, tiles);
        const int64_t count = tiles[NT - 1], per = (count + NT - 1) / NT;
        mine = 0;
        if (static_cast<int64_t>(tid) * per < count) {
            int r, mt;
            tile_at(p, tid * per, r, mt);
            Request q(p, r);
            int n = tile_count<TM>(q.rows(p));
            const int64_t stop = min(count, (tid + 1) * per);
            for (int64_t i = tid * per;;) {
                mine += units_of(p, q, mt);
                if (++i == stop) break;
                if (++mt == n) {
                    mt = 0;
                    do {
                        q = Request(p, ++r);
                        n = tile_count<TM>(q.rows(p));
                    } while (n == 0 && r < p.s.R - 1);
                }
            }
        }
        block_sums<NT>(mine, units);
        if (tid < 32) {
            const int64_t total = units[NT - 1] * p.s.Hkv;
            const int64_t range = max((total + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(p.least));
            const int64_t u0 = range * blockIdx.x;
            Start st = {};
            st.per = range;
            st.any = u0 < total;
            if (st.any) {
                st.left = min(range, total - u0);
                int64_t base;
                int r, mt;
                tile_at(p, find(p, u0 / p.s.Hkv, count, per, base), r, mt);  // a tile of the request
                const int c = r / each;
                int64_t first = c ? tiles[c - 1] : 0;  // its first tile's number
                for (int i = c * each; i < r; ++i) first += tile_count<TM>(Request(p, i).rows(p));
                const int64_t w0 = before(p, first, per);
                const int64_t w1 = before(p, first + tile_count<TM>(Request(p, r).rows(p)), per);
                const int64_t in = u0 - w0 * p.s.Hkv, one = w1 - w0;
                st.kh = static_cast<int>(in / one);
                const int64_t x = w0 + in - st.kh * one;
                const int64_t tile = find(p, x, count, per, base);
                st.r = r;
                st.mt = static_cast<int>(tile - first);
                st.off = static_cast<int>(x - base);
            }
            if (tid == 0) start = st;
        }
        __syncthreads();
    }
};

// Ranges that the tile of segment g touches when it starts in this block's range: `done` units of
// the range were taken with the segment's last one.
template <int OVER>
__device__ __forceinline__ int ranges_of(const Segment& g, int64_t done, int64_t per) {
    const int64_t end = done + (g.steps - g.b);  // the tile's end, in units from the range's start
    return static_cast<int>((end + per - 1) / per);
}

}  // namespace prefill
}  // namespace la
