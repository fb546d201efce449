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
    float2* ml;    // [blocks][2][TM] their maxima (to base 2) and sums; a negative sum: no part
    int4* desc;    // [blocks][2] the cut tile whose first step is in the block's range: {request, key head, first row, rows}, {ranges, -, -, -}
    unsigned* status;
    int withhold;    // test hook: a block that gets no queries (-1: none), and the polls of its wait for them
    unsigned limit;
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
    int none;           // the starts go back: no request is done
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
    // Of a tile's queries, outputs and of the step that its border cuts: as much as 192 positions.
    static constexpr int kTile = 192;
    // A tile of few steps is not cut, and the others by four steps at least: joining costs more than they
    // would take (bf16, 4 short requests: 15 us, 27 us cut by the step).  And a range is at least about a small tile, so that it has one.
    static constexpr int kWhole = KT == 128 ? 12 : 16, kCut = 4, kLeast = 320;
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

// Finds a block's range, by all its NT threads.  What it costs is paid by the smallest calls, and it
// is code that runs once: so sums over warps and the search in them are left to the two warps that look for borders.
template <int TM, int KT, int NT>
struct Planner {
    static_assert(NT / 32 <= 32, "a lane a warp");
    int64_t sums[NT];     // of costs over chunks of requests, inclusive within a warp
    int64_t warps[NT / 32];
    Range range;

    __device__ __forceinline__ static int64_t scan(int64_t x, int lane) {  // inclusive, over a warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        return x;
    }

    // The border at cost u < total, by a warp, from the sum `s` of the costs of lane's and earlier warps' chunks; `end`
    // gets the cost up to its tile's end.
    __device__ __forceinline__ Place locate(const Args& p, int64_t u, int64_t s, int64_t& end) const {
        const int lane = threadIdx.x & 31, each = (p.s.R + NT - 1) / NT;
        // the warp, the chunk, and with more than one request in it the request whose cost passes u
        const int w = min(__popc(__ballot_sync(0xffffffffu, s <= u)), NT / 32 - 1);
        int64_t before = w ? __shfl_sync(0xffffffffu, s, max(w - 1, 0)) : 0;
        s = before + sums[32 * w + lane];
        const int c = min(__popc(__ballot_sync(0xffffffffu, s <= u)), 31);
        if (c) before = __shfl_sync(0xffffffffu, s, c - 1);
        int r = (32 * w + c) * each;
        const int r1 = min(r + each, p.s.R);
        while (each > 1) {  // 32 requests at once
            int64_t x = 0;
            if (r + lane < r1) {
                const Cost<TM, KT> cost(p, Request(p, r + lane));
                x = cost(cost.tiles) * p.s.Hkv;
            }
            x = before + scan(x, lane);
            const int n = __popc(__ballot_sync(0xffffffffu, x <= u));
            if (n) before = __shfl_sync(0xffffffffu, x, n - 1);
            r += n;
            if (n < 32 || r >= r1) break;
        }
        r = min(r, p.s.R - 1);
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
        bool bad = false, back = false;
        for (int i = 0; i < each; ++i) {
            const int r = tid * each + i;
            if (r >= p.s.R) break;
            const Request q(p, r);
            bad |= q.bad;
            back |= p.starts[r + 1] < p.starts[r];
            const Cost<TM, KT> cost(p, q);
            x += cost(cost.tiles);
        }
        x = scan(x * p.s.Hkv, lane);
        sums[tid] = x;
        if (lane == 31) warps[warp] = x;
        if (bad && blockIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
        // Starts that go back can name more rows than there are.  Nothing is done, however long that would take.
        const bool none = __syncthreads_or(back);
        if (warp < 2) {  // one finds the first border, one the last
            const int64_t s = scan(lane < NT / 32 && !none ? warps[min(lane, NT / 32 - 1)] : 0, lane);
            const int64_t total = __shfl_sync(0xffffffffu, s, 31);
            const int64_t per = max(divide(total + gridDim.x - 1, gridDim.x), static_cast<int64_t>(Cost<TM, KT>::kLeast));
            const int64_t u = per * (blockIdx.x + warp);
            Place at = {p.s.R, 0, 0, 0};
            int64_t end = 0;
            if (u < total) at = locate(p, u, s, end);
            if (lane == 0) {
                if (warp == 0) {
                    range.from = at;
                    range.any = u < total;
                    range.none = none;
                } else {
                    range.to = at;
                    range.ranges = u < total ? static_cast<int>(divide(end - 1, per)) - static_cast<int>(blockIdx.x) + 1 : 0;
                }
            }
        }
        __syncthreads();
    }
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The columns of [i, i + 32), a bit each, in which a row sees a value that is not finite in a key
// tile, if that is one in which such values were replaced: one that some row from position
// `first` to `last` sees in part.  COMMON: positions that all rows see were replaced too.
template <typename T, int D, int KT, bool COMMON>
__device__ __noinline__ uint32_t odd_columns(const Args& p, const T* V, int r, int kh, int first, int last, int end,
                                             int tile, int from, int pos, int i) {
    const int x0 = tile * KT, mask = (1 << p.s.log2p) - 1;
    const int* table = p.table + static_cast<int64_t>(r) * p.s.max_pages;
    uint32_t bits = 0;
    bool all = x0 + KT - 1 <= first && (p.s.window == 0 || x0 > last - p.s.window) && x0 + KT <= end;
    for (int x = x0; all && x < x0 + KT; x += mask + 1)
        all = static_cast<unsigned>(table[x >> p.s.log2p]) < static_cast<unsigned>(p.s.num_pages);
    if (all) return 0;
    for (int x = max(x0, max(from + 1, 0)); x < min(x0 + KT, min(pos + 1, end)); ++x) {
        const int page = table[x >> p.s.log2p];
        if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.s.num_pages)) continue;
        if (!COMMON && x <= first && (p.s.window == 0 || x > last - p.s.window)) continue;
        const T* v = V + (((static_cast<int64_t>(page) * p.s.Hkv + kh) << p.s.log2p) + (x & mask)) * D + i;
        for (int y = 0; y < 32; ++y)
            if (!(fabsf(to_f<T>(v[y])) < INFINITY)) bits |= 1u << y;
    }
    return bits;
}

// Joins the partial sums of the cut tile that starts in range blockIdx.x: a warp a row.
constexpr int kJoinWarps = 8, kJoinRows = 32;
template <typename T, int D, int TM>
__global__ void __launch_bounds__(kJoinWarps * 32) prefill_join_kernel(const Args p, T* __restrict__ out) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int ranges = p.desc[2 * blockIdx.x + 1].x;
    if (ranges == 0) return;
    const int4 d = p.desc[2 * blockIdx.x];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Request rq(p, d.x);
    constexpr int E = D / 32, N = 4;
    for (int i = warp; i < kJoinRows; i += kJoinWarps) {
        const int row = blockIdx.y * kJoinRows + i, m = d.z + row;
        if (m >= d.w) return;
        float top = -INFINITY, sum = 0.f, o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        for (int x0 = 0; x0 < ranges; x0 += N) {
            float2 ml[N];
            float v[N][E];
#pragma unroll
            for (int x = 0; x < N; ++x) {
                const int64_t at = (2 * (static_cast<int64_t>(blockIdx.x) + x0 + x) + (x0 + x == 0 ? 1 : 0)) * TM + row;
                ml[x] = x0 + x < ranges ? p.ml[at] : make_float2(-INFINITY, -1.f);
#pragma unroll
                for (int e = 0; e < E; ++e) v[x][e] = x0 + x < ranges ? p.part[at * D + lane + 32 * e] : 0.f;
            }
#pragma unroll
            for (int x = 0; x < N; ++x) {
                const float y = fmaxf(top, ml[x].x);
                const float f = top == y ? 1.f : exp2_approx(top - y);
                // a part whose scores are NaN carries them on; what is infinite or NaN in a part comes through a factor
                // of 0 too, as it does in a tile that is not cut; what a block without a part has not written does not
                const float h = ml[x].x == -INFINITY ? (ml[x].y != ml[x].y ? 1.f : 0.f) : ml[x].x == y ? 1.f : exp2_approx(ml[x].x - y);
                const bool none = ml[x].y < 0.f;
                sum = sum * f + ml[x].y * h;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = o[e] * f + (none ? 0.f : v[x][e] * h);
                top = y;
            }
        }
        const bool good = sum > 0.f || sum != sum;
        const int token = token_of(p, m);
        const int64_t at = (static_cast<int64_t>(rq.first) + token) * p.s.Hq + static_cast<int64_t>(d.y) * p.G + (m - token * p.G);
#pragma unroll
        for (int e = 0; e < E; ++e) out[at * D + lane + 32 * e] = from_f<T>(good ? o[e] / sum : o[e]);
        if (lane == 0 && p.lse) p.lse[at] = good ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    }
}

// Launches the join behind the kernel whose ranges it joins, as its programmatic dependent.
template <typename T, int D, int TM>
cudaError_t launch_join(const Args& p, T* out, int ranges, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ranges, TM / kJoinRows);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, prefill_join_kernel<T, D, TM>, p, out);
    note_launch();
    return e;
}

// Scratch of `ranges` ranges: partial sums, their maxima and sums, and the cut tiles.
inline size_t part_bytes(int D, int TM, int ranges) { return sizeof(float) * 2 * ranges * TM * D; }
inline size_t ml_bytes(int TM, int ranges) { return sizeof(float2) * 2 * ranges * TM; }
inline size_t scratch_bytes(int D, int TM, int ranges) { return part_bytes(D, TM, ranges) + ml_bytes(TM, ranges) + sizeof(int4) * 2 * ranges; }
inline void set_scratch(Args& p, uint8_t* base, int D, int TM, int ranges) {
    p.part = reinterpret_cast<float*>(base);
    p.ml = reinterpret_cast<float2*>(base + part_bytes(D, TM, ranges));
    p.desc = reinterpret_cast<int4*>(base + part_bytes(D, TM, ranges) + ml_bytes(TM, ranges));
}

// The end of a block's work, by all its NT threads: the cut tile whose first step is in its range, a
// range without a step, and rows of no request (T: the outputs' type).
template <typename T, int D, int TM, int KT, int NT>
__device__ __forceinline__ void finish_range(const Args& p, const Range& range, bool complete, T* out) {
    const int tid = threadIdx.x;
    if (range.any && tid == 0 && complete) {
        Walk<TM, KT> walk(p, range);
        Segment g, last = {};
        while (walk.next(p, g)) last = g;
        if (last.b > 0 && last.a == 0 && !last.whole()) {
            p.desc[2 * blockIdx.x] = make_int4(last.r, last.kh, last.m0, last.rows);
            p.desc[2 * blockIdx.x + 1] = make_int4(range.ranges, 0, 0, 0);
        }
    }
    // a range inside a tile that has no whole step adds nothing to it
    if (range.any && range.from.a > 0 && range.from.a == range.to.a && range.from.r == range.to.r && range.from.kh == range.to.kh &&
        range.from.mt == range.to.mt)
        for (int i = tid; i < TM; i += NT) p.ml[2 * static_cast<int64_t>(blockIdx.x) * TM + i] = make_float2(-INFINITY, -1.f);
    if (p.fill) {
        const int64_t wide = static_cast<int64_t>(p.s.Hq) * D * sizeof(T) / 16;
        const auto clear = [&](int64_t t0, int64_t t1) {
            if (p.fill & 1)
                for (int64_t e = t0 * wide + tid; e < t1 * wide; e += NT) reinterpret_cast<uint4*>(out)[e] = make_uint4(0u, 0u, 0u, 0u);
            if (p.fill & 2)
                for (int64_t e = t0 * p.s.Hq + tid; e < t1 * p.s.Hq; e += NT) p.lse[e] = -INFINITY;
        };
        // Rows before the first request and behind the last one, by all blocks, 16 at a time.  Starts that go back may name
        // rows many times over, so then all rows are cleared, once.
        const bool some = p.s.R && !range.none;
        const int first = some ? min(max(p.starts[0], 0), p.s.T) : 0, last = some ? min(max(p.starts[p.s.R], 0), p.s.T) : 0;
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
            const int64_t from = side ? last : 0, to = side ? p.s.T : first;
            for (int64_t t0 = from + 16 * static_cast<int64_t>(blockIdx.x); t0 < to; t0 += 16 * static_cast<int64_t>(gridDim.x))
                clear(t0, min(t0 + 16, to));
        }
        for (int r = blockIdx.x; some && r < p.s.R; r += gridDim.x) {
            const Request rq(p, r);
            if (rq.pad && rq.n) clear(rq.first, rq.first + rq.n);
        }
    }
}

}  // namespace prefill
}  // namespace la
