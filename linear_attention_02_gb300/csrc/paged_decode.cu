// paged_decode.cu -- attention of one new token over a paged key-value cache:
// per request r and query head,
//     out = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m},  s_j = scale q . k_j
// over the request's own positions (its pages, then its own new row), and
// lse = m + ln sum_j e^{s_j - m}.  Query head h reads key head h / (Hq / Hkv).
//
// Bound by memory: every key and value is read once for all query heads that
// share it (2 D elements a position and key head).  The unit of work is a step:
// 16 positions of one key head, for up to 16 of its query heads.  The steps of
// all requests, request-major, are cut into equal ranges, one per warp of a grid
// that fills the GPU once, whatever the lengths: each block sums up the requests'
// step counts from their lengths on the device, so a captured call follows them.
//
// A warp works alone.  Each lane copies (cp.async) exactly the 16-byte pieces it
// will use itself as matrix operands, a ring of steps ahead, so there is no
// barrier and no exchange: scores are m16n8k16 products of the query heads (rows)
// with 8 keys, values m16n8k16 products of the weights with 16 value rows, with
// the contraction index and the output columns in the order in which the pieces
// lie in memory.  fp32 storage takes m16n8k8 tf32 products of two-term splits
// (three products; relative error 2^-21).  bf16 storage: q, k, v are exact
// operands; the weights are fp32 and go in as three bf16 terms (24 bits), so no
// precision is lost against fp32 arithmetic.  The warp-level matrix instruction
// is enough here: a step of 16 x 64 bf16 keys and values is 4 KB of memory
// traffic, about 170 cycles of an SM's share of the bandwidth, and 32 products.
//
// The maximum is kept lazily: it is raised, and the sums rescaled, only when a
// score passes it by more than 2^8, so most steps need no exchange between lanes.
// A range that starts or ends inside a request leaves partial sums, which a second
// small kernel joins in the order of the ranges.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "la_common.cuh"
#include "la_launch.h"
#include "la_plan.h"

namespace la {
namespace {

constexpr int kWarps = 4;       // warps of a block
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 16;       // positions of a step
constexpr int kTile = 16;       // query heads of a step
constexpr float kSlack = 8.f;   // log2 by which a score may pass the maximum kept

template <typename T, int D>
struct Lay {
    static constexpr int ES = sizeof(T);
    static constexpr int KC = D * ES / 64;              // 16-byte pieces of a key row per lane
    static constexpr int VPL = D * ES >= 128 ? 16 / ES : 8 / ES;  // values of a row piece
    static constexpr int VB = VPL * ES;                 // its bytes
    static constexpr int NI = D / (8 * VPL);            // pieces of a value row per lane
    static constexpr int KBYTES = 2 * KC * 512, VBYTES = 4 * NI * VB * 32;
    static constexpr int STAGE = KBYTES + VBYTES;       // bytes of a step
    static_assert(STAGE == 2 * kStep * D * ES, "a step");
    static constexpr int STAGES = STAGE >= 4096 ? 3 : 6;
    static constexpr int SMEM = kWarps * STAGES * STAGE;
    static constexpr int BLOCKS = STAGE <= 4096 ? 4 : STAGE == 8192 ? 2 : 1;  // per SM
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(on ? 8 : 0) : "memory");
}
template <int B>
__device__ __forceinline__ void cpv(uint32_t dst, const void* src, bool on) {
    if constexpr (B == 16) cp16(dst, src, on);
    else cp8(dst, src, on);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// x = hi + lo: hi the top 11 significant bits, lo the exact rest (the product
// takes its top 11 bits).  An infinity gives a NaN: see exact_scores.
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t& hi, uint32_t& lo) {
    hi = x & 0xFFFFE000u;
    lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
}

struct PagedArgs {
    PagedShape s;
    int G, HT, tiles_per_kh;    // query heads a key head, columns of a request, tiles of a key head
    int append, direct;         // direct: descriptors by column, else by worker
    const int *table, *lens;
    float *out, *lse, *part;
    int4* desc;                 // {first worker, ranges, its slot, column} of a split column; ranges 0: none
    unsigned* status;
};

// A request's positions in steps: [j0, j1) of 16 absolute positions each.
struct Row {
    int len, total, first, j0, j1;
    bool pad, bad;
    __device__ Row(const PagedArgs& p, int r) {
        len = p.lens[r];
        pad = len < 0;
        const int64_t cap = static_cast<int64_t>(p.s.max_pages) << p.s.log2p;
        bad = p.append ? len >= cap : len > cap;
        if (pad) len = 0, bad = false;
        if (len > cap) len = static_cast<int>(cap);
        total = pad ? 0 : len + p.append;
        first = p.s.window && p.s.window < total ? total - p.s.window : 0;
        j0 = first / kStep;
        j1 = max((total + kStep - 1) / kStep, j0 + 1);
    }
    __device__ int steps() const { return pad ? 0 : j1 - j0; }
};

// A warp's place in the steps.
struct Cursor {
    int r, col, j;
    Row row;
    __device__ Cursor(const PagedArgs& p, int r_) : r(r_), col(0), j(0), row(p, r_) {}
    __device__ void advance(const PagedArgs& p) {
        if (++j < row.j1) return;
        if (++col == p.HT) {
            col = 0;
            do {
                ++r;
                row = Row(p, min(r, p.s.R - 1));
            } while (row.pad && r < p.s.R - 1);
        }
        j = row.j0;
    }
};

// The warp's share: steps [u0, u0 + left) of all, `per` a warp; its first step is
// step u0 - base of request r.  Every block sums up all requests (R lengths from
// L2), each warp finds its place from the block's sums.
struct Share {
    int64_t left, per, base;
    int r;
};
__device__ __forceinline__ Share find_share(const PagedArgs& p, int worker, int workers, int min_per) {
    __shared__ int64_t s_sum[kThreads];
    const int tid = threadIdx.x, lane = tid & 31;
    const int chunk = (p.s.R + kThreads - 1) / kThreads;  // requests of a thread
    int64_t sum = 0;
    for (int i = 0; i < chunk; ++i) {
        const int r = tid * chunk + i;
        if (r < p.s.R) sum += Row(p, r).steps();
    }
    s_sum[tid] = sum;
    __syncthreads();
    // inclusive sums of the threads' chunks, each warp for itself
    int64_t pre[kThreads / 32], total = 0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) {
        int64_t x = s_sum[k * 32 + lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        pre[k] = x + total;
        total = __shfl_sync(0xffffffffu, pre[k], 31);
    }
    Share w;
    total *= p.HT;
    w.per = max(static_cast<int64_t>(min_per), (total + workers - 1) / workers);
    const int64_t u0 = worker * w.per;
    w.left = max(static_cast<int64_t>(0), min(w.per, total - u0));
    w.base = 0;
    w.r = 0;
    if (w.left == 0) return w;
    // the chunk with step u0, then the request in it
    int at = 0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) {
        const unsigned behind = __ballot_sync(0xffffffffu, pre[k] * p.HT <= u0);
        at += __popc(behind);
        const int n = __popc(behind);
        if (n) w.base = __shfl_sync(0xffffffffu, pre[k], n - 1) * p.HT;
    }
    int r = at * chunk;
    for (;; r += 32) {  // 32 requests at once
        const int mine = r + lane;
        int64_t x = mine < p.s.R ? Row(p, mine).steps() : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        const unsigned behind = __ballot_sync(0xffffffffu, w.base + x * p.HT <= u0);
        const int n = __popc(behind);
        const int64_t skip = n ? __shfl_sync(0xffffffffu, x, n ? n - 1 : 0) * p.HT : 0;
        w.base += skip;
        if (n < 32 || r + 32 >= p.s.R) {
            w.r = min(r + n, p.s.R - 1);
            return w;
        }
    }
}

// fp32 scores of a step by plain products, for the step whose split products gave
// a NaN (an infinite key or query): the lane's 8 scores from the warp's pieces in
// the ring and the query rows in memory.
template <int D>
__device__ __noinline__ void exact_scores(const uint8_t* st, const float* q, int heads, float (&s)[2][4]) {
    constexpr int KC = Lay<float, D>::KC;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    __syncwarp();  // every lane's pieces have come
    for (int n = 0; n < 2; ++n)
        for (int e = 0; e < 4; ++e) {
            const int h = g + 8 * (e >> 1), key = 2 * t + (e & 1);
            float x = 0.f;
            if (h < heads)
                for (int c = 0; c < D; ++c)  // value c is word c % 4 of piece c / 16 of lane (key, c / 4 % 4)
                    x += q[h * D + c] * reinterpret_cast<const float*>(
                                            st + (n * KC + c / 16) * 512 + (key * 4 + c / 4 % 4) * 16)[c & 3];
            s[n][e] = x;
        }
    __syncwarp();  // before any lane copies into this stage again
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, Lay<T, D>::BLOCKS)
paged_decode_kernel(const T* __restrict__ q, const T* __restrict__ kn, const T* __restrict__ vn, T* K, T* V,
                    const PagedArgs p, int min_per) {
    using Ly = Lay<T, D>;
    constexpr int KC = Ly::KC, VPL = Ly::VPL, VB = Ly::VB, NI = Ly::NI, NT = D / 8, STAGES = Ly::STAGES;
    constexpr bool kBf16 = sizeof(T) == 2;
    extern __shared__ __align__(16) uint8_t sm[];
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, warp = threadIdx.x >> 5;
    const int workers = gridDim.x * kWarps, worker = blockIdx.x * kWarps + warp;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Share sh = find_share(p, worker, workers, min_per);
    if (!p.direct && lane == 0) p.desc[worker] = make_int4(0, 0, 0, 0);
    if (sh.left == 0) return;
    uint8_t* ring = sm + warp * (STAGES * Ly::STAGE);
    const uint32_t ring32 = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    const int row16 = 1 << p.s.log2p;
    bool bad = false;

    Cursor ld(p, sh.r);
    {
        const int64_t off = static_cast<int64_t>(worker) * sh.per - sh.base;
        const int n = ld.row.steps();
        ld.col = static_cast<int>(off / n);
        ld.j = ld.row.j0 + static_cast<int>(off - static_cast<int64_t>(ld.col) * n);
    }
    Cursor cs = ld;
    bool whole = cs.j == cs.row.j0;  // the column's first step is this warp's
    bool first_seg = true;

    const auto page_of = [&](const Cursor& c) {  // page of the lane's position (lane & 15) of a step
        const int pos = c.j * kStep + (lane & 15);
        const int at = pos >> p.s.log2p;
        return pos < c.row.len && at < p.s.max_pages ? p.table[static_cast<int64_t>(c.r) * p.s.max_pages + at] : -1;
    };
    int64_t to_load = sh.left;
    int pg = page_of(ld);
    uint32_t seen[STAGES];  // positions that count, a bit each, of the steps in the ring, the current one first
#pragma unroll
    for (int s = 0; s < STAGES; ++s) seen[s] = 0;

    // Copies the lane's pieces of step `ld` into a stage and moves on; returns the
    // positions that count.
    const auto issue = [&](int stage) -> uint32_t {
        uint32_t mask = 0xFFFFu;
        if (to_load > 0) {
            const uint32_t kd = ring32 + stage * Ly::STAGE + lane * 16;
            const uint32_t vd = ring32 + stage * Ly::STAGE + Ly::KBYTES + lane * VB;
            const int pos0 = ld.j * kStep, kh = ld.col / p.tiles_per_kh;
            const int page = pg;
            const Cursor now = ld;
            ld.advance(p);
            if (--to_load > 0) pg = page_of(ld);
            const bool inside = p.s.log2p >= 4 && pos0 >= now.row.first && pos0 + kStep <= now.row.len &&
                                static_cast<unsigned>(page) < static_cast<unsigned>(p.s.num_pages);
            if (__all_sync(0xffffffffu, inside)) {  // one page, every position the request's
                const int64_t row = ((static_cast<int64_t>(page) * p.s.Hkv + kh) << p.s.log2p) + (pos0 & (row16 - 1));
                const T* kr = K + (row + g) * D + t * (16 / static_cast<int>(sizeof(T)));
                const T* vr = V + (row + 2 * t) * D + g * VPL;
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int i = 0; i < KC; ++i)
                        cp16(kd + (n * KC + i) * 512, kr + n * 8 * D + i * (64 / static_cast<int>(sizeof(T))), true);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        cpv<VB>(vd + (e * NI + i) * VB * 32, vr + ((e >> 1) * 8 + (e & 1)) * D + i * 8 * VPL, true);
            } else {
                const int mypos = pos0 + (lane & 15);
                const bool mine = mypos >= now.row.first && mypos < now.row.total;
                const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(p.s.num_pages);
                bad |= mine && mypos < now.row.len && !there;
                mask = __ballot_sync(0xffffffffu, mine && (there || mypos == now.row.len)) & 0xFFFFu;
                const int64_t nrow = static_cast<int64_t>(now.r) * p.s.Hkv + kh;
                const auto key_row = [&](int key, const T* pool, const T* fresh, bool& on) -> const T* {
                    const int pos = pos0 + key;
                    const int id = __shfl_sync(0xffffffffu, page, key);
                    on = mask >> key & 1u;
                    if (on && pos == now.row.len) return fresh + nrow * D;
                    const int64_t row = ((static_cast<int64_t>(id) * p.s.Hkv + kh) << p.s.log2p) + (pos & (row16 - 1));
                    return on ? pool + row * D : q;
                };
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    bool on;
                    const T* kr = key_row(8 * n + g, K, kn, on) + t * (16 / static_cast<int>(sizeof(T)));
#pragma unroll
                    for (int i = 0; i < KC; ++i)
                        cp16(kd + (n * KC + i) * 512, on ? kr + i * (64 / static_cast<int>(sizeof(T))) : q, on);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    bool on;
                    const T* vr = key_row((e >> 1) * 8 + 2 * t + (e & 1), V, vn, on) + g * VPL;
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        cpv<VB>(vd + (e * NI + i) * VB * 32, on ? vr + i * 8 * VPL : q, on);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return mask;
    };

    // query operands of a column: rows g and g + 8 of the tile (0 past the heads)
    uint4 qa[KC], qb[KC];
    const auto load_q = [&]() {
        const int kh = cs.col / p.tiles_per_kh, h0 = (cs.col - kh * p.tiles_per_kh) * kTile;
        const int64_t row = static_cast<int64_t>(cs.r) * p.s.Hq + kh * p.G + h0;
        const T* src = q + (row + g) * D + t * (16 / static_cast<int>(sizeof(T)));
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            const int off = i * (64 / static_cast<int>(sizeof(T)));
            qa[i] = h0 + g < p.G ? *reinterpret_cast<const uint4*>(src + off) : make_uint4(0, 0, 0, 0);
            qb[i] = h0 + g + 8 < p.G ? *reinterpret_cast<const uint4*>(src + 8 * D + off) : make_uint4(0, 0, 0, 0);
        }
    };

    float o[NT][4], m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    const auto clear = [&]() {
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
    };
    clear();
    load_q();
    const float sc = p.s.scale * 1.4426950408889634f;

#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) seen[s] = issue(s);
    int stage = 0;
    for (int64_t n_left = sh.left; n_left > 0; --n_left) {
        {
            const int to = stage + STAGES - 1;
            seen[STAGES - 1] = issue(to >= STAGES ? to - STAGES : to);
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
        const uint8_t* st = ring + stage * Ly::STAGE;

        // scores of 16 heads x 16 keys
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                const uint4 k = *reinterpret_cast<const uint4*>(st + (n * KC + i) * 512 + lane * 16);
                if constexpr (kBf16) {
                    mma_bf16(s[n], qa[i].x, qb[i].x, qa[i].y, qb[i].y, k.x, k.y);
                    mma_bf16(s[n], qa[i].z, qb[i].z, qa[i].w, qb[i].w, k.z, k.w);
                } else {
                    const uint32_t kw[4] = {k.x, k.y, k.z, k.w}, aw[4] = {qa[i].x, qa[i].y, qa[i].z, qa[i].w},
                                   bw[4] = {qb[i].x, qb[i].y, qb[i].z, qb[i].w};
#pragma unroll
                    for (int h = 0; h < 4; h += 2) {
                        uint32_t kh0, kl0, kh1, kl1, ah0, al0, ah1, al1, bh0, bl0, bh1, bl1;
                        split_tf32(kw[h], kh0, kl0);
                        split_tf32(kw[h + 1], kh1, kl1);
                        split_tf32(aw[h], ah0, al0);
                        split_tf32(aw[h + 1], ah1, al1);
                        split_tf32(bw[h], bh0, bl0);
                        split_tf32(bw[h + 1], bh1, bl1);
                        mma_tf32(s[n], ah0, bh0, ah1, bh1, kh0, kh1);
                        mma_tf32(s[n], ah0, bh0, ah1, bh1, kl0, kl1);
                        mma_tf32(s[n], al0, bl0, al1, bl1, kh0, kh1);
                    }
                }
            }
        }
        if constexpr (!kBf16) {
            bool nan = false;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) nan |= s[n][e] != s[n][e];
            if (__any_sync(0xffffffffu, nan)) {
                const int kh = cs.col / p.tiles_per_kh, h0 = (cs.col - kh * p.tiles_per_kh) * kTile;
                exact_scores<D>(st, q + (static_cast<int64_t>(cs.r) * p.s.Hq + kh * p.G + h0) * D, p.G - h0, s);
            }
        }
        const int pos0 = cs.j * kStep;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] *= sc;
        if (seen[0] != 0xFFFFu) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(seen[0] >> (8 * n + 2 * t + (e & 1)) & 1u)) s[n][e] = -INFINITY;
        }
        const float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
        const float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
        if (__any_sync(0xffffffffu, x0 > m0 + kSlack || x1 > m1 + kSlack)) {
            float y0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1)), y1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
            y0 = fmaxf(m0, fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, 2)));
            y1 = fmaxf(m1, fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, 2)));
            const float f0 = m0 == y0 ? 1.f : ex2(m0 - y0), f1 = m1 == y1 ? 1.f : ex2(m1 - y1);
            l0 *= f0;
            l1 *= f1;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                o[n][0] *= f0;
                o[n][1] *= f0;
                o[n][2] *= f1;
                o[n][3] *= f1;
            }
            m0 = y0;
            m1 = y1;
        }
        const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
        float w[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            w[n][0] = ex2(s[n][0] - z0);
            w[n][1] = ex2(s[n][1] - z0);
            w[n][2] = ex2(s[n][2] - z1);
            w[n][3] = ex2(s[n][3] - z1);
            l0 += w[n][0] + w[n][1];
            l1 += w[n][2] + w[n][3];
        }
        const uint8_t* vs = st + Ly::KBYTES + lane * VB;
        if constexpr (kBf16) {
            uint32_t a[3][4];  // three terms of the weights
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                float x = w[u >> 1][2 * (u & 1)], y = w[u >> 1][2 * (u & 1) + 1];
#pragma unroll
                for (int z = 0; z < 3; ++z) {
                    a[z][u] = pack2(x, y);
                    x -= __uint_as_float(a[z][u] << 16);
                    y -= __uint_as_float(a[z][u] & 0xFFFF0000u);
                }
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                uint32_t v[4][VPL / 2];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (VB == 16) {
                        const uint4 f = *reinterpret_cast<const uint4*>(vs + (e * NI + i) * VB * 32);
                        v[e][0] = f.x, v[e][1] = f.y, v[e][2] = f.z, v[e][3] = f.w;
                    } else {
                        const uint2 f = *reinterpret_cast<const uint2*>(vs + (e * NI + i) * VB * 32);
                        v[e][0] = f.x, v[e][1] = f.y;
                    }
                }
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                    const uint32_t b0 = __byte_perm(v[0][j / 2], v[1][j / 2], sel);
                    const uint32_t b1 = __byte_perm(v[2][j / 2], v[3][j / 2], sel);
#pragma unroll
                    for (int z = 0; z < 3; ++z)
                        mma_bf16(o[i * VPL + j], a[z][0], a[z][1], a[z][2], a[z][3], b0, b1);
                }
            }
        } else {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                uint32_t ah[4], al[4];  // keys 2t (operand k = t) and 2t + 1 (k = t + 4)
                split_tf32(__float_as_uint(w[n][0]), ah[0], al[0]);
                split_tf32(__float_as_uint(w[n][2]), ah[1], al[1]);
                split_tf32(__float_as_uint(w[n][1]), ah[2], al[2]);
                split_tf32(__float_as_uint(w[n][3]), ah[3], al[3]);
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const uint4 v0 = *reinterpret_cast<const uint4*>(vs + ((2 * n) * NI + i) * VB * 32);
                    const uint4 v1 = *reinterpret_cast<const uint4*>(vs + ((2 * n + 1) * NI + i) * VB * 32);
                    const uint32_t x0w[4] = {v0.x, v0.y, v0.z, v0.w}, x1w[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t h0, c0, h1, c1;
                        split_tf32(x0w[j], h0, c0);
                        split_tf32(x1w[j], h1, c1);
                        mma_tf32(o[i * 4 + j], ah[0], ah[1], ah[2], ah[3], h0, h1);
                        mma_tf32(o[i * 4 + j], ah[0], ah[1], ah[2], ah[3], c0, c1);
                        mma_tf32(o[i * 4 + j], al[0], al[1], al[2], al[3], h0, h1);
                    }
                }
            }
        }

        // the new row goes into the cache, once a key head
        if (p.append && cs.row.len >= pos0 && cs.row.len < pos0 + kStep && cs.col % p.tiles_per_kh == 0) {
            const int kh = cs.col / p.tiles_per_kh, at = cs.row.len >> p.s.log2p;
            const int id = at < p.s.max_pages ? p.table[static_cast<int64_t>(cs.r) * p.s.max_pages + at] : -1;
            if (static_cast<unsigned>(id) < static_cast<unsigned>(p.s.num_pages)) {
                constexpr int PIECES = D * static_cast<int>(sizeof(T)) / 16;
                const int64_t to = ((static_cast<int64_t>(id) * p.s.Hkv + kh) << p.s.log2p) + (cs.row.len & (row16 - 1));
                const int64_t from = static_cast<int64_t>(cs.r) * p.s.Hkv + kh;
                if (lane < PIECES) {
                    reinterpret_cast<uint4*>(K + to * D)[lane] = reinterpret_cast<const uint4*>(kn + from * D)[lane];
                    reinterpret_cast<uint4*>(V + to * D)[lane] = reinterpret_cast<const uint4*>(vn + from * D)[lane];
                }
            } else {
                bad = true;
            }
        }

        const bool col_end = cs.j + 1 == cs.row.j1;
        if (col_end || n_left == 1) {  // end of the column, or of the warp's range inside it
            bad |= cs.row.bad;
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            const int kh = cs.col / p.tiles_per_kh, h0 = (cs.col - kh * p.tiles_per_kh) * kTile;
            const int64_t row0 = static_cast<int64_t>(cs.r) * p.s.Hq + kh * p.G + h0;
            const bool done = whole && col_end;
            const int slot = first_seg ? 0 : 1;
            float* part = p.part + (static_cast<int64_t>(worker) * 2 + slot) * kTile * (D + 2);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int h = g + 8 * half;
                if (h0 + h >= p.G) continue;
                const float l = half ? l1 : l0, m = half ? m1 : m0;
                const float f = done ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
                float* dst = done ? p.out + (row0 + h) * D : part + h * D;
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int j = 0; j < VPL; j += 4) {
                            const int b = i * VPL + j, e = 2 * half + c;
                            const int d = (2 * t + c + 8 * i) * VPL + j;
                            *reinterpret_cast<float4*>(dst + d) =
                                make_float4(o[b][e] * f, o[b + 1][e] * f, o[b + 2][e] * f, o[b + 3][e] * f);
                        }
                if (t == 0) {
                    if (!done) {
                        part[kTile * D + 2 * h] = m;
                        part[kTile * D + 2 * h + 1] = l;
                    } else if (p.lse) {
                        p.lse[row0 + h] = (m + log2f(l)) * 0.6931471805599453f;
                    }
                }
            }
            if (lane == 0) {
                const int64_t index = p.direct ? static_cast<int64_t>(cs.r) * p.HT + cs.col : worker;
                if (whole && !col_end) {  // first range of a split column
                    const int64_t rest = cs.row.j1 - (cs.j + 1);
                    p.desc[index] = make_int4(worker, static_cast<int>(1 + (rest + sh.per - 1) / sh.per), slot,
                                              p.direct ? 0 : cs.r * p.HT + cs.col);
                } else if (whole && p.direct) {
                    p.desc[index] = make_int4(0, 0, 0, 0);
                }
            }
            first_seg = false;
            if (n_left > 1) {
                cs.advance(p);
                whole = true;
                clear();
                load_q();
            }
        } else {
            ++cs.j;
        }
        if (++stage == STAGES) stage = 0;
#pragma unroll
        for (int s = 0; s + 1 < STAGES; ++s) seen[s] = seen[s + 1];
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (bad) atomicOr(p.status, kStatusBadIndex);
}

// Joins the ranges of a split column, one block a query head: the maximum of the
// ranges' maxima, then sums scaled to it, in the order of the ranges within each
// of the block's warps and of the warps.
template <int D>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const PagedArgs p) {
    __shared__ float s_m[kWarps], s_l[kWarps], s_a[kWarps][D];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t index = blockIdx.x;
    const int h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t col = index;
    if (p.direct && p.lens[index / p.HT] < 0) return;
    const int4 d = p.desc[index];
    if (d.y == 0) return;
    if (!p.direct) col = d.w;
    const int64_t r = col / p.HT;
    const int c = static_cast<int>(col - r * p.HT), kh = c / p.tiles_per_kh, h0 = (c - kh * p.tiles_per_kh) * kTile;
    if (h0 + h >= p.G) return;
    constexpr int E = D / 32;
    float m = -INFINITY, l = 0.f, a[E];
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = 0.f;
    const int each = (d.y + kWarps - 1) / kWarps, i1 = min(d.y, (warp + 1) * each);
#pragma unroll 4
    for (int i = warp * each; i < i1; ++i) {
        const float* part = p.part + ((static_cast<int64_t>(d.x) + i) * 2 + (i ? 0 : d.z)) * kTile * (D + 2);
        const float pm = part[kTile * D + 2 * h], pl = part[kTile * D + 2 * h + 1];
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = part[h * D + lane + 32 * e];
        const float x = fmaxf(m, pm);
        const float f = m == x ? 1.f : ex2(m - x), g = pm == -INFINITY ? 0.f : pm == x ? 1.f : ex2(pm - x);
        l = l * f + pl * g;
#pragma unroll
        for (int e = 0; e < E; ++e) a[e] = a[e] * f + v[e] * g;
        m = x;
    }
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) s_a[warp][lane + 32 * e] = a[e];
    __syncthreads();
    const int64_t row = r * p.s.Hq + kh * p.G + h0 + h;
    for (int i = threadIdx.x; i < D; i += kThreads) {
        float x = -INFINITY, tl = 0.f, ta = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) x = fmaxf(x, s_m[w]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = s_m[w] == -INFINITY ? (s_l[w] != s_l[w] ? 1.f : 0.f) : s_m[w] == x ? 1.f : ex2(s_m[w] - x);
            tl += s_l[w] * f;
            ta += s_a[w][i] * f;
        }
        p.out[row * D + i] = tl > 0.f || tl != tl ? ta / tl : 0.f;
        if (i == 0 && p.lse) p.lse[row] = (x + log2f(tl)) * 0.6931471805599453f;
    }
}

}  // namespace

// Ranges are of at least this many steps, so that few partial sums are written.
constexpr int kMinSteps = 4;

template <typename T, int D>
cudaError_t paged_decode_step(const LaunchCtx& c, const T* q, const T* k, const T* v, T* K, T* V,
                              const int* table, const int* lens, float* out, float* lse,
                              const PagedShape& s) {
    using Ly = Lay<T, D>;
    auto* kernel = paged_decode_kernel<T, D>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::SMEM);
    if (e != cudaSuccess) return e;
    const int blocks = Ly::BLOCKS * c.num_sms, workers = blocks * kWarps;
    PagedArgs p = {};
    p.s = s;
    p.G = s.Hq / s.Hkv;
    p.tiles_per_kh = (p.G + kTile - 1) / kTile;
    p.HT = s.Hkv * p.tiles_per_kh;
    p.append = k ? 1 : 0;
    p.table = table;
    p.lens = lens;
    p.out = out;
    p.lse = lse;
    p.status = c.status_word;
    const int64_t cols = static_cast<int64_t>(s.R) * p.HT;
    p.direct = cols <= workers;
    uint8_t* base = nullptr;
    const size_t part = sizeof(float) * workers * 2 * kTile * (D + 2);
    e = scratch_alloc(c, reinterpret_cast<void**>(&base), part + sizeof(int4) * workers);
    if (e != cudaSuccess) return e;
    p.part = reinterpret_cast<float*>(base);
    p.desc = reinterpret_cast<int4*>(base + part);
    kernel<<<blocks, kThreads, Ly::SMEM, c.stream>>>(q, k, v, K, V, p, kMinSteps);
    note_launch(2);
    e = cudaGetLastError();
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(p.direct ? cols : workers), std::min(p.G, kTile));
        cfg.blockDim = dim3(kThreads);
        cfg.stream = c.stream;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, paged_join_kernel<D>, p);
    }
    scratch_free(c, base);
    return e;
}

#define LA_INST_PD(T, D)                                                                          \
    template cudaError_t paged_decode_step<T, D>(const LaunchCtx&, const T*, const T*, const T*, T*, \
                                                 T*, const int*, const int*, float*, float*,      \
                                                 const PagedShape&);
LA_INST_PD(float, 32) LA_INST_PD(float, 64) LA_INST_PD(float, 128)
LA_INST_PD(__nv_bfloat16, 32) LA_INST_PD(__nv_bfloat16, 64) LA_INST_PD(__nv_bfloat16, 128)

}  // namespace la
