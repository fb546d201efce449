// paged_decode.cu -- attention of one new token over a paged key-value cache:
// per request r and query head,
//     out = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m},  s_j = scale q . k_j
// over the request's own positions (its pages, then its own new row), and
// lse = m + ln sum_j e^{s_j - m}.  Query head h reads key head h / (Hq / Hkv).
//
// Bound by memory: every key and value is read once for up to 16 query heads that
// share it (2 D elements a position and key head).  The unit of work is a step:
// 16 positions of one key head, for up to 16 of its query heads.  The steps of
// all requests, request-major, are cut into equal ranges, one to four for each warp of
// a grid that fills the GPU once, whatever the lengths: each block sums up the requests'
// step counts from their lengths on the device, so a captured call follows them.  A
// warp's first range has its own number, the next ones are taken from a counter.
//
// A warp works alone, on a ring of steps of its own in shared memory that TMA fills
// (one box of 16 rows x 128 bytes at a time, 128-byte swizzle), so blocks have no
// barrier.  (Filled by cp.async, 16 bytes a lane, the same kernel stayed at 5.2 TB/s
// whatever it computed: the load pipe held back the reads behind the copies.)
// Steps that are not 16 positions of one page (a request's ends, its new row, pages
// of fewer than 16) are copied by the lanes, each the pieces it will read.  Scores
// are products of the query heads (rows) with 8 keys, outputs products of the
// weights with 16 value rows; the contraction index and the output columns are in
// such an order that a lane's operands are 16-byte pieces of the rows, read without
// bank conflicts.
// bf16 storage: m16n8k16; q, k, v are exact operands, the weights are fp32 and go
// in as three bf16 terms (24 bits), so no precision is lost against fp32
// arithmetic.  fp32 storage: m16n8k8 tf32 products of splits.  Queries, keys and weights
// go in as two terms split by rounding, which keep 23 of 24 bits: a term of a score is
// off by 2^-22 of itself, no more than D fp32 additions leave, and a weight by 2^-23, half
// of what the approximate power that makes it leaves.  Values go in as two terms, the
// second rounded: off by 2^-22 at most, to either side (cut off, half of all values came
// out smaller by a bit or two); where a request sees no more than kExact positions, so that
// no sum hides it, a third term, in bf16, carries the rest.  With all three always, a step
// takes 2% longer at D = 64 (328 us against 321 us at 64 x 16 x 4096) and 11% at 128 (436 us
// against 394 us at 64 x 8 key heads x 4096).
// With up to 8 query heads a key head (kHeads = 8), the operand's rows 8 to 15 hold a
// second term of the same heads instead of nothing; with more, they hold heads 8 to 15
// (and the product of two second terms is left out), and heads past 16 take further passes.
// The warp-level matrix instruction is enough here: a step of 16 x 64 bf16 keys
// and values is 4 KB of memory traffic, about 170 cycles of an SM's share of the
// bandwidth, against 24 small products.
//
// Each step's outputs are summed by the matrix unit from zero and added to the running
// sums in fp32 (summed on through a whole range, the unit's truncation left an error
// of 3.4e-6 at 4096 positions; so it is 2.6e-7, at the same time).  The maximum is kept
// lazily: it is raised, and the sums rescaled, only when a score passes it by more than
// 2^8, so most steps need no exchange between lanes.  A range that starts or ends inside a request leaves partial sums, which a second
// small kernel joins in the order of the ranges.
//
// Measured on the GPU (measured copy bandwidth 6.79 TB/s): 256 requests x 16 heads x 4096
// positions, D = 64, bf16: 670 us, 6.4 TB/s.  64 requests x 4096 positions: bf16, D = 128,
// 4 key heads, 5.2 TB/s with 8 query heads each and 4.7 TB/s with 16 (with G > 16 the bytes
// are read ceil(G / 16) times); fp32, 6.6 TB/s at 16 key heads, D = 64, 5.6 at D = 32, 5.4 at 8
// key heads, D = 128, and 3.8 with 12 query heads each; bf16, D = 32, 5.1 TB/s: there a
// step's chain of products and exponentials on the few warps that shared memory leaves
// room for bounds it.  A small call (4 requests, up to 300 positions) takes 8.7 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "la_common.cuh"
#include "la_launch.h"
#include "la_plan.h"
#include "tc_common.cuh"

namespace la {
namespace {

constexpr int kStep = 16;       // positions of a step
constexpr float kSlack = 8.f;   // log2 by which a score may pass the maximum kept
constexpr int kExact = 32;      // positions up to which fp32 values are weighted with all their bits

// A step in shared memory: 16 key rows, then 16 value rows, each as atoms of 16 rows
// x AB bytes in which 16-byte chunk c of row r lies at chunk c ^ (r & 7) (AB = 128),
// or c ^ (r / 2 & 3) (AB = 64).  Lane (g, t) = lane / 4, lane % 4 reads KC pieces of
// keys g and g + 8 (chunks 2 t and 2 t + 1 of each atom; t of a 64-byte row) and NI
// pieces of VPL values of rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9 (chunk g of each atom).
template <typename T, int D>
struct Lay {
    static constexpr int ES = sizeof(T);
    static constexpr int AB = D * ES >= 128 ? 128 : 64;
    static constexpr int ATOMS = D * ES / AB, ATOM = kStep * AB;
    static constexpr int KC = D * ES / 64;
    static constexpr int VB = AB / 8, VPL = VB / ES, NI = ATOMS;  // bytes and values of a value piece
    static constexpr int HALF = ATOMS * ATOM, STAGE = 2 * HALF;   // bytes of the keys, of a step
    // Warps of a block, blocks of an SM and steps of a ring fill the SM's shared memory
    // with about 192 KB: enough warps to hide a step's chain of products, exponentials
    // and products, and as many steps ahead as is left.  Measured, TB/s: 4 KB steps
    // 6.50 with 12 warps x 4, 6.35 with 16 x 3; 8 KB steps (D = 128, bf16) 5.76 with
    // 8 x 3, 5.3 with 12 x 2, 5.66 with 6 x 4; 16 KB steps 6.14 with 6 x 2, 5.57 with 4 x 3.
    static constexpr int WARPS = STAGE == 16384 ? 6 : 4, THREADS = 32 * WARPS;
    static constexpr int BLOCKS = STAGE == 2048 ? 4 : STAGE == 4096 ? 3 : STAGE == 8192 ? 2 : 1;
    static constexpr int STAGES = STAGE == 2048 ? 6 : STAGE == 4096 ? 4 : STAGE == 8192 ? 3 : 2;
    static constexpr int SMEM = WARPS * STAGES * STAGE + 1024;
    static_assert(STAGES <= 8, "the loader is never two ranges ahead");
    // the chunk (of the whole row) and the place of the lane's key piece i in key tile n
    static __device__ __forceinline__ int kchunk(int t, int i) { return AB == 128 ? (i / 2) * 8 + 2 * t + i % 2 : t; }
    static __device__ __forceinline__ int kat(int g, int t, int n, int i) {
        if constexpr (AB == 128) return (i / 2) * ATOM + (8 * n + g) * 128 + (((2 * t + i % 2) ^ g) << 4);
        else return (8 * n + g) * 64 + ((t ^ (g >> 1 & 3)) << 4);
    }
    // the place of the lane's value piece i of row vrow(t, e)
    static __device__ __forceinline__ int vrow(int t, int e) { return 2 * t + (e & 1) + 8 * (e >> 1); }
    static __device__ __forceinline__ int vat(int g, int t, int e, int i) {
        if constexpr (AB == 128) return HALF + i * ATOM + vrow(t, e) * 128 + ((g ^ (2 * t + (e & 1))) << 4);
        else return HALF + vrow(t, e) * 64 + (((g >> 1) ^ t) << 4) + (g & 1) * 8;
    }
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// x = hi + lo, exactly: the top 11 significant bits and the other 13, of which a product
// takes 11.  An infinity gives a NaN.
__device__ __forceinline__ void split_tf32(uint32_t x, uint32_t& hi, uint32_t& lo) {
    hi = x & 0xFFFFE000u;
    lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi));
}
// x = hi + lo in two terms: hi rounded to nearest, so that lo fits its 11 bits but for
// one at most and has either sign.  An infinity gives a NaN: see exact_scores.
__device__ __forceinline__ void split_tf32_rn(uint32_t x, uint32_t& hi, uint32_t& lo) {
    hi = (x + 0x1000u) & 0xFFFFE000u;
    lo = __float_as_uint(__uint_as_float(x) - __uint_as_float(hi));
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// Ranges a warp: 4, so that warps that run ahead take more of them (690 us against
// 700 us with 2, 256 x 16 x 4096 x 64), but 2 below kFour steps a warp, since each
// range may leave partial sums (95 us against 105 us at 6 x 4 key heads of up to
// 65535 positions, D = 128), and 1 below kTwo: a few ranges more than warps would
// cost a whole range's time.  A range that is followed by another then has at least
// kTwo / 2 steps, more than the loader runs ahead.
constexpr int kTwo = 16, kFour = 64;

struct PagedArgs {
    PagedShape s;
    int G, HT, tiles_per_kh;    // query heads a key head, columns of a request, columns of a key head
    int tma;                    // the pools have tensor maps
    int append, direct;         // direct: descriptors by column, else by range
    int heads;                  // rows of a partial result: the column's query heads
    int max_ranges;
    unsigned* next;             // ranges taken beyond the first of each warp (null: one each is enough)
    const int *table, *lens;
    float *out, *lse;
    int fill;                   // what rows without a request get: bit 0, out 0; bit 1, lse -infinity
    float* part;                // [ranges][2][heads x (D + 4)]: output sums [heads][D], then maximum, sum of each head
    int4* desc;                 // {first range, ranges, its slot, column} of a split column; ranges 0: none
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
        j1 = max((total + kStep - 1) / kStep, j0 + 1);  // positions stay below 2^30
    }
    __device__ int steps() const { return pad ? 0 : j1 - j0; }
};

// A warp's place in the steps.
struct Cursor {
    int r, kh, tile, j;  // request, key head, tile of its query heads, step
    Row row;
    __device__ Cursor(const PagedArgs& p, int r_, int64_t off) : r(r_), row(p, r_) {
        const int n = row.steps(), col = static_cast<int>(off / n);
        j = row.j0 + static_cast<int>(off - static_cast<int64_t>(col) * n);
        kh = col / p.tiles_per_kh;
        tile = col - kh * p.tiles_per_kh;
    }
    __device__ int col(const PagedArgs& p) const { return kh * p.tiles_per_kh + tile; }
    __device__ void advance(const PagedArgs& p) {
        if (++j < row.j1) return;
        if (++tile == p.tiles_per_kh) tile = 0, ++kh;
        if (kh == p.s.Hkv) {
            kh = 0;
            do {
                ++r;
                row = Row(p, min(r, p.s.R - 1));
            } while (row.pad && r < p.s.R - 1);
        }
        j = row.j0;
    }
};

// Inclusive sums of the steps of all requests, chunk by chunk of requests (a chunk
// a thread); returns their total.  Every block does it for itself (R lengths from L2).
template <int kThreads>
__device__ __forceinline__ int64_t sum_steps(const PagedArgs& p, int64_t* s_pre) {
    const int tid = threadIdx.x, lane = tid & 31;
    const int chunk = (p.s.R + kThreads - 1) / kThreads;
    int64_t x = 0;
    for (int i = 0; i < chunk; ++i) {
        const int r = tid * chunk + i;
        if (r < p.s.R) x += Row(p, r).steps();
    }
    x *= p.HT;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    s_pre[tid] = x;
    __syncthreads();
    int64_t before = 0;
    for (int w = 0; w < tid / 32; ++w) before += s_pre[w * 32 + 31];
    __syncthreads();
    s_pre[tid] = x + before;
    __syncthreads();
    return s_pre[kThreads - 1];
}

// The request with step u0 < total, and its first step's number.  For a whole warp.
template <int kThreads>
__device__ __forceinline__ int locate(const PagedArgs& p, const int64_t* s_pre, int64_t u0, int64_t& base) {
    const int lane = threadIdx.x & 31, chunk = (p.s.R + kThreads - 1) / kThreads;
    int at = 0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) at += __popc(__ballot_sync(0xffffffffu, s_pre[k * 32 + lane] <= u0));
    base = at ? s_pre[at - 1] : 0;
    for (int r = at * chunk;; r += 32) {  // 32 requests at once
        const int mine = r + lane;
        int64_t x = mine < p.s.R ? static_cast<int64_t>(Row(p, mine).steps()) * p.HT : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        const int n = __popc(__ballot_sync(0xffffffffu, base + x <= u0));
        const int64_t skip = __shfl_sync(0xffffffffu, x, n ? n - 1 : 0);
        if (n) base += skip;
        if (n < 32 || r + 32 >= p.s.R) return min(r + n, p.s.R - 1);
    }
}

// fp32 scores of a step by plain products, for the step whose split products gave
// a NaN (an infinite key or query): the lane's scores of a head (x of keys 2 t and
// 2 t + 1 of key tile n) from the step in shared memory and the query row in memory.
template <int D>
__device__ __noinline__ float2 exact_scores(const uint8_t* st, const float* q, bool on, int n, float sign) {
    const int t = threadIdx.x & 3;
    float x[2] = {0.f, 0.f};
    __syncwarp();  // every lane's copies have come
    if (on)
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * n + 2 * t + e;
            for (int c = 0; c < D; ++c)
                x[e] += sign * q[c] * reinterpret_cast<const float*>(
                                          st + c / 32 * Lay<float, D>::ATOM + r * 128 + ((c / 4 % 8 ^ (r & 7)) << 4))[c & 3];
        }
    __syncwarp();
    return make_float2(x[0], x[1]);
}

// kHeads: 8 or 16 query heads a step.
template <typename T, int D, int kHeads>
__global__ void __launch_bounds__(Lay<T, D>::THREADS, Lay<T, D>::BLOCKS)
paged_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    const T* __restrict__ q, const T* __restrict__ kn, const T* __restrict__ vn, T* K, T* V,
                    const PagedArgs p) {
    using Ly = Lay<T, D>;
    constexpr int KC = Ly::KC, VPL = Ly::VPL, VB = Ly::VB, NI = Ly::NI, ROWS = kHeads / 8, NT = D / 8;
    constexpr int STAGES = Ly::STAGES, PE = 16 / static_cast<int>(sizeof(T));  // values of 16 bytes
    constexpr int kWarps = Ly::WARPS, kThreads = Ly::THREADS;
    constexpr bool kBf16 = sizeof(T) == 2;
    extern __shared__ uint8_t sm_raw[];
    __shared__ uint64_t s_bar[kWarps][STAGES];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, warp = threadIdx.x >> 5;
    const int workers = gridDim.x * kWarps, worker = blockIdx.x * kWarps + warp;
    __shared__ int64_t s_pre[kThreads];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint64_t* bar = s_bar[warp];
    if (lane == 0) {
        for (int s = 0; s < STAGES; ++s) tc::mbar_init(bar + s, 1);
        tc::fence_mbar_init();
    }
    const int64_t total = sum_steps<kThreads>(p, s_pre);
    const int64_t each = total / workers;  // steps of a warp
    const int64_t cuts = static_cast<int64_t>(workers) * (p.next == nullptr || each < kTwo ? 1 : each < kFour ? 2 : 4);
    const int64_t per = max(static_cast<int64_t>(1), (total + cuts - 1) / cuts);
    const int ranges = static_cast<int>((total + per - 1) / per);
    if (!p.direct && lane == 0)
        for (int i = worker; i < p.max_ranges; i += workers)
            if (i >= ranges) p.desc[i] = make_int4(0, 0, 0, 0);
    if (worker >= ranges) return;
    const auto range_steps = [&](int i) { return static_cast<int>(min(per, total - i * per)); };
    // the number of the range after this one (its lane 0 asks ahead of time)
    const auto ask = [&]() { return p.next && lane == 0 ? workers + static_cast<int>(atomicAdd(p.next, 1u)) : INT_MAX; };
    uint8_t* ring = sm + warp * (STAGES * Ly::STAGE);
    const int off_mask = (1 << p.s.log2p) - 1;
    bool bad = false;

    int64_t base;
    int range = worker, after = ask();          // the range in work; the loader's next one
    const int row_at = locate<kThreads>(p, s_pre, range * per, base);
    Cursor ld(p, row_at, range * per - base);
    Cursor cs = ld, nx = ld;                    // nx: where the loader began its range, when it is ahead
    int nx_range = range;
    int n_left = range_steps(range);            // steps of the range in work
    bool whole = cs.j == cs.row.j0;             // the column's first step is this range's
    bool first_seg = true;
    if (!p.direct && lane == 0) p.desc[range] = make_int4(0, 0, 0, 0);

    const auto page_of = [&](const Cursor& c) {  // page of the lane's position (lane & 15) of a step
        const int pos = c.j * kStep + (lane & 15);
        const int at = pos >> p.s.log2p;
        return pos < c.row.len ? p.table[static_cast<int64_t>(c.r) * p.s.max_pages + at] : -1;
    };
    int to_load = n_left;                       // steps of the loader's range not yet copied
    int pg = page_of(ld);
    uint32_t seen[STAGES];  // positions that count, a bit each, of the steps in the ring, the current one first
#pragma unroll
    for (int s = 0; s < STAGES; ++s) seen[s] = 0;

    // Copies step `ld` into a stage and moves on; returns the positions that count and
    // whether lanes copied it.
    constexpr uint32_t kByLanes = 0x10000u;
    const auto issue = [&](int stage) -> uint32_t {
        uint32_t mask = 0xFFFFu;
        if (to_load > 0) {
            uint8_t* dst = ring + stage * Ly::STAGE;
            const int pos0 = ld.j * kStep, page = pg;
            const bool inside = p.tma && pos0 >= ld.row.first && pos0 + kStep <= ld.row.len &&
                                static_cast<unsigned>(page) < static_cast<unsigned>(p.s.num_pages);
            if (__all_sync(0xffffffffu, inside)) {  // 16 positions of one page, and all lanes are done with the stage
                if (lane == 0) {
                    const int y = pos0 & off_mask, z = page * p.s.Hkv + ld.kh;
                    tc::mbar_arrive_expect_tx(bar + stage, Ly::STAGE);
#pragma unroll
                    for (int a = 0; a < Ly::ATOMS; ++a) {
                        tc::tma_load_3d(dst + a * Ly::ATOM, &kmap, bar + stage, a * 8 * PE, y, z);
                        tc::tma_load_3d(dst + Ly::HALF + a * Ly::ATOM, &vmap, bar + stage, a * 8 * PE, y, z);
                    }
                }
            } else {
                if (lane == 0) tc::mbar_arrive(bar + stage);
                const uint32_t d32 = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
                const int mypos = pos0 + (lane & 15), len = ld.row.len;
                const bool mine = mypos >= ld.row.first && mypos < ld.row.total;
                const bool there = static_cast<unsigned>(page) < static_cast<unsigned>(p.s.num_pages);
                bad |= mine && mypos < len && !there;
                mask = __ballot_sync(0xffffffffu, mine && (there || mypos == len)) & 0xFFFFu;
                const int64_t nrow = static_cast<int64_t>(ld.r) * p.s.Hkv + ld.kh;
                const auto key_row = [&](int key, const T* pool, const T* fresh, bool& on) -> const T* {
                    const int pos = pos0 + key;
                    const int id = __shfl_sync(0xffffffffu, page, key);
                    on = mask >> key & 1u;
                    if (on && pos == len) return fresh + nrow * D;
                    const int64_t row = ((static_cast<int64_t>(id) * p.s.Hkv + ld.kh) << p.s.log2p) + (pos & off_mask);
                    return on ? pool + row * D : q;
                };
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    bool on;
                    const T* kr = key_row(8 * n + g, K, kn, on);
#pragma unroll
                    for (int i = 0; i < KC; ++i)
                        cp16(d32 + Ly::kat(g, t, n, i), on ? kr + Ly::kchunk(t, i) * PE : q, on);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    bool on;
                    const T* vr = key_row(Ly::vrow(t, e), V, vn, on);
#pragma unroll
                    for (int i = 0; i < NI; ++i) cpv<VB>(d32 + Ly::vat(g, t, e, i), on ? vr + (g + 8 * i) * VPL : q, on);
                }
                mask |= kByLanes;
            }
            if (--to_load > 0) {
                ld.advance(p);
                pg = page_of(ld);
            } else {  // on to the next range
                const int i = __shfl_sync(0xffffffffu, after, 0);
                if (i < ranges) {
                    const int r = locate<kThreads>(p, s_pre, i * per, base);
                    ld = Cursor(p, r, i * per - base);
                    pg = page_of(ld);
                    nx = ld;
                    nx_range = i;
                    to_load = range_steps(i);
                    after = ask();
                }
            }
        }
        return mask;
    };

    // query operands of a column: head g, and g + 8 with 16 heads (0 past the heads);
    // a negative scale goes into their sign, so that larger products stay larger
    // scores.  fp32 with 8 heads keeps both terms of the split.
    constexpr int QT = kBf16 ? ROWS : 2;
    const uint32_t flip = p.s.scale < 0.f ? (kBf16 ? 0x80008000u : 0x80000000u) : 0u;
    const float sc = fabsf(p.s.scale) * 1.4426950408889634f;
    uint32_t qf[QT][KC][4];
    const auto load_q = [&]() {
        const int h0 = cs.tile * kHeads;
        const int64_t row = static_cast<int64_t>(cs.r) * p.s.Hq + cs.kh * p.G + h0;
        const T* src = q + (row + g) * D;
#pragma unroll
        for (int z = 0; z < ROWS; ++z)
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (h0 + 8 * z + g < p.G) u = *reinterpret_cast<const uint4*>(src + 8 * z * D + Ly::kchunk(t, i) * PE);
                const uint32_t w[4] = {u.x ^ flip, u.y ^ flip, u.z ^ flip, u.w ^ flip};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if constexpr (!kBf16 && ROWS == 1) split_tf32_rn(w[x], qf[0][i][x], qf[1][i][x]);
                    else qf[z][i][x] = w[x];
                }
            }
    };

    // of head g (and g + 8): output sums, maximum (log2), sum of the weights of the lane's positions
    float o[NT][2 * ROWS], m[ROWS], l[ROWS];
    const auto clear = [&]() {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 2 * ROWS; ++e) o[i][e] = 0.f;
#pragma unroll
        for (int z = 0; z < ROWS; ++z) m[z] = -INFINITY, l[z] = 0.f;
    };
    const auto add = [](float(&to)[2 * ROWS], const float(&d)[4]) {  // rows 8 to 15: a second term, or heads
        if constexpr (ROWS == 1) {
            to[0] += d[0] + d[2];
            to[1] += d[1] + d[3];
        } else {
            to[0] += d[0], to[1] += d[1], to[2] += d[2], to[3] += d[3];
        }
    };
    clear();
    load_q();

#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) seen[s] = issue(s);
    int stage = 0;
    uint32_t phase = 0, limit = tcf::kWaitLimit;
    bool bad_wait = false;
    while (true) {
        {
            const int to = stage + STAGES - 1;
            seen[STAGES - 1] = issue(to >= STAGES ? to - STAGES : to);
        }
        const bool by_lanes = seen[0] & kByLanes;
        if (by_lanes) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            seen[0] &= 0xFFFFu;
        }
        if (!tc::mbar_wait(bar + stage, phase, limit)) {  // a copy never came: report it and go on
            bad_wait = true;
            limit = 1;
        }
        const uint8_t* st = ring + stage * Ly::STAGE;

        // scores of 16 keys: s[n][2 z + e] of head g + 8 z, key 8 n + 2 t + e
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
        for (int i = 0; i < KC; ++i) {
            uint32_t kw[2][4];
            float from0[2][4] = {};  // fp32 storage: each 64 bytes of the rows from zero, then added in fp32
            float(&d)[2][4] = kBf16 ? s : from0;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const uint4 k = *reinterpret_cast<const uint4*>(st + Ly::kat(g, t, n, i));
                kw[n][0] = k.x, kw[n][1] = k.y, kw[n][2] = k.z, kw[n][3] = k.w;
            }
#pragma unroll
            for (int h = 0; h < 4; h += 2) {
                if constexpr (kBf16) {
#pragma unroll
                    for (int n = 0; n < 2; ++n)
                        mma_bf16(d[n], qf[0][i][h], ROWS == 2 ? qf[ROWS - 1][i][h] : 0u, qf[0][i][h + 1],
                                 ROWS == 2 ? qf[ROWS - 1][i][h + 1] : 0u, kw[n][h], kw[n][h + 1]);
                } else {
                    uint32_t kh[2][2], kl[2][2];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        split_tf32_rn(kw[n][h], kh[n][0], kl[n][0]);
                        split_tf32_rn(kw[n][h + 1], kh[n][1], kl[n][1]);
                    }
                    if constexpr (ROWS == 1) {  // rows: both terms of q
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            mma_tf32(d[n], qf[0][i][h], qf[1][i][h], qf[0][i][h + 1], qf[1][i][h + 1], kh[n][0], kh[n][1]);
#pragma unroll
                        for (int n = 0; n < 2; ++n)
                            mma_tf32(d[n], qf[0][i][h], qf[1][i][h], qf[0][i][h + 1], qf[1][i][h + 1], kl[n][0], kl[n][1]);
                    } else {
                        uint32_t ah[4], al[4];
                        split_tf32_rn(qf[0][i][h], ah[0], al[0]);
                        split_tf32_rn(qf[1][i][h], ah[1], al[1]);
                        split_tf32_rn(qf[0][i][h + 1], ah[2], al[2]);
                        split_tf32_rn(qf[1][i][h + 1], ah[3], al[3]);
#pragma unroll
                        for (int n = 0; n < 2; ++n) mma_tf32(d[n], ah[0], ah[1], ah[2], ah[3], kh[n][0], kh[n][1]);
#pragma unroll
                        for (int n = 0; n < 2; ++n) mma_tf32(d[n], ah[0], ah[1], ah[2], ah[3], kl[n][0], kl[n][1]);
#pragma unroll
                        for (int n = 0; n < 2; ++n) mma_tf32(d[n], al[0], al[1], al[2], al[3], kh[n][0], kh[n][1]);
                    }
                }
            }
            if constexpr (!kBf16) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[n][e] += d[n][e];
            }
        }
        if constexpr (!kBf16) {
            bool nan = false;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                if constexpr (ROWS == 1) s[n][0] += s[n][2], s[n][1] += s[n][3];
#pragma unroll
                for (int e = 0; e < 2 * ROWS; ++e) nan |= s[n][e] != s[n][e];
            }
            if (__any_sync(0xffffffffu, nan)) {
#pragma unroll
                for (int z = 0; z < ROWS; ++z) {
                    const int h = cs.tile * kHeads + 8 * z + g;
                    const float* src = q + (static_cast<int64_t>(cs.r) * p.s.Hq + cs.kh * p.G + h) * D;
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float2 x = exact_scores<D>(st, src, h < p.G, n, flip ? -1.f : 1.f);
                        s[n][2 * z] = x.x, s[n][2 * z + 1] = x.y;
                    }
                }
            }
        }
        // to base 2, rounded once for the maximum and for the weights alike: the largest
        // score's weight is exactly 1, so a single position's row comes out bit for bit
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2 * ROWS; ++e) s[n][e] *= sc;
        if (seen[0] != 0xFFFFu) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2 * ROWS; ++e)
                    if (!(seen[0] >> (8 * n + 2 * t + (e & 1)) & 1u)) s[n][e] = -INFINITY;
        }
        bool up = false;
        float top[ROWS];
#pragma unroll
        for (int z = 0; z < ROWS; ++z) {
            top[z] = fmaxf(fmaxf(s[0][2 * z], s[0][2 * z + 1]), fmaxf(s[1][2 * z], s[1][2 * z + 1]));
            up |= top[z] > m[z] + kSlack;
        }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int z = 0; z < ROWS; ++z) {
                float y = fmaxf(top[z], __shfl_xor_sync(0xffffffffu, top[z], 1));
                y = fmaxf(m[z], fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2)));
                const float f = m[z] == y ? 1.f : ex2(m[z] - y);
                m[z] = y;
                l[z] *= f;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    o[i][2 * z] *= f;
                    o[i][2 * z + 1] *= f;
                }
            }
        }
        // weights; all of them 0 while no score is above -infinity
#pragma unroll
        for (int z = 0; z < ROWS; ++z) {
            const float at = m[z] == -INFINITY ? 0.f : m[z];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                s[n][2 * z] = ex2(s[n][2 * z] - at);
                s[n][2 * z + 1] = ex2(s[n][2 * z + 1] - at);
                l[z] += s[n][2 * z] + s[n][2 * z + 1];
            }
        }
        if constexpr (kBf16) {
            uint32_t w[3][ROWS][2];  // three terms of the weights
#pragma unroll
            for (int z = 0; z < ROWS; ++z)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    float x = s[n][2 * z], y = s[n][2 * z + 1];
#pragma unroll
                    for (int u = 0; u < 3; ++u) {
                        w[u][z][n] = pack2(x, y);
                        x -= __uint_as_float(w[u][z][n] << 16);
                        y -= __uint_as_float(w[u][z][n] & 0xFFFF0000u);
                    }
                }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                uint32_t v[4][VPL / 2];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (VB == 16) {
                        const uint4 f = *reinterpret_cast<const uint4*>(st + Ly::vat(g, t, e, i));
                        v[e][0] = f.x, v[e][1] = f.y, v[e][2] = f.z, v[e][3] = f.w;
                    } else {
                        const uint2 f = *reinterpret_cast<const uint2*>(st + Ly::vat(g, t, e, i));
                        v[e][0] = f.x, v[e][1] = f.y;
                    }
                }
                float d[VPL][4];
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
                    const uint32_t b0 = __byte_perm(v[0][j / 2], v[1][j / 2], sel);
                    const uint32_t b1 = __byte_perm(v[2][j / 2], v[3][j / 2], sel);
                    d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
                    if constexpr (ROWS == 1) {  // rows: the first two terms, then the third
                        mma_bf16(d[j], w[0][0][0], w[1][0][0], w[0][0][1], w[1][0][1], b0, b1);
                        mma_bf16(d[j], w[2][0][0], 0u, w[2][0][1], 0u, b0, b1);
                    } else {
#pragma unroll
                        for (int u = 0; u < 3; ++u)
                            mma_bf16(d[j], w[u][0][0], w[u][ROWS - 1][0], w[u][0][1], w[u][ROWS - 1][1], b0, b1);
                    }
                }
#pragma unroll
                for (int j = 0; j < VPL; ++j) add(o[i * VPL + j], d[j]);
            }
        } else {
            uint32_t wh[2][ROWS][2], wl[2][ROWS][2];  // keys 2t (operand k = t) and 2t + 1 (k = t + 4) of each tile
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int z = 0; z < ROWS; ++z)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        split_tf32_rn(__float_as_uint(s[n][2 * z + e]), wh[n][z][e], wl[n][z][e]);
            // half a unit of the second term, or 0 where a third one takes what the unit cuts off
            const uint32_t half = cs.row.total - cs.row.first <= kExact ? 0u : 0x1000u;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                uint32_t v[4][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint4 f = *reinterpret_cast<const uint4*>(st + Ly::vat(g, t, e, i));
                    v[e][0] = f.x, v[e][1] = f.y, v[e][2] = f.z, v[e][3] = f.w;
                }
                float d[4][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
                if (half == 0u) {
                    const uint32_t a0 = pack2(s[0][0], s[0][1]), a2 = pack2(s[1][0], s[1][1]);
                    const uint32_t a1 = ROWS == 2 ? pack2(s[0][2], s[0][3]) : 0u, a3 = ROWS == 2 ? pack2(s[1][2], s[1][3]) : 0u;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t r[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t hi, lo;
                            split_tf32(v[e][j], hi, lo);
                            r[e] = __float_as_uint(__uint_as_float(lo) - __uint_as_float(lo & 0xFFFFE000u));
                        }
                        mma_bf16(d[j], a0, a1, a2, a3, __byte_perm(r[0], r[1], 0x7632u), __byte_perm(r[2], r[3], 0x7632u));
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t h[4], c[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        split_tf32(v[e][j], h[e], c[e]);
                        c[e] += half;
                    }
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        constexpr int Z = ROWS - 1;
                        if constexpr (ROWS == 1) {  // rows: both terms of the weights
                            mma_tf32(d[j], wh[n][0][0], wl[n][0][0], wh[n][0][1], wl[n][0][1], c[2 * n], c[2 * n + 1]);
                            mma_tf32(d[j], wh[n][0][0], wl[n][0][0], wh[n][0][1], wl[n][0][1], h[2 * n], h[2 * n + 1]);
                        } else {
                            mma_tf32(d[j], wh[n][0][0], wh[n][Z][0], wh[n][0][1], wh[n][Z][1], c[2 * n], c[2 * n + 1]);
                            mma_tf32(d[j], wl[n][0][0], wl[n][Z][0], wl[n][0][1], wl[n][Z][1], h[2 * n], h[2 * n + 1]);
                            mma_tf32(d[j], wh[n][0][0], wh[n][Z][0], wh[n][0][1], wh[n][Z][1], h[2 * n], h[2 * n + 1]);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) add(o[i * 4 + j], d[j]);
            }
        }

        // the new row goes into the cache, once a key head
        if (p.append && cs.row.len >> 4 == cs.j && cs.tile == 0) {
            const int at = cs.row.len >> p.s.log2p;
            const int id = at < p.s.max_pages ? p.table[static_cast<int64_t>(cs.r) * p.s.max_pages + at] : -1;
            if (static_cast<unsigned>(id) < static_cast<unsigned>(p.s.num_pages)) {
                constexpr int PIECES = D * static_cast<int>(sizeof(T)) / 16;
                const int64_t to = ((static_cast<int64_t>(id) * p.s.Hkv + cs.kh) << p.s.log2p) + (cs.row.len & off_mask);
                const int64_t from = static_cast<int64_t>(cs.r) * p.s.Hkv + cs.kh;
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
            const int h0 = cs.tile * kHeads;
            const int64_t row0 = static_cast<int64_t>(cs.r) * p.s.Hq + cs.kh * p.G + h0;
            const bool done = whole && col_end;
            const int slot = first_seg ? 0 : 1;
            float* part = p.part + (static_cast<int64_t>(range) * 2 + slot) * p.heads * (D + 4);
#pragma unroll
            for (int z = 0; z < ROWS; ++z) {
                float sum = l[z] + __shfl_xor_sync(0xffffffffu, l[z], 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const int h = g + 8 * z;
                if (h0 + h < p.G) {
                    const float f = done ? (sum > 0.f || sum != sum ? 1.f / sum : 0.f) : 1.f;
                    float* dst = done ? p.out + (row0 + h) * D : part + h * D;
#pragma unroll
                    for (int i = 0; i < NI; ++i)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int j = 0; j < VPL; j += 4) {
                                float y[4];
#pragma unroll
                                for (int x = 0; x < 4; ++x) {
                                    y[x] = o[i * VPL + j + x][2 * z + c] * f;
                                }
                                *reinterpret_cast<float4*>(dst + (2 * t + c + 8 * i) * VPL + j) =
                                    make_float4(y[0], y[1], y[2], y[3]);
                            }
                    if (t == 0) {
                        if (!done) {
                            part[p.heads * D + 2 * h] = m[z];
                            part[p.heads * D + 2 * h + 1] = sum;
                        } else if (p.lse) {
                            p.lse[row0 + h] = (m[z] + log2f(sum)) * 0.6931471805599453f;
                        }
                    }
                }
            }
            if (lane == 0) {
                const int col = cs.r * p.HT + cs.col(p), index = p.direct ? col : range;
                if (whole && !col_end) {  // first range of a split column
                    const int64_t rest = cs.row.j1 - (cs.j + 1);
                    p.desc[index] = make_int4(range, static_cast<int>(1 + (rest + per - 1) / per), slot, col);
                } else if (whole && p.direct) {
                    p.desc[index] = make_int4(0, 0, 0, 0);
                }
            }
            first_seg = false;
            if (n_left > 1) {
                cs.advance(p);
                whole = true;
            } else {
                if (nx_range == range) break;  // the loader found no further range
                cs = nx;
                range = nx_range;
                n_left = range_steps(range) + 1;
                whole = cs.j == cs.row.j0;
                first_seg = true;
                if (!p.direct && lane == 0) p.desc[range] = make_int4(0, 0, 0, 0);
            }
            clear();
            load_q();
        } else {
            ++cs.j;
        }
        --n_left;
        if (by_lanes) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before TMA writes there again
        if (++stage == STAGES) stage = 0, phase ^= 1u;
#pragma unroll
        for (int s = 0; s + 1 < STAGES; ++s) seen[s] = seen[s + 1];
    }
    if (bad) atomicOr(p.status, kStatusBadIndex);
    if (bad_wait) atomicOr(p.status, tcf::kErrWait);
}

// Joins the ranges of a split column, one block a query head: the maximum of the
// ranges' maxima, then sums scaled to it, in the order of the ranges within each
// of the block's warps and of the warps.
template <int D, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_join_kernel(const PagedArgs p) {
    __shared__ float s_m[kJoinWarps], s_l[kJoinWarps], s_a[kJoinWarps][D];
    if (p.fill && blockIdx.y == 0)  // rows without a request, under the kernel before
        for (int r = blockIdx.x; r < p.s.R; r += gridDim.x)
            if (p.lens[r] < 0) {
                const int64_t row = static_cast<int64_t>(r) * p.s.Hq;
                for (int i = threadIdx.x; (p.fill & 1) && i < p.s.Hq * (D / 4); i += kJoinWarps * 32)
                    reinterpret_cast<float4*>(p.out + row * D)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int i = threadIdx.x; (p.fill & 2) && i < p.s.Hq; i += kJoinWarps * 32) p.lse[row + i] = -INFINITY;
            }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t index = blockIdx.x;
    const int h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t col = index;
    const int len = p.direct ? p.lens[index / p.HT] : 0;
    const int4 d = p.desc[index];  // unwritten for a row without a request
    if (len < 0 || d.y == 0) return;
    if (!p.direct) col = d.w;
    const int64_t r = col / p.HT;
    const int c = static_cast<int>(col - r * p.HT), kh = c / p.tiles_per_kh, h0 = (c - kh * p.tiles_per_kh) * p.heads;
    if (h0 + h >= p.G) return;
    constexpr int E = D / 32;
    float m = -INFINITY, l = 0.f, a[E];
#pragma unroll
    for (int e = 0; e < E; ++e) a[e] = 0.f;
    const int each = (d.y + kJoinWarps - 1) / kJoinWarps, i1 = min(d.y, (warp + 1) * each);
    // Ranges fetched at once: 8 where a column has many (13.2 us against 14.2 us with 4 at
    // 16 requests x 16 heads x 4000 positions), else 4 (48.9 us against 50.2 us with 8 at 64
    // requests x 4 x 16 heads, D = 64).
    constexpr int N = kJoinWarps == 16 ? 8 : 4;
    for (int i0 = warp * each; i0 < i1; i0 += N) {
        float pm[N], pl[N], v[N][E];
#pragma unroll
        for (int x = 0; x < N; ++x) {
            const int i = i0 + x;
            const float* part = p.part + ((static_cast<int64_t>(d.x) + i) * 2 + (i ? 0 : d.z)) * p.heads * (D + 4);
            pm[x] = i < i1 ? part[p.heads * D + 2 * h] : -INFINITY;
            pl[x] = i < i1 ? part[p.heads * D + 2 * h + 1] : 0.f;
            const float* row = part + h * D + lane * E;
            if constexpr (E == 4) {
                const float4 f = i < i1 ? *reinterpret_cast<const float4*>(row) : make_float4(0.f, 0.f, 0.f, 0.f);
                v[x][0] = f.x, v[x][1] = f.y, v[x][E - 2] = f.z, v[x][E - 1] = f.w;
            } else if constexpr (E == 2) {
                const float2 f = i < i1 ? *reinterpret_cast<const float2*>(row) : make_float2(0.f, 0.f);
                v[x][0] = f.x, v[x][E - 1] = f.y;
            } else {
                v[x][0] = i < i1 ? *row : 0.f;
            }
        }
#pragma unroll
        for (int x = 0; x < N; ++x) {
            const float y = fmaxf(m, pm[x]);
            const float f = m == y ? 1.f : ex2(m - y), g = pm[x] == -INFINITY ? 0.f : pm[x] == y ? 1.f : ex2(pm[x] - y);
            l = l * f + pl[x] * g;
#pragma unroll
            for (int e = 0; e < E; ++e) a[e] = a[e] * f + v[x][e] * g;
            m = y;
        }
    }
    if (lane == 0) s_m[warp] = m, s_l[warp] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) s_a[warp][lane * E + e] = a[e];
    __syncthreads();
    const int64_t row = r * p.s.Hq + kh * p.G + h0 + h;
    for (int i = threadIdx.x; i < D; i += kJoinWarps * 32) {
        float x = -INFINITY, tl = 0.f, ta = 0.f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) x = fmaxf(x, s_m[w]);
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            const float f = s_m[w] == -INFINITY ? (s_l[w] != s_l[w] ? 1.f : 0.f) : s_m[w] == x ? 1.f : ex2(s_m[w] - x);
            tl += s_l[w] * f;
            ta += s_a[w][i] * f;
        }
        p.out[row * D + i] = tl > 0.f || tl != tl ? ta / tl : 0.f;
        if (i == 0 && p.lse) p.lse[row] = (x + log2f(tl)) * 0.6931471805599453f;
    }
}

}  // namespace

namespace {

// Map over a pool [num_pages * Hkv][page_size][D] with a box of 16 rows x AB bytes.
template <typename T, int D>
cudaError_t pool_map(CUtensorMap* m, const void* pool, const PagedShape& s) {
    using Ly = Lay<T, D>;
    tcf::EncodeTiled enc = tcf::encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t page = 1ull << s.log2p;
    cuuint64_t dims[3] = {D, page, static_cast<cuuint64_t>(s.num_pages) * s.Hkv};
    cuuint64_t strides[2] = {D * sizeof(T), page * D * sizeof(T)};
    cuuint32_t box[3] = {Ly::AB / sizeof(T), kStep, 1}, es[3] = {1, 1, 1};
    const CUresult r = enc(m, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                           const_cast<void*>(pool), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           Ly::AB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Grid, ranges and scratch of a call; pure arithmetic.
struct Plan {
    int blocks, workers, tiles_per_kh, heads, max_ranges;
    int64_t cols, most;  // columns; steps at most
    bool single;         // one range a warp at most
    size_t part, desc, bytes;
};
template <typename T, int D, int kHeads>
Plan plan_of(const PagedShape& s, int num_sms) {
    Plan n = {};
    const int G = s.Hq / s.Hkv;
    n.blocks = Lay<T, D>::BLOCKS * num_sms;
    n.workers = n.blocks * Lay<T, D>::WARPS;
    n.tiles_per_kh = (G + kHeads - 1) / kHeads;
    n.heads = std::min(G, kHeads);
    n.cols = static_cast<int64_t>(s.R) * s.Hkv * n.tiles_per_kh;
    n.most = n.cols * ((static_cast<int64_t>(s.max_pages) << s.log2p) / kStep + 2);
    n.single = n.most < static_cast<int64_t>(n.workers) * kTwo;
    n.max_ranges = n.single ? n.workers : n.workers * 4;
    n.part = plan::up256(sizeof(float) * n.max_ranges * 2 * n.heads * (D + 4));
    n.desc = sizeof(int4) * n.max_ranges;
    n.bytes = n.part + n.desc + 16;
    return n;
}

template <typename T, int D, int kHeads>
cudaError_t launch(const LaunchCtx& c, const T* q, const T* k, const T* v, T* K, T* V, const int* table,
                   const int* lens, float* out, float* lse, const PagedShape& s, int fill) {
    using Ly = Lay<T, D>;
    auto* kernel = paged_decode_kernel<T, D, kHeads>;
    const Plan n = plan_of<T, D, kHeads>(s, c.num_sms);
    if (n.most / n.workers >= INT_MAX) return cudaErrorInvalidValue;  // a range's steps are counted in 32 bits
    int per_sm = 1;
    cudaError_t e = resident_blocks<paged_decode_kernel<T, D, kHeads>>(c.device, Ly::THREADS, Ly::SMEM, &per_sm);
    if (e != cudaSuccess) return e;
    PagedArgs p = {};
    p.s = s;
    p.G = s.Hq / s.Hkv;
    p.tiles_per_kh = n.tiles_per_kh;
    p.HT = s.Hkv * n.tiles_per_kh;
    p.append = k ? 1 : 0;
    p.table = table;
    p.lens = lens;
    p.out = out;
    p.lse = lse;
    p.fill = fill;
    p.status = c.status_word;
    p.max_ranges = n.max_ranges;
    p.heads = n.heads;
    p.direct = n.cols <= n.max_ranges;
    CUtensorMap kmap = {}, vmap = {};
    p.tma = s.log2p >= 4 && s.num_pages > 0 && static_cast<int64_t>(s.num_pages) * s.Hkv < INT_MAX;
    if (p.tma && ((e = pool_map<T, D>(&kmap, K, s)) != cudaSuccess || (e = pool_map<T, D>(&vmap, V, s)) != cudaSuccess))
        return e;
    uint8_t* base = nullptr;
    if ((e = scratch_alloc(c, reinterpret_cast<void**>(&base), n.bytes)) != cudaSuccess) return e;
    p.part = reinterpret_cast<float*>(base);
    p.desc = reinterpret_cast<int4*>(base + n.part);
    if (!n.single) {
        p.next = reinterpret_cast<unsigned*>(base + n.part + n.desc);
        e = cudaMemsetAsync(p.next, 0, 4, c.stream);
    }
    if (e == cudaSuccess) {
        kernel<<<n.blocks, Ly::THREADS, Ly::SMEM, c.stream>>>(kmap, vmap, q, k, v, K, V, p);
        note_launch();
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(p.direct ? n.cols : n.max_ranges), n.heads);
        // Warps by the ranges that a column can be cut into, so that each fetches its own at
        // once: 653 us with 2, 656 us with 4 at 256 x 16 key heads (2 ranges a column), 106 us
        // with 4, 107 us with 2 at 48 requests (about 10), 8.1 us with 8, 8.6 us with 16 at 4 x 4
        // (about 20).  But 4 at most where the blocks fill the GPU anyway (48.9 us against
        // 53.7 us with 8 at 64 x 4 x 16 heads).
        const int64_t most = std::min((n.most + n.cols - 1) / n.cols, n.max_ranges / n.cols + 2);
        const bool few = n.cols * n.heads <= 2 * static_cast<int64_t>(c.num_sms);
        const int warps = most <= 8 ? 2 : most <= 16 || !few ? 4 : most <= 32 ? 8 : 16;
        cfg.blockDim = dim3(32 * warps);
        cfg.stream = c.stream;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg,
                               warps == 2   ? paged_join_kernel<D, 2>
                               : warps == 4 ? paged_join_kernel<D, 4>
                               : warps == 8 ? paged_join_kernel<D, 8>
                                            : paged_join_kernel<D, 16>,
                               p);
        note_launch();
    }
    scratch_free(c, base);
    return e;
}

}  // namespace

template <typename T, int D>
cudaError_t paged_decode_step(const LaunchCtx& c, const T* q, const T* k, const T* v, T* K, T* V,
                              const int* table, const int* lens, float* out, float* lse,
                              const PagedShape& s, int fill) {
    return s.Hq / s.Hkv <= 8 ? launch<T, D, 8>(c, q, k, v, K, V, table, lens, out, lse, s, fill)
                             : launch<T, D, 16>(c, q, k, v, K, V, table, lens, out, lse, s, fill);
}

size_t paged_decode_scratch(const PagedShape& s, int D, bool bf16, int num_sms) {
    if (s.R == 0 || s.Hq == 0) return 0;
#define LA_PD_PLAN(T, d) \
    if (D == d) return s.Hq / s.Hkv <= 8 ? plan_of<T, d, 8>(s, num_sms).bytes : plan_of<T, d, 16>(s, num_sms).bytes;
    if (bf16) {
        LA_PD_PLAN(__nv_bfloat16, 32) LA_PD_PLAN(__nv_bfloat16, 64) LA_PD_PLAN(__nv_bfloat16, 128)
    } else {
        LA_PD_PLAN(float, 32) LA_PD_PLAN(float, 64) LA_PD_PLAN(float, 128)
    }
#undef LA_PD_PLAN
    return SIZE_MAX;
}

#define LA_INST_PD(T, D)                                                                          \
    template cudaError_t paged_decode_step<T, D>(const LaunchCtx&, const T*, const T*, const T*, T*, \
                                                 T*, const int*, const int*, float*, float*,      \
                                                 const PagedShape&, int);
LA_INST_PD(float, 32) LA_INST_PD(float, 64) LA_INST_PD(float, 128)
LA_INST_PD(__nv_bfloat16, 32) LA_INST_PD(__nv_bfloat16, 64) LA_INST_PD(__nv_bfloat16, 128)

}  // namespace la
