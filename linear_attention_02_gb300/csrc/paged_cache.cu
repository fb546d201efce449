// paged_cache.cu -- bookkeeping of the paged key-value cache: block tables and
// slot maps from request lengths, and rows of keys and values into their slots.
//
// A pool holds num_pages pages [Hkv][page_size][D] of keys and as many of
// values.  Position p of request r lives on page block_table[r][p / page_size]
// at offset p % page_size; its slot number is page * page_size + offset.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "la_common.cuh"
#include "la_launch.h"
#include "la_plan.h"

namespace la {
namespace {

constexpr int kMapThreads = 256;
constexpr int kMapShared = plan::kMapShared;

// One request's lengths made valid: cached and new positions that fit a table
// row of `cap` positions; `rows` keeps the given count of new rows.  A negative cached
// length without new rows is a row of the batch without a request, and not bad.
struct Request {
    int cached, fit, rows, old_pages, need;
    bool bad;
    __device__ Request(int c, int n, int log2p, int max_pages) {
        const int64_t cap = static_cast<int64_t>(max_pages) << log2p;
        bad = n < 0 || (c < 0 && n > 0) || static_cast<int64_t>(c) + n > cap;
        c = max(c, 0);
        rows = max(n, 0);
        cached = static_cast<int>(c < cap ? c : cap);
        const int64_t room = cap - cached;
        fit = static_cast<int>(rows < room ? rows : room);
        const int64_t m = (1 << log2p) - 1;
        old_pages = static_cast<int>((cached + m) >> log2p);
        need = static_cast<int>((static_cast<int64_t>(cached) + fit + m) >> log2p) - old_pages;
    }
};

struct MapArgs {
    const int *cached, *fresh, *free_pages;
    int R, num_free, log2p, num_pages, max_pages, max_tokens;
    int *table, *slots, *starts, *counts;
    int2* sums;  // [R + 1] running sums (rows, pages) in memory, for more than kMapShared requests
    unsigned* status;
};

__device__ __forceinline__ int clamp_int(int64_t x) { return static_cast<int>(min(x, static_cast<int64_t>(INT_MAX))); }

// Running sums of new rows and of wanted pages before every request, and after the
// last: sums[0 .. R], cut to INT_MAX.  Returns whether a request's lengths are bad.
template <int NT>
__device__ __forceinline__ bool map_sums(const MapArgs& p, int2* sums) {
    __shared__ int64_t s_row[NT / 32], s_page[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, each = (p.R + NT - 1) / NT, r0 = tid * each;
    bool bad = false;
    int64_t rows = 0, pages = 0;
    for (int i = 0; i < each; ++i) {
        if (r0 + i >= p.R) break;
        const Request q(p.cached[r0 + i], p.fresh[r0 + i], p.log2p, p.max_pages);
        bad |= q.bad;
        rows += q.rows;
        pages += q.need;
    }
    int64_t a = rows, b = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) a += x, b += y;
    }
    if (lane == 31) s_row[tid / 32] = a, s_page[tid / 32] = b;
    __syncthreads();
    a -= rows;
    b -= pages;
    for (int w = 0; w < tid / 32; ++w) a += s_row[w], b += s_page[w];
    for (int i = 0; i < each; ++i) {
        if (r0 + i >= p.R) break;
        sums[r0 + i] = make_int2(clamp_int(a), clamp_int(b));
        const Request q(p.cached[r0 + i], p.fresh[r0 + i], p.log2p, p.max_pages);
        a += q.rows;
        b += q.need;
    }
    if (tid == NT - 1) {  // its sums end after the last request, whether it has any or not
        int64_t x = 0, y = 0;
        for (int w = 0; w < NT / 32; ++w) x += s_row[w], y += s_page[w];
        sums[p.R] = make_int2(clamp_int(x), clamp_int(y));
    }
    return bad;
}

// Fills the outputs from the running sums: rows, opened pages and requests in turn
// over all threads; a row or page finds its request by bisection.
__device__ __forceinline__ bool map_fill(const MapArgs& p, const int2* sums) {
    const int id = blockIdx.x * kMapThreads + threadIdx.x, all = gridDim.x * kMapThreads;
    const int rows = sums[p.R].x, pages = sums[p.R].y, mask = (1 << p.log2p) - 1;
    bool bad = rows > p.max_tokens;
    const auto find = [&](int i, bool by_page) {  // last request whose sum before it is <= i
        int lo = 0, hi = p.R;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            const int2 s = sums[mid];
            if ((by_page ? s.y : s.x) <= i) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    const auto free_page = [&](int i) {  // -1 where there is none
        const int f = i < p.num_free ? p.free_pages[i] : -1;
        return static_cast<unsigned>(f) < static_cast<unsigned>(p.num_pages) ? f : -1;
    };
    // four rows a thread, with one look for their first request
    for (int64_t i0 = 4 * static_cast<int64_t>(id); i0 < p.max_tokens; i0 += 4 * static_cast<int64_t>(all)) {
        const int n = min(4, p.max_tokens - static_cast<int>(i0));
        int out[4] = {-1, -1, -1, -1};
        if (i0 < rows) {
            int r = find(static_cast<int>(i0), false), end = sums[r + 1].x;
            Request q(p.cached[r], p.fresh[r], p.log2p, p.max_pages);
            for (int x = 0; x < n; ++x) {
                const int i = static_cast<int>(i0) + x;
                if (i >= rows) break;
                while (i >= end) {
                    end = sums[++r + 1].x;
                    q = Request(p.cached[r], p.fresh[r], p.log2p, p.max_pages);
                }
                const int j = i - sums[r].x;
                if (j >= q.fit) continue;
                const int64_t pos = static_cast<int64_t>(q.cached) + j;
                const int col = static_cast<int>(pos >> p.log2p);
                const int page = col < q.old_pages ? p.table[static_cast<int64_t>(r) * p.max_pages + col]
                                                   : free_page(clamp_int(static_cast<int64_t>(sums[r].y) + col - q.old_pages));
                if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages))
                    out[x] = (page << p.log2p) + static_cast<int>(pos & mask);
                else
                    bad = true;
            }
        }
        int* dst = p.slots + i0;
        if (n == 4 && (reinterpret_cast<uintptr_t>(p.slots) & 15u) == 0) {
            *reinterpret_cast<int4*>(dst) = make_int4(out[0], out[1], out[2], out[3]);
        } else {
            for (int x = 0; x < n; ++x) dst[x] = out[x];
        }
    }
    for (int64_t i = id; i < pages; i += all) {
        const int r = find(static_cast<int>(i), true), page = free_page(static_cast<int>(i));
        const Request q(p.cached[r], p.fresh[r], p.log2p, p.max_pages);
        bad |= page < 0;
        p.table[static_cast<int64_t>(r) * p.max_pages + q.old_pages + (i - sums[r].y)] = page;
    }
    for (int64_t r = id; r <= p.R; r += all) p.starts[r] = sums[r].x;
    if (id == 0) p.counts[0] = rows, p.counts[1] = pages;
    return bad;
}

// Up to kMapShared requests: every block adds up all lengths for itself (two loads a
// request from L2, one block-wide sum), so that one launch does it all.
__global__ void __launch_bounds__(kMapThreads) page_map_kernel(const MapArgs p) {
    __shared__ int2 s_sums[kMapShared + 1];
    bool bad = map_sums<kMapThreads>(p, s_sums);
    __syncthreads();
    bad |= map_fill(p, s_sums);
    if (bad) atomicOr(p.status, kStatusBadIndex);
}

// More requests: one block adds up, a second kernel fills.
__global__ void __launch_bounds__(1024) page_sums_kernel(const MapArgs p) {
    if (map_sums<1024>(p, p.sums)) atomicOr(p.status, kStatusBadIndex);
}
__global__ void __launch_bounds__(kMapThreads) page_fill_kernel(const MapArgs p) {
    if (map_fill(p, p.sums)) atomicOr(p.status, kStatusBadIndex);
}

// A thread moves one 16-byte piece of a key row and of a value row.
__global__ void paged_append_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                                    uint4* __restrict__ K, uint4* __restrict__ V,
                                    const int* __restrict__ slots, int64_t n, int Hkv, int row16,
                                    int log2p, int64_t num_slots, unsigned* status) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    const int64_t per = static_cast<int64_t>(Hkv) * row16;
    const int64_t t = i / per;
    const int e = static_cast<int>(i - t * per), h = e / row16, c = e - h * row16;
    const int slot = slots[t];
    if (slot < 0 || slot >= num_slots) {
        if (slot != -1) atomicOr(status, kStatusBadIndex);
        return;
    }
    const int64_t page = slot >> log2p, off = slot & ((1 << log2p) - 1);
    const int64_t to = ((((page * Hkv + h) << log2p) + off)) * row16 + c;
    K[to] = k[i];
    V[to] = v[i];
}

}  // namespace

cudaError_t page_map(const LaunchCtx& c, const int* cached, const int* fresh, int R,
                     const int* free_pages, int num_free, int log2p, int num_pages, int* table,
                     int max_pages, int* slots, int max_tokens, int* starts, int* counts) {
    MapArgs p = {cached, fresh, free_pages, R, num_free, log2p, num_pages, max_pages, max_tokens,
                 table, slots, starts, counts, nullptr, c.status_word};
    // four rows a thread, or a request a thread, up to two blocks an SM
    const int64_t work = std::max<int64_t>((static_cast<int64_t>(max_tokens) + 3) / 4, R + 1);
    const int blocks = static_cast<int>(std::min<int64_t>((work + kMapThreads - 1) / kMapThreads, 2 * c.num_sms));
    if (R <= kMapShared) {
        page_map_kernel<<<blocks, kMapThreads, 0, c.stream>>>(p);
        note_launch();
        return cudaGetLastError();
    }
    cudaError_t e = scratch_alloc(c, reinterpret_cast<void**>(&p.sums), plan::page_map_scratch(R));
    if (e != cudaSuccess) return e;
    page_sums_kernel<<<1, 1024, 0, c.stream>>>(p);
    page_fill_kernel<<<blocks, kMapThreads, 0, c.stream>>>(p);
    note_launch(2);
    e = cudaGetLastError();
    scratch_free(c, p.sums);
    return e;
}

cudaError_t paged_append(const LaunchCtx& c, const void* k, const void* v, void* K, void* V,
                         const int* slots, int T, int Hkv, int row_bytes, int log2p, int num_pages) {
    const int row16 = row_bytes / 16;
    const int64_t n = static_cast<int64_t>(T) * Hkv * row16;
    paged_append_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, c.stream>>>(
        static_cast<const uint4*>(k), static_cast<const uint4*>(v), static_cast<uint4*>(K),
        static_cast<uint4*>(V), slots, n, Hkv, row16, log2p, static_cast<int64_t>(num_pages) << log2p,
        c.status_word);
    note_launch();
    return cudaGetLastError();
}

}  // namespace la
