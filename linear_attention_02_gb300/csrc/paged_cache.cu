// paged_cache.cu -- bookkeeping of the paged key-value cache: block tables and
// slot maps from request lengths, and rows of keys and values into their slots.
//
// A pool holds num_pages pages [Hkv][page_size][D] of keys and as many of
// values.  Position p of request r lives on page block_table[r][p / page_size]
// at offset p % page_size; its slot number is page * page_size + offset.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>

#include "la_common.cuh"
#include "la_launch.h"
#include "la_plan.h"

namespace la {
namespace {

constexpr int kMapThreads = 1024;

// One request's lengths made valid: cached and new positions that fit a table
// row of `cap` positions; `rows` keeps the given count of new rows.
struct Request {
    int cached, fit, rows, old_pages, need;
    bool bad;
    __device__ Request(int c, int n, int log2p, int max_pages) {
        const int64_t cap = static_cast<int64_t>(max_pages) << log2p;
        bad = c < 0 || n < 0 || static_cast<int64_t>(c) + n > cap;
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

__global__ void __launch_bounds__(kMapThreads)
page_map_kernel(const int* __restrict__ cached, const int* __restrict__ fresh, int R,
                const int* __restrict__ free_pages, int num_free, int log2p, int num_pages,
                int* __restrict__ table, int max_pages, int* __restrict__ slots, int max_tokens,
                int* __restrict__ starts, int* __restrict__ counts, unsigned* status) {
    __shared__ int64_t s_tok, s_page;
    bool bad = false;
    if (threadIdx.x == 0) s_tok = s_page = 0;
    __syncthreads();
    for (int r = 0; r < R; ++r) {
        const Request q(cached[r], fresh[r], log2p, max_pages);
        bad |= q.bad;
        const int64_t tok = s_tok, pg = s_page;
        if (threadIdx.x == 0) starts[r] = static_cast<int>(min(tok, static_cast<int64_t>(INT_MAX)));
        for (int i = threadIdx.x; i < q.need; i += kMapThreads) {
            int id = pg + i < num_free ? free_pages[pg + i] : -1;
            if (id < 0 || id >= num_pages) id = -1, bad = true;
            table[static_cast<int64_t>(r) * max_pages + q.old_pages + i] = id;
        }
        for (int j = threadIdx.x; j < q.rows; j += kMapThreads) {
            if (tok + j >= max_tokens) {
                bad = true;
                break;
            }
            int slot = -1;
            if (j < q.fit) {
                const int64_t pos = static_cast<int64_t>(q.cached) + j;
                const int col = static_cast<int>(pos >> log2p);
                int id = -1;
                if (col < q.old_pages) id = table[static_cast<int64_t>(r) * max_pages + col];
                else if (pg + col - q.old_pages < num_free) id = free_pages[pg + col - q.old_pages];
                if (id >= 0 && id < num_pages) slot = (id << log2p) + static_cast<int>(pos & ((1 << log2p) - 1));
                else bad = true;
            }
            slots[tok + j] = slot;
        }
        __syncthreads();
        if (threadIdx.x == 0) s_tok += q.rows, s_page += q.need;
        __syncthreads();
    }
    const int64_t tok = s_tok, pg = s_page;
    for (int64_t j = tok + threadIdx.x; j < max_tokens; j += kMapThreads) slots[j] = -1;
    if (tok > max_tokens) bad = true;
    if (threadIdx.x == 0) {
        starts[R] = counts[0] = static_cast<int>(min(tok, static_cast<int64_t>(INT_MAX)));
        counts[1] = static_cast<int>(min(pg, static_cast<int64_t>(INT_MAX)));
    }
    if (bad) atomicOr(status, kStatusBadIndex);
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
    page_map_kernel<<<1, kMapThreads, 0, c.stream>>>(cached, fresh, R, free_pages, num_free, log2p,
                                                    num_pages, table, max_pages, slots, max_tokens,
                                                    starts, counts, c.status_word);
    note_launch();
    return cudaGetLastError();
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
