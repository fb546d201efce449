// paged_prefill.cu -- attention of each request's new tokens over its pages: query i of
// request r stands at position p = cached_lens[r] + i, whose key is in the cache already, and
//     out = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m},  s_j = scale q . k_j,
// over the positions j <= p (of these the last `window`); lse = m + ln sum_j e^{s_j - m}.
// Query head h reads key head h / (Hq / Hkv).
//
// The rows of a request and key head are its tokens' query heads, token after token; a block
// takes 16 of them and walks over the keys that any of them sees, 32 at a time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "la_common.cuh"
#include "la_launch.h"
#include "la_plan.h"

namespace la {
namespace {

constexpr int kRows = 16, kKeys = 32, kThreads = 128;

struct PrefillArgs {
    PrefillShape s;
    int G;
    const int *table, *lens, *starts;
    float* lse;
    int fill;
    unsigned* status;
};

// A request's rows and positions made valid.
struct Request {
    int first, n, cached;  // its first row, its rows (0: none), positions before them
    int64_t end;           // positions that its table has room for
    bool bad, pad;
    __device__ Request(const PrefillArgs& p, int r) {
        const int a = p.starts[r], b = p.starts[r + 1], len = p.lens[r];
        first = min(max(a, 0), p.s.T);
        const int last = min(max(b, first), p.s.T);
        n = last - first;
        pad = len < 0;
        cached = max(len, 0);
        end = static_cast<int64_t>(p.s.max_pages) << p.s.log2p;
        bad = a != first || b != last || (!pad && n > 0 && static_cast<int64_t>(cached) + n > end);
        if (cached > end) cached = static_cast<int>(end);
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) paged_prefill_kernel(const T* __restrict__ q, const T* __restrict__ K,
                                                                 const T* __restrict__ V, T* __restrict__ out,
                                                                 const PrefillArgs p) {
    __shared__ float s_q[kRows][D], s_k[kKeys][D + 1], s_v[kKeys][D];
    __shared__ int s_page[kKeys];
    constexpr int E = D / 32, W = kRows / 4;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kh = blockIdx.y;
    int64_t tile = blockIdx.x;
    int r = 0;
    bool bad = false, found = false;
    for (; r < p.s.R; ++r) {
        const Request a(p, r);
        bad |= a.bad;
        const int64_t tiles = a.pad ? 0 : (static_cast<int64_t>(a.n) * p.G + kRows - 1) / kRows;
        if (tile < tiles) {
            found = true;
            break;
        }
        tile -= tiles;
    }
    if (bad && threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
    // rows without a request
    if (p.fill && kh == 0) {
        const int64_t last = p.s.R ? min(max(p.starts[p.s.R], 0), p.s.T) : 0;
        for (int64_t i = last + blockIdx.x; i < p.s.T; i += gridDim.x)
            for (int e = threadIdx.x; e < p.s.Hq * D; e += kThreads) {
                if (p.fill & 1) out[i * p.s.Hq * D + e] = from_f<T>(0.f);
                if ((p.fill & 2) && e < p.s.Hq) p.lse[i * p.s.Hq + e] = -INFINITY;
            }
        for (int x = blockIdx.x; x < p.s.R; x += gridDim.x) {
            const Request a(p, x);
            if (!a.pad) continue;
            for (int64_t e = threadIdx.x; e < static_cast<int64_t>(a.n) * p.s.Hq * D; e += kThreads) {
                if (p.fill & 1) out[static_cast<int64_t>(a.first) * p.s.Hq * D + e] = from_f<T>(0.f);
                if ((p.fill & 2) && e < static_cast<int64_t>(a.n) * p.s.Hq) p.lse[static_cast<int64_t>(a.first) * p.s.Hq + e] = -INFINITY;
            }
        }
    }
    if (!found) return;
    const Request a(p, r);
    const int64_t m0 = tile * kRows, rows = static_cast<int64_t>(a.n) * p.G;
    const auto row_of = [&](int64_t m) {  // in q and out
        return (static_cast<int64_t>(a.first) + m / p.G) * p.s.Hq + static_cast<int64_t>(kh) * p.G + m % p.G;
    };
    for (int i = threadIdx.x; i < kRows * D; i += kThreads) {
        const int64_t m = m0 + i / D;
        s_q[i / D][i % D] = m < rows ? to_f<T>(q[row_of(m) * D + i % D]) : 0.f;
    }
    int64_t pos[W];
    float mx[W], sum[W], o[W][E];
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int64_t m = m0 + warp * W + w;
        pos[w] = m < rows ? a.cached + m / p.G : -1;
        mx[w] = -INFINITY, sum[w] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[w][e] = 0.f;
    }
    const int64_t first = a.cached + m0 / p.G, last = a.cached + (min(m0 + kRows, rows) - 1) / p.G;
    const int64_t lo = p.s.window ? max(first - p.s.window + 1, static_cast<int64_t>(0)) : 0;
    const float c = p.s.scale * 1.4426950408889634f;
    for (int64_t k0 = lo; k0 <= last && k0 < a.end; k0 += kKeys) {
        __syncthreads();
        if (threadIdx.x < kKeys) {
            const int64_t x = k0 + threadIdx.x;
            int page = -1;
            if (x <= last && x < a.end) {
                page = p.table[static_cast<int64_t>(r) * p.s.max_pages + (x >> p.s.log2p)];
                if (static_cast<unsigned>(page) >= static_cast<unsigned>(p.s.num_pages)) page = -1, bad = true;
            }
            s_page[threadIdx.x] = page;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kKeys * D; i += kThreads) {
            const int j = i / D, d = i % D, page = s_page[j];
            const int64_t at = page < 0 ? 0 : (((static_cast<int64_t>(page) * p.s.Hkv + kh) << p.s.log2p) +
                                               ((k0 + j) & ((1 << p.s.log2p) - 1))) * D + d;
            s_k[j][d] = page < 0 ? 0.f : to_f<T>(K[at]);
            s_v[j][d] = page < 0 ? 0.f : to_f<T>(V[at]);
        }
        __syncthreads();
        const int64_t x = k0 + lane;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            float s = 0.f;
#pragma unroll 8
            for (int d = 0; d < D; ++d) s = fmaf(s_q[warp * W + w][d], s_k[lane][d], s);
            const bool seen = s_page[lane] >= 0 && x <= pos[w] && (p.s.window == 0 || x > pos[w] - p.s.window);
            s = seen ? s * c : -INFINITY;
            float top = s;
#pragma unroll
            for (int k = 16; k; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
            const float was = mx[w];
            mx[w] = fmaxf(was, top);
            const float f = was == mx[w] ? 1.f : exp2f(was - mx[w]), e = seen ? exp2f(s - mx[w]) : 0.f;
            float t = e;
#pragma unroll
            for (int k = 16; k; k >>= 1) t += __shfl_xor_sync(0xffffffffu, t, k);
            sum[w] = sum[w] * f + t;
#pragma unroll
            for (int i = 0; i < E; ++i) o[w][i] *= f;
            const unsigned who = __ballot_sync(0xffffffffu, seen);
            for (int j = 0; j < kKeys; ++j) {
                const float y = __shfl_sync(0xffffffffu, e, j);
                if (who >> j & 1u) {  // a value that the row does not see may be anything
#pragma unroll
                    for (int i = 0; i < E; ++i) o[w][i] = fmaf(y, s_v[j][lane + 32 * i], o[w][i]);
                }
            }
        }
    }
    if (bad) atomicOr(p.status, kStatusBadIndex);
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int64_t m = m0 + warp * W + w;
        if (m >= rows) continue;
        const bool some = sum[w] > 0.f || sum[w] != sum[w];
#pragma unroll
        for (int i = 0; i < E; ++i) out[row_of(m) * D + lane + 32 * i] = from_f<T>(some ? o[w][i] / sum[w] : 0.f);
        if (lane == 0 && p.lse) p.lse[row_of(m)] = some ? (mx[w] + log2f(sum[w])) * 0.6931471805599453f : -INFINITY;
    }
}

}  // namespace

template <typename T, int D>
cudaError_t paged_prefill(const LaunchCtx& c, const T* q, const T* K, const T* V, const int* table,
                          const int* lens, const int* starts, T* out, float* lse,
                          const PrefillShape& s, int fill) {
    if constexpr (sizeof(T) == 2) return paged_prefill_tc<D>(c, q, K, V, table, lens, starts, out, lse, s, fill);
    PrefillArgs p = {s, s.Hq / s.Hkv, table, lens, starts, lse, fill, c.status_word};
    const int64_t tiles = (static_cast<int64_t>(s.T) * p.G + kRows - 1) / kRows + s.R;
    paged_prefill_kernel<T, D><<<dim3(static_cast<unsigned>(tiles), s.Hkv), kThreads, 0, c.stream>>>(q, K, V, out, p);
    note_launch();
    return cudaGetLastError();
}

#define LA_INST_PP(T, D)                                                                               \
    template cudaError_t paged_prefill<T, D>(const LaunchCtx&, const T*, const T*, const T*, const int*, \
                                             const int*, const int*, T*, float*, const PrefillShape&, int);
LA_INST_PP(float, 32) LA_INST_PP(float, 64) LA_INST_PP(float, 128)
LA_INST_PP(__nv_bfloat16, 32) LA_INST_PP(__nv_bfloat16, 64) LA_INST_PP(__nv_bfloat16, 128)

}  // namespace la
