// paged_decode.cu -- attention of one new token over a paged key-value cache:
// per request r and query head,
//     out = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m},  s_j = scale q . k_j,  m = max_j s_j
// over the request's own positions (its pages, then its own new row), and
// lse = m + ln sum_j e^{s_j - m}.  Query head h reads key head h / (Hq / Hkv).
//
// A warp takes one query head of one request, its lanes the head's columns.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_common.cuh"
#include "la_launch.h"
#include "la_plan.h"

namespace la {
namespace {

template <typename T, int D>
__global__ void __launch_bounds__(128)
paged_decode_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, T* K,
                    T* V, const int* __restrict__ table, const int* __restrict__ lens,
                    float* __restrict__ out, float* __restrict__ lse, PagedShape s, unsigned* status) {
    constexpr int E = D / 32;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 32;
    if (row >= static_cast<int64_t>(s.R) * s.Hq) return;
    const int lane = threadIdx.x & 31, r = static_cast<int>(row / s.Hq), h = static_cast<int>(row % s.Hq);
    const int G = s.Hq / s.Hkv, kh = h / G;
    int len = lens[r];
    if (len < 0) return;
    const int64_t cap = static_cast<int64_t>(s.max_pages) << s.log2p;
    bool bad = k ? len >= cap : len > cap;
    if (len > cap) len = static_cast<int>(cap);
    const int total = len + (k ? 1 : 0);
    const int j0 = s.window && s.window < total ? total - s.window : 0;
    float qv[E], acc[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qv[e] = to_f(q[row * D + lane + 32 * e]) * s.scale;
        acc[e] = 0.f;
    }
    const int64_t nrow = (static_cast<int64_t>(r) * s.Hkv + kh) * D;
    for (int j = j0; j < total; ++j) {
        const T *kp, *vp;
        if (j == len) {
            kp = k + nrow;
            vp = v + nrow;
        } else {
            const int id = table[static_cast<int64_t>(r) * s.max_pages + (j >> s.log2p)];
            if (id < 0 || id >= s.num_pages) {
                bad = true;
                continue;
            }
            const int64_t at = ((((static_cast<int64_t>(id) * s.Hkv + kh) << s.log2p) +
                                 (j & ((1 << s.log2p) - 1)))) * D;
            kp = K + at;
            vp = V + at;
        }
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x = fmaf(qv[e], to_f(kp[lane + 32 * e]), x);
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        const float mn = fmaxf(m, x);
        const float f = m == mn ? 1.f : expf(m - mn), p = x == mn ? 1.f : expf(x - mn);
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(p, to_f(vp[lane + 32 * e]), acc[e] * f);
        m = mn;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) out[row * D + lane + 32 * e] = l > 0.f ? acc[e] / l : 0.f;
    if (lse && lane == 0) lse[row] = m + logf(l);
    if (k && h % G == 0) {  // the new row goes into the cache
        const int id = len < cap ? table[static_cast<int64_t>(r) * s.max_pages + (len >> s.log2p)] : -1;
        if (id >= 0 && id < s.num_pages) {
            const int64_t at = ((((static_cast<int64_t>(id) * s.Hkv + kh) << s.log2p) +
                                 (len & ((1 << s.log2p) - 1)))) * D;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                K[at + lane + 32 * e] = k[nrow + lane + 32 * e];
                V[at + lane + 32 * e] = v[nrow + lane + 32 * e];
            }
        } else {
            bad = true;
        }
    }
    if (bad) atomicOr(status, kStatusBadIndex);
}

}  // namespace

template <typename T, int D>
cudaError_t paged_decode_step(const LaunchCtx& c, const T* q, const T* k, const T* v, T* K, T* V,
                              const int* table, const int* lens, float* out, float* lse,
                              const PagedShape& s) {
    const int64_t rows = static_cast<int64_t>(s.R) * s.Hq;
    paged_decode_kernel<T, D><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, c.stream>>>(
        q, k, v, K, V, table, lens, out, lse, s, c.status_word);
    note_launch();
    return cudaGetLastError();
}

#define LA_INST_PD(T, D)                                                                          \
    template cudaError_t paged_decode_step<T, D>(const LaunchCtx&, const T*, const T*, const T*, T*, \
                                                 T*, const int*, const int*, float*, float*,      \
                                                 const PagedShape&);
LA_INST_PD(float, 32) LA_INST_PD(float, 64) LA_INST_PD(float, 128)
LA_INST_PD(__nv_bfloat16, 32) LA_INST_PD(__nv_bfloat16, 64) LA_INST_PD(__nv_bfloat16, 128)

}  // namespace la
