// gated_scan.cu -- the gated linear recurrence over token-major rows [B][N][C],
// one decay per token and channel:
//     decay form   h_t = a_t h_{t-1} + x_t
//     logit form   h_t = s_t h_{t-1} + (1 - s_t) x_t,  s_t = sigmoid(a_t)
// forward, backward and the single-token step.  The state is fp32.
//
// A thread walks one channel of one sequence from its first row to its last.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "la_common.cuh"
#include "la_launch.h"
#include "la_plan.h"

namespace la {
namespace {

constexpr int kScanThreads = 128;

// s = sigmoid(z), c = 1 - s = sigmoid(-z), each from the exponential that does not overflow.
__device__ __forceinline__ void sigmoid_pair(float z, float& s, float& c) {
    const float e = expf(-fabsf(z)), r = 1.f / (1.f + e);
    s = z >= 0.f ? r : e * r;
    c = z >= 0.f ? e * r : r;
}

// Decay, its complement factor on x, of one element.
template <bool kLogit>
__device__ __forceinline__ void gate(float a, float& s, float& c) {
    if constexpr (kLogit) {
        sigmoid_pair(a, s, c);
    } else {
        s = a;
        c = 1.f;
    }
}

// Rows [t0, t1) of sequence `seq` (global row numbers over all batch rows).
__device__ __forceinline__ void seq_rows(const int* starts, int seq, int N, int64_t& t0, int64_t& t1) {
    if (starts) {
        t0 = min(max(starts[seq], 0), N);
        t1 = min(max(starts[seq + 1], static_cast<int>(t0)), N);
    } else {
        t0 = static_cast<int64_t>(seq) * N;
        t1 = t0 + N;
    }
}

template <typename T, bool kLogit>
__global__ void scan_forward_kernel(const T* __restrict__ A, const T* __restrict__ X, T* __restrict__ O,
                                    int N, int C, const int* __restrict__ starts,
                                    const float* __restrict__ h_init, float* __restrict__ h_final,
                                    float* __restrict__ hs) {
    const int c = blockIdx.y * kScanThreads + threadIdx.x;
    if (c >= C) return;
    const int seq = blockIdx.x;
    int64_t t0, t1;
    seq_rows(starts, seq, N, t0, t1);
    float h = h_init ? h_init[static_cast<int64_t>(seq) * C + c] : 0.f;
    for (int64_t t = t0; t < t1; ++t) {
        float s, m;
        gate<kLogit>(to_f(A[t * C + c]), s, m);
        if (hs) hs[t * C + c] = h;
        h = fmaf(s, h, m * to_f(X[t * C + c]));
        if (O) O[t * C + c] = from_f<T>(h);
    }
    if (h_final) h_final[static_cast<int64_t>(seq) * C + c] = h;
}

// hs[t] = h_{t-1}.
template <typename T, bool kLogit>
__global__ void scan_backward_kernel(const T* __restrict__ A, const T* __restrict__ X,
                                     const T* __restrict__ G, T* __restrict__ dA, T* __restrict__ dX,
                                     int N, int C, const int* __restrict__ starts,
                                     const float* __restrict__ dh_final, float* __restrict__ dh_init,
                                     const float* __restrict__ hs) {
    const int c = blockIdx.y * kScanThreads + threadIdx.x;
    if (c >= C) return;
    const int seq = blockIdx.x;
    int64_t t0, t1;
    seq_rows(starts, seq, N, t0, t1);
    float carry = dh_final ? dh_final[static_cast<int64_t>(seq) * C + c] : 0.f;
    for (int64_t t = t1 - 1; t >= t0; --t) {
        const int64_t i = t * C + c;
        float s, m;
        gate<kLogit>(to_f(A[i]), s, m);
        const float g = to_f(G[i]) + carry, hp = hs[i];
        dX[i] = from_f<T>(m * g);
        dA[i] = from_f<T>(kLogit ? s * m * g * (hp - to_f(X[i])) : g * hp);
        carry = s * g;
    }
    if (dh_init) dh_init[static_cast<int64_t>(seq) * C + c] = carry;
}

template <typename T, bool kLogit>
__global__ void scan_step_kernel(const T* __restrict__ a, const T* __restrict__ x, float* __restrict__ h,
                                 T* __restrict__ out, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kScanThreads + threadIdx.x;
    if (i >= n) return;
    float s, m;
    gate<kLogit>(to_f(a[i]), s, m);
    const float y = fmaf(s, h[i], m * to_f(x[i]));
    h[i] = y;
    out[i] = from_f<T>(y);
}

}  // namespace

template <typename T>
cudaError_t gated_scan_forward(const LaunchCtx& c, const T* A, const T* X, T* O, const ScanShape& s,
                               const float* h_init, float* h_final, float* /*Ckpt*/) {
    const int seqs = s.starts ? s.num_seqs : s.B;
    const dim3 grid(seqs, (s.C + kScanThreads - 1) / kScanThreads);
    auto* k = s.logit ? scan_forward_kernel<T, true> : scan_forward_kernel<T, false>;
    k<<<grid, kScanThreads, 0, c.stream>>>(A, X, O, s.N, s.C, s.starts, h_init, h_final, nullptr);
    note_launch();
    return cudaGetLastError();
}

template <typename T>
cudaError_t gated_scan_backward(const LaunchCtx& c, const T* A, const T* X, const T* G, T* dA, T* dX,
                                const ScanShape& s, const float* h_init, const float* dh_final,
                                float* dh_init, const float* /*Ckpt*/) {
    const int seqs = s.starts ? s.num_seqs : s.B;
    float* hs = nullptr;
    cudaError_t e = scratch_alloc(c, reinterpret_cast<void**>(&hs),
                                  sizeof(float) * static_cast<size_t>(s.B) * s.N * s.C);
    if (e != cudaSuccess) return e;
    const dim3 grid(seqs, (s.C + kScanThreads - 1) / kScanThreads);
    auto* f = s.logit ? scan_forward_kernel<T, true> : scan_forward_kernel<T, false>;
    f<<<grid, kScanThreads, 0, c.stream>>>(A, X, nullptr, s.N, s.C, s.starts, h_init, nullptr, hs);
    auto* k = s.logit ? scan_backward_kernel<T, true> : scan_backward_kernel<T, false>;
    k<<<grid, kScanThreads, 0, c.stream>>>(A, X, G, dA, dX, s.N, s.C, s.starts, dh_final, dh_init, hs);
    note_launch(2);
    e = cudaGetLastError();
    scratch_free(c, hs);
    return e;
}

template <typename T>
cudaError_t gated_scan_step(const LaunchCtx& c, const T* a, const T* x, float* h, T* out, int64_t n,
                            bool logit) {
    auto* k = logit ? scan_step_kernel<T, true> : scan_step_kernel<T, false>;
    k<<<static_cast<unsigned>((n + kScanThreads - 1) / kScanThreads), kScanThreads, 0, c.stream>>>(a, x, h,
                                                                                             out, n);
    note_launch();
    return cudaGetLastError();
}

#define LA_INST_SCAN(T)                                                                               \
    template cudaError_t gated_scan_forward<T>(const LaunchCtx&, const T*, const T*, T*,              \
                                               const ScanShape&, const float*, float*, float*);       \
    template cudaError_t gated_scan_backward<T>(const LaunchCtx&, const T*, const T*, const T*, T*,   \
                                                T*, const ScanShape&, const float*, const float*,     \
                                                float*, const float*);                                \
    template cudaError_t gated_scan_step<T>(const LaunchCtx&, const T*, const T*, float*, T*, int64_t, \
                                            bool);
LA_INST_SCAN(float) LA_INST_SCAN(__nv_bfloat16)

}  // namespace la
