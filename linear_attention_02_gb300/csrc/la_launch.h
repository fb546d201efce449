// la_launch.h -- host-side launchers behind the C ABI (internal).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace la {

constexpr int kMaxDevices = 64;

// Everything a launcher needs from the device it runs on.
struct LaunchCtx {
    cudaStream_t stream;
    int num_sms;
    int device;                  // its ordinal, below kMaxDevices
    cudaMemPool_t pool;          // library-owned pool for stream-ordered scratch
    unsigned int* status_word;   // device error word for bounded waits
    // test hook (la_debug_withhold_publication): the unit whose look-back flag the next
    // tensor-core causal or gated scan launch leaves unset (-1: none), and its flag-poll
    // limit (0: default)
    int withhold_unit;
    unsigned spin_limit;
};

// Allows `kernel` its shared memory on a device and returns its resident blocks per
// SM, both asked of the runtime once per device and kernel.
template <auto kernel>
cudaError_t resident_blocks(int device, int threads, int smem, int* per_sm) {
    static std::atomic<int> known[kMaxDevices];
    int n = known[device].load(std::memory_order_acquire);
    if (n == 0) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
        if (e != cudaSuccess) return e;
        if (n == 0) return cudaErrorLaunchOutOfResources;
        known[device].store(n, std::memory_order_release);
    }
    *per_sm = n;
    return cudaSuccess;
}

// Counts one kernel launch (la_kernel_launch_count).
void note_launch(int n = 1);

// Sets the text returned by la_last_error_message() on this host thread.
void set_error_message(const char* msg);

// Bit of the device error word: an index read from device memory (a request
// length, a page number, a slot) was out of range and its access was skipped.
constexpr unsigned kStatusBadIndex = 0x100u;

// Optional checkpoints kept by the causal forward for the backward: the fp32
// state [S | Z] (D*M + D words) of every head before every kCkptChunks-th chunk
// of 128 tokens, laid out [BH][ceil(chunks / kCkptChunks)][D*M + D]; slot 0
// (the zero state) is never written or read.
constexpr int kCkptChunks = 8;

// Scratch bytes the tensor-core launchers take from the pool for one call
// (what la_workspace_bytes reports; the launchers allocate exactly these).
size_t causal_forward_tc_scratch(int D, int BH, int N, int num_sms);
size_t causal_backward_tc64_scratch(int BH, int N, int num_sms, bool out_given, bool den_given,
                                    bool ckpt_given);
size_t noncausal_forward_tc_f32_scratch(int BH, int N, int num_sms);

// Stream-ordered scratch from the library pool.  Returns cudaSuccess or the error.
cudaError_t scratch_alloc(const LaunchCtx& c, void** p, size_t bytes);
// One block whose bounded waits expire and set their bits in c.status_word.
cudaError_t selftest_expired_waits(const LaunchCtx& c);
void scratch_free(const LaunchCtx& c, void* p);

// Each launcher returns cudaSuccess or the first CUDA error it met.
template <typename T, int D, int M>
cudaError_t causal_forward(const LaunchCtx& c, const T* Q, const T* K, const T* V, T* O, int BH,
                           int N, const float* S_init, const float* Z_init, float* S_final,
                           float* Z_final, float* Den);

// Tensor-core causal forward for bf16 storage with D = M in {64, 128}.
template <int D, int M>
cudaError_t causal_forward_tc(const LaunchCtx& c, const __nv_bfloat16* Q, const __nv_bfloat16* K,
                              const __nv_bfloat16* V, __nv_bfloat16* O, int BH, int N,
                              const float* S_init, const float* Z_init, float* S_final,
                              float* Z_final, float* Den, float* Ckpt);

// Tensor-core retention forward (decay, no normaliser) for bf16 storage with D = M in {64, 128}.
template <int D, int M>
cudaError_t retention_forward_tc(const LaunchCtx& c, const __nv_bfloat16* Q, const __nv_bfloat16* K,
                                 const __nv_bfloat16* V, __nv_bfloat16* O, const float* gamma_head,
                                 const float* gates, int BH, int H, int N, const float* S_init,
                                 float* S_final);
size_t retention_forward_tc_scratch(int D, int BH, int N, int num_sms);

// Tensor-core causal backward for bf16 storage with D = M = 64; Den (the
// forward's normaliser per token) and Ckpt (its state checkpoints) may be null.
cudaError_t causal_backward_tc64(const LaunchCtx& c, const __nv_bfloat16* Q, const __nv_bfloat16* K,
                                 const __nv_bfloat16* V, const __nv_bfloat16* O,
                                 const __nv_bfloat16* G, __nv_bfloat16* dQ, __nv_bfloat16* dK,
                                 __nv_bfloat16* dV, int BH, int N, const float* Den,
                                 const float* Ckpt);

template <typename T, int D, int M>
cudaError_t causal_backward(const LaunchCtx& c, const T* Q, const T* K, const T* V, const T* O,
                            const T* G, T* dQ, T* dK, T* dV, int BH, int N);

// Tensor-core non-causal forward for fp32 storage with D = M = 64 (fp32
// operands split into two bf16 terms).
cudaError_t noncausal_forward_tc_f32(const LaunchCtx& c, const float* Q, const float* K,
                                     const float* V, float* O, int BH, int N);

template <typename T, int D, int M>
cudaError_t noncausal_forward(const LaunchCtx& c, const T* Q, const T* K, const T* V, T* O,
                              int BH, int N);

// Tensor-core non-causal backward for fp32 storage with D = M = 64 (O nullable).
cudaError_t noncausal_backward_tc_f32(const LaunchCtx& c, const float* Q, const float* K,
                                      const float* V, const float* O, const float* G, float* dQ,
                                      float* dK, float* dV, int BH, int N);
size_t noncausal_backward_tc_f32_scratch(int BH, int N, int num_sms);

template <typename T, int D, int M>
cudaError_t noncausal_backward(const LaunchCtx& c, const T* Q, const T* K, const T* V, const T* O,
                               const T* G, T* dQ, T* dK, T* dV, int BH, int N);

// Softmax attention decode step with a KV cache (M = D): appends k, v at
// position T_len of the caches, then attends over positions 0..T_len.
template <typename T, int D>
cudaError_t softmax_decode_step(const LaunchCtx& c, const T* q, const T* k, const T* v, T* Kc,
                                T* Vc, int T_len, int T_max, float* out, int BH);

// Retention (decayed, unnormalised linear attention) forward on the CUDA cores:
// gamma_head [H] or gates [BH][N] (per token) or neither (decay 1).
template <typename T, int D, int M>
cudaError_t retention_forward(const LaunchCtx& c, const T* Q, const T* K, const T* V, T* O,
                              const float* gamma_head, const float* gates, int BH, int H, int N,
                              const float* S_init, float* S_final);

// One retention decode step: S = gamma S + k v^T, out = S^T q.
template <typename T, int D, int M>
cudaError_t retention_step(const LaunchCtx& c, const T* q, const T* k, const T* v,
                           const float* gamma_head, const float* gate, float* S, float* out, int BH,
                           int H);

// Attention with the degree-2 polynomial similarity (q . k)^2 through its
// explicit feature map, D = 32, causal or over all tokens.
template <typename T, int M>
cudaError_t poly2_forward(const LaunchCtx& c, const T* Q, const T* K, const T* V, T* O, int BH,
                          int N, bool causal);

// The same on the tensor core for bf16 storage and M = 64 (D^2 = 1024 features).
cudaError_t poly2_forward_tc(const LaunchCtx& c, const __nv_bfloat16* Q, const __nv_bfloat16* K,
                             const __nv_bfloat16* V, __nv_bfloat16* O, int BH, int N, bool causal);

// Below, `fill`: which outputs get 0 in rows of no packed sequence (forward: Out; backward:
// bit 0 dA, bit 1 dX), or in rows without a request (bit 0: 0 to out, bit 1: -infinity to lse).
// Rows of a gated scan: [B][N][C], or with `starts` (device, [num_seqs + 1]) one
// row axis (B = 1) cut into packed sequences.
struct ScanShape {
    int B, N, C;
    bool logit;  // gates are logits (decay sigmoid(a), input scaled by 1 - decay)
    const int* starts;
    int num_seqs;
};
template <typename T>
cudaError_t gated_scan_forward(const LaunchCtx& c, const T* A, const T* X, T* O, const ScanShape& s,
                               const float* h_init, float* h_final, float* Ckpt, bool fill);
template <typename T>
cudaError_t gated_scan_backward(const LaunchCtx& c, const T* A, const T* X, const T* G, T* dA, T* dX,
                                const ScanShape& s, const float* h_init, const float* dh_final,
                                float* dh_init, const float* Ckpt, int fill);
template <typename T>
cudaError_t gated_scan_step(const LaunchCtx& c, const T* a, const T* x, float* h, T* out, int64_t n,
                            bool logit);

// Scratch bytes of a forward or backward call (ckpt: checkpoints are given).
size_t gated_scan_scratch(int B, int N, int C, bool backward, bool ckpt);

// Block table and slot map from request lengths (page_size = 1 << log2p).
cudaError_t page_map(const LaunchCtx& c, const int* cached, const int* fresh, int R,
                     const int* free_pages, int num_free, int log2p, int num_pages, int* table,
                     int max_pages, int* slots, int max_tokens, int* starts, int* counts);

// Rows [T][Hkv][row_bytes] of keys and values into their slots of the pools.
cudaError_t paged_append(const LaunchCtx& c, const void* k, const void* v, void* K, void* V,
                         const int* slots, int T, int Hkv, int row_bytes, int log2p, int num_pages);

// One decode step over the paged cache.
struct PagedShape {
    int R, Hq, Hkv, num_pages, log2p, max_pages, window;
    float scale;
};
// Its scratch bytes (the shape's num_pages, window and scale do not matter).
size_t paged_decode_scratch(const PagedShape& s, int D, bool bf16, int num_sms);
template <typename T, int D>
cudaError_t paged_decode_step(const LaunchCtx& c, const T* q, const T* k, const T* v, T* K, T* V,
                              const int* table, const int* lens, float* out, float* lse,
                              const PagedShape& s, int fill);

template <typename T, int D, int M>
cudaError_t decode_step(const LaunchCtx& c, const T* q, const T* k, const T* v, float* S,
                        float* Z, float* out, int BH);

}  // namespace la
