// la_api.cu -- the C ABI declared in include/linattn.h: argument validation,
// per-device context (SM count, scratch pool, device error word) and dispatch
// to the kernels for each (dtype, D, M).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "la_launch.h"
#include "la_plan.h"
#include "linattn.h"

namespace la {

namespace {

std::atomic<uint64_t> g_launches{0};
std::atomic<int> g_withhold_unit{-1};     // test hook, consumed by the next call
std::atomic<unsigned> g_spin_limit{0};
thread_local char g_msg[512] = "";

la_status fail(la_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
    va_end(ap);
    return s;
}

la_status cuda_fail(cudaError_t e, const char* where) {
    return fail(LA_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

struct DeviceState {
    std::atomic<bool> ready{false};  // set (release) once the fields below are filled
    int num_sms = 0;
    cudaMemPool_t pool = nullptr;
    unsigned int* status_word = nullptr;
};
DeviceState g_dev[kMaxDevices];
std::mutex g_dev_mu;

la_status get_ctx(cudaStream_t stream, LaunchCtx* ctx) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    if (dev < 0 || dev >= kMaxDevices) return fail(LA_ERR_CUDA, "device ordinal %d out of range", dev);
    DeviceState& d = g_dev[dev];
    if (!d.ready.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lk(g_dev_mu);
        if (!d.ready.load(std::memory_order_relaxed)) {
            int sms = 0;
            if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)))
                return cuda_fail(e, "cudaDeviceGetAttribute");
            cudaMemPoolProps props;
            memset(&props, 0, sizeof(props));
            props.allocType = cudaMemAllocationTypePinned;
            props.location.type = cudaMemLocationTypeDevice;
            props.location.id = dev;
            cudaMemPool_t pool = nullptr;
            if ((e = cudaMemPoolCreate(&pool, &props))) return cuda_fail(e, "cudaMemPoolCreate");
            uint64_t keep = ~0ull;  // keep freed scratch in the pool between calls
            if ((e = cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep)))
                return cuda_fail(e, "cudaMemPoolSetAttribute");
            unsigned int* word = nullptr;
            if ((e = cudaMalloc(&word, 256))) return cuda_fail(e, "cudaMalloc(status word)");
            if ((e = cudaMemset(word, 0, 256))) return cuda_fail(e, "cudaMemset(status word)");
            d.num_sms = sms;
            d.pool = pool;
            d.status_word = word;
            d.ready.store(true, std::memory_order_release);
        }
    }
    ctx->stream = stream;
    ctx->withhold_unit = g_withhold_unit.exchange(-1);
    ctx->spin_limit = g_spin_limit.exchange(0u);
    ctx->num_sms = d.num_sms;
    ctx->device = dev;
    ctx->pool = d.pool;
    ctx->status_word = d.status_word;
    return LA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

bool head_ok(int x) { return x == 32 || x == 64 || x == 128; }

// Common shape/pointer checks.  `ptrs` must be non-null and 16-byte aligned
// whenever the work is non-empty.
la_status check_common(const char* fn, int B, int H, int N, int D, int M, la_dtype dt,
                       const void* const* ptrs, const char* const* names, int nptr,
                       bool* empty) {
    if (B < 0 || H < 0 || N < 0)
        return fail(LA_ERR_INVALID_ARG, "%s: negative size B=%d H=%d N=%d", fn, B, H, N);
    if (dt != LA_DTYPE_F32 && dt != LA_DTYPE_BF16)
        return fail(LA_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dt);
    if (!head_ok(D) || !head_ok(M))
        return fail(LA_ERR_UNSUPPORTED, "%s: D=%d M=%d, supported head sizes are 32, 64, 128", fn,
                    D, M);
    const unsigned long long bhn = (unsigned long long)B * H * N;
    if (bhn * (unsigned long long)(D > M ? D : M) >= (1ull << 40))
        return fail(LA_ERR_INVALID_ARG, "%s: tensor too large", fn);
    if ((unsigned long long)B * H >= (1ull << 31))
        return fail(LA_ERR_INVALID_ARG, "%s: B*H too large", fn);
    *empty = bhn == 0;
    if (*empty) return LA_OK;
    for (int i = 0; i < nptr; ++i) {
        if (!ptrs[i]) return fail(LA_ERR_INVALID_ARG, "%s: %s is NULL", fn, names[i]);
        if (!aligned16(ptrs[i]))
            return fail(LA_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", fn, names[i]);
    }
    return LA_OK;
}

la_status check_optional(const char* fn, const void* p, const char* name) {
    if (p && !aligned16(p)) return fail(LA_ERR_INVALID_ARG, "%s: %s is not 16-byte aligned", fn, name);
    return LA_OK;
}

la_status finish(cudaError_t e, const char* fn) {
    if (e != cudaSuccess) return cuda_fail(e, fn);
    return LA_OK;
}

// Checks a list of required device pointers against an alignment in bytes.
la_status check_ptrs(const char* fn, const void* const* ptrs, const char* const* names, int n,
                     unsigned align) {
    for (int i = 0; i < n; ++i) {
        if (!ptrs[i]) return fail(LA_ERR_INVALID_ARG, "%s: %s is NULL", fn, names[i]);
        if (reinterpret_cast<uintptr_t>(ptrs[i]) & (align - 1))
            return fail(LA_ERR_INVALID_ARG, "%s: %s is not %u-byte aligned", fn, names[i], align);
    }
    return LA_OK;
}

// Sizes, dtype and packed sequences of a gated scan call.
la_status check_scan(const char* fn, int B, int N, int C, la_dtype dt, la_gate_form form,
                     const int* starts, int num_seqs) {
    if (B < 0 || N < 0 || C < 0 || num_seqs < 0)
        return fail(LA_ERR_INVALID_ARG, "%s: negative size B=%d N=%d C=%d num_seqs=%d", fn, B, N, C,
                    num_seqs);
    if (dt != LA_DTYPE_F32 && dt != LA_DTYPE_BF16)
        return fail(LA_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dt);
    if (form != LA_GATE_DECAY && form != LA_GATE_LOGIT)
        return fail(LA_ERR_UNSUPPORTED, "%s: unknown gate form %d", fn, (int)form);
    if (starts && B != 1)
        return fail(LA_ERR_INVALID_ARG, "%s: packed sequences need B == 1, got %d", fn, B);
    if (!starts && num_seqs != 0)
        return fail(LA_ERR_INVALID_ARG, "%s: num_seqs=%d without seq_starts", fn, num_seqs);
    if (reinterpret_cast<uintptr_t>(starts) & 3u)
        return fail(LA_ERR_INVALID_ARG, "%s: seq_starts is not 4-byte aligned", fn);
    // rows of a last tile and borders of sequences are counted in 32 bits, the latter beside two flags
    const unsigned long long rows = (unsigned long long)B * N;
    if (N > INT_MAX - plan::kScanTile || num_seqs >= (1 << 29) - 1 || rows >= (1ull << 40) ||
        (C && rows * C >= (1ull << 40)) ||
        (unsigned long long)(starts ? num_seqs : B) * C >= (1ull << 40))
        return fail(LA_ERR_INVALID_ARG, "%s: tensor too large", fn);
    return LA_OK;
}

// to = from (or zeros): the state of sequences without a row.
cudaError_t copy_state(cudaStream_t st, float* to, const float* from, size_t words) {
    if (!to || words == 0) return cudaSuccess;
    return from ? cudaMemcpyAsync(to, from, words * sizeof(float), cudaMemcpyDeviceToDevice, st)
                : cudaMemsetAsync(to, 0, words * sizeof(float), st);
}

size_t elem_bytes(la_dtype dt) { return dt == LA_DTYPE_F32 ? 4 : 2; }

// The outputs whose padding a call fills, a bit each of `all`.
la_status check_fill(const char* fn, int fill, int all) {
    return fill & ~all ? fail(LA_ERR_INVALID_ARG, "%s: fill=%d", fn, fill) : LA_OK;
}

// log2 of a supported page size, or -1.
int page_log2(int page_size) {
    for (int b = 0; b <= 10; ++b)
        if (page_size == 1 << b) return b;
    return -1;
}

// Page size and pool size of a paged cache call.
la_status check_pages(const char* fn, int num_pages, int page_size, int* log2p) {
    *log2p = page_log2(page_size);
    if (*log2p < 0)
        return fail(LA_ERR_UNSUPPORTED, "%s: page_size=%d, supported are powers of two up to 1024", fn,
                    page_size);
    if (num_pages < 0 || (unsigned long long)num_pages * page_size >= (1ull << 31))
        return fail(LA_ERR_INVALID_ARG, "%s: num_pages=%d of %d positions: negative, or 2^31 slots or more",
                    fn, num_pages, page_size);
    return LA_OK;
}

// Calls F::template run<T, D, M>(args...) for the runtime (dtype, D, M).
template <class F, class... A>
cudaError_t dispatch(la_dtype dt, int D, int M, A... a) {
#define LA_CASE_DM(T, d, m) \
    if (D == d && M == m) return F::template run<T, d, m>(a...);
#define LA_CASE_T(T)                                                                  \
    LA_CASE_DM(T, 32, 32) LA_CASE_DM(T, 32, 64) LA_CASE_DM(T, 32, 128)                \
    LA_CASE_DM(T, 64, 32) LA_CASE_DM(T, 64, 64) LA_CASE_DM(T, 64, 128)                \
    LA_CASE_DM(T, 128, 32) LA_CASE_DM(T, 128, 64) LA_CASE_DM(T, 128, 128)
    if (dt == LA_DTYPE_F32) {
        LA_CASE_T(float)
    } else {
        LA_CASE_T(__nv_bfloat16)
    }
#undef LA_CASE_T
#undef LA_CASE_DM
    return cudaErrorInvalidValue;
}

// bf16 with D = M in {64, 128} runs on the tensor cores; every other shape
// and fp32 storage runs the CUDA-core kernels.
template <typename T, int D, int M>
struct UseTensorCores {
    static constexpr bool value = false;
};
template <>
struct UseTensorCores<__nv_bfloat16, 64, 64> {
    static constexpr bool value = true;
};
template <>
struct UseTensorCores<__nv_bfloat16, 128, 128> {
    static constexpr bool value = true;
};

struct FwdCausal {
    template <typename T, int D, int M>
    static cudaError_t run(const LaunchCtx* c, const void* Q, const void* K, const void* V, void* O,
                           int BH, int N, const float* Si, const float* Zi, float* Sf, float* Zf,
                           float* Den, float* Ckpt) {
        if constexpr (UseTensorCores<T, D, M>::value)
            return causal_forward_tc<D, M>(*c, (const T*)Q, (const T*)K, (const T*)V, (T*)O, BH, N,
                                           Si, Zi, Sf, Zf, Den, Ckpt);
        else
            return causal_forward<T, D, M>(*c, (const T*)Q, (const T*)K, (const T*)V, (T*)O, BH, N,
                                           Si, Zi, Sf, Zf, Den);
    }
};
struct BwdCausal {
    template <typename T, int D, int M>
    static cudaError_t run(const LaunchCtx* c, const void* Q, const void* K, const void* V,
                           const void* O, const void* G, void* dQ, void* dK, void* dV, int BH, int N,
                           const float* Den, const float* Ckpt) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value && D == 64 && M == 64)
            return causal_backward_tc64(*c, (const T*)Q, (const T*)K, (const T*)V, (const T*)O,
                                        (const T*)G, (T*)dQ, (T*)dK, (T*)dV, BH, N, Den, Ckpt);
        else
            return causal_backward<T, D, M>(*c, (const T*)Q, (const T*)K, (const T*)V,
                                            (const T*)O, (const T*)G, (T*)dQ, (T*)dK, (T*)dV, BH,
                                            N);
    }
};
struct FwdNoncausal {
    template <typename T, int D, int M>
    static cudaError_t run(const LaunchCtx* c, const void* Q, const void* K, const void* V, void* O,
                           int BH, int N) {
        if constexpr (std::is_same<T, float>::value && D == 64 && M == 64)
            return noncausal_forward_tc_f32(*c, (const T*)Q, (const T*)K, (const T*)V, (T*)O, BH, N);
        else
            return noncausal_forward<T, D, M>(*c, (const T*)Q, (const T*)K, (const T*)V, (T*)O, BH,
                                              N);
    }
};
struct BwdNoncausal {
    template <typename T, int D, int M>
    static cudaError_t run(const LaunchCtx* c, const void* Q, const void* K, const void* V,
                           const void* O, const void* G, void* dQ, void* dK, void* dV, int BH, int N) {
        if constexpr (std::is_same<T, float>::value && D == 64 && M == 64)
            return noncausal_backward_tc_f32(*c, (const T*)Q, (const T*)K, (const T*)V, (const T*)O,
                                             (const T*)G, (T*)dQ, (T*)dK, (T*)dV, BH, N);
        else
            return noncausal_backward<T, D, M>(*c, (const T*)Q, (const T*)K, (const T*)V, (const T*)O,
                                               (const T*)G, (T*)dQ, (T*)dK, (T*)dV, BH, N);
    }
};
struct FwdRetention {
    template <typename T, int D, int M>
    static cudaError_t run(const LaunchCtx* c, const void* Q, const void* K, const void* V, void* O,
                           const float* gh, const float* gt, int BH, int H, int N, const float* Si,
                           float* Sf) {
        if constexpr (UseTensorCores<T, D, M>::value)
            return retention_forward_tc<D, M>(*c, (const T*)Q, (const T*)K, (const T*)V, (T*)O, gh,
                                              gt, BH, H, N, Si, Sf);
        else
            return retention_forward<T, D, M>(*c, (const T*)Q, (const T*)K, (const T*)V, (T*)O, gh,
                                              gt, BH, H, N, Si, Sf);
    }
};
struct RetentionStep {
    template <typename T, int D, int M>
    static cudaError_t run(const LaunchCtx* c, const void* q, const void* k, const void* v,
                           const float* gh, const float* gt, float* S, float* out, int BH, int H) {
        return retention_step<T, D, M>(*c, (const T*)q, (const T*)k, (const T*)v, gh, gt, S, out, BH,
                                       H);
    }
};
struct Decode {
    template <typename T, int D, int M>
    static cudaError_t run(const LaunchCtx* c, const void* q, const void* k, const void* v,
                           float* S, float* Z, float* out, int BH) {
        return decode_step<T, D, M>(*c, (const T*)q, (const T*)k, (const T*)v, S, Z, out, BH);
    }
};

// Writes zeros (or the initial state) to S_final/Z_final for an N == 0 forward.
cudaError_t empty_forward_state(cudaStream_t st, size_t bh, int D, int M, const float* Si,
                                const float* Zi, float* Sf, float* Zf) {
    if (!Sf || bh == 0) return cudaSuccess;
    const size_t sb = bh * D * M * sizeof(float), zb = bh * D * sizeof(float);
    cudaError_t e;
    if (Si) {
        if ((e = cudaMemcpyAsync(Sf, Si, sb, cudaMemcpyDeviceToDevice, st))) return e;
        return cudaMemcpyAsync(Zf, Zi, zb, cudaMemcpyDeviceToDevice, st);
    }
    if ((e = cudaMemsetAsync(Sf, 0, sb, st))) return e;
    return cudaMemsetAsync(Zf, 0, zb, st);
}

}  // namespace

void note_launch(int n) { g_launches.fetch_add((uint64_t)n, std::memory_order_relaxed); }

void set_error_message(const char* msg) { snprintf(g_msg, sizeof(g_msg), "%s", msg); }

cudaError_t scratch_alloc(const LaunchCtx& c, void** p, size_t bytes) {
    if (bytes == 0) bytes = 256;
    return cudaMallocFromPoolAsync(p, bytes, c.pool, c.stream);
}

void scratch_free(const LaunchCtx& c, void* p) {
    if (p) cudaFreeAsync(p, c.stream);
}

// Scratch bytes of one call, following the same dispatch as the entry points.
size_t workspace_for(const char* op, int BH, int N, int D, int M, la_dtype dt, unsigned saved,
                     int sms) {
    const bool bf16 = dt == LA_DTYPE_BF16;
    if (!strcmp(op, "la_forward_causal")) {
        if (bf16 && D == M && (D == 64 || D == 128)) return causal_forward_tc_scratch(D, BH, N, sms);
        return plan::ffma_causal_forward(BH, N, D, M, sms);
    }
    if (!strcmp(op, "la_backward_causal")) {
        if (bf16 && D == 64 && M == 64)
            return causal_backward_tc64_scratch(BH, N, sms, saved & LA_SAVED_OUT, saved & LA_SAVED_DEN,
                                                saved & LA_SAVED_CKPT);
        return plan::ffma_causal_backward(BH, N, D, M, sms);
    }
    if (!strcmp(op, "la_forward_noncausal")) {
        if (!bf16 && D == 64 && M == 64) return noncausal_forward_tc_f32_scratch(BH, N, sms);
        return plan::ffma_noncausal_forward(BH, N, D, M, sms);
    }
    if (!strcmp(op, "la_backward_noncausal"))
        return !bf16 && D == 64 && M == 64 ? noncausal_backward_tc_f32_scratch(BH, N, sms)
                                           : plan::ffma_noncausal_backward(BH, N, D, M, sms);
    if (!strcmp(op, "la_forward_poly2")) {
        if (D != 32 || (M != 32 && M != 64)) return SIZE_MAX;
        return bf16 && M == 64 ? plan::poly2_tc_scratch(BH, N) : plan::poly2_scratch(BH, N, M, sms);
    }
    if (!strcmp(op, "la_forward_retention"))
        return bf16 && D == M && (D == 64 || D == 128) ? retention_forward_tc_scratch(D, BH, N, sms)
                                                       : plan::ffma_retention_forward(BH, N, D, M, sms);
    if (!strcmp(op, "la_retention_decode_step")) return 0;
    if (!strcmp(op, "la_softmax_decode_step"))  // N is the cache position T: T + 1 positions
        return D == M ? plan::softmax_decode_scratch(BH, N + 1, D, sms) : SIZE_MAX;
    if (!strcmp(op, "la_decode_step") || !strcmp(op, "la_forward_noncausal_noalloc")) return 0;
    return SIZE_MAX;
}

}  // namespace la

using namespace la;

extern "C" {

size_t la_workspace_bytes(const char* op, int B, int H, int N, int D, int M, la_dtype dtype,
                          unsigned saved, int num_sms) {
    static const char* fn = "la_workspace_bytes";
    if (!op) return fail(LA_ERR_INVALID_ARG, "%s: op is NULL", fn), SIZE_MAX;
    if (B < 0 || H < 0 || N < 0)
        return fail(LA_ERR_INVALID_ARG, "%s: negative size B=%d H=%d N=%d", fn, B, H, N), SIZE_MAX;
    if (dtype != LA_DTYPE_F32 && dtype != LA_DTYPE_BF16)
        return fail(LA_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype), SIZE_MAX;
    if (!head_ok(D) || !head_ok(M))
        return fail(LA_ERR_UNSUPPORTED, "%s: D=%d M=%d, supported head sizes are 32, 64, 128", fn, D,
                    M),
               SIZE_MAX;
    if ((unsigned long long)B * H >= (1ull << 31))
        return fail(LA_ERR_INVALID_ARG, "%s: B*H too large", fn), SIZE_MAX;
    const int BH = B * H;
    if (workspace_for(op, 1, 1, D, M, dtype, saved, 1) == SIZE_MAX)
        return fail(LA_ERR_INVALID_ARG, "%s: unknown op \"%s\" or unsupported shape", fn, op), SIZE_MAX;
    if (!strcmp(op, "la_decode_step")) N = 1;
    const bool cache_op = !strcmp(op, "la_softmax_decode_step");  // N = T may be 0
    if (BH == 0 || (N == 0 && !cache_op)) return 0;
    if (num_sms <= 0) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, fn), SIZE_MAX;
    }
    return workspace_for(op, BH, N, D, M, dtype, saved, num_sms);
}

size_t la_scratch_peak_bytes(int reset) {
    static const char* fn = "la_scratch_peak_bytes";
    LaunchCtx ctx;
    if (get_ctx(nullptr, &ctx) != LA_OK) return SIZE_MAX;
    unsigned long long v = 0;
    cudaError_t e = cudaMemPoolGetAttribute(ctx.pool, cudaMemPoolAttrUsedMemHigh, &v);
    if (e != cudaSuccess) return cuda_fail(e, fn), SIZE_MAX;
    if (reset) {
        unsigned long long zero = 0;
        if ((e = cudaMemPoolSetAttribute(ctx.pool, cudaMemPoolAttrUsedMemHigh, &zero)) != cudaSuccess)
            return cuda_fail(e, fn), SIZE_MAX;
    }
    return (size_t)v;
}


la_status la_forward_causal(const void* Q, const void* K, const void* V, void* Out, int B, int H,
                            int N, int D, int M, la_dtype dtype, const float* S_init,
                            const float* Z_init, float* S_final, float* Z_final, float* Den,
                            float* Ckpt, void* stream) {
    static const char* fn = "la_forward_causal";
    const void* p[] = {Q, K, V, Out};
    const char* nm[] = {"Q", "K", "V", "Out"};
    bool empty = false;
    la_status s = check_common(fn, B, H, N, D, M, dtype, p, nm, 4, &empty);
    if (s != LA_OK) return s;
    if ((S_init == nullptr) != (Z_init == nullptr))
        return fail(LA_ERR_INVALID_ARG, "%s: S_init and Z_init must both be given or both NULL", fn);
    if ((S_final == nullptr) != (Z_final == nullptr))
        return fail(LA_ERR_INVALID_ARG, "%s: S_final and Z_final must both be given or both NULL", fn);
    if ((s = check_optional(fn, S_init, "S_init")) || (s = check_optional(fn, Z_init, "Z_init")) ||
        (s = check_optional(fn, S_final, "S_final")) || (s = check_optional(fn, Z_final, "Z_final")) ||
        (s = check_optional(fn, Den, "Den")) || (s = check_optional(fn, Ckpt, "Ckpt")))
        return s;
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    const size_t bh = (size_t)B * H;
    if (empty) return finish(empty_forward_state(ctx.stream, bh, D, M, S_init, Z_init, S_final, Z_final), fn);
    return finish(dispatch<FwdCausal>(dtype, D, M, &ctx, Q, K, V, Out, (int)bh, N, S_init, Z_init,
                                      S_final, Z_final, Den, Ckpt),
                  fn);
}

la_status la_backward_causal(const void* Q, const void* K, const void* V, const void* Out,
                             const void* dOut, void* dQ, void* dK, void* dV, int B, int H, int N,
                             int D, int M, la_dtype dtype, const float* Den, const float* Ckpt,
                             void* stream) {
    static const char* fn = "la_backward_causal";
    const void* p[] = {Q, K, V, dOut, dQ, dK, dV};
    const char* nm[] = {"Q", "K", "V", "dOut", "dQ", "dK", "dV"};
    bool empty = false;
    la_status s = check_common(fn, B, H, N, D, M, dtype, p, nm, 7, &empty);
    if (s != LA_OK) return s;
    if ((s = check_optional(fn, Out, "Out")) || (s = check_optional(fn, Den, "Den")) ||
        (s = check_optional(fn, Ckpt, "Ckpt")))
        return s;
    if (empty) return LA_OK;
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    return finish(dispatch<BwdCausal>(dtype, D, M, &ctx, Q, K, V, Out, dOut, dQ, dK, dV,
                                      (int)((size_t)B * H), N, Den, Ckpt),
                  fn);
}

size_t la_causal_ckpt_floats(int B, int H, int N, int D, int M) {
    if (B <= 0 || H <= 0 || N <= 0 || D <= 0 || M <= 0) return 0;
    const size_t chunks = ((size_t)N + 127) / 128;
    return (size_t)B * H * ((chunks + kCkptChunks - 1) / kCkptChunks) * ((size_t)D * M + D);
}

la_status la_forward_noncausal(const void* Q, const void* K, const void* V, void* Out, int B,
                               int H, int N, int D, int M, la_dtype dtype, void* stream) {
    static const char* fn = "la_forward_noncausal";
    const void* p[] = {Q, K, V, Out};
    const char* nm[] = {"Q", "K", "V", "Out"};
    bool empty = false;
    la_status s = check_common(fn, B, H, N, D, M, dtype, p, nm, 4, &empty);
    if (s != LA_OK || empty) return s;
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    return finish(dispatch<FwdNoncausal>(dtype, D, M, &ctx, Q, K, V, Out, (int)((size_t)B * H), N),
                  fn);
}

la_status la_backward_noncausal(const void* Q, const void* K, const void* V, const void* Out,
                                const void* dOut, void* dQ, void* dK, void* dV, int B, int H, int N,
                                int D, int M, la_dtype dtype, void* stream) {
    static const char* fn = "la_backward_noncausal";
    const void* p[] = {Q, K, V, dOut, dQ, dK, dV};
    const char* nm[] = {"Q", "K", "V", "dOut", "dQ", "dK", "dV"};
    bool empty = false;
    la_status s = check_common(fn, B, H, N, D, M, dtype, p, nm, 7, &empty);
    if (s != LA_OK) return s;
    if ((s = check_optional(fn, Out, "Out"))) return s;
    if (empty) return LA_OK;
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    return finish(dispatch<BwdNoncausal>(dtype, D, M, &ctx, Q, K, V, Out, dOut, dQ, dK, dV,
                                         (int)((size_t)B * H), N),
                  fn);
}

la_status la_decode_step(const void* q, const void* k, const void* v, float* S, float* Z,
                         float* out, int B, int H, int D, int M, la_dtype dtype, void* stream) {
    static const char* fn = "la_decode_step";
    const void* p[] = {q, k, v, S, Z, out};
    const char* nm[] = {"q", "k", "v", "S", "Z", "out"};
    bool empty = false;
    la_status s = check_common(fn, B, H, 1, D, M, dtype, p, nm, 6, &empty);
    if (s != LA_OK || empty) return s;
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    return finish(dispatch<Decode>(dtype, D, M, &ctx, q, k, v, S, Z, out, (int)((size_t)B * H)), fn);
}

la_status la_forward_retention(const void* Q, const void* K, const void* V, void* Out, int B,
                               int H, int N, int D, int M, la_dtype dtype, const float* gamma_head,
                               const float* gates, const float* S_init, float* S_final,
                               void* stream) {
    static const char* fn = "la_forward_retention";
    const void* p[] = {Q, K, V, Out};
    const char* nm[] = {"Q", "K", "V", "Out"};
    bool empty = false;
    la_status s = check_common(fn, B, H, N, D, M, dtype, p, nm, 4, &empty);
    if (s != LA_OK) return s;
    if (gamma_head && gates)
        return fail(LA_ERR_INVALID_ARG, "%s: give gamma_head or gates, not both", fn);
    if ((s = check_optional(fn, S_init, "S_init")) || (s = check_optional(fn, S_final, "S_final")))
        return s;
    if (((uintptr_t)gamma_head | (uintptr_t)gates) & 3u)
        return fail(LA_ERR_INVALID_ARG, "%s: gamma_head / gates not 4-byte aligned", fn);
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    const size_t bh = (size_t)B * H;
    if (empty) {
        if (!S_final || bh == 0) return LA_OK;
        const size_t sb = bh * D * M * sizeof(float);
        return finish(S_init ? cudaMemcpyAsync(S_final, S_init, sb, cudaMemcpyDeviceToDevice, ctx.stream)
                             : cudaMemsetAsync(S_final, 0, sb, ctx.stream),
                      fn);
    }
    return finish(dispatch<FwdRetention>(dtype, D, M, &ctx, Q, K, V, Out, gamma_head, gates, (int)bh,
                                         H, N, S_init, S_final),
                  fn);
}

la_status la_retention_decode_step(const void* q, const void* k, const void* v,
                                   const float* gamma_head, const float* gate, float* S, float* out,
                                   int B, int H, int D, int M, la_dtype dtype, void* stream) {
    static const char* fn = "la_retention_decode_step";
    const void* p[] = {q, k, v, S, out};
    const char* nm[] = {"q", "k", "v", "S", "out"};
    bool empty = false;
    la_status s = check_common(fn, B, H, 1, D, M, dtype, p, nm, 5, &empty);
    if (s != LA_OK || empty) return s;
    if (gamma_head && gate) return fail(LA_ERR_INVALID_ARG, "%s: give gamma_head or gate, not both", fn);
    if (((uintptr_t)gamma_head | (uintptr_t)gate) & 3u)
        return fail(LA_ERR_INVALID_ARG, "%s: gamma_head / gate not 4-byte aligned", fn);
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    return finish(dispatch<RetentionStep>(dtype, D, M, &ctx, q, k, v, gamma_head, gate, S, out,
                                          (int)((size_t)B * H), H),
                  fn);
}

la_status la_forward_poly2(const void* Q, const void* K, const void* V, void* Out, int B, int H,
                           int N, int D, int M, la_dtype dtype, int causal, void* stream) {
    static const char* fn = "la_forward_poly2";
    const void* p[] = {Q, K, V, Out};
    const char* nm[] = {"Q", "K", "V", "Out"};
    bool empty = false;
    la_status s = check_common(fn, B, H, N, D, M, dtype, p, nm, 4, &empty);
    if (s != LA_OK) return s;
    if (D != 32 || (M != 32 && M != 64))
        return fail(LA_ERR_UNSUPPORTED, "%s: D=%d M=%d, the degree-2 feature map is built for D = 32, "
                    "M in {32, 64}", fn, D, M);
    if (empty) return LA_OK;
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    const int BH = B * H;
    const bool c = causal != 0;
    cudaError_t e;
    if (dtype == LA_DTYPE_F32)
        e = M == 32 ? poly2_forward<float, 32>(ctx, (const float*)Q, (const float*)K, (const float*)V,
                                               (float*)Out, BH, N, c)
                    : poly2_forward<float, 64>(ctx, (const float*)Q, (const float*)K, (const float*)V,
                                               (float*)Out, BH, N, c);
    else
        e = M == 32 ? poly2_forward<__nv_bfloat16, 32>(ctx, (const __nv_bfloat16*)Q, (const __nv_bfloat16*)K,
                                                       (const __nv_bfloat16*)V, (__nv_bfloat16*)Out, BH, N, c)
                    : poly2_forward_tc(ctx, (const __nv_bfloat16*)Q, (const __nv_bfloat16*)K,
                                       (const __nv_bfloat16*)V, (__nv_bfloat16*)Out, BH, N, c);
    return finish(e, fn);
}

la_status la_softmax_decode_step(const void* q, const void* k, const void* v, void* K_cache,
                                 void* V_cache, int T, int T_max, float* out, int B, int H, int D,
                                 int M, la_dtype dtype, void* stream) {
    static const char* fn = "la_softmax_decode_step";
    const void* p[] = {q, k, v, K_cache, V_cache, out};
    const char* nm[] = {"q", "k", "v", "K_cache", "V_cache", "out"};
    bool empty = false;
    la_status s = check_common(fn, B, H, 1, D, M, dtype, p, nm, 6, &empty);
    if (s != LA_OK) return s;
    if (D != M)
        return fail(LA_ERR_UNSUPPORTED, "%s: D=%d M=%d, the KV-cache step needs D == M", fn, D, M);
    if (T < 0 || T >= T_max)
        return fail(LA_ERR_INVALID_ARG, "%s: cache position T=%d must satisfy 0 <= T < T_max=%d", fn,
                    T, T_max);
    if ((unsigned long long)B * H * T_max * D >= (1ull << 40))
        return fail(LA_ERR_INVALID_ARG, "%s: cache too large", fn);
    if (empty) return LA_OK;
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    const int BH = B * H;
    cudaError_t e = cudaErrorInvalidValue;
#define LA_SD_CASE(Ty, d)                                                                       \
    if (D == d)                                                                                 \
        e = softmax_decode_step<Ty, d>(ctx, (const Ty*)q, (const Ty*)k, (const Ty*)v, (Ty*)K_cache, \
                                       (Ty*)V_cache, T, T_max, out, BH);
    if (dtype == LA_DTYPE_F32) {
        LA_SD_CASE(float, 32) else LA_SD_CASE(float, 64) else LA_SD_CASE(float, 128)
    } else {
        LA_SD_CASE(__nv_bfloat16, 32) else LA_SD_CASE(__nv_bfloat16, 64) else LA_SD_CASE(__nv_bfloat16, 128)
    }
#undef LA_SD_CASE
    return finish(e, fn);
}

size_t la_gated_scan_workspace_bytes(int backward, int B, int N, int C, la_dtype dtype, int ckpt_given) {
    static const char* fn = "la_gated_scan_workspace_bytes";
    la_status s = check_scan(fn, B, N, C, dtype, LA_GATE_DECAY, nullptr, 0);
    if (s != LA_OK) return SIZE_MAX;
    if ((size_t)B * N * C == 0) return 0;
    return gated_scan_scratch(B, N, C, backward != 0, ckpt_given != 0);
}

size_t la_paged_decode_workspace_bytes(int R, int Hq, int Hkv, int D, int page_size, int max_pages,
                                       la_dtype dtype, int num_sms) {
    static const char* fn = "la_paged_decode_workspace_bytes";
    int log2p = 0;
    if (check_pages(fn, 0, page_size, &log2p) != LA_OK) return SIZE_MAX;
    if (dtype != LA_DTYPE_F32 && dtype != LA_DTYPE_BF16)
        return fail(LA_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype), SIZE_MAX;
    if (!head_ok(D))
        return fail(LA_ERR_UNSUPPORTED, "%s: D=%d, supported head sizes are 32, 64, 128", fn, D), SIZE_MAX;
    if (R < 0 || Hq < 0 || Hkv < 0 || max_pages < 0 || (Hq && (Hkv == 0 || Hq % Hkv)) ||
        (unsigned long long)max_pages * page_size >= (1ull << 30))
        return fail(LA_ERR_INVALID_ARG, "%s: sizes R=%d Hq=%d Hkv=%d max_pages=%d", fn, R, Hq, Hkv, max_pages),
               SIZE_MAX;
    if ((unsigned long long)R * Hq * D >= (1ull << 31))
        return fail(LA_ERR_INVALID_ARG, "%s: tensor too large", fn), SIZE_MAX;
    if (num_sms <= 0) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, fn), SIZE_MAX;
    }
    const PagedShape sh = {R, Hq, Hkv, 0, log2p, max_pages, 0, 1.f};
    return paged_decode_scratch(sh, D, dtype == LA_DTYPE_BF16, num_sms);
}

size_t la_page_map_workspace_bytes(int R) {
    if (R < 0 || R >= (1 << 30))
        return fail(LA_ERR_INVALID_ARG, "la_page_map_workspace_bytes: R=%d: negative, or 2^30 requests or more", R),
               SIZE_MAX;
    return plan::page_map_scratch(R);
}

size_t la_gated_scan_ckpt_floats(int B, int N, int C) {
    if (B <= 0 || N <= 0 || C <= 0) return 0;
    return (size_t)B * (((size_t)N + plan::kScanTile - 1) / plan::kScanTile) * (size_t)C;
}

static la_status scan_forward(const void* A, const void* X, void* Out, int B, int N, int C,
                              la_dtype dtype, la_gate_form form, const int* seq_starts, int num_seqs,
                              const float* h_init, float* h_final, float* Ckpt, bool fill,
                              void* stream) {
    static const char* fn = "la_forward_gated_scan";
    la_status s = check_scan(fn, B, N, C, dtype, form, seq_starts, num_seqs);
    if (s != LA_OK) return s;
    if ((s = check_optional(fn, h_init, "h_init")) || (s = check_optional(fn, h_final, "h_final")) ||
        (s = check_optional(fn, Ckpt, "Ckpt")))
        return s;
    const size_t states = (size_t)(seq_starts ? num_seqs : B) * C;
    const bool empty = (size_t)B * N * C == 0 || (seq_starts && num_seqs == 0);
    const bool clear = fill && seq_starts && num_seqs == 0 && (size_t)N * C != 0;  // no row has a sequence
    if (empty && !clear && (!h_final || states == 0)) return LA_OK;
    if (!empty || clear) {
        const void* p[] = {A, X, Out};
        const char* nm[] = {"A", "X", "Out"};
        if ((s = check_ptrs(fn, p, nm, 3, 16)) != LA_OK) return s;
    }
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    if (clear) return finish(cudaMemsetAsync(Out, 0, elem_bytes(dtype) * N * C, ctx.stream), fn);
    if (empty) return finish(copy_state(ctx.stream, h_final, h_init, states), fn);
    const ScanShape sh = {B, N, C, form == LA_GATE_LOGIT, seq_starts, num_seqs};
    using bf = __nv_bfloat16;
    return finish(dtype == LA_DTYPE_F32
                      ? gated_scan_forward<float>(ctx, (const float*)A, (const float*)X, (float*)Out, sh,
                                                  h_init, h_final, Ckpt, fill)
                      : gated_scan_forward<bf>(ctx, (const bf*)A, (const bf*)X, (bf*)Out, sh, h_init,
                                               h_final, Ckpt, fill),
                  fn);
}

la_status la_forward_gated_scan(const void* A, const void* X, void* Out, int B, int N, int C,
                                la_dtype dtype, la_gate_form form, const int* seq_starts, int num_seqs,
                                const float* h_init, float* h_final, float* Ckpt, void* stream) {
    return scan_forward(A, X, Out, B, N, C, dtype, form, seq_starts, num_seqs, h_init, h_final, Ckpt, false, stream);
}

la_status la_forward_gated_scan_padded(const void* A, const void* X, void* Out, int B, int N, int C,
                                       la_dtype dtype, la_gate_form form, const int* seq_starts, int num_seqs,
                                       const float* h_init, float* h_final, float* Ckpt, int fill, void* stream) {
    if (la_status s = check_fill("la_forward_gated_scan", fill, 1)) return s;
    return scan_forward(A, X, Out, B, N, C, dtype, form, seq_starts, num_seqs, h_init, h_final, Ckpt, fill != 0, stream);
}

static la_status scan_backward(const void* A, const void* X, const void* dOut, void* dA, void* dX,
                               int B, int N, int C, la_dtype dtype, la_gate_form form,
                               const int* seq_starts, int num_seqs, const float* h_init,
                               const float* dh_final, float* dh_init, const float* Ckpt, int fill, void* stream) {
    static const char* fn = "la_backward_gated_scan";
    la_status s = check_scan(fn, B, N, C, dtype, form, seq_starts, num_seqs);
    if (s != LA_OK) return s;
    if ((s = check_optional(fn, h_init, "h_init")) || (s = check_optional(fn, dh_final, "dh_final")) ||
        (s = check_optional(fn, dh_init, "dh_init")) || (s = check_optional(fn, Ckpt, "Ckpt")))
        return s;
    const size_t states = (size_t)(seq_starts ? num_seqs : B) * C;
    const bool empty = (size_t)B * N * C == 0 || (seq_starts && num_seqs == 0);
    const bool clear = fill && seq_starts && num_seqs == 0 && (size_t)N * C != 0;  // no row has a sequence
    if (empty && !clear && (!dh_init || states == 0)) return LA_OK;
    if (!empty || clear) {
        const void* p[] = {A, X, dOut, dA, dX};
        const char* nm[] = {"A", "X", "dOut", "dA", "dX"};
        if ((s = check_ptrs(fn, p, nm, 5, 16)) != LA_OK) return s;
    }
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    if (clear) {
        const size_t bytes = elem_bytes(dtype) * N * C;
        cudaError_t e = fill & 1 ? cudaMemsetAsync(dA, 0, bytes, ctx.stream) : cudaSuccess;
        if (e == cudaSuccess && (fill & 2)) e = cudaMemsetAsync(dX, 0, bytes, ctx.stream);
        return finish(e, fn);
    }
    if (empty) return finish(copy_state(ctx.stream, dh_init, dh_final, states), fn);
    const ScanShape sh = {B, N, C, form == LA_GATE_LOGIT, seq_starts, num_seqs};
    using bf = __nv_bfloat16;
    return finish(dtype == LA_DTYPE_F32
                      ? gated_scan_backward<float>(ctx, (const float*)A, (const float*)X,
                                                   (const float*)dOut, (float*)dA, (float*)dX, sh, h_init,
                                                   dh_final, dh_init, Ckpt, fill)
                      : gated_scan_backward<bf>(ctx, (const bf*)A, (const bf*)X, (const bf*)dOut, (bf*)dA,
                                                (bf*)dX, sh, h_init, dh_final, dh_init, Ckpt, fill),
                  fn);
}

la_status la_backward_gated_scan(const void* A, const void* X, const void* dOut, void* dA, void* dX,
                                 int B, int N, int C, la_dtype dtype, la_gate_form form,
                                 const int* seq_starts, int num_seqs, const float* h_init,
                                 const float* dh_final, float* dh_init, const float* Ckpt,
                                 void* stream) {
    return scan_backward(A, X, dOut, dA, dX, B, N, C, dtype, form, seq_starts, num_seqs, h_init, dh_final, dh_init,
                         Ckpt, 0, stream);
}

la_status la_backward_gated_scan_padded(const void* A, const void* X, const void* dOut, void* dA, void* dX,
                                        int B, int N, int C, la_dtype dtype, la_gate_form form,
                                        const int* seq_starts, int num_seqs, const float* h_init,
                                        const float* dh_final, float* dh_init, const float* Ckpt, int fill,
                                        void* stream) {
    if (la_status s = check_fill("la_backward_gated_scan", fill, 3)) return s;
    return scan_backward(A, X, dOut, dA, dX, B, N, C, dtype, form, seq_starts, num_seqs, h_init, dh_final, dh_init,
                         Ckpt, fill, stream);
}

la_status la_gated_scan_decode_step(const void* a, const void* x, float* h, void* out, int B, int C,
                                    la_dtype dtype, la_gate_form form, void* stream) {
    static const char* fn = "la_gated_scan_decode_step";
    la_status s = check_scan(fn, B, 1, C, dtype, form, nullptr, 0);
    if (s != LA_OK) return s;
    const int64_t n = (int64_t)B * C;
    if (n == 0) return LA_OK;
    const void* p[] = {a, x, h, out};
    const char* nm[] = {"a", "x", "h", "out"};
    if ((s = check_ptrs(fn, p, nm, 4, 16)) != LA_OK) return s;
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    using bf = __nv_bfloat16;
    const bool lg = form == LA_GATE_LOGIT;
    return finish(dtype == LA_DTYPE_F32
                      ? gated_scan_step<float>(ctx, (const float*)a, (const float*)x, h, (float*)out, n, lg)
                      : gated_scan_step<bf>(ctx, (const bf*)a, (const bf*)x, h, (bf*)out, n, lg),
                  fn);
}

la_status la_page_map(const int* cached_lens, const int* new_lens, int R, const int* free_pages,
                      int num_free, int page_size, int num_pages, int* block_table, int max_pages,
                      int* slot_map, int max_tokens, int* seq_starts, int* counts, void* stream) {
    static const char* fn = "la_page_map";
    int log2p = 0;
    la_status s = check_pages(fn, num_pages, page_size, &log2p);
    if (s != LA_OK) return s;
    if (R < 0 || num_free < 0 || max_pages < 0 || max_tokens < 0)
        return fail(LA_ERR_INVALID_ARG, "%s: negative size R=%d num_free=%d max_pages=%d max_tokens=%d", fn,
                    R, num_free, max_pages, max_tokens);
    if (R >= (1 << 30)) return fail(LA_ERR_INVALID_ARG, "%s: R=%d: 2^30 requests or more", fn, R);
    if ((unsigned long long)max_pages * page_size >= (1ull << 31))
        return fail(LA_ERR_INVALID_ARG, "%s: max_pages=%d of %d positions: 2^31 positions or more", fn,
                    max_pages, page_size);
    const void* p[] = {seq_starts, counts, cached_lens, new_lens, block_table, free_pages, slot_map};
    const char* nm[] = {"seq_starts", "counts", "cached_lens", "new_lens", "block_table", "free_pages",
                        "slot_map"};
    const bool need[] = {true, true, R > 0, R > 0, R > 0 && max_pages > 0, num_free > 0, max_tokens > 0};
    for (int i = 0; i < 7; ++i)
        if (need[i] && (s = check_ptrs(fn, p + i, nm + i, 1, 4)) != LA_OK) return s;
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    return finish(page_map(ctx, cached_lens, new_lens, R, free_pages, num_free, log2p, num_pages,
                           block_table, max_pages, slot_map, max_tokens, seq_starts, counts),
                  fn);
}

la_status la_paged_append(const void* k, const void* v, void* K_pages, void* V_pages,
                          const int* slot_map, int T, int Hkv, int D, int num_pages, int page_size,
                          la_dtype dtype, void* stream) {
    static const char* fn = "la_paged_append";
    int log2p = 0;
    la_status s = check_pages(fn, num_pages, page_size, &log2p);
    if (s != LA_OK) return s;
    if (T < 0 || Hkv < 0) return fail(LA_ERR_INVALID_ARG, "%s: negative size T=%d Hkv=%d", fn, T, Hkv);
    if (dtype != LA_DTYPE_F32 && dtype != LA_DTYPE_BF16)
        return fail(LA_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
    if (!head_ok(D))
        return fail(LA_ERR_UNSUPPORTED, "%s: D=%d, supported head sizes are 32, 64, 128", fn, D);
    if ((unsigned long long)T * Hkv * D >= (1ull << 40) || (unsigned long long)Hkv * D >= (1ull << 31) ||
        (unsigned long long)num_pages * page_size * (Hkv ? Hkv : 1) >= (1ull << 40) / D)
        return fail(LA_ERR_INVALID_ARG, "%s: tensor too large", fn);
    if (T == 0 || Hkv == 0) return LA_OK;
    const void* p[] = {k, v, K_pages, V_pages};
    const char* nm[] = {"k", "v", "K_pages", "V_pages"};
    if ((s = check_ptrs(fn, p, nm, num_pages ? 4 : 2, 16)) != LA_OK) return s;
    const void* sp[] = {slot_map};
    const char* sn[] = {"slot_map"};
    if ((s = check_ptrs(fn, sp, sn, 1, 4)) != LA_OK) return s;
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    return finish(paged_append(ctx, k, v, K_pages, V_pages, slot_map, T, Hkv,
                               D * (dtype == LA_DTYPE_F32 ? 4 : 2), log2p, num_pages),
                  fn);
}

static la_status paged_step(const void* q, const void* k, const void* v, void* K_pages,
                            void* V_pages, const int* block_table, const int* cached_lens, float* out,
                            float* lse, int R, int Hq, int Hkv, int D, int num_pages, int page_size,
                            int max_pages, int window, float scale, la_dtype dtype, int fill,
                            void* stream) {
    static const char* fn = "la_paged_decode_step";
    int log2p = 0;
    la_status s = check_pages(fn, num_pages, page_size, &log2p);
    if (s != LA_OK) return s;
    if (R < 0 || Hq < 0 || Hkv < 0 || max_pages < 0 || window < 0)
        return fail(LA_ERR_INVALID_ARG, "%s: negative size R=%d Hq=%d Hkv=%d max_pages=%d window=%d", fn, R,
                    Hq, Hkv, max_pages, window);
    if (dtype != LA_DTYPE_F32 && dtype != LA_DTYPE_BF16)
        return fail(LA_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
    if (!head_ok(D))
        return fail(LA_ERR_UNSUPPORTED, "%s: D=%d, supported head sizes are 32, 64, 128", fn, D);
    if (Hq && (Hkv == 0 || Hq % Hkv))
        return fail(LA_ERR_INVALID_ARG, "%s: Hq=%d query heads over Hkv=%d key heads: not a multiple", fn,
                    Hq, Hkv);
    if (!std::isfinite(scale * 1.4426950408889634f))  // scores are taken to base 2
        return fail(LA_ERR_INVALID_ARG, "%s: scale=%g, or its product with log2 e, is not finite", fn, scale);
    if ((k == nullptr) != (v == nullptr))
        return fail(LA_ERR_INVALID_ARG, "%s: k and v must both be given or both NULL", fn);
    if ((unsigned long long)max_pages * page_size >= (1ull << 30))
        return fail(LA_ERR_INVALID_ARG, "%s: max_pages=%d of %d positions: 2^30 positions or more", fn,
                    max_pages, page_size);
    if ((unsigned long long)R * Hq * D >= (1ull << 31) ||
        (unsigned long long)num_pages * page_size * (Hkv ? Hkv : 1) >= (1ull << 40) / D)
        return fail(LA_ERR_INVALID_ARG, "%s: tensor too large", fn);
    if (R && Hkv && k && Hq == 0)
        return fail(LA_ERR_INVALID_ARG, "%s: new rows but no query heads (la_paged_append appends alone)", fn);
    if (R == 0 || Hq == 0) return LA_OK;
    const void* p[] = {q, out, K_pages, V_pages};
    const char* nm[] = {"q", "out", "K_pages", "V_pages"};
    if ((s = check_ptrs(fn, p, nm, num_pages ? 4 : 2, 16)) != LA_OK) return s;
    if ((s = check_optional(fn, k, "k")) || (s = check_optional(fn, v, "v"))) return s;
    const void* ip[] = {cached_lens, block_table};
    const char* in[] = {"cached_lens", "block_table"};
    if ((s = check_ptrs(fn, ip, in, max_pages ? 2 : 1, 4)) != LA_OK) return s;
    if ((fill & 2) && !lse) return fail(LA_ERR_INVALID_ARG, "%s: lse is NULL", fn);
    if (reinterpret_cast<uintptr_t>(lse) & 3u)
        return fail(LA_ERR_INVALID_ARG, "%s: lse is not 4-byte aligned", fn);
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    const PagedShape sh = {R, Hq, Hkv, num_pages, log2p, max_pages, window,
                           scale == 0.f ? 1.f / sqrtf((float)D) : scale};
    cudaError_t e = cudaErrorInvalidValue;
#define LA_PD_CASE(Ty, d)                                                                              \
    if (D == d)                                                                                        \
        e = paged_decode_step<Ty, d>(ctx, (const Ty*)q, (const Ty*)k, (const Ty*)v, (Ty*)K_pages,      \
                                     (Ty*)V_pages, block_table, cached_lens, out, lse, sh, fill);
    if (dtype == LA_DTYPE_F32) {
        LA_PD_CASE(float, 32) else LA_PD_CASE(float, 64) else LA_PD_CASE(float, 128)
    } else {
        LA_PD_CASE(__nv_bfloat16, 32) else LA_PD_CASE(__nv_bfloat16, 64) else LA_PD_CASE(__nv_bfloat16, 128)
    }
#undef LA_PD_CASE
    return finish(e, fn);
}

la_status la_paged_decode_step(const void* q, const void* k, const void* v, void* K_pages,
                               void* V_pages, const int* block_table, const int* cached_lens, float* out,
                               float* lse, int R, int Hq, int Hkv, int D, int num_pages, int page_size,
                               int max_pages, int window, float scale, la_dtype dtype, void* stream) {
    return paged_step(q, k, v, K_pages, V_pages, block_table, cached_lens, out, lse, R, Hq, Hkv, D, num_pages,
                      page_size, max_pages, window, scale, dtype, 0, stream);
}

la_status la_paged_decode_step_padded(const void* q, const void* k, const void* v, void* K_pages,
                                      void* V_pages, const int* block_table, const int* cached_lens, float* out,
                                      float* lse, int R, int Hq, int Hkv, int D, int num_pages, int page_size,
                                      int max_pages, int window, float scale, la_dtype dtype, int fill,
                                      void* stream) {
    if (la_status s = check_fill("la_paged_decode_step", fill, 3)) return s;
    return paged_step(q, k, v, K_pages, V_pages, block_table, cached_lens, out, lse, R, Hq, Hkv, D, num_pages,
                      page_size, max_pages, window, scale, dtype, fill, stream);
}

// A call of the rotary family: its tensors in the order of RotaryShape, checked.
static la_status rotary_shape(const char* fn, RotaryShape* sh, const void* const* ptrs, const char* const* names,
                              int tensors, int B, int N, int Hq, int Hk, int D, const int64_t* strides,
                              const int* positions, int position_rows, int first_position, const uint64_t* freqs,
                              int rot, float magnitude, la_rotary_layout layout, la_dtype dtype, int fill, bool* empty) {
    if (B < 0 || N < 0 || Hq < 0 || Hk < 0)
        return fail(LA_ERR_INVALID_ARG, "%s: negative size B=%d N=%d Hq=%d Hk=%d", fn, B, N, Hq, Hk);
    if (dtype != LA_DTYPE_F32 && dtype != LA_DTYPE_BF16)
        return fail(LA_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
    if (!head_ok(D))
        return fail(LA_ERR_UNSUPPORTED, "%s: D=%d, supported head sizes are 32, 64, 128", fn, D);
    if (layout != LA_ROTARY_HALF && layout != LA_ROTARY_INTERLEAVED)
        return fail(LA_ERR_UNSUPPORTED, "%s: unknown layout %d", fn, (int)layout);
    if (rot < 2 || rot > D || rot % 2)
        return fail(LA_ERR_INVALID_ARG, "%s: rot=%d must be even, from 2 to D=%d", fn, rot, D);
    if (!std::isfinite(magnitude)) return fail(LA_ERR_INVALID_ARG, "%s: magnitude=%g is not finite", fn, magnitude);
    // positions of no token are an array without an element, which may be NULL
    const bool no_token = B == 0 || N == 0;
    if (positions || (no_token && position_rows != 0) ? position_rows != 1 && position_rows != B : position_rows != 0)
        return fail(LA_ERR_INVALID_ARG, "%s: position_rows=%d with %s must be %s", fn, position_rows,
                    positions ? "positions" : "no positions", positions ? "1 or B" : "0");
    if (positions ? first_position != 0 : first_position < 0 || (long long)first_position + N > INT_MAX)
        return fail(LA_ERR_INVALID_ARG, "%s: first_position=%d: given beside positions, negative, or past 2^31 with N=%d",
                    fn, first_position, N);
    if (la_status s = check_fill(fn, fill, 3)) return s;
    // tiles of tokens are counted in 32 bits
    const unsigned long long tokens = (unsigned long long)B * N;
    if (tokens >= (1ull << 30) || (unsigned long long)Hq * D >= (1ull << 30) || (unsigned long long)Hk * D >= (1ull << 30) ||
        tokens * ((unsigned long long)Hq + Hk) * D >= (1ull << 40))
        return fail(LA_ERR_INVALID_ARG, "%s: tensor too large", fn);
    *empty = tokens == 0 || Hq + Hk == 0;
    RotaryShape& r = *sh;
    r = {};
    r.B = B, r.N = N, r.Hq = Hq, r.Hk = Hk, r.D = D, r.rot = rot;
    r.interleaved = layout == LA_ROTARY_INTERLEAVED;
    r.freqs = freqs, r.positions = positions, r.pos_batch = position_rows > 1 ? N : 0, r.first = first_position;
    r.mag = magnitude, r.fill = fill, r.tensors = tensors;
    if (*empty) return LA_OK;
    const size_t es = elem_bytes(dtype);
    for (int i = 0; i < tensors; ++i) {
        const int H = i % 2 ? Hk : Hq;
        if (H == 0) continue;
        if (!ptrs[i]) return fail(LA_ERR_INVALID_ARG, "%s: %s is NULL", fn, names[i]);
        if (reinterpret_cast<uintptr_t>(ptrs[i]) % es)
            return fail(LA_ERR_INVALID_ARG, "%s: %s is not %zu-byte aligned", fn, names[i], es);
        r.ptr[i] = ptrs[i];
        const int64_t dense[3] = {(int64_t)H * N * D, D, (int64_t)N * D};  // [B][H][N][D]
        const int sizes[3] = {B, N, H};
        for (int d = 0; d < 3; ++d) {
            const int64_t x = strides ? strides[3 * i + d] : dense[d];
            if (x >= (1ll << 40) || x <= -(1ll << 40))
                return fail(LA_ERR_INVALID_ARG, "%s: %s has stride %lld", fn, names[i], (long long)x);
            r.strides[i][d] = sizes[d] > 1 ? x : 0;  // the stride of a single row is no one's
        }
    }
    const void* p[] = {freqs};
    const char* nm[] = {"freqs"};
    if (la_status s = check_ptrs(fn, p, nm, 1, 8)) return s;
    if (reinterpret_cast<uintptr_t>(positions) & 3u)
        return fail(LA_ERR_INVALID_ARG, "%s: positions is not 4-byte aligned", fn);
    return LA_OK;
}

static la_status norm_args(const char* fn, RotaryShape* sh, const float* q_weight, const float* k_weight, float eps) {
    if (!(eps > 0.f) || !std::isfinite(eps)) return fail(LA_ERR_INVALID_ARG, "%s: eps=%g must be positive and finite", fn, eps);
    if ((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight)) & 3u)
        return fail(LA_ERR_INVALID_ARG, "%s: q_weight or k_weight is not 4-byte aligned", fn);
    sh->w[0] = q_weight, sh->w[1] = k_weight, sh->eps = eps;
    return LA_OK;
}

static la_status run_rotary(const char* fn, const RotaryShape& sh, la_dtype dtype, bool norm, void* stream) {
    LaunchCtx ctx;
    if (la_status s = get_ctx((cudaStream_t)stream, &ctx)) return s;
    return finish(rotary(ctx, sh, dtype == LA_DTYPE_BF16, norm), fn);
}

la_status la_rotary_frequencies(int rot, double base, la_rotary_scaling scaling, double factor, double original_len,
                                double beta_fast, double beta_slow, uint64_t* freqs, float* magnitude) {
    static const char* fn = "la_rotary_frequencies";
    if (rot < 2 || rot % 2 || rot > 128) return fail(LA_ERR_INVALID_ARG, "%s: rot=%d must be even, from 2 to 128", fn, rot);
    if (!std::isfinite(base) || !(base >= 1.0)) return fail(LA_ERR_INVALID_ARG, "%s: base=%g must be at least 1", fn, base);
    if (scaling < LA_ROTARY_UNSCALED || scaling > LA_ROTARY_BY_PARTS)
        return fail(LA_ERR_UNSUPPORTED, "%s: unknown scaling %d", fn, (int)scaling);
    if (scaling != LA_ROTARY_UNSCALED && (!std::isfinite(factor) || !(factor >= 1.0)))
        return fail(LA_ERR_INVALID_ARG, "%s: factor=%g must be at least 1", fn, factor);
    if (scaling == LA_ROTARY_BY_PARTS &&
        !(std::isfinite(original_len) && original_len > 0 && std::isfinite(beta_fast) && std::isfinite(beta_slow) &&
          beta_fast > beta_slow))
        return fail(LA_ERR_INVALID_ARG, "%s: original_len=%g must be positive and beta_fast=%g above beta_slow=%g", fn,
                    original_len, beta_fast, beta_slow);
    if (!freqs || !magnitude) return fail(LA_ERR_INVALID_ARG, "%s: freqs or magnitude is NULL", fn);
    const double two_pi = 6.283185307179586;
    const double to_turns = 0.15915494309189535, to_turns_rest = -9.839338337591243e-18;  // 1 / 2 pi in two terms
    if (scaling == LA_ROTARY_BASE && rot > 2) base *= std::pow(factor, (double)rot / (rot - 2));
    if (!std::isfinite(base)) return fail(LA_ERR_INVALID_ARG, "%s: factor=%g makes the base infinite", fn, factor);
    for (int i = 0; i < rot / 2; ++i) {
        double theta = std::pow(base, -2.0 * i / rot);
        if (scaling == LA_ROTARY_LINEAR) theta /= factor;
        if (scaling == LA_ROTARY_BY_PARTS) {
            const double turns = original_len * theta / two_pi;
            const double keep = std::fmin(1.0, std::fmax(0.0, (turns - beta_slow) / (beta_fast - beta_slow)));
            theta = theta / factor * (1.0 - keep) + theta * keep;
        }
        // theta <= 1, so below a turn; the product's rounding goes into the second term
        const double hi = theta * to_turns, lo = std::fma(theta, to_turns, -hi) + theta * to_turns_rest;
        freqs[i] = (uint64_t)std::ldexp(hi, 64) + (uint64_t)(int64_t)std::llrint(std::ldexp(lo, 64));
    }
    *magnitude = scaling == LA_ROTARY_BY_PARTS ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return LA_OK;
}

la_status la_forward_rotary(const void* q, const void* k, void* q_out, void* k_out, int B, int N, int Hq, int Hk,
                            int D, const int64_t* strides, const int* positions, int position_rows,
                            int first_position, const uint64_t* freqs, int rot, float magnitude,
                            la_rotary_layout layout, la_dtype dtype, int fill, void* stream) {
    static const char* fn = "la_forward_rotary";
    const void* p[] = {q, k, q_out, k_out};
    const char* nm[] = {"q", "k", "q_out", "k_out"};
    RotaryShape sh;
    bool empty;
    la_status s = rotary_shape(fn, &sh, p, nm, 4, B, N, Hq, Hk, D, strides, positions, position_rows, first_position,
                               freqs, rot, magnitude, layout, dtype, fill, &empty);
    return s != LA_OK || empty ? s : run_rotary(fn, sh, dtype, false, stream);
}

la_status la_backward_rotary(const void* dq_out, const void* dk_out, void* dq, void* dk, int B, int N, int Hq, int Hk,
                             int D, const int64_t* strides, const int* positions, int position_rows,
                             int first_position, const uint64_t* freqs, int rot, float magnitude,
                             la_rotary_layout layout, la_dtype dtype, int fill, void* stream) {
    static const char* fn = "la_backward_rotary";
    const void* p[] = {dq_out, dk_out, dq, dk};
    const char* nm[] = {"dq_out", "dk_out", "dq", "dk"};
    RotaryShape sh;
    bool empty;
    la_status s = rotary_shape(fn, &sh, p, nm, 4, B, N, Hq, Hk, D, strides, positions, position_rows, first_position,
                               freqs, rot, magnitude, layout, dtype, fill, &empty);
    sh.backward = true;
    return s != LA_OK || empty ? s : run_rotary(fn, sh, dtype, false, stream);
}

la_status la_forward_norm_rotary(const void* q, const void* k, const float* q_weight, const float* k_weight,
                                 void* q_out, void* k_out, int B, int N, int Hq, int Hk, int D, const int64_t* strides,
                                 const int* positions, int position_rows, int first_position, const uint64_t* freqs,
                                 int rot, float magnitude, la_rotary_layout layout, float eps, la_dtype dtype,
                                 int fill, void* stream) {
    static const char* fn = "la_forward_norm_rotary";
    const void* p[] = {q, k, q_out, k_out};
    const char* nm[] = {"q", "k", "q_out", "k_out"};
    RotaryShape sh;
    bool empty;
    la_status s = rotary_shape(fn, &sh, p, nm, 4, B, N, Hq, Hk, D, strides, positions, position_rows, first_position,
                               freqs, rot, magnitude, layout, dtype, fill, &empty);
    if (s != LA_OK || (s = norm_args(fn, &sh, q_weight, k_weight, eps)) != LA_OK || empty) return s;
    return run_rotary(fn, sh, dtype, true, stream);
}

la_status la_backward_norm_rotary(const void* q, const void* k, const void* dq_out, const void* dk_out,
                                  const float* q_weight, const float* k_weight, void* dq, void* dk, float* dq_weight,
                                  float* dk_weight, int B, int N, int Hq, int Hk, int D, const int64_t* strides,
                                  const int* positions, int position_rows, int first_position, const uint64_t* freqs,
                                  int rot, float magnitude, la_rotary_layout layout, float eps, la_dtype dtype,
                                  int fill, void* stream) {
    static const char* fn = "la_backward_norm_rotary";
    const void* p[] = {q, k, dq_out, dk_out, dq, dk};
    const char* nm[] = {"q", "k", "dq_out", "dk_out", "dq", "dk"};
    RotaryShape sh;
    bool empty;
    la_status s = rotary_shape(fn, &sh, p, nm, 6, B, N, Hq, Hk, D, strides, positions, position_rows, first_position,
                               freqs, rot, magnitude, layout, dtype, fill, &empty);
    if (s != LA_OK || (s = norm_args(fn, &sh, q_weight, k_weight, eps)) != LA_OK) return s;
    if ((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 3u)
        return fail(LA_ERR_INVALID_ARG, "%s: dq_weight or dk_weight is not 4-byte aligned", fn);
    if (empty && !dq_weight && !dk_weight) return LA_OK;
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    if (empty) {  // sums over no rows
        cudaError_t e = dq_weight ? cudaMemsetAsync(dq_weight, 0, sizeof(float) * D, ctx.stream) : cudaSuccess;
        if (e == cudaSuccess && dk_weight) e = cudaMemsetAsync(dk_weight, 0, sizeof(float) * D, ctx.stream);
        return finish(e, fn);
    }
    sh.backward = true;
    return finish(norm_rotary_grad(ctx, sh, dtype == LA_DTYPE_BF16, dq_weight, dk_weight), fn);
}

size_t la_norm_rotary_workspace_bytes(int B, int N, int Hq, int Hk, int D, int num_sms) {
    static const char* fn = "la_norm_rotary_workspace_bytes";
    if (!head_ok(D))
        return fail(LA_ERR_UNSUPPORTED, "%s: D=%d, supported head sizes are 32, 64, 128", fn, D), SIZE_MAX;
    if (B < 0 || N < 0 || Hq < 0 || Hk < 0 || (unsigned long long)B * N >= (1ull << 30) ||
        (unsigned long long)Hq * D >= (1ull << 30) || (unsigned long long)Hk * D >= (1ull << 30) ||
        (unsigned long long)B * N * ((unsigned long long)Hq + Hk) * D >= (1ull << 40))
        return fail(LA_ERR_INVALID_ARG, "%s: sizes B=%d N=%d Hq=%d Hk=%d", fn, B, N, Hq, Hk), SIZE_MAX;
    if (num_sms <= 0) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, fn), SIZE_MAX;
    }
    return rotary_grad_scratch(B, N, Hq, Hk, D, true, num_sms);
}

// Sizes of a prefill call.
static la_status check_prefill(const char* fn, int T, int R, int Hq, int Hkv, int D, int num_pages, int page_size,
                               int max_pages, int window, la_dtype dtype, int* log2p) {
    la_status s = check_pages(fn, num_pages, page_size, log2p);
    if (s != LA_OK) return s;
    if (T < 0 || R < 0 || Hq < 0 || Hkv < 0 || max_pages < 0 || window < 0)
        return fail(LA_ERR_INVALID_ARG, "%s: negative size T=%d R=%d Hq=%d Hkv=%d max_pages=%d window=%d", fn, T, R, Hq,
                    Hkv, max_pages, window);
    if (dtype != LA_DTYPE_F32 && dtype != LA_DTYPE_BF16)
        return fail(LA_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
    if (!head_ok(D))
        return fail(LA_ERR_UNSUPPORTED, "%s: D=%d, supported head sizes are 32, 64, 128", fn, D);
    if (Hq && (Hkv == 0 || Hq % Hkv))
        return fail(LA_ERR_INVALID_ARG, "%s: Hq=%d query heads over Hkv=%d key heads: not a multiple", fn, Hq, Hkv);
    if ((unsigned long long)max_pages * page_size >= (1ull << 30))
        return fail(LA_ERR_INVALID_ARG, "%s: max_pages=%d of %d positions: 2^30 positions or more", fn, max_pages, page_size);
    if (R >= (1 << 20)) return fail(LA_ERR_INVALID_ARG, "%s: R=%d: 2^20 requests or more", fn, R);
    // rows of a request and head are counted in 32 bits
    if (T >= (1 << 30) || (unsigned long long)T * Hq >= (1ull << 30) || Hkv >= (1 << 16) ||
        (unsigned long long)num_pages * page_size * (Hkv ? Hkv : 1) >= (1ull << 40) / D)
        return fail(LA_ERR_INVALID_ARG, "%s: tensor too large", fn);
    return LA_OK;
}

size_t la_paged_prefill_workspace_bytes(int D, la_dtype dtype, int num_sms) {
    static const char* fn = "la_paged_prefill_workspace_bytes";
    if (dtype != LA_DTYPE_F32 && dtype != LA_DTYPE_BF16)
        return fail(LA_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype), SIZE_MAX;
    if (!head_ok(D))
        return fail(LA_ERR_UNSUPPORTED, "%s: D=%d, supported head sizes are 32, 64, 128", fn, D), SIZE_MAX;
    if (num_sms <= 0) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&num_sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return cuda_fail(e, fn), SIZE_MAX;
    }
    return paged_prefill_scratch(D, dtype == LA_DTYPE_BF16, num_sms);
}

la_status la_paged_prefill(const void* q, const void* K_pages, const void* V_pages, const int* block_table,
                           const int* cached_lens, const int* seq_starts, void* out, float* lse, int T, int R, int Hq,
                           int Hkv, int D, int num_pages, int page_size, int max_pages, int window, float scale,
                           la_dtype dtype, int fill, void* stream) {
    static const char* fn = "la_paged_prefill";
    int log2p = 0;
    la_status s = check_prefill(fn, T, R, Hq, Hkv, D, num_pages, page_size, max_pages, window, dtype, &log2p);
    if (s != LA_OK || (s = check_fill(fn, fill, 3)) != LA_OK) return s;
    if (!std::isfinite(scale * 1.4426950408889634f))  // scores are taken to base 2
        return fail(LA_ERR_INVALID_ARG, "%s: scale=%g, or its product with log2 e, is not finite", fn, scale);
    if (T == 0 || Hq == 0 || (R == 0 && !fill)) return LA_OK;
    const void* p[] = {q, out, K_pages, V_pages};
    const char* nm[] = {"q", "out", "K_pages", "V_pages"};
    if ((s = check_ptrs(fn, p, nm, num_pages ? 4 : 2, 16)) != LA_OK) return s;
    const void* ip[] = {cached_lens, seq_starts, block_table};
    const char* in[] = {"cached_lens", "seq_starts", "block_table"};
    if (R && (s = check_ptrs(fn, ip, in, max_pages ? 3 : 2, 4)) != LA_OK) return s;
    if ((fill & 2) && !lse) return fail(LA_ERR_INVALID_ARG, "%s: lse is NULL", fn);
    if (reinterpret_cast<uintptr_t>(lse) & 3u)
        return fail(LA_ERR_INVALID_ARG, "%s: lse is not 4-byte aligned", fn);
    LaunchCtx ctx;
    if ((s = get_ctx((cudaStream_t)stream, &ctx)) != LA_OK) return s;
    const PrefillShape sh = {T, R, Hq, Hkv, num_pages, log2p, max_pages, window,
                             scale == 0.f ? 1.f / sqrtf((float)D) : scale};
    cudaError_t e = cudaErrorInvalidValue;
#define LA_PP_CASE(Ty, d)                                                                               \
    if (D == d)                                                                                         \
        e = paged_prefill<Ty, d>(ctx, (const Ty*)q, (const Ty*)K_pages, (const Ty*)V_pages, block_table, \
                                 cached_lens, seq_starts, (Ty*)out, lse, sh, fill);
    if (dtype == LA_DTYPE_F32) {
        LA_PP_CASE(float, 32) else LA_PP_CASE(float, 64) else LA_PP_CASE(float, 128)
    } else {
        LA_PP_CASE(__nv_bfloat16, 32) else LA_PP_CASE(__nv_bfloat16, 64) else LA_PP_CASE(__nv_bfloat16, 128)
    }
#undef LA_PP_CASE
    return finish(e, fn);
}

la_status la_selftest_expired_waits(void* stream) {
    LaunchCtx ctx;
    la_status s = get_ctx((cudaStream_t)stream, &ctx);
    if (s != LA_OK) return s;
    return finish(selftest_expired_waits(ctx), "la_selftest_expired_waits");
}

la_status la_debug_withhold_publication(int unit, unsigned spin_limit) {
    if (unit < 0 || spin_limit == 0)
        return fail(LA_ERR_INVALID_ARG, "la_debug_withhold_publication: unit %d, spin limit %u", unit,
                    spin_limit);
    g_spin_limit.store(spin_limit);
    g_withhold_unit.store(unit);
    return LA_OK;
}

la_status la_check_device_status(void* stream) {
    LaunchCtx ctx;
    la_status s = get_ctx((cudaStream_t)stream, &ctx);
    if (s != LA_OK) return s;
    cudaError_t e = cudaStreamSynchronize(ctx.stream);
    if (e != cudaSuccess) return cuda_fail(e, "la_check_device_status");
    unsigned int word = 0;
    if ((e = cudaMemcpy(&word, ctx.status_word, sizeof(word), cudaMemcpyDeviceToHost)))
        return cuda_fail(e, "la_check_device_status");
    if (word) {
        const unsigned int zero = 0;
        if ((e = cudaMemcpy(ctx.status_word, &zero, sizeof(zero), cudaMemcpyHostToDevice)))
            return cuda_fail(e, "la_check_device_status");
        if (!(word & ~kStatusBadIndex))
            return fail(LA_ERR_BAD_INDEX, "a length, page or slot read from device memory was out of range "
                        "(code 0x%x)", word);
        return fail(LA_ERR_TIMEOUT, "a bounded device wait gave up (code 0x%x)", word);
    }
    return LA_OK;
}

const char* la_status_string(la_status status) {
    switch (status) {
        case LA_OK: return "LA_OK";
        case LA_ERR_INVALID_ARG: return "LA_ERR_INVALID_ARG";
        case LA_ERR_UNSUPPORTED: return "LA_ERR_UNSUPPORTED";
        case LA_ERR_CUDA: return "LA_ERR_CUDA";
        case LA_ERR_TIMEOUT: return "LA_ERR_TIMEOUT";
        case LA_ERR_BAD_INDEX: return "LA_ERR_BAD_INDEX";
    }
    return "LA_ERR_UNKNOWN";
}

const char* la_last_error_message(void) { return g_msg; }

uint64_t la_kernel_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

}  // extern "C"
