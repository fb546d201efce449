// gated_scan_impl.cuh -- the launches of the gated scan in one storage type (LA_SCAN_T, set by the
// including file) and the single-token step.
#include "gated_scan.cuh"

namespace la {
namespace {

using namespace scan;

// Scratch of one pass: ticket, A, B, end states (unless they go to the caller's
// checkpoints), all unset at first.
struct Parts {
    size_t states, bytes;
};
Parts parts_of(int B, int N, int C, bool own_incl) {
    const size_t tiles = (static_cast<size_t>(N) + TILE - 1) / TILE;
    Parts s = {};
    s.states = tiles > 1 ? static_cast<size_t>(B) * tiles * C : 0;
    s.bytes = s.states ? 4 * (4 + (own_incl ? 3 : 2) * s.states) : 0;
    return s;
}

// Map over a [B][N][C] tensor with a box of 128 rows x 128 bytes.
template <typename T>
cudaError_t stream_map(CUtensorMap* m, const T* base, int B, int N, int C) {
    tcf::EncodeTiled enc = tcf::encoder();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(C), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(B)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(C) * sizeof(T), static_cast<cuuint64_t>(N) * C * sizeof(T)};
    cuuint32_t box[3] = {static_cast<cuuint32_t>(Geo<T>::CB), TILE, 1}, es[3] = {1, 1, 1};
    const CUresult r = enc(m, sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                           const_cast<T*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// One pass along the rows (forward, or the backward's carry).  `own_incl` is
// true when the pass keeps its chain's end states in scratch.
template <typename T, bool kBwd>
cudaError_t launch(const LaunchCtx& c, Args<T> a, bool logit, bool own_incl) {
    constexpr int STREAMS = kBwd ? 3 : 2;
    const bool packed = a.starts != nullptr;
    const bool vec = static_cast<size_t>(a.C) * sizeof(T) % 16 == 0;
    const size_t tiles = (static_cast<size_t>(a.N) + TILE - 1) / TILE;
    const size_t ncb = (static_cast<size_t>(a.C) + Geo<T>::CB - 1) / Geo<T>::CB;
    if (static_cast<size_t>(a.B) * tiles * ncb >= (1ull << 31)) return cudaErrorInvalidValue;
    a.tiles = static_cast<int>(tiles);
    a.ncb = static_cast<int>(ncb);
    a.total = static_cast<unsigned>(a.B * tiles * ncb);
    a.status = c.status_word;

    Maps maps = {};
    const T* streams[3] = {a.A, a.X, a.G};
    for (int i = 0; vec && i < STREAMS; ++i)
        if (cudaError_t m = stream_map<T>(&maps.m[i], streams[i], a.B, a.N, a.C)) return m;
    const T* outs[2] = {kBwd ? a.dA : a.O, a.dX};
    for (int i = 0; vec && !packed && i < 2; ++i)
        if (cudaError_t m = outs[i] ? stream_map<T>(&maps.o[i], outs[i], a.B, a.N, a.C) : cudaSuccess) return m;

    const Parts s = parts_of(a.B, a.N, a.C, own_incl);
    uint8_t* base = nullptr;
    cudaError_t e = cudaSuccess;
    if (s.bytes && (e = scratch_alloc(c, reinterpret_cast<void**>(&base), s.bytes)) != cudaSuccess) return e;
    if (tiles > 1) {
        a.ticket = reinterpret_cast<unsigned*>(base);
        a.aggA = reinterpret_cast<float*>(base) + 4;
        a.aggB = a.aggA + s.states;
        if (own_incl) a.incl = a.aggB + s.states;
        else e = cudaMemsetAsync(a.incl, 0xFF, s.states * 4, c.stream);
    }
    if (s.bytes && e == cudaSuccess) e = cudaMemsetAsync(base, 0xFF, s.bytes, c.stream);

#define LA_SCAN_RUN(K, SMEM)                                                                       \
    {                                                                                              \
        int per = 1;                                                                               \
        if (e == cudaSuccess) e = resident_blocks<K>(c.device, NT, SMEM, &per);                    \
        if (e == cudaSuccess) {                                                                    \
            K<<<std::min<unsigned>(a.total, per * c.num_sms), NT, SMEM, c.stream>>>(a, maps);      \
            note_launch();                                                                         \
            e = cudaGetLastError();                                                                \
        }                                                                                          \
    }
#define LA_SCAN_GO(L, P, V)                                                                        \
    if (logit == L && packed == P && vec == V) {                                                   \
        constexpr int smem = static_cast<int>(smem_bytes<T, P, STREAMS>());                        \
        if constexpr (kBwd) LA_SCAN_RUN((scan_backward_kernel<T, L, P, V>), smem)                  \
        else LA_SCAN_RUN((scan_forward_kernel<T, L, P, V>), smem)                                  \
    }
    LA_SCAN_GO(false, false, false) LA_SCAN_GO(false, false, true) LA_SCAN_GO(false, true, false)
    LA_SCAN_GO(false, true, true) LA_SCAN_GO(true, false, false) LA_SCAN_GO(true, false, true)
    LA_SCAN_GO(true, true, false) LA_SCAN_GO(true, true, true)
#undef LA_SCAN_RUN
#undef LA_SCAN_GO
    scratch_free(c, base);
    return e;
}

template <typename T>
Args<T> args_of(const ScanShape& s, const T* A, const T* X) {
    Args<T> a = {};
    a.A = A;
    a.X = X;
    a.B = s.B;
    a.N = s.N;
    a.C = s.C;
    a.starts = s.starts;
    a.S = s.num_seqs;
    return a;
}

}  // namespace

template <typename T>
cudaError_t gated_scan_forward(const LaunchCtx& c, const T* A, const T* X, T* O, const ScanShape& s,
                               const float* h_init, float* h_final, float* Ckpt) {
    Args<T> a = args_of<T>(s, A, X);
    a.O = O;
    a.init = h_init;
    a.fin = h_final;
    a.incl = Ckpt;
    return launch<T, false>(c, a, s.logit, Ckpt == nullptr);
}

template <typename T>
cudaError_t gated_scan_backward(const LaunchCtx& c, const T* A, const T* X, const T* G, T* dA, T* dX,
                                const ScanShape& s, const float* h_init, const float* dh_final,
                                float* dh_init, const float* Ckpt) {
    float* states = nullptr;
    cudaError_t e = cudaSuccess;
    const size_t tiles = (static_cast<size_t>(s.N) + TILE - 1) / TILE;
    if (!Ckpt && tiles > 1) {  // the forward's tile states, without its output
        e = scratch_alloc(c, reinterpret_cast<void**>(&states), sizeof(float) * s.B * tiles * s.C);
        if (e == cudaSuccess) e = gated_scan_forward<T>(c, A, X, nullptr, s, h_init, nullptr, states);
    }
    if (e == cudaSuccess) {
        Args<T> a = args_of<T>(s, A, X);
        a.G = G;
        a.dA = dA;
        a.dX = dX;
        a.h_init = h_init;
        a.init = dh_final;
        a.fin = dh_init;
        a.states = Ckpt ? Ckpt : states;
        e = launch<T, true>(c, a, s.logit, true);
    }
    scratch_free(c, states);
    return e;
}

size_t LA_SCAN_SCRATCH(int B, int N, int C, bool backward, bool ckpt) {
    const size_t pass = parts_of(B, N, C, backward || !ckpt).bytes;
    if (!backward || ckpt || N <= TILE) return pass;
    // the states, and on top of them the larger of the two passes, one after the other
    const size_t fwd = parts_of(B, N, C, false).bytes;
    return sizeof(float) * B * ((static_cast<size_t>(N) + TILE - 1) / TILE) * C + std::max(pass, fwd);
}

namespace {

// The single-token step: 16 bytes a thread where the element count allows it,
// one element otherwise (the last elements of an odd count).
template <typename T, bool kLogit>
__global__ void scan_step_kernel(const T* __restrict__ a, const T* __restrict__ x, float* __restrict__ h,
                                 T* __restrict__ out, int64_t n) {
    constexpr int VEC = Geo<T>::VEC;
    const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x) * VEC;
    if (i0 + VEC <= n) {
        float av[VEC], xv[VEC], hv[VEC];
        unpack(*reinterpret_cast<const uint4*>(a + i0), av);
        unpack(*reinterpret_cast<const uint4*>(x + i0), xv);
#pragma unroll
        for (int v = 0; v < VEC; v += 4) {
            const float4 f = *reinterpret_cast<const float4*>(h + i0 + v);
            hv[v] = f.x, hv[v + 1] = f.y, hv[v + 2] = f.z, hv[v + 3] = f.w;
        }
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float d = kLogit ? sigmoid(av[v]) : av[v];
            hv[v] = fmaf(d, hv[v], kLogit ? (1.f - d) * xv[v] : xv[v]);
        }
#pragma unroll
        for (int v = 0; v < VEC; v += 4)
            *reinterpret_cast<float4*>(h + i0 + v) = make_float4(hv[v], hv[v + 1], hv[v + 2], hv[v + 3]);
        *reinterpret_cast<uint4*>(out + i0) = pack(hv);
        return;
    }
    for (int64_t i = i0; i < n; ++i) {
        const float d = kLogit ? sigmoid(to_f(a[i])) : to_f(a[i]);
        const float y = fmaf(d, h[i], kLogit ? (1.f - d) * to_f(x[i]) : to_f(x[i]));
        h[i] = y;
        out[i] = from_f<T>(y);
    }
}

}  // namespace

template <typename T>
cudaError_t gated_scan_step(const LaunchCtx& c, const T* a, const T* x, float* h, T* out, int64_t n,
                            bool logit) {
    auto* k = logit ? scan_step_kernel<T, true> : scan_step_kernel<T, false>;
    constexpr int per = NT * Geo<T>::VEC;
    k<<<static_cast<unsigned>((n + per - 1) / per), NT, 0, c.stream>>>(a, x, h, out, n);
    note_launch();
    return cudaGetLastError();
}

using LA_T = LA_SCAN_T;
template cudaError_t gated_scan_forward<LA_T>(const LaunchCtx&, const LA_T*, const LA_T*, LA_T*, const ScanShape&,
                                              const float*, float*, float*);
template cudaError_t gated_scan_backward<LA_T>(const LaunchCtx&, const LA_T*, const LA_T*, const LA_T*, LA_T*, LA_T*,
                                               const ScanShape&, const float*, const float*, float*, const float*);
template cudaError_t gated_scan_step<LA_T>(const LaunchCtx&, const LA_T*, const LA_T*, float*, LA_T*, int64_t, bool);

}  // namespace la
