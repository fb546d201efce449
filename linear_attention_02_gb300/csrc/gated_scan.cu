// gated_scan.cu -- the gated scan's calls, and its single-token step.
#include "gated_scan.cuh"

namespace la {
namespace {

using namespace scan;

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

__global__ void unset_kernel(unsigned* a, size_t na, unsigned* b, size_t nb) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const size_t id = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x, all = static_cast<size_t>(gridDim.x) * 256;
    const auto fill = [&](unsigned* to, size_t n) {
        const size_t n4 = n / 4;
        for (size_t i = id; i < n4; i += all) reinterpret_cast<uint4*>(to)[i] = make_uint4(kUnset, kUnset, kUnset, kUnset);
        if (id < n % 4) to[4 * n4 + id] = kUnset;
    };
    fill(a, na);
    fill(b, nb);
}

}  // namespace

namespace scan {
cudaError_t unset_words(const LaunchCtx& c, unsigned* a, size_t na, unsigned* b, size_t nb) {
    const size_t blocks = (std::max(na, nb) / 4 + 256) / 256;
    unset_kernel<<<static_cast<unsigned>(std::min<size_t>(blocks, 4 * c.num_sms)), 256, 0, c.stream>>>(a, na, b, nb);
    note_launch();
    return cudaGetLastError();
}
}  // namespace scan

template <typename T>
cudaError_t gated_scan_forward(const LaunchCtx& c, const T* A, const T* X, T* O, const ScanShape& s,
                               const float* h_init, float* h_final, float* Ckpt, bool fill) {
    Args<T> a = args_of<T>(s, A, X);
    a.O = O;
    a.init = h_init;
    a.fin = h_final;
    a.incl = Ckpt;
    a.fill = fill ? 1 : 0;
    return launch<T, false>(c, a, s.logit, Ckpt == nullptr);
}

template <typename T>
cudaError_t gated_scan_backward(const LaunchCtx& c, const T* A, const T* X, const T* G, T* dA, T* dX,
                                const ScanShape& s, const float* h_init, const float* dh_final,
                                float* dh_init, const float* Ckpt, int fill) {
    float* states = nullptr;
    cudaError_t e = cudaSuccess;
    const size_t tiles = (static_cast<size_t>(s.N) + TILE - 1) / TILE;
    if (!Ckpt && tiles > 1) {  // the forward's tile states, without its output
        e = scratch_alloc(c, reinterpret_cast<void**>(&states), sizeof(float) * s.B * tiles * s.C);
        if (e == cudaSuccess) e = gated_scan_forward<T>(c, A, X, nullptr, s, h_init, nullptr, states, false);
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
        a.fill = fill;
        e = launch<T, true>(c, a, s.logit, true);
    }
    scratch_free(c, states);
    return e;
}

size_t gated_scan_scratch(int B, int N, int C, bool backward, bool ckpt) {
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
        for (int v = 0; v < VEC; v += 4) {
            float d[4], h4[4];
            const float x4[4] = {xv[v], xv[v + 1], xv[v + 2], xv[v + 3]};
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = av[v + i], h4[i] = hv[v + i];
            if constexpr (kLogit) gate(d, d);
            step<kLogit>(h4, d, x4);
#pragma unroll
            for (int i = 0; i < 4; ++i) hv[v + i] = h4[i];
        }
#pragma unroll
        for (int v = 0; v < VEC; v += 4)
            *reinterpret_cast<float4*>(h + i0 + v) = make_float4(hv[v], hv[v + 1], hv[v + 2], hv[v + 3]);
        *reinterpret_cast<uint4*>(out + i0) = pack(hv);
        return;
    }
    for (int64_t i = i0; i < n; ++i) {
        float d[2] = {to_f(a[i]), 0.f}, y[2] = {h[i], 0.f};
        const float xi[2] = {to_f(x[i]), 0.f};
        if constexpr (kLogit) gate(d, d);
        step<kLogit>(y, d, xi);
        h[i] = y[0];
        out[i] = from_f<T>(y[0]);
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

#define LA_INST_SCAN(T)                                                                               \
    template cudaError_t gated_scan_forward<T>(const LaunchCtx&, const T*, const T*, T*,              \
                                               const ScanShape&, const float*, float*, float*, bool); \
    template cudaError_t gated_scan_backward<T>(const LaunchCtx&, const T*, const T*, const T*, T*,   \
                                                T*, const ScanShape&, const float*, const float*,     \
                                                float*, const float*, int);                           \
    template cudaError_t gated_scan_step<T>(const LaunchCtx&, const T*, const T*, float*, T*, int64_t, \
                                            bool);
LA_INST_SCAN(float) LA_INST_SCAN(__nv_bfloat16)

}  // namespace la
