// gated_scan_impl.cuh -- the launch of one pass of the gated scan, in the storage type
// LA_SCAN_T and the direction LA_SCAN_BWD that the including file sets.
#include "gated_scan.cuh"

namespace la {
namespace scan {

// Map over a [B][N][C] tensor with a box of 128 rows x 128 bytes.
template <typename T>
static cudaError_t stream_map(CUtensorMap* m, const T* base, int B, int N, int C) {
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
    a.withhold = static_cast<unsigned>(c.withhold_unit);
    a.spin_limit = c.spin_limit ? c.spin_limit : tcf::kSpinLimit;
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
        e = unset_words(c, reinterpret_cast<unsigned*>(base), s.bytes / 4, own_incl ? nullptr : reinterpret_cast<unsigned*>(a.incl),
                        own_incl ? 0 : s.states);
    }
    // After the kernel that unsets the words, this one may start before that has ended.
    cudaLaunchAttribute early[1];
    early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(NT);
    cfg.stream = c.stream;
    cfg.attrs = early;
    cfg.numAttrs = tiles > 1 ? 1 : 0;

#define LA_SCAN_RUN(K, SMEM)                                                                       \
    {                                                                                              \
        int per = 1;                                                                               \
        if (e == cudaSuccess) e = resident_blocks<K>(c.device, NT, SMEM, &per);                    \
        if (e == cudaSuccess) {                                                                    \
            cfg.gridDim = dim3(std::min<unsigned>(a.total, per * c.num_sms));                      \
            cfg.dynamicSmemBytes = SMEM;                                                           \
            e = cudaLaunchKernelEx(&cfg, K, static_cast<const Args<T>>(a), static_cast<const Maps>(maps)); \
            note_launch();                                                                         \
        }                                                                                          \
    }
#define LA_SCAN_WIN(L, P, V, W)                                                                    \
    if constexpr (kBwd) LA_SCAN_RUN((scan_backward_kernel<T, L, P, V, W>), smem)                   \
    else LA_SCAN_RUN((scan_forward_kernel<T, L, P, V, W>), smem)
#define LA_SCAN_GO(L, P, V)                                                                        \
    if (logit == L && packed == P && vec == V) {                                                   \
        constexpr int smem = static_cast<int>(smem_bytes<T, P, V, STREAMS>());                        \
        constexpr int blocks = kBwd ? backward_blocks<T>() : forward_blocks<T, L>();               \
        if (static_cast<size_t>(blocks) * c.num_sms > kDeep * a.B * ncb) { LA_SCAN_WIN(L, P, V, kFar) } \
        else { LA_SCAN_WIN(L, P, V, kNear) }                                                       \
    }
    LA_SCAN_GO(false, false, false) LA_SCAN_GO(false, false, true) LA_SCAN_GO(false, true, false)
    LA_SCAN_GO(false, true, true) LA_SCAN_GO(true, false, false) LA_SCAN_GO(true, false, true)
    LA_SCAN_GO(true, true, false) LA_SCAN_GO(true, true, true)
#undef LA_SCAN_RUN
#undef LA_SCAN_WIN
#undef LA_SCAN_GO
    scratch_free(c, base);
    return e;
}

template cudaError_t launch<LA_SCAN_T, LA_SCAN_BWD>(const LaunchCtx&, Args<LA_SCAN_T>, bool, bool);

}  // namespace scan
}  // namespace la
