// rotary.cu -- rotary positions of queries and keys, with or without a norm of every head
// in the same pass, and the gradients of both.
//
// Pair i of a row at position p turns by the angle p theta_i:
//     (y0, y1) = mag (x0 cos - x1 sin, x0 sin + x1 cos),
// its gradient by the opposite angle.  The norm before it is n = x r w with
// r = 1 / sqrt(mean x^2 + eps); with g the gradient turned back and u = x r, h = g w,
//     dx = r (h - u mean(u h)),   dw = sum over rows of g u.
//
// Angles.  theta_i is kept as a whole number f_i of 2^-64 turns, so that the phase of any
// position is p f_i modulo 2^64: an integer product, exact for every position.  Its upper
// 32 bits are taken to the nearest quarter turn and a rest of at most an eighth, whose
// sine and cosine are those of an fp32 number with a rounding of 2^-25 of itself: an angle
// is off by 2.4e-8 at most, whether the position is 1 or 2^31.
//
// Bound by memory: a row is read once and written once (with the norm's gradient, two are
// read).  A thread holds one unit of a row: two pieces of 16 bytes whose elements are paired
// with each other (half layout) or among themselves; D / (2 VEC) neighbouring lanes hold a
// row and sum up its squares between them.  A block takes a tile of tokens with all heads
// of the queries or of the keys, works out the tile's sines and cosines once for all heads
// into shared memory, and has four rows a thread in flight.  Rows that are not 16-byte aligned, or whose
// rotated part is not a whole number of units, take units of two single elements.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "la_common.cuh"
#include "la_launch.h"
#include "la_plan.h"

namespace la {
namespace {

constexpr int kThreads = 256;

// Sine and cosine of a phase in units of 2^-32 turns.
__device__ __forceinline__ void turn(uint32_t phase, float& s, float& c) {
    const uint32_t quarter = (phase + 0x20000000u) >> 30;                   // nearest
    const int rest = static_cast<int>(phase - (quarter << 30));             // within +- 2^29
    float a, b;
    sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &a, &b);   // rest / 2^31 half turns
    s = quarter & 1 ? b : a;
    c = quarter & 1 ? a : b;
    if (quarter & 2) s = -s;
    if ((quarter + 1) & 2) c = -c;
}

template <typename T, int VEC>
struct Piece;  // VEC elements in one access
template <>
struct Piece<float, 4> { using type = float4; };
template <>
struct Piece<__nv_bfloat16, 8> { using type = uint4; };
template <>
struct Piece<float, 1> { using type = float; };
template <>
struct Piece<__nv_bfloat16, 1> { using type = __nv_bfloat16; };

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const typename Piece<T, VEC>::type& p, float* x) {
    if constexpr (VEC == 1) {
        x[0] = to_f<T>(p);
    } else if constexpr (sizeof(T) == 4) {
        x[0] = p.x, x[1] = p.y, x[2] = p.z, x[3] = p.w;
    } else {
        const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
}
template <typename T, int VEC>
__device__ __forceinline__ typename Piece<T, VEC>::type pack(const float* x) {
    if constexpr (VEC == 1) {
        return from_f<T>(x[0]);
    } else if constexpr (sizeof(T) == 4) {
        return make_float4(x[0], x[1], x[2], x[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// One side of a call, the queries or the keys.
struct Side {
    const void *x, *g;  // input rows; with a norm's gradient also the gradient's rows
    void* y;
    int64_t xs[3], gs[3], ys[3];  // strides in elements: batch row, token, head
    const float* w;
    float* part;                  // partial sums of dw, one row of D a block (null: none)
    int H, fill, tile, tiles, blocks;  // tokens of a tile; tiles of all batch rows; blocks
};

struct RotaryArgs {
    Side side[2];
    int B, N, rot, interleaved, backward;
    const uint64_t* freqs;
    const int* pos;
    int64_t pos_batch;
    int first;
    float mag, eps;
};

enum { kPlain, kNorm, kNormGrad };

template <typename T, int D, int VEC, int MODE>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs p) {
    using P = typename Piece<T, VEC>::type;
    constexpr int UNITS = D / (2 * VEC);                 // of a row
    constexpr int LANES = UNITS < 32 ? UNITS : 32;       // that hold it
    constexpr int EACH = UNITS / LANES;                  // units of a lane
    constexpr int ROWS = kThreads / LANES;               // rows a block has at once
    constexpr int FLY = (EACH > 1 ? 2 : MODE == kNormGrad ? 2 : 4);  // rows of a thread in flight
    constexpr int E = 2 * VEC;                           // elements of a unit
    extern __shared__ float2 s_trig[];                   // [tile][rot / 2]: cosine, sine
    const bool second = static_cast<int>(blockIdx.x) >= p.side[0].blocks;
    const Side& sd = p.side[second];
    const int block = blockIdx.x - (second ? p.side[0].blocks : 0);
    const int lane = threadIdx.x % LANES, row0 = threadIdx.x / LANES;
    const int pairs = p.rot / 2, rotated = pairs / VEC;  // units that turn
    const T* x = static_cast<const T*>(sd.x);
    const T* g = static_cast<const T*>(sd.g);
    T* y = static_cast<T*>(sd.y);

    int at[EACH], to[EACH], unit[EACH];                  // first elements of a unit's pieces
    float w[MODE == kPlain ? 1 : EACH * E], dw[MODE == kNormGrad ? EACH * E : 1];
#pragma unroll
    for (int u = 0; u < EACH; ++u) {
        unit[u] = lane + u * LANES;
        const bool half = !p.interleaved && unit[u] < rotated;
        at[u] = unit[u] * (half ? VEC : E);
        to[u] = at[u] + (half ? pairs : VEC);
        if constexpr (MODE != kPlain) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                w[u * E + i] = sd.w ? sd.w[at[u] + i] : 1.f;
                w[u * E + VEC + i] = sd.w ? sd.w[to[u] + i] : 1.f;
            }
        }
        if constexpr (MODE == kNormGrad) {
#pragma unroll
            for (int i = 0; i < E; ++i) dw[u * E + i] = 0.f;
        }
    }
    // tokens of the tile run fastest where they are nearer to each other than heads
    const bool by_token = sd.xs[1] < sd.xs[2] || sd.H == 1;
    const int per = (p.N + sd.tile - 1) / sd.tile;       // tiles of a batch row

    for (int tile = block; tile < sd.tiles; tile += sd.blocks) {
        const int b = tile / per, n0 = (tile - b * per) * sd.tile;
        const int tokens = min(sd.tile, p.N - n0), rows = tokens * sd.H;
        const int* pos = p.pos ? p.pos + b * p.pos_batch + n0 : nullptr;
        // The first rows are on their way while the sines are worked out.
        P px[FLY][EACH][2], pg[MODE == kNormGrad ? FLY : 1][EACH][2];
        int hd[FLY], tk[FLY];
        const auto load = [&](int base) {
#pragma unroll
            for (int f = 0; f < FLY; ++f) {
                const int i = base + row0 + f * ROWS;
                tk[f] = -1;
                if (i >= rows) continue;
                const int a = by_token ? i / tokens : i / sd.H;
                tk[f] = by_token ? i - a * tokens : a;
                hd[f] = by_token ? a : i - a * sd.H;
                const int64_t n = n0 + tk[f];
                const T* row = x + b * sd.xs[0] + n * sd.xs[1] + hd[f] * sd.xs[2];
                const T* grow = MODE == kNormGrad ? g + b * sd.gs[0] + n * sd.gs[1] + hd[f] * sd.gs[2] : nullptr;
#pragma unroll
                for (int u = 0; u < EACH; ++u) {
                    px[f][u][0] = *reinterpret_cast<const P*>(row + at[u]);
                    px[f][u][1] = *reinterpret_cast<const P*>(row + to[u]);
                    if constexpr (MODE == kNormGrad) {
                        pg[f][u][0] = *reinterpret_cast<const P*>(grow + at[u]);
                        pg[f][u][1] = *reinterpret_cast<const P*>(grow + to[u]);
                    }
                }
            }
        };
        load(0);
        __syncthreads();  // the last tile's rows have read its sines
        for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
            const int t = i / pairs;
            const int n = pos ? pos[t] : p.first + n0 + t;
            const uint64_t ph = static_cast<uint64_t>(static_cast<int64_t>(n)) * p.freqs[i - t * pairs] + 0x80000000u;
            float s, c;
            turn(static_cast<uint32_t>(ph >> 32), s, c);
            s_trig[i] = make_float2(c * p.mag, (p.backward ? -s : s) * p.mag);
        }
        __syncthreads();
        for (int base = 0; base < rows; base += FLY * ROWS) {
            if (base) load(base);
#pragma unroll
            for (int f = 0; f < FLY; ++f) {
                const int t = tk[f];
                const bool live = t >= 0 && !(pos && pos[t] < 0);  // a row of a token
                float v[EACH * E];
#pragma unroll
                for (int u = 0; u < EACH; ++u) {
                    if (!live) {
#pragma unroll
                        for (int i = 0; i < E; ++i) v[u * E + i] = 0.f;
                    } else {
                        unpack<T, VEC>(px[f][u][0], v + u * E);
                        unpack<T, VEC>(px[f][u][1], v + u * E + VEC);
                    }
                }
                float r = 1.f;
                if constexpr (MODE != kPlain) {
                    float q = 0.f;
#pragma unroll
                    for (int i = 0; i < EACH * E; ++i) q = fmaf(v[i], v[i], q);
#pragma unroll
                    for (int o = LANES / 2; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
                    r = 1.f / sqrtf(q * (1.f / D) + p.eps);
                }
                float z[MODE == kNormGrad ? EACH * E : 1];
                float mean = 0.f;
#pragma unroll
                for (int u = 0; u < EACH; ++u) {
                    float* m = v + u * E;  // what is turned
                    if constexpr (MODE == kNorm) {
#pragma unroll
                        for (int i = 0; i < E; ++i) m[i] = m[i] * r * w[u * E + i];
                    }
                    if constexpr (MODE == kNormGrad) {
                        m = z + u * E;
                        if (!live) {
#pragma unroll
                            for (int i = 0; i < E; ++i) m[i] = 0.f;
                        } else {
                            unpack<T, VEC>(pg[f][u][0], m);
                            unpack<T, VEC>(pg[f][u][1], m + VEC);
                        }
                    }
                    if (live && unit[u] < rotated) {
                        const float2* cs = s_trig + t * pairs + unit[u] * VEC;
                        if (p.interleaved) {
#pragma unroll
                            for (int i = 0; i < VEC; ++i) {
                                const float2 a = cs[i];
                                const float m0 = m[2 * i], m1 = m[2 * i + 1];
                                m[2 * i] = m0 * a.x - m1 * a.y;
                                m[2 * i + 1] = m0 * a.y + m1 * a.x;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < VEC; ++i) {
                                const float2 a = cs[i];
                                const float m0 = m[i], m1 = m[VEC + i];
                                m[i] = m0 * a.x - m1 * a.y;
                                m[VEC + i] = m0 * a.y + m1 * a.x;
                            }
                        }
                    }
                    if constexpr (MODE == kNormGrad) {
#pragma unroll
                        for (int i = 0; i < E; ++i) {
                            float& n = v[u * E + i];
                            n *= r;
                            dw[u * E + i] = fmaf(m[i], n, dw[u * E + i]);
                            m[i] *= w[u * E + i];
                            mean = fmaf(m[i], n, mean);
                        }
                    }
                }
                if constexpr (MODE == kNormGrad) {
#pragma unroll
                    for (int o = LANES / 2; o; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
                    mean *= 1.f / D;
#pragma unroll
                    for (int i = 0; i < EACH * E; ++i) v[i] = r * (z[i] - v[i] * mean);
                }
                if (live || (t >= 0 && sd.fill)) {
                    T* out = y + b * sd.ys[0] + static_cast<int64_t>(n0 + t) * sd.ys[1] + hd[f] * sd.ys[2];
                    if (!live) {  // whatever the weights are
#pragma unroll
                        for (int i = 0; i < EACH * E; ++i) v[i] = 0.f;
                    }
#pragma unroll
                    for (int u = 0; u < EACH; ++u) {
                        *reinterpret_cast<P*>(out + at[u]) = pack<T, VEC>(v + u * E);
                        *reinterpret_cast<P*>(out + to[u]) = pack<T, VEC>(v + u * E + VEC);
                    }
                }
            }
        }
    }
    if constexpr (MODE == kNormGrad) {
        // The block's sums: units over the block's rows, in the order of the rows.
        if (sd.part == nullptr) return;
        float* s_dw = reinterpret_cast<float*>(s_trig);  // [ROWS][D + 1]
        __syncthreads();
#pragma unroll
        for (int u = 0; u < EACH; ++u)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s_dw[row0 * (D + 1) + at[u] + i] = dw[u * E + i];
                s_dw[row0 * (D + 1) + to[u] + i] = dw[u * E + VEC + i];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += kThreads) {
            float a = 0.f;
            for (int i = 0; i < ROWS; ++i) a += s_dw[i * (D + 1) + c];
            sd.part[static_cast<int64_t>(block) * D + c] = a;
        }
    }
}

// dw of a side: its blocks' sums, added up by 32 threads a column in a fixed order.
__global__ void __launch_bounds__(1024) rotary_weight_kernel(const float* q_part, const float* k_part, int q_blocks,
                                                             int k_blocks, int D, float* dwq, float* dwk) {
    __shared__ float s_sum[32][33];
    const int cols = D / 32, side = blockIdx.x / cols, c0 = (blockIdx.x - side * cols) * 32;
    const float* part = side ? k_part : q_part;
    float* dw = side ? dwk : dwq;
    const int blocks = side ? k_blocks : q_blocks, x = threadIdx.x & 31, i0 = threadIdx.x >> 5;
    if (dw == nullptr) return;
    float a = 0.f;
    for (int i = i0; i < blocks; i += 32) a += part[static_cast<int64_t>(i) * D + c0 + x];
    s_sum[i0][x] = a;
    __syncthreads();
    a = s_sum[x][i0];  // column i0, partial sum x
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if (x == 0) dw[c0 + i0] = a;
}

// Largest common piece: every row's units are whole 16-byte pieces.
bool aligned(const RotaryShape& s, int rot, int vec, int es) {
    if (rot % (2 * vec)) return false;
    for (int i = 0; i < s.tensors; ++i) {
        if (s.ptr[i] == nullptr) continue;
        if (reinterpret_cast<uintptr_t>(s.ptr[i]) & 15u) return false;
        for (int d = 0; d < 3; ++d)
            if (s.strides[i][d] % (16 / es)) return false;
    }
    return true;
}

template <typename T, int D, int VEC, int MODE>
cudaError_t launch(const LaunchCtx& c, const RotaryShape& s, float* dwq, float* dwk) {
    constexpr int UNITS = D / (2 * VEC), LANES = UNITS < 32 ? UNITS : 32, ROWS = kThreads / LANES;
    RotaryArgs p = {};
    p.B = s.B, p.N = s.N, p.rot = s.rot, p.interleaved = s.interleaved, p.backward = s.backward;
    p.freqs = s.freqs, p.pos = s.positions, p.pos_batch = s.pos_batch, p.first = s.first;
    p.mag = s.mag, p.eps = s.eps;
    int smem = 0;
    for (int i = 0; i < 2; ++i) {
        Side& d = p.side[i];
        const int H = i ? s.Hk : s.Hq;
        d.H = H;
        // tensors: q, k, [gradients of q, k,] outputs of q, k
        const int out = MODE == kNormGrad ? 4 : 2;
        d.x = s.ptr[i], d.g = s.ptr[2 + i], d.y = const_cast<void*>(s.ptr[out + i]);
        for (int j = 0; j < 3; ++j) d.xs[j] = s.strides[i][j], d.gs[j] = s.strides[2 + i][j], d.ys[j] = s.strides[out + i][j];
        d.w = s.w[i];
        d.fill = s.fill >> i & 1;
        if (H == 0) continue;
        // A tile's rows: enough for a few turns of the block where the call is large, few where
        // it is small, so that all SMs have some.
        const int64_t all = static_cast<int64_t>(s.B) * s.N * H;
        const int64_t want = std::min<int64_t>(std::max<int64_t>(all / (8 * c.num_sms), ROWS), 8 * ROWS);
        int64_t tile = std::max<int64_t>(1, want / H);
        tile = std::min<int64_t>(std::min<int64_t>(tile, 64), s.N);
        d.tile = static_cast<int>(tile);
        const int64_t tiles = (s.N + tile - 1) / tile * s.B;
        if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
        d.tiles = static_cast<int>(tiles);
        d.blocks = d.tiles;
        if (MODE == kNormGrad) d.blocks = std::min(d.tiles, rotary_grad_blocks(c.num_sms));
        smem = std::max(smem, static_cast<int>(tile) * (s.rot / 2) * 8);
    }
    float* part = nullptr;
    if (MODE == kNormGrad) {
        smem = std::max(smem, ROWS * (D + 1) * 4);
        if (dwq || dwk) {
            cudaError_t e = scratch_alloc(c, reinterpret_cast<void**>(&part), rotary_grad_scratch(s.B, s.N, s.Hq, s.Hk, D, dwq || dwk, c.num_sms));
            if (e != cudaSuccess) return e;
            if (dwq) p.side[0].part = part;
            if (dwk) p.side[1].part = part + static_cast<int64_t>(rotary_grad_blocks(c.num_sms)) * D;
        }
    }
    static_assert(ROWS * (D + 1) * 4 <= 160 * 1024, "shared memory");
    auto* kernel = rotary_kernel<T, D, VEC, MODE>;
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && p.side[0].blocks + p.side[1].blocks > 0) {
        kernel<<<p.side[0].blocks + p.side[1].blocks, kThreads, smem, c.stream>>>(p);
        note_launch();
        e = cudaGetLastError();
    }
    if (MODE == kNormGrad && (dwq || dwk)) {
        if (e == cudaSuccess) {
            rotary_weight_kernel<<<2 * (D / 32), 1024, 0, c.stream>>>(part, p.side[1].part, p.side[0].blocks,
                                                                     p.side[1].blocks, D, dwq, dwk);
            note_launch();
            e = cudaGetLastError();
        }
        scratch_free(c, part);
    }
    return e;
}

template <typename T, int D, int MODE>
cudaError_t by_alignment(const LaunchCtx& c, const RotaryShape& s, float* dwq, float* dwk) {
    constexpr int VEC = 16 / sizeof(T);
    return aligned(s, s.rot, VEC, sizeof(T)) ? launch<T, D, VEC, MODE>(c, s, dwq, dwk)
                                             : launch<T, D, 1, MODE>(c, s, dwq, dwk);
}

template <typename T, int MODE>
cudaError_t by_size(const LaunchCtx& c, const RotaryShape& s, float* dwq, float* dwk) {
    if (s.D == 32) return by_alignment<T, 32, MODE>(c, s, dwq, dwk);
    if (s.D == 64) return by_alignment<T, 64, MODE>(c, s, dwq, dwk);
    return by_alignment<T, 128, MODE>(c, s, dwq, dwk);
}

}  // namespace

int rotary_grad_blocks(int num_sms) { return 4 * num_sms; }

size_t rotary_grad_scratch(int B, int N, int Hq, int Hk, int D, bool weights, int num_sms) {
    if (!weights || static_cast<int64_t>(B) * N * (Hq + Hk) == 0) return 0;
    return 2 * sizeof(float) * rotary_grad_blocks(num_sms) * D;
}

cudaError_t rotary(const LaunchCtx& c, const RotaryShape& s, bool bf16, bool norm) {
    using bf = __nv_bfloat16;
    if (norm) return bf16 ? by_size<bf, kNorm>(c, s, nullptr, nullptr) : by_size<float, kNorm>(c, s, nullptr, nullptr);
    return bf16 ? by_size<bf, kPlain>(c, s, nullptr, nullptr) : by_size<float, kPlain>(c, s, nullptr, nullptr);
}

cudaError_t norm_rotary_grad(const LaunchCtx& c, const RotaryShape& s, bool bf16, float* dwq, float* dwk) {
    return bf16 ? by_size<__nv_bfloat16, kNormGrad>(c, s, dwq, dwk) : by_size<float, kNormGrad>(c, s, dwq, dwk);
}

}  // namespace la
