// gated_scan.cuh -- the gated linear recurrence over token-major rows [B][N][C],
// one decay per token and channel:
//     decay form   h_t = a_t h_{t-1} + x_t
//     logit form   h_t = s_t h_{t-1} + (1 - s_t) x_t,  s_t = sigmoid(a_t)
// and its gradient (g_t the whole gradient at h_t; m_t = 1 or 1 - s_t):
//     c_t = s_t (dOut_t + c_{t+1}),  g_t = dOut_t + c_{t+1},  dX_t = m_t g_t,
//     dA_t = g_t h_{t-1}  or  s_t (1 - s_t) g_t (h_{t-1} - x_t).
// A run of rows acts on the state that enters it as h -> A h + B, so runs
// combine: (A1, B1) then (A2, B2) is (A1 A2, A2 B1 + B2); the gradient's carry c
// runs through the rows backwards with the same A.
//
// The kernels are bound by memory: every element is read once and written once
// (forward 2 streams in, 1 out; backward 3 in, 2 out).  A tile is 128 rows x 128
// bytes of a row, filled by TMA and worked by 128 threads; a thread owns 8 rows x 16
// bytes.  Per tile: each thread sums its 8 rows up to (A, B);
// one thread per channel folds the 16 row groups, gets the state that enters the
// tile from the tile before (below), and hands each row group its state; then
// each thread runs its rows and writes them.
//
// Tiles of the same channels in time form a chain.  A tile publishes the end
// state of each channel, and its (A, B) before that where the tile before is not
// done; the next tile looks back over up to 4 or 16 tiles at once to the nearest
// end state and applies the (A, B) in between in order.  The result is the same
// whichever it finds, since the end state of a tile is always fma(A, state
// before, B).  A published word is its own flag: the arrays start as all ones, a
// NaN that no arithmetic gives, so neither side needs a fence (flags beside the
// data, with their fences, took 1.5 us a tile in series: 786 us at 65536 x 2048).
// Tiles are numbered in time order and taken by an atomic ticket, so a tile only
// waits for tiles that running blocks hold, each block working its own in
// ascending order: the lowest unfinished one can always go on.
//
// Measured on the GPU (the copy bandwidth is 6.79 TB/s), decay form: fp32, 4 x 8192 x
// 1024, forward 68 us (6.0 TB/s), backward 106 us (6.3 TB/s); bf16, the same rows, 40 us
// and 68 us (5.0 and 4.9 TB/s); bf16, 65536 x 2048, 142 us and 243 us (5.7 and 5.5 TB/s).
// Logit form, bf16: 51 and 78 us, 177 and 285 us; fp32 69 and 107 us.
// What is lost is the chain's wait: without it the same kernels take 63, 103, 34, 59,
// 121 and 205 us, and in the logit form 42, 70, 140 and 244 us.  A word takes 1.3 us from one SM to another, more while the memory is busy,
// and a tile waits for the slowest of those before it.  It is worst with few channel
// blocks (B C / 64 below the number of SMs), where many tiles of one chain are under
// way.  Blocks of a cluster reading each other's (A, B) in shared memory did not help
// (172 us, and 81 us for the fp32 rows, against 169 us and 68 us at that stage), nor
// did more or fewer blocks, or copying the next tile under the wait.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "la_common.cuh"
#include "la_launch.h"
#include "la_plan.h"
#include "tc_common.cuh"

namespace la {
namespace scan {

constexpr int NT = 128;                 // threads
constexpr int R = 8;                    // rows of a thread
constexpr int LANES = 8;                // threads across a row: 128 bytes
constexpr int RG = NT / LANES;          // row groups of a tile
constexpr int TILE = RG * R;            // rows of a tile
// Blocks per SM, by shared memory (42 KB forward, 63 KB backward a block) and registers.
// A block waits for its copy, then for the chain: more blocks with one stage each beat
// fewer with two (51 us against 58 us forward at 4 x 8192 x 1024 bf16).
template <typename T, bool kLogit>
constexpr int forward_blocks() { return sizeof(T) == 2 && kLogit ? 4 : 5; }
template <typename T>
constexpr int backward_blocks() { return sizeof(T) == 2 ? 3 : 4; }
static_assert(TILE == plan::kScanTile, "checkpoints lie at tile borders");

template <typename T>
struct Geo {
    static constexpr int VEC = 16 / static_cast<int>(sizeof(T));  // channels of a thread
    static constexpr int CB = LANES * VEC;                        // channels of a tile
};

constexpr int kBegin = 1 << 30, kEnd = 1 << 29, kOwner = kEnd - 1;  // packed row info; kOwner: no sequence

template <typename T>
struct Args {
    const T *A, *X, *G;
    T *O, *dA, *dX;
    int B, N, C, tiles, ncb;
    unsigned total;             // B * tiles * ncb
    const int* starts;          // packed sequences
    int S;
    int fill;                   // outputs that get 0 in rows of no sequence: bit 0 O or dA, bit 1 dX
    const float* init;          // forward: h_init; backward: dh_final (state entering the chain)
    float* fin;                 // forward: h_final; backward: dh_init
    const float* h_init;        // backward: the forward's h_init
    const float* states;        // backward: the forward's end state of each tile, [B][tiles][C]
    float *incl, *aggA, *aggB;  // chain of this direction: end states and (A, B), [B][tiles][C]
    unsigned* ticket;           // tiles taken - 1; null: one tile a chain, blocks take tiles by number
    unsigned withhold;          // test hook: a tile (in the chain's order) that publishes nothing (-1: none)
    unsigned spin_limit;        // polls of a look-back before it gives up
    unsigned* status;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {  // the rest of the 16 is 0
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// A thread's 16 bytes as fp32 values, and back (round to nearest even).
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
}

// Arithmetic on a thread's channels, two to an instruction (each rounded as by itself):
// d = a b, d = a b + c, d = a + k.
__device__ __forceinline__ uint64_t two(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void both(uint64_t x, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
template <int V>
__device__ __forceinline__ void mul(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
        uint64_t r;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(two(a[v], a[v + 1])), "l"(two(b[v], b[v + 1])));
        both(r, d[v], d[v + 1]);
    }
}
template <int V>
__device__ __forceinline__ void fma(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
        uint64_t r;
        asm("fma.rn.f32x2 %0, %1, %2, %3;"
            : "=l"(r)
            : "l"(two(a[v], a[v + 1])), "l"(two(b[v], b[v + 1])), "l"(two(c[v], c[v + 1])));
        both(r, d[v], d[v + 1]);
    }
}
template <int V>
__device__ __forceinline__ void add(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
#pragma unroll
    for (int v = 0; v < V; v += 2) {
        uint64_t r;
        asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(two(a[v], a[v + 1])), "l"(two(b[v], b[v + 1])));
        both(r, d[v], d[v + 1]);
    }
}
template <int V>
__device__ __forceinline__ void fill(float (&d)[V], float x) {
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = x;
}
// The logit form's gate as one value v without cancellation: with e = 2^(-z log2 e),
// s = 1 / (1 + e) and 1 - s = e s, v is s where s < 1/2 and -(1 - s) elsewhere (sign bit
// set, -0 where s is 1): the smaller of the two keeps all its bits (1.f - s has lost them
// from z = 17 up), the larger is one less the smaller.  Relative error of the smaller up
// to (|z| + 6) 2^-23: two roundings of the exponent, the approximate power (2^-22.5) and
// reciprocal (2^-23), two roundings.  An overflow of the power gives s = 0.
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
template <int V>
__device__ __forceinline__ void gate(float (&v)[V], const float (&z)[V]) {
    float k[V], e[V];
    fill(k, -1.4426950408889634f);
    mul(e, z, k);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = tcf::ex2_approx(e[i]);
    fill(k, 1.f);
    add(k, e, k);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float s = rcp_approx(k[i]);
        v[i] = e[i] < 1.f ? -e[i] * s : s;
    }
}
__device__ __forceinline__ bool mostly_open(float v) { return __float_as_int(v) < 0; }  // s >= 1/2

// A row's effect on the state: d h + x; in the logit form h - (1 - s)(h - x) or
// x + s (h - x), whichever has the smaller factor.
// With the factors s and 1.f - s instead the passes take 7% less (4 x 8192 x 1024 bf16: 51
// and 77 us against 55 and 83 us), but lose the input of channels with a long memory and
// their gradients.
template <bool kLogit, int V>
__device__ __forceinline__ void step(float (&h)[V], const float (&d)[V], const float (&x)[V]) {
    if constexpr (kLogit) {
        float u[V], k[V];
        fill(k, -1.f);
        fma(u, x, k, h);
#pragma unroll
        for (int v = 0; v < V; ++v) k[v] = mostly_open(d[v]) ? h[v] : x[v];
        fma(h, d, u, k);
    } else {
        fma(h, d, h, x);
    }
}
// A = d A, the decay's product: A - (1 - s) A or s A.
template <bool kLogit, int V>
__device__ __forceinline__ void shrink(float (&A)[V], const float (&d)[V]) {
    if constexpr (kLogit) {
        float k[V];
#pragma unroll
        for (int v = 0; v < V; ++v) k[v] = mostly_open(d[v]) ? A[v] : 0.f;
        fma(A, d, A, k);
    } else {
        mul(A, A, d);
    }
}

// A row's decays: v in the logit form, else the gate a itself.
template <bool kLogit, int V>
__device__ __forceinline__ const float (&decay_of(const float (&s)[V], const float (&a)[V]))[V] {
    if constexpr (kLogit) return s;
    else return a;
}

// A tile's place: batch row, time tile, channel block.
struct Place {
    int b, k, cb;
};

template <typename T, bool kRev>
__device__ __forceinline__ Place place_of(const Args<T>& p, unsigned tile) {
    const unsigned per = static_cast<unsigned>(p.B) * p.ncb;
    const unsigned k = tile / per, rem = tile - k * per;
    Place q;
    q.b = static_cast<int>(rem / p.ncb);
    q.cb = static_cast<int>(rem - q.b * p.ncb);
    q.k = kRev ? p.tiles - 1 - static_cast<int>(k) : static_cast<int>(k);
    return q;
}

// Tensor maps of the streams (A, X, dOut) and outputs (Out; dA, dX) for rows that are
// 16-byte aligned.
struct Maps {
    CUtensorMap m[3], o[2];
};

// A thread's 16 bytes of row r of its row group in stream s of a stage.
template <int s>
__device__ __forceinline__ uint4& piece(uint4* stage, int r) {
    return stage[s * TILE * LANES + (static_cast<int>(threadIdx.x) / LANES * R + r) * LANES + threadIdx.x % LANES];
}

// Rows that are not 16-byte aligned: the aligned 16-byte chunks that cover a row's 128
// bytes, up to 9, lie in 36 words, 8 words apart more from row group to row group, so
// that the 4 rows that a warp reads at once are in different banks.
constexpr int kLoosePitch = 36, kLooseGroup = R * kLoosePitch + 8, kLooseWords = RG * kLooseGroup;

template <bool kVec>
constexpr int stream_bytes() { return kVec ? TILE * LANES * 16 : kLooseWords * 4; }

// Copies a tile's streams into a stage.  kVec: by TMA, a box of 128 rows x 128 bytes
// a stream, which thread 0 asks for when all threads are done with the stage (values
// past N and C come as 0).  Otherwise the 8 lanes of a row copy its chunks (cp.async,
// cut at the end of the tensor; channel by channel the backward took 40 us against
// 30 us at 5003 x 1001 fp32).
template <typename T, bool kVec, int STREAMS>
__device__ __forceinline__ void issue(const Args<T>& p, const Maps& maps, const Place& q, uint4* stage,
                                      uint64_t* bar) {
    constexpr int VEC = Geo<T>::VEC, CB = Geo<T>::CB;
    const int tid = threadIdx.x, lane = tid % LANES, rg = tid / LANES;
    if constexpr (kVec) {
        if (tid == 0) {
            tc::mbar_arrive_expect_tx(bar, STREAMS * TILE * LANES * 16);
#pragma unroll
            for (int s = STREAMS - 1; s >= 0; --s) {
                if (s == STREAMS - 2) tc::tma_store_wait_read();  // outputs leave from the other slots
                tc::tma_load_3d(stage + s * TILE * LANES, &maps.m[s], bar, q.cb * CB, q.k * TILE, q.b);
            }
        }
    } else {
        const T* src[3] = {p.A, p.X, p.G};
        const int64_t total = static_cast<int64_t>(p.B) * p.N * p.C;
        const int width = min(CB, p.C - q.cb * CB);
        const uint32_t dst = tc::smem_u32(stage) + 4 * (rg * kLooseGroup) + 16 * lane;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = q.k * TILE + rg * R + r;
            const int64_t e0 = (static_cast<int64_t>(q.b) * p.N + t) * p.C + q.cb * CB;
            const int off = static_cast<int>(e0 & (VEC - 1)), used = t < p.N ? off + width : 0;
            const int64_t from = e0 - off + lane * VEC;
            const auto bytes = [&](int first) {  // of the chunk of elements first .. first + VEC - 1 of the row
                const int64_t left = total - (e0 - off + first);
                return first < used ? static_cast<int>(min(left, static_cast<int64_t>(VEC))) * static_cast<int>(sizeof(T)) : 0;
            };
            const int n = bytes(lane * VEC), n8 = lane == 0 ? bytes(8 * VEC) : 0;
#pragma unroll
            for (int s = 0; s < STREAMS; ++s) {
                const uint32_t to = dst + 4 * (s * kLooseWords + r * kLoosePitch);
                cp16(to, n ? src[s] + from : src[s], n);
                if (n8) cp16(to + 128, src[s] + from + 8 * VEC, n8);
            }
        }
    }
}

// A thread's channels of row r of its row group in stream s.
template <typename T, bool kVec, int s>
__device__ __forceinline__ void fetch(const Args<T>& p, const Place& q, uint4* stage, int r, float (&x)[Geo<T>::VEC]) {
    constexpr int VEC = Geo<T>::VEC;
    if constexpr (kVec) {
        unpack(piece<s>(stage, r), x);
    } else {
        const int lane = threadIdx.x % LANES, rg = threadIdx.x / LANES;
        const unsigned row = static_cast<unsigned>(q.b) * p.N + q.k * TILE + rg * R + r;
        const T* from = reinterpret_cast<const T*>(reinterpret_cast<const uint32_t*>(stage) + s * kLooseWords +
                                                   rg * kLooseGroup + r * kLoosePitch) +
                        (row * static_cast<unsigned>(p.C) & (VEC - 1)) + lane;
#pragma unroll
        for (int v = 0; v < VEC; ++v) x[v] = to_f(from[LANES * v]);
    }
}
template <typename T, bool kVec>
__device__ __forceinline__ void landed(const Args<T>& p, uint64_t* bar, uint32_t phase) {
    if constexpr (kVec) {
        if (!tc::mbar_wait(bar, phase, tcf::kWaitLimit)) atomicOr(p.status, tcf::kErrWait);
    } else {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();  // the lanes of a row read each other's chunks
    }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_row(T* dst, const Args<T>& p, const Place& q, int t,
                                          const float (&y)[Geo<T>::VEC]) {
    constexpr int VEC = Geo<T>::VEC, CB = Geo<T>::CB;
    const int lane = threadIdx.x % LANES;
    const int64_t row = (static_cast<int64_t>(q.b) * p.N + t) * p.C;
    if constexpr (kVec) {
        const int c = q.cb * CB + lane * VEC;
        if (c < p.C) *reinterpret_cast<uint4*>(dst + row + c) = pack(y);
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const int c = q.cb * CB + lane + LANES * v;
            if (c < p.C) dst[row + c] = from_f<T>(y[v]);
        }
    }
}

// A thread's channels of a [..][C] fp32 row (0 past C, or without a row).
template <typename T, bool kVec>
__device__ __forceinline__ void load_state(const float* row, const Args<T>& p, const Place& q,
                                           float (&y)[Geo<T>::VEC]) {
    const int lane = threadIdx.x % LANES;
#pragma unroll
    for (int v = 0; v < Geo<T>::VEC; ++v) {
        const int c = q.cb * Geo<T>::CB + (kVec ? lane * Geo<T>::VEC + v : lane + LANES * v);
        y[v] = row && c < p.C ? row[c] : 0.f;
    }
}
template <typename T, bool kVec>
__device__ __forceinline__ void add_state(const float* row, const Args<T>& p, const Place& q,
                                          float (&y)[Geo<T>::VEC]) {
    const int lane = threadIdx.x % LANES;
#pragma unroll
    for (int v = 0; v < Geo<T>::VEC; ++v) {
        const int c = q.cb * Geo<T>::CB + (kVec ? lane * Geo<T>::VEC + v : lane + LANES * v);
        if (c < p.C) y[v] += row[c];
    }
}
template <typename T, bool kVec>
__device__ __forceinline__ void save_state(float* row, const Args<T>& p, const Place& q,
                                           const float (&y)[Geo<T>::VEC]) {
    const int lane = threadIdx.x % LANES;
#pragma unroll
    for (int v = 0; v < Geo<T>::VEC; ++v) {
        const int c = q.cb * Geo<T>::CB + (kVec ? lane * Geo<T>::VEC + v : lane + LANES * v);
        if (c < p.C) row[c] = y[v];
    }
}

// Shared rows [RG][CB] of per-channel values.
template <typename T, bool kVec>
__device__ __forceinline__ void put(float* sm, const float (&y)[Geo<T>::VEC]) {
    constexpr int VEC = Geo<T>::VEC, CB = Geo<T>::CB;
    float* row = sm + (threadIdx.x / LANES) * CB;
    const int lane = threadIdx.x % LANES;
    if constexpr (kVec) {
#pragma unroll
        for (int v = 0; v < VEC; v += 4)
            *reinterpret_cast<float4*>(row + lane * VEC + v) = make_float4(y[v], y[v + 1], y[v + 2], y[v + 3]);
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) row[lane + LANES * v] = y[v];
    }
}
template <typename T, bool kVec>
__device__ __forceinline__ void get(const float* sm, float (&y)[Geo<T>::VEC]) {
    constexpr int VEC = Geo<T>::VEC, CB = Geo<T>::CB;
    const float* row = sm + (threadIdx.x / LANES) * CB;
    const int lane = threadIdx.x % LANES;
    if constexpr (kVec) {
#pragma unroll
        for (int v = 0; v < VEC; v += 4) {
            const float4 f = *reinterpret_cast<const float4*>(row + lane * VEC + v);
            y[v] = f.x, y[v + 1] = f.y, y[v + 2] = f.z, y[v + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) y[v] = row[lane + LANES * v];
    }
}

// Packed sequences: info[row] = owner | kBegin | kEnd of a tile's rows, and each
// row group's "a row begins" / "a row ends" bits.  An owner outside 0 .. S-1
// becomes kOwner (a row of no sequence, which begins and ends itself).
template <typename T>
__device__ __forceinline__ void row_info(const Args<T>& p, int k, int* info, unsigned* grp) {
    constexpr int LR = TILE / 32, PER = R / LR;  // rows of a lane, lanes of a row group
    static_assert(TILE == 32 * LR && R == LR * PER && (PER == 1 || PER == 2), "lanes over rows");
    const int tid = threadIdx.x, row0 = k * TILE;
    for (int i = tid; i <= TILE; i += NT) info[i] = -1;
    // f0, the first boundary i in 0 .. S with starts[i] >= row0 (S + 1 if none): 32
    // probes a round trip, every warp for itself
    int f0 = 0, f1 = p.S + 1;
    while (f1 - f0 > 0) {
        const int step = (f1 - f0 + 31) / 32, i = f0 + (tid & 31) * step;
        const bool before = i < f1 && min(max(p.starts[i], 0), p.N) < row0;
        const int n = __popc(__ballot_sync(0xffffffffu, before));  // probes before the tile
        f1 = n < 32 ? min(f1, f0 + n * step) : f1;
        f0 = n ? f0 + (n - 1) * step + 1 : f0;
        if (n == 0) break;
    }
    __syncthreads();
    for (int i = f0 + tid; i <= p.S; i += NT) {
        const int r = min(max(p.starts[i], 0), p.N) - row0;
        if (r > TILE) break;
        if (r >= 0) atomicMax(&info[r], i);  // of equal boundaries the last: the sequence with rows
    }
    __syncthreads();
    if (tid < 32) {  // owners: running maximum over the rows
        int m[LR + 1], run = f0 - 1, top = -1;
#pragma unroll
        for (int r = 0; r < LR; ++r) m[r] = info[tid * LR + r];
        // the row behind the lane's own, from its lane: that word of info is written below
        m[LR] = __shfl_down_sync(0xffffffffu, m[0], 1);
        if (tid == 31) m[LR] = info[TILE];
#pragma unroll
        for (int r = 0; r < LR; ++r) top = max(top, m[r]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, top, o);
            if (tid >= o) top = max(top, up);
        }
        const int up = __shfl_up_sync(0xffffffffu, top, 1);
        if (tid) run = max(run, up);
        unsigned g = 0;
#pragma unroll
        for (int r = 0; r < LR; ++r) {
            const int t = row0 + tid * LR + r;
            run = max(run, m[r]);
            const bool none = run < 0 || run >= p.S || t >= p.N;
            const bool b = none || m[r] >= 0, e = none || m[r + 1] >= 0 || t + 1 >= p.N;
            info[tid * LR + r] = (none ? kOwner : run) | (b ? kBegin : 0) | (e ? kEnd : 0);
            g |= (b ? 1u : 0u) | (e ? 2u : 0u);
        }
        if (PER == 2) g |= __shfl_xor_sync(0xffffffffu, g, 1);
        if (tid % PER == 0) grp[tid / PER] = g;
    }
    __syncthreads();
}

constexpr unsigned kUnset = 0xFFFFFFFFu;  // a word that nothing has been published in
// Tiles looked back over at once.  The smaller suits chains of which up to kDeep tiles
// are under way (65536 x 2048 bf16: forward 142 us with 4, 146 us with 8, 159 us with
// 16: each more costs two words a tile and registers), the larger those of few channels,
// whose many tiles advance by a window a round trip (65536 x 256: 44 us against 94 us).
constexpr int kNear = 4, kFar = 16, kDeep = 48;

__device__ __forceinline__ unsigned ld_relaxed(const float* p) {
    unsigned v;
    asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_relaxed(float* p, float x) {
    unsigned v = __float_as_uint(x);
    if (v == kUnset) v = 0x7FFFFFFFu;  // a NaN that came in with the caller's state
    asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// What a channel knows of the tiles before its chain tile i: the (A, B) of up to
// kWindow of them, nearest first.  Fetched when the tile begins, under its copy.
template <int kWindow>
struct Window {
    unsigned a[kWindow], b[kWindow], near;  // near: the end state of the tile before
};
template <typename T, int kWindow>
__device__ __forceinline__ void peek(Window<kWindow>& w, const Args<T>& p, int i, int64_t at, int64_t step, bool on) {
#pragma unroll
    for (int d = 0; d < kWindow; ++d) {
        const bool in = on && d < i - 1;
        w.a[d] = in ? ld_relaxed(p.aggA + at + (i - 1 - d) * step) : kUnset;
        w.b[d] = in ? ld_relaxed(p.aggB + at + (i - 1 - d) * step) : kUnset;
    }
    w.near = on && i > 0 ? ld_relaxed(p.incl + at + (i - 1) * step) : kUnset;
}

// The state that enters chain tile i > 0 (numbered in the chain's direction) of
// a channel; `at` is the channel's place in tile 0, tiles are `step` words apart.
// Publishes the tile's own (A, B) first if the tile before is not done (quiet: its
// end state is out).  The (A, B) that are out without a gap, nearest first, lead to
// the end state before them, the first to come; each round trip reads that one, the
// nearest end state and what is still missing (all words of the window every time
// slowed the copies down: 210 us against 268 us at 65536 x 2048).
template <typename T, int kWindow>
__device__ float look_back(const Args<T>& p, Window<kWindow>& w, int i, int64_t at, int64_t step, float At, float Bt,
                           bool quiet) {
    if (w.near != kUnset) return __uint_as_float(w.near);
    if (!quiet) {
        st_relaxed(p.aggA + at + i * step, At);
        st_relaxed(p.aggB + at + i * step, Bt);
    }
    for (unsigned spin = 0; spin < p.spin_limit; ++spin) {
        int n = 0;
#pragma unroll
        for (int d = 0; d < kWindow; ++d)
            if (n == d && w.a[d] != kUnset && w.b[d] != kUnset) n = d + 1;
        const unsigned far = ld_relaxed(p.incl + at + (i - 1 - n) * step);
        const unsigned near = n ? ld_relaxed(p.incl + at + (i - 1) * step) : kUnset;
        float h = __uint_as_float(far);
        if (far == kUnset && near == kUnset) {
#pragma unroll
            for (int d = 0; d < kWindow; ++d) {
                if (d < i - 1 && (w.a[d] == kUnset || w.b[d] == kUnset)) {
                    w.a[d] = ld_relaxed(p.aggA + at + (i - 1 - d) * step);
                    w.b[d] = ld_relaxed(p.aggB + at + (i - 1 - d) * step);
                }
            }
            if (spin > 256) __nanosleep(100);
            continue;
        }
        if (near != kUnset) return __uint_as_float(near);
#pragma unroll
        for (int d = kWindow - 1; d >= 0; --d)
            if (d < n) h = fmaf(__uint_as_float(w.a[d]), h, __uint_as_float(w.b[d]));
        return h;
    }
    atomicOr(p.status, tcf::kErrLookback);  // the tiles before never came: report it and go on
    return 0.f;
}

template <typename T, bool kPacked, bool kVec, int STREAMS>
constexpr size_t smem_bytes() {
    return static_cast<size_t>(STREAMS) * stream_bytes<kVec>() + sizeof(float) * STREAMS * RG * Geo<T>::CB +
           (kPacked ? sizeof(int) * (TILE + 4 + RG) : 0) + 16;
}

// Scratch of one pass: ticket, A, B, end states (unless they go to the caller's
// checkpoints), all unset at first.
struct Parts {
    size_t states, bytes;
};
inline Parts parts_of(int B, int N, int C, bool own_incl) {
    const size_t tiles = (static_cast<size_t>(N) + TILE - 1) / TILE;
    Parts s = {};
    s.states = tiles > 1 ? static_cast<size_t>(B) * tiles * C : 0;
    s.bytes = s.states ? 4 * (4 + (own_incl ? 3 : 2) * s.states) : 0;
    return s;
}

// Unsets na words at a and nb words at b (16-byte aligned) by one kernel, which a pass
// launched behind it may overlap until its griddepcontrol.wait.
cudaError_t unset_words(const LaunchCtx& c, unsigned* a, size_t na, unsigned* b, size_t nb);

// One pass along the rows (forward, or the backward's carry); defined in
// gated_scan_impl.cuh, compiled in a file of its own for each type and direction.
// `own_incl`: the pass keeps its chain's end states in scratch.
template <typename T, bool kBwd>
cudaError_t launch(const LaunchCtx& c, Args<T> a, bool logit, bool own_incl);

// States of empty packed sequences (to = from, or 0), over all warps of the grid.
template <typename T>
__device__ __forceinline__ void empty_sequences(const Args<T>& p, const float* from, float* to) {
    if (!to) return;
    const int lane = threadIdx.x & 31, all = gridDim.x * (NT / 32);
    for (int i = blockIdx.x * (NT / 32) + threadIdx.x / 32; i < p.S; i += all) {
        const int a = min(max(p.starts[i], 0), p.N), b = min(max(p.starts[i + 1], 0), p.N);
        if (a < b) continue;
        const int64_t row = static_cast<int64_t>(i) * p.C;
        for (int c = lane; c < p.C; c += 32) to[row + c] = from ? from[row + c] : 0.f;
    }
}

// Zeros to the rows before the first packed sequence and behind the last one, over all
// threads of the grid: two runs of memory.
template <typename T>
__device__ __forceinline__ void clear_padding(const Args<T>& p, T* out, bool on) {
    if (!on) return;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * NT + threadIdx.x, all = static_cast<int64_t>(gridDim.x) * NT;
    const int a = min(max(p.starts[0], 0), p.N), b = max(min(max(p.starts[p.S], 0), p.N), a);
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        constexpr int VEC = Geo<T>::VEC;
        const int64_t from = static_cast<int64_t>(i ? b : 0) * p.C, to = static_cast<int64_t>(i ? p.N : a) * p.C;
        const int64_t v0 = (from + VEC - 1) / VEC, v1 = to / VEC;  // whole 16-byte pieces
        for (int64_t v = v0 + id; v < v1; v += all) reinterpret_cast<uint4*>(out)[v] = make_uint4(0, 0, 0, 0);
        if (id < VEC) {
            const int64_t head = from + id, tail = v1 * VEC + id;
            if (head < min(v0 * VEC, to)) out[head] = from_f<T>(0.f);
            if (tail >= from && tail < to) out[tail] = from_f<T>(0.f);
        }
    }
}

// One channel's fold over the row groups: the tile's (A, B), and whether a row
// group replaces the state (its "begin" bit, or for the backward pass "end").
template <int CB, bool kPacked, bool kRev>
__device__ __forceinline__ bool fold(const float* a, const float* b, const unsigned* grp, float& At,
                                     float& Bt) {
    At = 1.f, Bt = 0.f;
    bool cut = false;
#pragma unroll 8
    for (int g0 = 0; g0 < RG; ++g0) {
        const int g = kRev ? RG - 1 - g0 : g0;
        const float A = a[g * CB], B = b[g * CB];
        const bool x = kPacked && (grp[g] & (kRev ? 2u : 1u));
        Bt = x ? B : fmaf(A, Bt, B);
        At *= A;
        cut |= x;
    }
    return cut;
}

template <typename T, bool kLogit, bool kPacked, bool kVec, int kWindow>
__global__ void __launch_bounds__(NT, forward_blocks<T, kLogit>())
scan_forward_kernel(const Args<T> p, const __grid_constant__ Maps maps) {
    constexpr int VEC = Geo<T>::VEC, CB = Geo<T>::CB;
    extern __shared__ __align__(128) uint8_t sm[];
    uint4* stage = reinterpret_cast<uint4*>(sm);
    float* sa = reinterpret_cast<float*>(sm + 2 * stream_bytes<kVec>());
    float* sb = sa + RG * CB;
    int* info = reinterpret_cast<int*>(sb + RG * CB);
    unsigned* grp = reinterpret_cast<unsigned*>(info + (kPacked ? TILE + 4 : 0));
    unsigned* snext = grp + (kPacked ? RG : 0);
    const int tid = threadIdx.x, rg = tid / LANES;

    __shared__ uint64_t bar;
    uint32_t phase = 0;
    if (kVec && tid == 0) {
        tc::mbar_init(&bar, 1);
        tc::fence_mbar_init();
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the chain's words are unset
    unsigned tile = blockIdx.x;
    if (p.ticket) {
        if (tid == 0) *snext = atomicAdd(p.ticket, 1u) + 1u;
        __syncthreads();
        tile = *snext;
        __syncthreads();
    }
    if constexpr (kPacked) {
        empty_sequences(p, p.init, p.fin);
        clear_padding(p, p.O, p.fill & 1);
    }
    if (tile < p.total) issue<T, kVec, 2>(p, maps, place_of<T, false>(p, tile), stage, &bar);
    while (tile < p.total) {
        const Place q = place_of<T, false>(p, tile);
        if constexpr (kPacked) row_info<T>(p, q.k, info, grp);
        const int t0 = q.k * TILE + rg * R, c = q.cb * CB + tid;
        const bool on = tid < CB && c < p.C;  // this thread has a channel of the chain
        const int64_t at = static_cast<int64_t>(q.b) * p.tiles * p.C + c;
        Window<kWindow> win;
        peek<T, kWindow>(win, p, q.k, at, p.C, on);
        landed<T, kVec>(p, &bar, phase);
        phase ^= 1u;
        // The thread's rows as one map (A, B); rows past N change nothing.
        float s[kLogit ? R : 1][VEC];
        float A[VEC], Bv[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) A[v] = 1.f, Bv[v] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float a[VEC], x[VEC];
            fetch<T, kVec, 0>(p, q, stage, r, a);
            fetch<T, kVec, 1>(p, q, stage, r, x);
            if constexpr (kLogit) gate(s[r], a);
            const float(&d)[VEC] = decay_of<kLogit>(s[kLogit ? r : 0], a);
            if (t0 + r < p.N) {
                if constexpr (kPacked) {
                    const int w = info[rg * R + r], o = w & kOwner;
                    if (w & kBegin)
                        load_state<T, kVec>(p.init && o != kOwner ? p.init + static_cast<int64_t>(o) * p.C : nullptr,
                                            p, q, Bv);
                }
                shrink<kLogit>(A, d);
                step<kLogit>(Bv, d, x);
            }
        }
        put<T, kVec>(sa, A);
        put<T, kVec>(sb, Bv);
        __syncthreads();
        unsigned mine = 0;
        if (on) {
            const bool last = q.k + 1 == p.tiles;
            float At, Bt, h = 0.f;
            const bool cut = fold<CB, kPacked, false>(sa + tid, sb + tid, grp, At, Bt), mute = tile == p.withhold;
            float* out = p.incl + at + static_cast<int64_t>(q.k) * p.C;
            if (cut && !last && !mute) st_relaxed(out, Bt);
            if (q.k) h = look_back<T, kWindow>(p, win, q.k, at, p.C, At, Bt, cut || mute);
            else if (!kPacked && p.init) h = p.init[static_cast<int64_t>(q.b) * p.C + c];
            const float end = cut ? Bt : fmaf(At, h, Bt);
            // The next tile is taken as late as the copy allows: a block that took it
            // earlier would hold up the chain with it.
            if (tid == 0) mine = p.ticket ? atomicAdd(p.ticket, 1u) + 1u : tile + gridDim.x;
            if (!last && !cut && !mute) st_relaxed(out, end);
            if (!kPacked && last && p.fin) p.fin[static_cast<int64_t>(q.b) * p.C + c] = end;
#pragma unroll 8
            for (int g = 0; g < RG; ++g) {
                const float ga = sa[g * CB + tid], gb = sb[g * CB + tid];
                sa[g * CB + tid] = h;
                h = kPacked && (grp[g] & 1u) ? gb : fmaf(ga, h, gb);
            }
        }
        __syncthreads();
        if (p.O || (kPacked && p.fin)) {
            float h[VEC];
            get<T, kVec>(sa, h);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (t0 + r >= p.N) break;
                float a[VEC], x[VEC];
                fetch<T, kVec, 0>(p, q, stage, r, a);
                fetch<T, kVec, 1>(p, q, stage, r, x);
                const int w = kPacked ? info[rg * R + r] : 0, o = w & kOwner;
                if (kPacked && (w & kBegin))
                    load_state<T, kVec>(p.init && o != kOwner ? p.init + static_cast<int64_t>(o) * p.C : nullptr, p,
                                        q, h);
                step<kLogit>(h, decay_of<kLogit>(s[kLogit ? r : 0], a), x);
                if (kVec && !kPacked) piece<0>(stage, r) = pack(h);
                else if (p.O && (!kPacked || o != kOwner)) store_row<T, kVec>(p.O, p, q, t0 + r, h);
                if (kPacked && (w & kEnd) && o != kOwner && p.fin)
                    save_state<T, kVec>(p.fin + static_cast<int64_t>(o) * p.C, p, q, h);
            }
        }
        if (kVec && !kPacked && p.O) tc::fence_proxy_async();
        if (tid == 0) *snext = mine;
        __syncthreads();  // every thread is done with the stage and info
        const unsigned next = *snext;
        if (kVec && !kPacked && p.O && tid == 0) {
            tc::tma_store_3d(&maps.o[0], stage, q.cb * CB, q.k * TILE, q.b);
            tc::tma_store_commit();
        }
        if (next < p.total) issue<T, kVec, 2>(p, maps, place_of<T, false>(p, next), stage, &bar);
        tile = next;
    }
    if (kVec && !kPacked && tid == 0) tc::tma_store_wait_read();  // the block's memory outlives its outputs
}

// Backward: the forward state enters each tile from its checkpoint (no chain);
// the carry c comes down the chain from the last tile.
template <typename T, bool kLogit, bool kPacked, bool kVec, int kWindow>
__global__ void __launch_bounds__(NT, backward_blocks<T>())
scan_backward_kernel(const Args<T> p, const __grid_constant__ Maps maps) {
    constexpr int VEC = Geo<T>::VEC, CB = Geo<T>::CB;
    extern __shared__ __align__(128) uint8_t sm[];
    uint4* stage = reinterpret_cast<uint4*>(sm);
    float* sa = reinterpret_cast<float*>(sm + 3 * stream_bytes<kVec>());
    float* sb = sa + RG * CB;
    float* sc = sb + RG * CB;
    int* info = reinterpret_cast<int*>(sc + RG * CB);
    unsigned* grp = reinterpret_cast<unsigned*>(info + (kPacked ? TILE + 4 : 0));
    unsigned* snext = grp + (kPacked ? RG : 0);
    const int tid = threadIdx.x, rg = tid / LANES;

    __shared__ uint64_t bar;
    uint32_t phase = 0;
    if (kVec && tid == 0) {
        tc::mbar_init(&bar, 1);
        tc::fence_mbar_init();
    }
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the chain's words are unset
    unsigned tile = blockIdx.x;
    if (p.ticket) {
        if (tid == 0) *snext = atomicAdd(p.ticket, 1u) + 1u;
        __syncthreads();
        tile = *snext;
        __syncthreads();
    }
    if constexpr (kPacked) {
        empty_sequences(p, p.init, p.fin);
        clear_padding(p, p.dA, p.fill & 1);
        clear_padding(p, p.dX, p.fill & 2);
    }
    if (tile < p.total) issue<T, kVec, 3>(p, maps, place_of<T, true>(p, tile), stage, &bar);
    while (tile < p.total) {
        const Place q = place_of<T, true>(p, tile);
        if constexpr (kPacked) row_info<T>(p, q.k, info, grp);
        const int t0 = q.k * TILE + rg * R, c = q.cb * CB + tid, i = p.tiles - 1 - q.k;
        const bool on = tid < CB && c < p.C;  // this thread has a channel of the chain
        const int64_t at = static_cast<int64_t>(q.b) * p.tiles * p.C + c;
        Window<kWindow> win;
        peek<T, kWindow>(win, p, i, at, p.C, on);
        float h0 = 0.f;  // the state that enters the tile
        if (on && q.k) h0 = p.states[at + static_cast<int64_t>(q.k - 1) * p.C];
        else if (on && !kPacked && p.h_init) h0 = p.h_init[static_cast<int64_t>(q.b) * p.C + c];
        landed<T, kVec>(p, &bar, phase);
        phase ^= 1u;
        float s[kLogit ? R : 1][VEC];
        float A[VEC], Bf[VEC], Br[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) A[v] = 1.f, Bf[v] = 0.f, Br[v] = 0.f;
        // forward over the rows: A, the state's Bf, and the carry's
        // Br = sum_i (s_0 .. s_i) dOut_i, up to the first row that ends a sequence
        bool live = true;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float a[VEC], x[VEC], g[VEC];
            fetch<T, kVec, 0>(p, q, stage, r, a);
            fetch<T, kVec, 1>(p, q, stage, r, x);
            fetch<T, kVec, 2>(p, q, stage, r, g);
            if constexpr (kLogit) gate(s[r], a);
            const float(&d)[VEC] = decay_of<kLogit>(s[kLogit ? r : 0], a);
            if (t0 + r < p.N) {
                const int w = kPacked ? info[rg * R + r] : 0, o = w & kOwner;
                if (kPacked && (w & kBegin))
                    load_state<T, kVec>(p.h_init && o != kOwner ? p.h_init + static_cast<int64_t>(o) * p.C : nullptr,
                                        p, q, Bf);
                if (kPacked && (w & kEnd) && p.init && o != kOwner)
                    add_state<T, kVec>(p.init + static_cast<int64_t>(o) * p.C, p, q, g);
                shrink<kLogit>(A, d);
                step<kLogit>(Bf, d, x);
                if (live) fma(Br, A, g, Br);
                if (kPacked && (w & kEnd)) live = false;
            }
        }
        put<T, kVec>(sa, A);
        put<T, kVec>(sb, Bf);
        put<T, kVec>(sc, Br);
        __syncthreads();
        unsigned mine = 0;
        if (on) {
            const bool last = q.k == 0;
            float At, Bt, y = 0.f, h = h0;
            const bool cut = fold<CB, kPacked, true>(sa + tid, sc + tid, grp, At, Bt), mute = tile == p.withhold;
            float* out = p.incl + at + static_cast<int64_t>(i) * p.C;
            if (cut && !last && !mute) st_relaxed(out, Bt);
            if (i) y = look_back<T, kWindow>(p, win, i, at, p.C, At, Bt, cut || mute);
            else if (!kPacked && p.init) y = p.init[static_cast<int64_t>(q.b) * p.C + c];
            const float end = cut ? Bt : fmaf(At, y, Bt);
            if (tid == 0) mine = p.ticket ? atomicAdd(p.ticket, 1u) + 1u : tile + gridDim.x;
            if (!last && !cut && !mute) st_relaxed(out, end);
            if (!kPacked && last && p.fin) p.fin[static_cast<int64_t>(q.b) * p.C + c] = end;
            // the carry entering each row group replaces its Br, from the last group down
#pragma unroll 8
            for (int g = RG - 1; g >= 0; --g) {
                const float ga = sa[g * CB + tid], gb = sc[g * CB + tid];
                sc[g * CB + tid] = y;
                y = kPacked && (grp[g] & 2u) ? gb : fmaf(ga, y, gb);
            }
#pragma unroll 8
            for (int g = 0; g < RG; ++g) {
                const float ga = sa[g * CB + tid], gb = sb[g * CB + tid];
                sa[g * CB + tid] = h;
                h = kPacked && (grp[g] & 1u) ? gb : fmaf(ga, h, gb);
            }
        }
        __syncthreads();
        // The rows' states are kept for H rows at a time, from the last ones up; the rows
        // before them are run through again.
        constexpr int H = kPacked && sizeof(T) == 2 ? R / 2 : R;
        float y[VEC];
        get<T, kVec>(sc, y);
#pragma unroll
        for (int r0 = R - H; r0 >= 0; r0 -= H) {
            float hp[H][VEC], h[VEC];
            get<T, kVec>(sa, h);
#pragma unroll
            for (int r = 0; r < r0 + H; ++r) {
                if (kPacked && (info[rg * R + r] & kBegin)) {
                    const int o = info[rg * R + r] & kOwner;
                    load_state<T, kVec>(p.h_init && o != kOwner ? p.h_init + static_cast<int64_t>(o) * p.C : nullptr,
                                        p, q, h);
                }
                if (r >= r0) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) hp[r >= r0 ? r - r0 : 0][v] = h[v];
                }
                if (r + 1 == r0 + H) break;
                float a[VEC], x[VEC];
                fetch<T, kVec, 0>(p, q, stage, r, a);
                fetch<T, kVec, 1>(p, q, stage, r, x);
                step<kLogit>(h, decay_of<kLogit>(s[kLogit ? r : 0], a), x);
            }
#pragma unroll
            for (int r = r0 + H - 1; r >= r0; --r) {
                if (t0 + r < p.N) {
                    float a[VEC], x[VEC], g[VEC];
                    fetch<T, kVec, 0>(p, q, stage, r, a);
                    fetch<T, kVec, 1>(p, q, stage, r, x);
                    fetch<T, kVec, 2>(p, q, stage, r, g);
                    const int w = kPacked ? info[rg * R + r] : 0, o = w & kOwner;
                    if (kPacked && (w & kEnd))
                        load_state<T, kVec>(p.init && o != kOwner ? p.init + static_cast<int64_t>(o) * p.C : nullptr, p,
                                            q, y);
                    const float(&d)[VEC] = decay_of<kLogit>(s[kLogit ? r : 0], a);
                    float da[VEC], dx[VEC];
                    add(dx, g, y);  // the whole gradient at h_t
                    if constexpr (kLogit) {
                        // with w the smaller of s and 1 - s and rest = (1 - w) dx: y and dX are
                        // w dx and rest in one order or the other, s (1 - s) dx is w rest
                        float u[VEC], k[VEC];
                        fill(k, -1.f);
                        fma(u, x, k, hp[r - r0]);
#pragma unroll
                        for (int v = 0; v < VEC; ++v) {
                            const float w = fabsf(d[v]), part = w * dx[v], rest = fmaf(-w, dx[v], dx[v]);
                            da[v] = w * rest * u[v];
                            y[v] = mostly_open(d[v]) ? rest : part;
                            dx[v] = mostly_open(d[v]) ? part : rest;
                        }
                    } else {
                        mul(y, d, dx);
                        mul(da, dx, hp[r - r0]);
                    }
                    if constexpr (kVec && !kPacked) {
                        piece<0>(stage, r) = pack(da);
                        piece<1>(stage, r) = pack(dx);
                    } else if (!kPacked || o != kOwner) {
                        store_row<T, kVec>(p.dA, p, q, t0 + r, da);
                        store_row<T, kVec>(p.dX, p, q, t0 + r, dx);
                    }
                    if (kPacked && (w & kBegin) && o != kOwner && p.fin)
                        save_state<T, kVec>(p.fin + static_cast<int64_t>(o) * p.C, p, q, y);
                }
            }
        }
        if (kVec && !kPacked) tc::fence_proxy_async();
        if (tid == 0) *snext = mine;
        __syncthreads();  // every thread is done with the stage and info
        const unsigned next = *snext;
        if (kVec && !kPacked && tid == 0) {
            tc::tma_store_3d(&maps.o[0], stage, q.cb * CB, q.k * TILE, q.b);
            tc::tma_store_3d(&maps.o[1], stage + TILE * LANES, q.cb * CB, q.k * TILE, q.b);
            tc::tma_store_commit();
        }
        if (next < p.total) issue<T, kVec, 3>(p, maps, place_of<T, true>(p, next), stage, &bar);
        tile = next;
    }
    if (kVec && !kPacked && tid == 0) tc::tma_store_wait_read();  // the block's memory outlives its outputs
}

}  // namespace scan
}  // namespace la
