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
// 32 bits are taken to the nearest quarter turn and a rest of at most an eighth, an fp32
// number with a rounding of 2^-25 of itself: an angle is off by 2.4e-8 at most from the position times the
// stored frequency, whether the position is 1 or 2^31.  (The frequency itself comes from a theta_i in double, so
// that theta_i's angle is off by another p theta_i 2^-53 or so: at most 1.6e-7 at position 2^31 for bases from 10^4
// to 10^6.)  Its sine and cosine are summed from their series.
//
// Bound by memory: a row is read once and written once (with the norm's gradient, two are
// read).  A thread holds one unit of a row: two pieces of 16 bytes whose elements are paired
// with each other (half layout) or each within itself (interleaved); D / (2 VEC) neighbouring lanes hold a
// row and sum up its squares between them.  Neighbouring lanes' pieces are neighbours, so that a warp
// touches whole lines (a lane's two pieces side by side: 27 us instead of 13 for 3001 x 32 x 128 fp32).
// A thread keeps to its token and takes every HS-th
// head of the queries, then of the keys: so a token's sines and cosines are worked out once for
// all of them, lie in registers, and a row costs no index arithmetic.  (With rows dealt
// out one by one, and the sines read from shared memory for each, the same work took twice the
// instructions: 389 us against 196 us for 65536 x (32 + 4) x 128 bf16.)  Products are on pairs of elements
// (fma.rn.f32x2).  As many blocks run as an SM has room for, and every thread keeps a few rows under way:
// cp.async into a ring of its own, which needs no barrier.  65536 x 36 x 128 bf16: 196 us, 6.2 TB/s;
// gradients of 4 x 8192 x 32 x 64 bf16: 70 us, 5.7 TB/s.
//
// Rows that are not 16-byte aligned, or whose rotated part ends inside a piece, take pieces of two elements,
// or single elements where two do not fit either.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "la_common.cuh"
#include "la_launch.h"
#include "la_plan.h"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kTrig = 3;  // a token's sines, in rows

// Sine and cosine of a phase in units of 2^-32 turns.
__device__ __forceinline__ void turn(uint32_t phase, float& s, float& c) {
    const uint32_t quarter = (phase + 0x20000000u) >> 30;                   // nearest
    const int rest = static_cast<int>(phase - (quarter << 30));             // within +- 2^29
    const float x = static_cast<float>(rest) * 4.656612873077393e-10f;      // half turns, within +- 1/4
    // Taylor's series of sin(pi x) and cos(pi x); their next terms are below 2e-9 there.
    const float z = x * x;
    const float a = x * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 0.08214589f, -0.5992645f), 2.550164f), -5.1677128f), 3.1415927f);
    const float b = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -0.025806891f, 0.23533063f), -1.3352628f), 4.058712f), -4.934802f), 1.f);
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
struct Piece<float, 2> { using type = float2; };
template <>
struct Piece<__nv_bfloat16, 2> { using type = uint32_t; };
template <>
struct Piece<float, 1> { using type = float; };
template <>
struct Piece<__nv_bfloat16, 1> { using type = __nv_bfloat16; };

template <typename T, int VEC>
__device__ __forceinline__ void unpack(const typename Piece<T, VEC>::type& p, float* x) {
    if constexpr (VEC == 1) {
        x[0] = to_f<T>(p);
    } else if constexpr (sizeof(T) == 4 && VEC == 2) {
        x[0] = p.x, x[1] = p.y;
    } else if constexpr (sizeof(T) == 4) {
        x[0] = p.x, x[1] = p.y, x[2] = p.z, x[3] = p.w;
    } else if constexpr (VEC == 2) {
        x[0] = __uint_as_float(p << 16), x[1] = __uint_as_float(p & 0xFFFF0000u);
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
    } else if constexpr (sizeof(T) == 4 && VEC == 2) {
        return make_float2(x[0], x[1]);
    } else if constexpr (sizeof(T) == 4) {
        return make_float4(x[0], x[1], x[2], x[3]);
    } else if constexpr (VEC == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[0], x[1]);
        return *reinterpret_cast<const uint32_t*>(&h);
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

// d = a b + c (or a b) on two elements; d may be an operand.
__device__ __forceinline__ void fma2(float* d, const float* a, const float* b, const float* c) {
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]), "f"(c[0]), "f"(c[1]));
}
__device__ __forceinline__ void mul2(float* d, const float* a, const float* b) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}

// One side of a call, the queries or the keys.
struct Side {
    const void *x, *g;  // input rows; with a norm's gradient also the gradient's rows
    void* y;
    int64_t xs[3], gs[3], ys[3];  // strides in elements: batch row, token, head
    const float* w;
    float* part;                  // partial sums of dw, one row of D a block (null: none)
    int H, fill;
    int tokens, tiles, blocks;    // of a tile; of all batch rows; that do this side (both sides the same if `both`)
};

struct RotaryArgs {
    Side side[2];
    int B, N, rot, backward;
    int both;                     // a block does both sides
    const uint64_t* freqs;
    const int* pos;
    int64_t pos_batch;
    int first;
    float mag, eps;
};

enum { kPlain, kNorm, kNormGrad };

template <typename T, int D, int VEC, int MODE>
struct Shape {
    static constexpr int UNITS = D / (2 * VEC);               // of a row
    static constexpr int LANES = UNITS < 32 ? UNITS : 32;     // that hold it
    static constexpr int EACH = UNITS / LANES;                // units of a lane
    static constexpr int ROWS = kThreads / LANES;             // rows a block has at once
    static constexpr int E = 2 * VEC;                         // elements of a unit
    static constexpr bool RING = VEC > 1;                     // rows come through shared memory
    static constexpr int PIECES = MODE == kNormGrad ? 4 : 2;  // of a row in a stage of a thread
    static constexpr int STAGES = MODE == kNormGrad ? 3 : 4;
    // Blocks of an SM: three where a thread's registers allow it without rows waiting for one another.  Measured, us, with
    // two and three: 65536 x 36 x 128 bf16 192, 204; 5003 x 16 x 64 fp32 9.9, 8.3, in pieces of two 13.3, 12.0.
    static constexpr int BLOCKS = MODE == kNormGrad || (sizeof(T) == 2 && VEC == 8) ? 2 : 3;
    static constexpr int RING_BYTES = RING ? STAGES * PIECES * VEC * static_cast<int>(sizeof(T)) * kThreads : 0;
    static constexpr int TABLE = 2 * ROWS * D;                // floats: two tables of [tokens][2][rot / 2]
    // Before the tables: frequencies, weights of both sides, positions of three tiles.
    static constexpr int HEAD = 64 * 8 + 2 * D * 4 + 3 * ROWS * 4;
    static constexpr int SMEM = HEAD + RING_BYTES + (TABLE > ROWS * (D + 1) ? TABLE : ROWS * (D + 1)) * 4;
};

template <int BYTES>
__device__ __forceinline__ void copy(void* to, const void* from, bool on) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
    if constexpr (BYTES == 16) {
        if (on) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
    } else {
        if (on) asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
    }
}

// INTER: pairs of neighbours, else of the two halves of the rotated part.
template <typename T, int D, int VEC, int MODE, bool INTER>
__global__ void __launch_bounds__(kThreads, (Shape<T, D, VEC, MODE>::BLOCKS)) rotary_kernel(const RotaryArgs p) {
    using P = typename Piece<T, VEC>::type;
    using S = Shape<T, D, VEC, MODE>;
    constexpr int LANES = S::LANES, EACH = S::EACH, ROWS = S::ROWS, E = S::E, ALL = EACH * E, STAGES = S::STAGES, PIECES = S::PIECES;
    extern __shared__ __align__(16) uint8_t s_raw[];
    P* ring = reinterpret_cast<P*>(s_raw) + threadIdx.x;      // [stage][piece][thread]
    uint64_t* s_freqs = reinterpret_cast<uint64_t*>(s_raw + S::RING_BYTES);
    float* s_w = reinterpret_cast<float*>(s_freqs + 64);      // [2][D]
    int* s_pos = reinterpret_cast<int*>(s_w + 2 * D);         // [3][ROWS]
    float* s_trig = reinterpret_cast<float*>(s_pos + 3 * ROWS);  // by turns: [tokens][2][rot / 2] cosines, sines
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES;
    const int pairs = p.rot / 2;
    constexpr bool WITHIN = VEC > 1 && INTER;                 // pairs lie in a piece, not across a unit's two
    const int only = !p.both && static_cast<int>(blockIdx.x) >= p.side[0].blocks ? 1 : 0, last = p.both ? 1 : only;  // sides
    const int block = blockIdx.x - only * p.side[0].blocks, blocks = p.side[only].blocks, tiles = p.side[only].tiles;
    const int per_tile = p.side[only].tokens;
    const int my = slot % per_tile, h0 = slot / per_tile, HS = ROWS / per_tile;  // token of the tile, first head, from head to head

    // Where a unit's pieces begin, and whether they turn.  Neighbouring lanes have neighbouring pieces, whatever the
    // layout, so that a warp's accesses are whole lines.
    int at[EACH], to[EACH];
    bool turns[EACH], turns2[EACH];
#pragma unroll
    for (int u = 0; u < EACH; ++u) {
        const int unit = lane + u * LANES;
        if constexpr (WITHIN) {
            at[u] = unit * VEC, to[u] = D / 2 + at[u];
            turns[u] = at[u] < p.rot, turns2[u] = to[u] < p.rot;
        } else {
            turns[u] = turns2[u] = unit * VEC < pairs;
            if (INTER) at[u] = 2 * unit, to[u] = at[u] + 1;
            else if (turns[u]) at[u] = unit * VEC, to[u] = pairs + at[u];
            else at[u] = pairs + unit * VEC, to[u] = D / 2 + unit * VEC;  // (D - rot) / 2 apart
        }
    }
    float dw[MODE == kNormGrad ? ALL : 1];
#pragma unroll
    for (int i = 0; i < (MODE == kNormGrad ? ALL : 1); ++i) dw[i] = 0.f;
    const int per = (p.N + per_tile - 1) / per_tile;            // tiles of a batch row

    // The loader runs STAGES - 1 rows ahead of the work, over heads, sides and tiles: every thread copies the
    // pieces that it will read itself, so no barrier is needed.
    int l_tile = block, l_side = only, l_h = 0, l_stage = 0;
    bool l_there = false;
    const T *l_x = nullptr, *l_g = nullptr;
    const auto l_base = [&]() {                               // the thread's token of tile l_tile, side l_side
        const int b = l_tile / per, n = (l_tile - b * per) * per_tile + my;
        const Side& sd = p.side[l_side];
        l_there = l_tile < tiles && n < p.N;
        l_x = static_cast<const T*>(sd.x) + b * sd.xs[0] + n * sd.xs[1];
        if constexpr (MODE == kNormGrad) l_g = static_cast<const T*>(sd.g) + b * sd.gs[0] + n * sd.gs[1];
    };
    const auto l_skip = [&]() {                               // past a side without heads, or done with
        while (l_tile < tiles && l_h >= p.side[l_side].H) {
            l_h = 0;
            if (++l_side > last) l_side = only, l_tile += blocks;
        }
        l_base();
    };
    const auto fetch = [&]() {
        if constexpr (S::RING) {
            if (l_tile < tiles) {
                const Side& sd = p.side[l_side];
                const int h = l_h + h0;
                const bool on = l_there && h < sd.H;
                const T* row = l_x + h * sd.xs[2];
                P* dst = ring + l_stage * PIECES * kThreads;
                copy<sizeof(P)>(dst, row + at[0], on);
                copy<sizeof(P)>(dst + kThreads, row + to[0], on);
                if constexpr (MODE == kNormGrad) {
                    const T* grow = l_g + h * sd.gs[2];
                    copy<sizeof(P)>(dst + 2 * kThreads, grow + at[0], on);
                    copy<sizeof(P)>(dst + 3 * kThreads, grow + to[0], on);
                }
                l_h += HS;
                if (l_h >= sd.H) l_skip();
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (++l_stage == STAGES) l_stage = 0;
        }
    };
    static_assert(!S::RING || EACH == 1, "a lane's unit");
    l_skip();
#pragma unroll 1
    for (int i = 0; S::RING && i < STAGES - 1; ++i) fetch();

    // Positions are fetched two tiles ahead, sines worked out one tile ahead, under the rows of the tile before:
    // so a tile starts with what lies in shared memory.
    const auto position = [&](int tile, int t) {              // of token t of a tile, which may be past the last
        const int b = tile / per, n = (tile - b * per) * per_tile + t;
        if (tile >= tiles || t >= per_tile || n >= p.N) return -1;
        return p.pos ? p.pos[b * p.pos_batch + n] : p.first + n;
    };
    const auto sines = [&](const int* pos, float* table) {
        int t = threadIdx.x / pairs, j = threadIdx.x - t * pairs;
        const int dt = kThreads / pairs, dj = kThreads - dt * pairs;
        for (; t < per_tile; t += dt, j += dj) {
            if (j >= pairs) {
                j -= pairs;
                if (++t >= per_tile) break;
            }
            const uint64_t ph = static_cast<uint64_t>(static_cast<int64_t>(pos[t])) * s_freqs[j] + 0x80000000u;
            float s, c;
            turn(static_cast<uint32_t>(ph >> 32), s, c);
            table[2 * t * pairs + j] = c * p.mag;
            table[(2 * t + 1) * pairs + j] = (p.backward ? -s : s) * p.mag;
        }
    };
    static_assert(ROWS <= kThreads, "a position a thread");
    for (int i = threadIdx.x; i < pairs; i += kThreads) s_freqs[i] = p.freqs[i];
    if constexpr (MODE != kPlain)
        for (int i = threadIdx.x; i < 2 * D; i += kThreads) s_w[i] = p.side[i / D].w ? p.side[i / D].w[i % D] : 1.f;
    if (static_cast<int>(threadIdx.x) < per_tile) {
        s_pos[threadIdx.x] = position(block, threadIdx.x);
        s_pos[ROWS + threadIdx.x] = position(block + blocks, threadIdx.x);
    }
    __syncthreads();
    sines(s_pos, s_trig);
    __syncthreads();

    int stage = 0;
    for (int tile = block, turn_no = 0, third = 0; tile < tiles; tile += blocks, turn_no ^= 1, third = third == 2 ? 0 : third + 1) {
        const int b = tile / per, n0 = (tile - b * per) * per_tile, tokens = min(per_tile, p.N - n0);
        const bool there = my < tokens;
        const bool live = there && s_pos[third * ROWS + my] >= 0;  // a row of a token
        const int ahead = static_cast<int>(threadIdx.x) < per_tile ? position(tile + 2 * blocks, threadIdx.x) : 0;
        const float* table = s_trig + turn_no * (per_tile * p.rot);
        float cs[EACH * VEC], sn[EACH * VEC];
#pragma unroll
        for (int u = 0; u < EACH; ++u) {
            // pairs of the first and the second half of the unit's
            const float* first = table + 2 * my * pairs + (WITHIN ? at[u] / 2 : (lane + u * LANES) * VEC);
            const float* second = first + (WITHIN ? D / 4 : VEC / 2);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const bool low = VEC == 1 || i < VEC / 2, on = there && (low ? turns[u] : turns2[u]);
                const float* pair = low ? first + i : second + (i - VEC / 2);
                cs[u * VEC + i] = on ? pair[0] : 1.f;
                sn[u * VEC + i] = on ? pair[pairs] : 0.f;
            }
        }
#pragma unroll 1
        for (int side = only; side <= last; ++side) {
            const Side& sd = p.side[side];
            float w[MODE == kPlain ? 1 : ALL];
            if constexpr (MODE != kPlain) {
#pragma unroll
                for (int u = 0; u < EACH; ++u)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        w[u * E + i] = s_w[side * D + at[u] + i];
                        w[u * E + VEC + i] = s_w[side * D + to[u] + i];
                    }
            }
            const int64_t n = n0 + my;
            T* y = static_cast<T*>(sd.y) + b * sd.ys[0] + n * sd.ys[1];
#pragma unroll 1
            for (int hb = 0; hb < sd.H; hb += HS) {           // the same for all threads of the block
                const int h = hb + h0;
                const bool mine = there && h < sd.H, count = live && mine;
                P px[EACH][PIECES];
                if constexpr (S::RING) {
                    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
#pragma unroll
                    for (int i = 0; i < PIECES; ++i) px[0][i] = ring[(stage * PIECES + i) * kThreads];
                    if (++stage == STAGES) stage = 0;
                    fetch();                                  // into the stage of the row before
                } else if (mine) {
                    const T* row = static_cast<const T*>(sd.x) + b * sd.xs[0] + n * sd.xs[1] + h * sd.xs[2];
                    const T* grow = MODE == kNormGrad ? static_cast<const T*>(sd.g) + b * sd.gs[0] + n * sd.gs[1] + h * sd.gs[2] : nullptr;
#pragma unroll
                    for (int u = 0; u < EACH; ++u) {
                        px[u][0] = *reinterpret_cast<const P*>(row + at[u]);
                        px[u][1] = *reinterpret_cast<const P*>(row + to[u]);
                        if constexpr (MODE == kNormGrad) {
                            px[u][2] = *reinterpret_cast<const P*>(grow + at[u]);
                            px[u][3] = *reinterpret_cast<const P*>(grow + to[u]);
                        }
                    }
                }
                float v[ALL], z[MODE == kNormGrad ? ALL : 1];
                float* m = MODE == kNormGrad ? z : v;         // what is turned
#pragma unroll
                for (int u = 0; u < EACH; ++u) {
                    unpack<T, VEC>(px[u][0], v + u * E);
                    unpack<T, VEC>(px[u][1], v + u * E + VEC);
                    if constexpr (MODE == kNormGrad) {
                        unpack<T, VEC>(px[u][2], z + u * E);
                        unpack<T, VEC>(px[u][3], z + u * E + VEC);
                    }
                }
                if (!count) {  // (also what was not loaded)
#pragma unroll
                    for (int i = 0; i < ALL; ++i) {
                        v[i] = 0.f;
                        if constexpr (MODE == kNormGrad) z[i] = 0.f;
                    }
                }
                float r = 1.f;
                if constexpr (MODE != kPlain) {
                    float q[2] = {0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < ALL; i += 2) fma2(q, v + i, v + i, q);
                    q[0] += q[1];
#pragma unroll
                    for (int o = LANES / 2; o; o >>= 1) q[0] += __shfl_xor_sync(0xffffffffu, q[0], o);
                    r = 1.f / sqrtf(q[0] * (1.f / D) + p.eps);
                }
                if constexpr (MODE == kNorm) {
#pragma unroll
                    for (int i = 0; i < ALL; i += 2) mul2(v + i, v + i, w + i);
                }
#pragma unroll
                for (int u = 0; u < EACH; ++u) {
                    float* e = m + u * E;
                    const float *c = cs + u * VEC, *s = sn + u * VEC;
                    // (what does not turn stays as it is, beside whatever else the row holds)
                    if constexpr (VEC == 1 || WITHIN) {
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            const float e0 = e[2 * i], e1 = e[2 * i + 1];
                            if (VEC == 1 || i < VEC / 2 ? turns[u] : turns2[u]) {
                                e[2 * i] = e0 * c[i] - e1 * s[i];
                                e[2 * i + 1] = e0 * s[i] + e1 * c[i];
                            }
                        }
                    } else if (turns[u]) {
#pragma unroll
                        for (int i = 0; i + 1 < VEC; i += 2) {
                            float t0[2], t1[2];
                            const float neg[2] = {-e[VEC + i], -e[VEC + i + 1]};
                            mul2(t0, e + i, c + i);
                            mul2(t1, e + i, s + i);
                            fma2(e + i, neg, s + i, t0);
                            fma2(e + VEC + i, e + VEC + i, c + i, t1);
                        }
                    }
                }
                if constexpr (MODE == kNorm) {
                    const float rr[2] = {r, r};
#pragma unroll
                    for (int i = 0; i < ALL; i += 2) mul2(v + i, v + i, rr);
                }
                if constexpr (MODE == kNormGrad) {
                    const float rr[2] = {r, r};
                    float mean[2] = {0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < ALL; i += 2) {
                        mul2(v + i, v + i, rr);
                        fma2(dw + i, z + i, v + i, dw + i);
                        mul2(z + i, z + i, w + i);
                        fma2(mean, z + i, v + i, mean);
                    }
                    mean[0] += mean[1];
#pragma unroll
                    for (int o = LANES / 2; o; o >>= 1) mean[0] += __shfl_xor_sync(0xffffffffu, mean[0], o);
                    mean[0] *= -1.f / D;
                    mean[1] = mean[0];
#pragma unroll
                    for (int i = 0; i < ALL; i += 2) {
                        fma2(v + i, v + i, mean, z + i);
                        mul2(v + i, v + i, rr);
                    }
                }
                if (count || (mine && sd.fill)) {
                    T* out = y + h * sd.ys[2];
                    if (!count) {  // whatever the weights are
#pragma unroll
                        for (int i = 0; i < ALL; ++i) v[i] = 0.f;
                    }
#pragma unroll
                    for (int u = 0; u < EACH; ++u) {
                        *reinterpret_cast<P*>(out + at[u]) = pack<T, VEC>(v + u * E);
                        *reinterpret_cast<P*>(out + to[u]) = pack<T, VEC>(v + u * E + VEC);
                    }
                }
            }
        }
        if (tile + blocks < tiles) {
            const int next = third == 2 ? 0 : third + 1;
            if (static_cast<int>(threadIdx.x) < per_tile) s_pos[(next == 2 ? 0 : next + 1) * ROWS + threadIdx.x] = ahead;
            sines(s_pos + next * ROWS, s_trig + (turn_no ^ 1) * (per_tile * p.rot));
            __syncthreads();
        }
    }
    if constexpr (S::RING) asm volatile("cp.async.wait_all;" ::: "memory");
    if constexpr (MODE == kNormGrad) {
        // The block's sums: units over the block's rows, in the order of the rows.
        float* part = p.side[only].part;
        if (part == nullptr) return;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < EACH; ++u)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s_trig[slot * (D + 1) + at[u] + i] = dw[u * E + i];
                s_trig[slot * (D + 1) + to[u] + i] = dw[u * E + VEC + i];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += kThreads) {
            float a = 0.f;
            for (int i = 0; i < ROWS; ++i) a += s_trig[i * (D + 1) + c];
            part[static_cast<int64_t>(block) * D + c] = a;
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

// Rows' pieces of `vec` elements lie on their boundaries, and turn as a whole or not at all.
bool aligned(const RotaryShape& s, int rot, int vec, int es) {
    if (rot % (s.interleaved ? vec : 2 * vec)) return false;
    for (int i = 0; i < s.tensors; ++i) {
        if (s.ptr[i] == nullptr) continue;
        if (reinterpret_cast<uintptr_t>(s.ptr[i]) % (vec * es)) return false;
        for (int d = 0; d < 3; ++d)
            if (s.strides[i][d] % vec) return false;
    }
    return true;
}

template <typename T, int D, int VEC, int MODE, bool INTER>
cudaError_t launch(const LaunchCtx& c, const RotaryShape& s, float* dwq, float* dwk) {
    using S = Shape<T, D, VEC, MODE>;
    RotaryArgs p = {};
    p.B = s.B, p.N = s.N, p.rot = s.rot, p.backward = s.backward;
    p.freqs = s.freqs, p.pos = s.positions, p.pos_batch = s.pos_batch, p.first = s.first;
    p.mag = s.mag, p.eps = s.eps;
    p.both = MODE != kNormGrad;
    // tensors: q, k, [gradients of q, k,] outputs of q, k
    constexpr int out = MODE == kNormGrad ? 4 : 2;
    for (int i = 0; i < 2; ++i) {
        Side& d = p.side[i];
        d.H = i ? s.Hk : s.Hq;
        d.x = s.ptr[i], d.g = s.ptr[2 + i], d.y = const_cast<void*>(s.ptr[out + i]);
        for (int j = 0; j < 3; ++j) d.xs[j] = s.strides[i][j], d.gs[j] = s.strides[2 + i][j], d.ys[j] = s.strides[out + i][j];
        d.w = s.w[i];
        d.fill = s.fill >> i & 1;
    }
    // As many blocks as an SM has room for, whose loaders never stop; with the gradient, whose sums are of one
    // side, dealt out by its work.
    const auto side_work = [&](int H) { return H ? static_cast<int64_t>(H) + kTrig : 0; };
    const int most = S::BLOCKS * c.num_sms;
    const int64_t q_work = side_work(s.Hq), work = q_work + side_work(s.Hk);
    const int q_blocks = static_cast<int>((most * q_work + work / 2) / work);
    int grid = 0, tokens = 1;
    for (int i = 0; i < (p.both ? 1 : 2); ++i) {
        Side& d = p.side[i];
        const int limit = p.both ? most : std::max(1, i ? most - q_blocks : q_blocks);
        if (!p.both && d.H == 0) continue;
        // Tokens of a tile: the power of two with the least time, counted in rows a thread for the block with most
        // tiles: its heads, a row or so for the tile's start, and its sines.
        double best = 0;
        for (int t = 1; t <= S::ROWS; t *= 2) {
            const int HS = S::ROWS / t;
            const auto rows = [&](int H) { return (H + HS - 1) / HS; };
            const int64_t tiles = (s.N + t - 1) / t * static_cast<int64_t>(s.B);
            const double cost = ((tiles + limit - 1) / limit) *
                                ((p.both ? rows(s.Hq) + rows(s.Hk) : rows(d.H)) + 1 + t * (s.rot / 2) / static_cast<double>(kThreads));
            if (t == 1 || cost < best) best = cost, d.tokens = t, d.tiles = static_cast<int>(tiles);
            if (tiles > INT32_MAX / 2 && t == 1) return cudaErrorInvalidValue;
        }
        d.blocks = std::min(d.tiles, limit);
        grid += d.blocks;
        tokens = std::max(tokens, d.tokens);
    }
    if (p.both) p.side[1].tokens = p.side[0].tokens, p.side[1].tiles = p.side[0].tiles, p.side[1].blocks = p.side[0].blocks;
    float* part = nullptr;
    if (MODE == kNormGrad && (dwq || dwk)) {
        cudaError_t e = scratch_alloc(c, reinterpret_cast<void**>(&part), rotary_grad_scratch(s.B, s.N, s.Hq, s.Hk, D, true, c.num_sms));
        if (e != cudaSuccess) return e;
        if (dwq) p.side[0].part = part;
        if (dwk) p.side[1].part = part + static_cast<int64_t>(rotary_grad_blocks(c.num_sms)) * D;
    }
    int smem = 2 * tokens * s.rot * static_cast<int>(sizeof(float));
    if (MODE == kNormGrad) smem = std::max(smem, S::ROWS * (D + 1) * 4);
    smem += S::HEAD + S::RING_BYTES;
    int per_sm = 0;
    cudaError_t e = resident_blocks<rotary_kernel<T, D, VEC, MODE, INTER>>(c.device, kThreads, S::SMEM, &per_sm);
    if (e == cudaSuccess) {
        rotary_kernel<T, D, VEC, MODE, INTER><<<grid, kThreads, smem, c.stream>>>(p);
        note_launch();
        e = cudaGetLastError();
    }
    if (MODE == kNormGrad && (dwq || dwk)) {
        if (e == cudaSuccess) {
            rotary_weight_kernel<<<2 * (D / 32), 1024, 0, c.stream>>>(part, p.side[1].part, p.side[0].blocks, p.side[1].blocks, D, dwq, dwk);
            note_launch();
            e = cudaGetLastError();
        }
        scratch_free(c, part);
    }
    return e;
}

// Pieces of 16 bytes, of two elements, or single ones.
template <typename T, int D, int MODE, bool INTER>
cudaError_t by_alignment(const LaunchCtx& c, const RotaryShape& s, float* dwq, float* dwk) {
    constexpr int VEC = 16 / sizeof(T);
    if (aligned(s, s.rot, VEC, sizeof(T))) return launch<T, D, VEC, MODE, INTER>(c, s, dwq, dwk);
    if (aligned(s, s.rot, 2, sizeof(T))) return launch<T, D, 2, MODE, INTER>(c, s, dwq, dwk);
    return launch<T, D, 1, MODE, INTER>(c, s, dwq, dwk);
}

template <typename T, int MODE, bool INTER>
cudaError_t by_size(const LaunchCtx& c, const RotaryShape& s, float* dwq, float* dwk) {
    if (s.D == 32) return by_alignment<T, 32, MODE, INTER>(c, s, dwq, dwk);
    if (s.D == 64) return by_alignment<T, 64, MODE, INTER>(c, s, dwq, dwk);
    return by_alignment<T, 128, MODE, INTER>(c, s, dwq, dwk);
}

template <int MODE>
cudaError_t by_type(const LaunchCtx& c, const RotaryShape& s, bool bf16, float* dwq, float* dwk) {
    using bf = __nv_bfloat16;
    if (s.interleaved) return bf16 ? by_size<bf, MODE, true>(c, s, dwq, dwk) : by_size<float, MODE, true>(c, s, dwq, dwk);
    return bf16 ? by_size<bf, MODE, false>(c, s, dwq, dwk) : by_size<float, MODE, false>(c, s, dwq, dwk);
}

}  // namespace

int rotary_grad_blocks(int num_sms) { return 2 * num_sms; }

size_t rotary_grad_scratch(int B, int N, int Hq, int Hk, int D, bool weights, int num_sms) {
    if (!weights || static_cast<int64_t>(B) * N * (Hq + Hk) == 0) return 0;
    return 2 * sizeof(float) * rotary_grad_blocks(num_sms) * D;
}

cudaError_t rotary(const LaunchCtx& c, const RotaryShape& s, bool bf16, bool norm) {
    return norm ? by_type<kNorm>(c, s, bf16, nullptr, nullptr) : by_type<kPlain>(c, s, bf16, nullptr, nullptr);
}

cudaError_t norm_rotary_grad(const LaunchCtx& c, const RotaryShape& s, bool bf16, float* dwq, float* dwk) {
    return by_type<kNormGrad>(c, s, bf16, dwq, dwk);
}

}  // namespace la
