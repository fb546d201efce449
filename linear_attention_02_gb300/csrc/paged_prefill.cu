// paged_prefill.cu -- attention of each request's new tokens over its pages: query i of
// request r stands at position p = cached_lens[r] + i, whose key is in the cache already, and
//     out = sum_j e^{s_j - m} v_j / sum_j e^{s_j - m},  s_j = scale q . k_j,
// over the positions j <= p (of these the last `window`); lse = m + ln sum_j e^{s_j - m}.
// Query head h reads key head h / (Hq / Hkv).  Here fp32; bf16 is paged_prefill_tc.cu.
//
// Bound by the matrix unit: fp32 operands enter tf32 products (m16n8k8) as two terms split by
// rounding, three products for each (the fourth, of two second terms, is below 2^-22 of the
// whole, 2^-24 in the mean).  A term of a score or an output is off by 2^-21 of itself at most, 2^-23 in the mean.
// The unit cuts off its sums: so scores are summed by it over 32 columns and outputs over a step, from zero,
// and those added to the running sums in fp32.  (Running sums in the tensor core's own memory are cut off in
// the same way; parts of them from zero, read back every step, were not tried.)
//
// A block takes a range of steps (prefill_plan.cuh): 128 rows of a request and key head, 16 a
// warp, against 32 key positions that cp.async brings a step ahead.  The contraction index and the output
// columns are in such an order that a lane's operands are 16-byte pieces of the rows, read
// without bank conflicts, and the weights of a lane are its operand of the second product.
//
// A value within 2^-12 of the largest fp32 number has an infinite first term.  Keeping it finite costs two
// operations a value (6% of the time), so a segment with a NaN among its outputs is computed again, from halved values.
//
// Measured: 16 prompts of 1024 tokens, 16 heads of 64: 763 us, 45 TFLOP/s; 8 x 1024 of 8 heads of 128: 437 us;
// 13 ragged requests up to 700 tokens with a window of 1000: 375 to 410 us (1940 with the products on the
// fp32 units), the matrix unit's pipe half full and what stalls most.  48 requests of 1 to 8 tokens over 500 to
// 16000 positions: 1390 us, as few rows leave most warps idle.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "la_common.cuh"
#include "la_launch.h"
#include "la_plan.h"
#include "prefill_plan.cuh"

namespace la {
namespace {

using prefill::Args;
using prefill::exp2_approx;
using prefill::Keys;
using prefill::Request;
using prefill::Segment;
using prefill::token_of;

constexpr int TM = 128, KT = 32, NT = 256;

template <int D>
struct Lay {
    // Strides of rows in words: of queries and keys 16 past a multiple of 32, of values 4, so that eight lanes
    // read eight different 16-byte places of the 128 bytes that shared memory delivers at once.
    static constexpr int KS = D + 16, VS = D + 4;
    static constexpr int STAGE = KT * (KS + VS);
    static constexpr int SMEM = (TM * KS + 2 * STAGE) * 4;
    static constexpr int BLOCKS = D == 128 ? 1 : 2;  // of an SM, by shared memory
};

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo: hi rounded to the 11 bits of an operand, the rest of either sign.  An infinity gives a NaN.
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}
// c += a b in three products of terms, the small ones first.
__device__ __forceinline__ void mma3(float (&c)[4], const uint32_t (&ah)[4], const uint32_t (&al)[4], float b0, float b1) {
    uint32_t h0, l0, h1, l1;
    split(b0, h0, l0);
    split(b1, h1, l1);
    mma(c, al, h0, h1);
    mma(c, ah, l0, l1);
    mma(c, ah, h0, h1);
}
__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void copy16(void* to, const void* from, bool on) {  // zeros if not on
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from),
                 "r"(on ? 16 : 0)
                 : "memory");
}

// Scores by plain products, for the step whose split products gave a NaN (an infinite key or query, where the
// definition may have an infinity): the lane's of rows g, g + 8 with keys 8 n + 2 t, 8 n + 2 t + 1.
template <int D>
__device__ __noinline__ float4 plain_scores(const float* q, const float* k, int n) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    for (int e = 0; e < 4; ++e) {
        const float *a = q + (g + 8 * (e >> 1)) * Lay<D>::KS, *b = k + (8 * n + 2 * t + (e & 1)) * Lay<D>::KS;
        for (int d = 0; d < D; ++d) x[e] += a[d] * b[d];
    }
    return make_float4(x[0], x[1], x[2], x[3]);
}

template <int D>
__global__ void __launch_bounds__(NT, Lay<D>::BLOCKS)
prefill_f32_kernel(const float* __restrict__ q, const float* __restrict__ K, const float* __restrict__ V, float* __restrict__ out,
                   const Args p) {
    using Ly = Lay<D>;
    using Plan = prefill::Planner<TM, KT, NT>;
    constexpr int KS = Ly::KS, VS = Ly::VS, GR = D / 32, CH = D / 4;
    extern __shared__ __align__(16) float sm[];
    __shared__ prefill::Range s_range;
    __shared__ uint32_t s_mask[2];      // keys of a stage that are on a page, a bit each
    __shared__ int s_odd;               // a value that was not finite was replaced
    float* s_q = sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (tid < 2) p.desc[2 * blockIdx.x + tid] = make_int4(0, 0, 0, 0);
    Plan& plan = *reinterpret_cast<Plan*>(sm);  // before anything else is in there
    plan.run(p);
    if (tid == 0) s_range = plan.range;
    __syncthreads();
    const prefill::Range range = s_range;
    const float c = p.s.scale * 1.4426950408889634f;
    const int off_mask = (1 << p.s.log2p) - 1;
    bool bad = false;

    if (range.any) {
        prefill::Walk<TM, KT> walk(p, range);
        Segment sg;
        while (walk.next(p, sg)) {
            const Request rq(p, sg.r);
            const Keys<KT> k(p, rq, sg.m0, min(sg.m0 + TM, sg.rows));
            const int* table = p.table + static_cast<int64_t>(sg.r) * p.s.max_pages;
            const auto load = [&](int j, int stage) {
                float *dk = sm + TM * KS + stage * Ly::STAGE, *dv = dk + KT * KS;
                const int x0 = (k.k0 + j) * KT;
#pragma unroll
                for (int i = 0; i < KT * CH / NT; ++i) {
                    const int e = tid + i * NT, y = e / CH, ch = e % CH, x = x0 + y;
                    int page = -1;
                    if (x >= k.lo && x < k.hi) page = table[x >> p.s.log2p];
                    const bool on = static_cast<unsigned>(page) < static_cast<unsigned>(p.s.num_pages);
                    const int64_t at = on ? ((((static_cast<int64_t>(page) * p.s.Hkv + sg.kh) << p.s.log2p) + (x & off_mask)) * D + 4 * ch) : 0;
                    copy16(dk + y * KS + 4 * ch, on ? K + at : q, on);
                    copy16(dv + y * VS + 4 * ch, on ? V + at : q, on);
                }
                if (warp == 0) {  // a key a lane
                    const int x = x0 + lane;
                    const bool in = x >= k.lo && x < k.hi;
                    const bool on = in && static_cast<unsigned>(table[x >> p.s.log2p]) < static_cast<unsigned>(p.s.num_pages);
                    bad |= in && !on;
                    const uint32_t m = __ballot_sync(0xffffffffu, on);
                    if (lane == 0) s_mask[stage] = m;
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            for (int e = tid; e < TM * CH; e += NT) {
                const int y = e / CH, ch = e % CH, m = sg.m0 + y, token = token_of(p, m);
                const bool on = m < sg.rows;
                const int64_t at = on ? (static_cast<int64_t>(rq.first) + token) * p.s.Hq + static_cast<int64_t>(sg.kh) * p.G + (m - token * p.G) : 0;
                copy16(s_q + y * KS + 4 * ch, q + at * D + 4 * ch, on);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");

            const int r0 = sg.m0 + 16 * warp, r1 = min(r0 + 16, sg.rows);  // the warp's rows
            const bool work = r0 < sg.rows;
            const int wfirst = rq.cached + token_of(p, work ? r0 : 0), wlast = rq.cached + token_of(p, work ? r1 - 1 : 0);
            const int wlo = p.s.window ? max(wfirst - p.s.window + 1, 0) : 0;
            int pos[2], from[2];  // of rows g and g + 8: they see positions past `from` up to `pos`
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                pos[i] = rq.cached + token_of(p, r0 + g + 8 * i);
                from[i] = p.s.window ? pos[i] - p.s.window : -1;
            }
            float top[2], sum[2], o[GR][4][4], half = 1.f;
#pragma unroll 1
            for (;; half = 0.5f) {
                load(sg.a, 0);
                if (tid == 0) s_odd = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) top[i] = -INFINITY, sum[i] = 0.f;
#pragma unroll
                for (int a = 0; a < GR; ++a)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[a][i][e] = 0.f;

#pragma unroll 1
                for (int j = sg.a; j < sg.b; ++j) {
                    const int stage = (j - sg.a) & 1, x0 = (k.k0 + j) * KT;
                    if (j + 1 < sg.b) load(j + 1, stage ^ 1);
                    else asm volatile("cp.async.commit_group;" ::: "memory");
                    asm volatile("cp.async.wait_group 1;" ::: "memory");  // all but the next step's
                    __syncthreads();
                    const float *sk = sm + TM * KS + stage * Ly::STAGE, *sv = sk + KT * KS;
                    const uint32_t mask = s_mask[stage];
                    const bool whole_tile = x0 + KT - 1 <= k.first && (p.s.window == 0 || x0 > k.last - p.s.window) && mask == 0xFFFFFFFFu;
                    if (!whole_tile || half < 1.f) {
                        // Values that a row does not see have weight 0, but 0 times an infinity or NaN is none: in tiles that
                        // some row sees in part they are replaced, and rows that do see them marked at the end.
                        float* v = const_cast<float*>(sv);
                        for (int e = tid; e < KT * CH; e += NT) {
                            float4* at = reinterpret_cast<float4*>(v + e / CH * VS + 4 * (e % CH));
                            float4 x = *at;
                            if (!whole_tile && !(fabsf(x.x) < INFINITY && fabsf(x.y) < INFINITY && fabsf(x.z) < INFINITY && fabsf(x.w) < INFINITY)) {
                                x.x = fabsf(x.x) < INFINITY ? x.x : 0.f, x.y = fabsf(x.y) < INFINITY ? x.y : 0.f;
                                x.z = fabsf(x.z) < INFINITY ? x.z : 0.f, x.w = fabsf(x.w) < INFINITY ? x.w : 0.f;
                                *at = x;
                                s_odd = 1;
                            }
                            if (half < 1.f) *at = make_float4(x.x * half, x.y * half, x.z * half, x.w * half);
                        }
                        __syncthreads();
                    }
                    if (work && x0 <= wlast && x0 + KT > wlo) {
                        // The unit cuts its sums off, 48 of them in a chain at D = 128, by 1.1e-6 of a score in all.  So those over 32
                        // columns start from zero and are added in fp32: 2.6e-7 (over 64: 4.8e-7; over 16: 1.6e-7, for 8% of the time).
                        float s[KT / 8][4], z[KT / 8][4];
                        const float* qa = s_q + (16 * warp + g) * KS + 4 * t;
                        const float* kb = sk + g * KS + 4 * t;
#pragma unroll
                        for (int d = 0; d < D; d += 16) {
                            const float4 a = *reinterpret_cast<const float4*>(qa + d), b = *reinterpret_cast<const float4*>(qa + 8 * KS + d);
                            uint32_t h[2][4], l[2][4];
                            split(a.x, h[0][0], l[0][0]), split(b.x, h[0][1], l[0][1]), split(a.y, h[0][2], l[0][2]), split(b.y, h[0][3], l[0][3]);
                            split(a.z, h[1][0], l[1][0]), split(b.z, h[1][1], l[1][1]), split(a.w, h[1][2], l[1][2]), split(b.w, h[1][3], l[1][3]);
#pragma unroll
                            for (int n = 0; n < KT / 8; ++n) {
                                const float4 f = *reinterpret_cast<const float4*>(kb + 8 * n * KS + d);
                                if (d % 32 == 0) z[n][0] = 0.f, z[n][1] = 0.f, z[n][2] = 0.f, z[n][3] = 0.f;
                                mma3(z[n], h[0], l[0], f.x, f.y);
                                mma3(z[n], h[1], l[1], f.z, f.w);
                                if ((d + 16) % 32) continue;
#pragma unroll
                                for (int e = 0; e < 4; ++e) s[n][e] = d < 32 ? z[n][e] : s[n][e] + z[n][e];
                            }
                        }
                        float nan = 0.f;
#pragma unroll
                        for (int n = 0; n < KT / 8; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) nan = max_nan(nan, s[n][e]);
                        if (__any_sync(0xffffffffu, nan != nan)) {
#pragma unroll
                            for (int n = 0; n < KT / 8; ++n) {
                                const float4 f = plain_scores<D>(s_q + 16 * warp * KS, sk, n);
                                // the others stay as they are, whatever rows they share the step with
                                s[n][0] = s[n][0] != s[n][0] ? f.x : s[n][0], s[n][1] = s[n][1] != s[n][1] ? f.y : s[n][1];
                                s[n][2] = s[n][2] != s[n][2] ? f.z : s[n][2], s[n][3] = s[n][3] != s[n][3] ? f.w : s[n][3];
                            }
                        }
                        const bool all = x0 + KT - 1 <= wfirst && (p.s.window == 0 || x0 > wlast - p.s.window) && mask == 0xFFFFFFFFu;
                        float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int n = 0; n < KT / 8; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int y = 8 * n + 2 * t + (e & 1), x = x0 + y;
                                s[n][e] *= c;
                                if (!all && !(x <= pos[e >> 1] && x > from[e >> 1] && (mask >> y & 1u))) s[n][e] = -INFINITY;
                                best[e >> 1] = fmaxf(best[e >> 1], s[n][e]);
                            }
                        float f[2], base[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            best[i] = fmaxf(best[i], __shfl_xor_sync(0xffffffffu, best[i], 1));
                            best[i] = fmaxf(best[i], __shfl_xor_sync(0xffffffffu, best[i], 2));
                            const float m = fmaxf(top[i], best[i]);
                            f[i] = m == top[i] ? 1.f : exp2_approx(top[i] - m);
                            top[i] = m;
                            base[i] = m == -INFINITY ? 0.f : m;
                            sum[i] *= f[i];
                        }
                        uint32_t wh[KT / 8][4], wl[KT / 8][4];  // a lane's weights, as the operand of the second product
#pragma unroll
                        for (int n = 0; n < KT / 8; ++n) {
                            float w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                w[e] = exp2_approx(s[n][e] - base[e >> 1]);
                                sum[e >> 1] += w[e];
                            }
                            split(w[0], wh[n][0], wl[n][0]), split(w[2], wh[n][1], wl[n][1]);
                            split(w[1], wh[n][2], wl[n][2]), split(w[3], wh[n][3], wl[n][3]);
                        }
                        const float* vb = sv + 2 * t * VS + 4 * g;
#pragma unroll
                        for (int a = 0; a < GR; ++a) {
                            float z[4][4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e) z[i][e] = 0.f;
#pragma unroll
                            for (int n = 0; n < KT / 8; ++n) {
                                const float4 u = *reinterpret_cast<const float4*>(vb + 8 * n * VS + 32 * a);
                                const float4 v = *reinterpret_cast<const float4*>(vb + (8 * n + 1) * VS + 32 * a);
                                mma3(z[0], wh[n], wl[n], u.x, v.x);
                                mma3(z[1], wh[n], wl[n], u.y, v.y);
                                mma3(z[2], wh[n], wl[n], u.z, v.z);
                                mma3(z[3], wh[n], wl[n], u.w, v.w);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i)
#pragma unroll
                                for (int e = 0; e < 4; ++e) o[a][i][e] = fmaf(o[a][i][e], f[e >> 1], z[i][e]);
                        }
                    }
                    __syncthreads();  // before the stage is filled again
                }
                bool nan = false;
#pragma unroll
                for (int a = 0; a < GR; ++a)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) nan |= o[a][i][e] != o[a][i][e];
                if (half < 1.f || !__syncthreads_or(nan)) break;
            }
            // the rows' outputs: 8 columns of each 32 a lane
            const bool whole = sg.whole();
            const int slot = 2 * blockIdx.x + (sg.a == 0 ? 1 : 0);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
                sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
                const int y = 16 * warp + g + 8 * i, m = sg.m0 + y;
                if (m >= sg.rows) continue;
                const bool good = sum[i] > 0.f || sum[i] != sum[i];
                const int token = token_of(p, m);
                const int64_t at = (static_cast<int64_t>(rq.first) + token) * p.s.Hq + static_cast<int64_t>(sg.kh) * p.G + (m - token * p.G);
                float* to = whole ? out + at * D : p.part + (static_cast<int64_t>(slot) * TM + y) * D;
                const float inv = (whole ? (good ? sum[i] : INFINITY) : 1.f) * half;
#pragma unroll
                for (int a = 0; a < GR; ++a) {
                    float v[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) v[x] = o[a][x & 3][2 * i + (x >> 2)] / inv;
                    if (s_odd) {  // rare: does this row see one of the replaced values?
                        uint32_t bits = 0;
                        for (int j = sg.a; j < sg.b; ++j)
                            bits |= prefill::odd_columns<float, D, KT, true>(p, V, sg.r, sg.kh, k.first, k.last, rq.end, k.k0 + j, from[i], pos[i], 32 * a);
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            if (bits >> (8 * t + x) & 1u) v[x] = __uint_as_float(0x7FFFFFFFu);
                    }
                    *reinterpret_cast<float4*>(to + 32 * a + 8 * t) = make_float4(v[0], v[1], v[2], v[3]);
                    *reinterpret_cast<float4*>(to + 32 * a + 8 * t + 4) = make_float4(v[4], v[5], v[6], v[7]);
                }
                if (t == 0) {
                    if (!whole) p.ml[static_cast<int64_t>(slot) * TM + y] = make_float2(top[i], sum[i]);
                    else if (p.lse) p.lse[at] = good ? (top[i] + log2f(sum[i])) * 0.6931471805599453f : -INFINITY;
                }
            }
            __syncthreads();  // before the next queries come
        }
        if (bad) atomicOr(p.status, kStatusBadIndex);
    }
    prefill::finish_range<float, D, TM, KT, NT>(p, range, true, out);
}

template <int D>
int ranges_of(int num_sms) { return Lay<D>::BLOCKS * num_sms; }

template <int D>
cudaError_t prefill_f32(const LaunchCtx& c, const float* q, const float* K, const float* V, const int* table, const int* lens,
                        const int* starts, float* out, float* lse, const PrefillShape& s, int fill) {
    Args p = {};
    prefill::set_group(p, s.Hq / s.Hkv, TM);
    p.s = s, p.table = table, p.lens = lens, p.starts = starts, p.lse = lse, p.fill = fill;
    p.status = c.status_word;
    int per_sm = 1;
    cudaError_t e = resident_blocks<prefill_f32_kernel<D>>(c.device, NT, Lay<D>::SMEM, &per_sm);
    if (e != cudaSuccess) return e;
    const int ranges = ranges_of<D>(c.num_sms);
    uint8_t* base = nullptr;
    if ((e = scratch_alloc(c, reinterpret_cast<void**>(&base), prefill::scratch_bytes(D, TM, ranges))) != cudaSuccess) return e;
    prefill::set_scratch(p, base, D, TM, ranges);
    prefill_f32_kernel<D><<<ranges, NT, Lay<D>::SMEM, c.stream>>>(q, K, V, out, p);
    note_launch();
    e = cudaGetLastError();
    if (e == cudaSuccess) e = prefill::launch_join<float, D, TM>(p, out, ranges, c.stream);
    scratch_free(c, base);
    return e;
}

}  // namespace

template <typename T, int D>
cudaError_t paged_prefill(const LaunchCtx& c, const T* q, const T* K, const T* V, const int* table,
                          const int* lens, const int* starts, T* out, float* lse,
                          const PrefillShape& s, int fill) {
    if constexpr (sizeof(T) == 2) return paged_prefill_tc<D>(c, q, K, V, table, lens, starts, out, lse, s, fill);
    else return prefill_f32<D>(c, q, K, V, table, lens, starts, out, lse, s, fill);
}

size_t paged_prefill_scratch(int D, bool bf16, int num_sms) {
    if (bf16) return paged_prefill_tc_scratch(D, num_sms);
    return prefill::scratch_bytes(D, TM, D == 32 ? ranges_of<32>(num_sms) : D == 64 ? ranges_of<64>(num_sms) : ranges_of<128>(num_sms));
}

#define LA_INST_PP(T, D)                                                                               \
    template cudaError_t paged_prefill<T, D>(const LaunchCtx&, const T*, const T*, const T*, const int*, \
                                             const int*, const int*, T*, float*, const PrefillShape&, int);
LA_INST_PP(float, 32) LA_INST_PP(float, 64) LA_INST_PP(float, 128)
LA_INST_PP(__nv_bfloat16, 32) LA_INST_PP(__nv_bfloat16, 64) LA_INST_PP(__nv_bfloat16, 128)

}  // namespace la
