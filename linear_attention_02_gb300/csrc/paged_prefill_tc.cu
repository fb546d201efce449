// paged_prefill_tc.cu -- attention of each request's new tokens over its pages, bf16, on the
// tensor core (the formulas are paged_prefill.cu's).
//
// Bound by the tensor core for long chunks (4 D operations a query head and visible
// position), by memory for a few tokens over long contexts.  One block an SM takes a range of
// steps (prefill_plan.cuh): 256 rows of a request and key head, as two subtiles of 128, against
// 128 key positions.  Warps:
//   0-3, 4-7  softmax of subtile 0 and 1, a row a thread, and the rows' outputs
//   8         every matrix product, issued by one thread
//   9, 10     keys and values by TMA, page by page, into a ring of tiles
//   11        the range's segments, worked out for all the others
//   12 to 15  queries, and the values of tiles that some row sees only in part
// S = Q K^T goes to tensor memory, a thread turns its row's 128 scores into weights there, and
// O += P V reads the weights from tensor memory.  The two subtiles take turns: while one's
// scores become weights, the tensor core works for the other.  The products are issued by an elected
// thread (by lane 0 of a diverged warp they took three times as long); two warps load, as one does not keep
// up with 2 KB copies of pages of 16 positions; they share a ring, whose stages serve either.
//
// Measured: chunks of 2048 tokens over 30 to 63 thousand positions, 32 heads of 128, 4 key heads: 2.12 to 2.32 ms
// from run to run (the power limit), 1.36 to 1.49 PFLOP/s.  32 prompts of 2048, 16 heads of 64: 451 us, 610
// TFLOP/s, bound by the softmax's latency: a step of 256 rows takes 1.86 us, in tiles of 512 steps 1.77 us, so it
// is not what a tile begins and ends with.  A subtile's step is 4096 exponentials a quarter of an SM (8 a clock,
// 512 cycles), loads and stores of tensor memory, and the wait for its next scores.  48 requests of 1 to 8 tokens
// over 500 to 16000 positions: 158 us, 5.2 TB/s.  Where the compiler puts code moves short tiles by up to 15%
// (a limit of the waits that was read from the arguments: 470 -> 540 us).
//
// The maximum is kept lazily: it is raised, and the sums so far rescaled in tensor memory, only when
// a score passes it by more than 2^8.  The weights are rounded to bf16 for the product with
// the values (2^-8 of a weight at most, which the rounding of the outputs equals); their sums are fp32
// sums of the unrounded ones.
//
// Values that a row does not see have weight 0, but 0 times an infinity or NaN is no 0.
// So in tiles that some row sees in part, warps 12 to 15 clear the value rows that no row
// sees, and replace what is not finite in those that some rows see by 0; a row that does see such an
// element gets NaN in that column at the end.  Value rows that all rows see stay as they are.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "la_common.cuh"
#include "la_launch.h"
#include "la_plan.h"
#include "prefill_plan.cuh"
#include "tc_common.cuh"

namespace la {
namespace {

using namespace la::tc;
using prefill::Args;
using prefill::Keys;
using prefill::Request;
using prefill::Segment;
using prefill::token_of;
using bf16 = __nv_bfloat16;

constexpr int TM = 256, KT = 128, NT = 512;
constexpr int kAux = 128;             // threads of warps 12 to 15
constexpr int kMasks = 16;            // steps whose masks are kept: more than the loader is ahead of the softmax
constexpr float kSlack = 8.f;         // log2 by which a score may pass the maximum kept
constexpr uint32_t kAtom = 16384;     // 128 rows x 128 bytes
// Polls of a wait for another role (a poll that fails takes 3.4 us, so about a minute; the queries' warps wait as long as
// a tile takes, a second for 10^8 positions), and of one for what is under way when a block ends: microseconds.
constexpr uint32_t kLimit = tcf::kWaitLimit, kDrain = 1u << 16;

template <int D>
struct Lay {
    static constexpr int DP = D == 128 ? 128 : 64;  // columns in shared memory: heads of 32 are padded with zeros
    static constexpr int ATOMS = DP / 64;
    static constexpr int TILE = ATOMS * kAtom;      // bytes of 128 rows
    static constexpr int STAGES = D == 128 ? 5 : 8;
    static constexpr int Q = 2 * TILE;
    static constexpr int SMEM = Q + STAGES * TILE + 1024;
    // Copies of the products' code, one for both subtiles or one each.  The whole kernel's code is more than the
    // instruction memory next to an SM's quarters holds, and short tiles run through most of it, so less of it is faster;
    // over long tiles the products' few addresses count.  Measured, us, with one and two: 32 x 2048 of 16 heads of 64 460,
    // 510; of 128, 256 over 65k of 16 heads 131, 127, long chunks 2277, 2199.
    static constexpr int COPIES = DP == 64 ? 1 : 2;
    static constexpr uint32_t T_O = 256;            // column of subtile 0's outputs in tensor memory
    // How often a stage has held values before tile `it` (an odd one) of the ring: keys and values
    // take turns in a stage if the stages are odd in number.
    __device__ static __forceinline__ uint32_t value_turn(uint32_t it) { return STAGES % 2 ? it / STAGES / 2 : it / STAGES; }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// (a0, a1) * (b, b) + (c, c)
__device__ __forceinline__ float2 fma2(float a0, float a1, float b, float c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %4};\n\tmov.b64 z, {%5, %5};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a0), "f"(a1), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// 32 columns of the thread's row, not waited for.
__device__ __forceinline__ void ld32(uint32_t taddr, float* v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// The wait for the loads above; their registers pass through it, so that no use moves before it.
__device__ __forceinline__ void ld_wait(float* v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 128; ++i) asm volatile("" : "+f"(v[i]));
}
// 32 bytes of a thread, at a 32-byte boundary if `wide`.
__device__ __forceinline__ void store32(void* to, const uint32_t (&v)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                     "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(to)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(to)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}
// 16 words of the thread's row, not waited for.
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Bits lo .. hi of a word, those of them that it has.
__device__ __forceinline__ uint32_t span(int lo, int hi) {
    const uint32_t to = hi < 0 ? 0u : hi >= 31 ? 0xFFFFFFFFu : (2u << hi) - 1u;
    return lo <= 0 ? to : lo > 31 ? 0u : to & (0xFFFFFFFFu << lo);
}
// Bits 15 and 31 where one of two bf16 values is an infinity or NaN (all exponent bits set).
__device__ __forceinline__ uint32_t not_finite2(uint32_t pair) { return ((pair & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// One lane of the warp, always the same: the compiler sees a single thread in what follows.
__device__ __forceinline__ bool elect() {
    uint32_t on;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(on));
    return on != 0;
}

// x * 0 + z for two bf16 values.
__device__ __forceinline__ uint32_t zero2(uint32_t x, uint32_t z) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(x), "r"(0u), "r"(z));
    return r;
}

// Products over K = 128 (or 64) elements in steps of 16, issued by one thread.  S += Q K^T: both operands
// with K along rows of 128 bytes, 64 elements an atom column.
#define LA_MMA_SS(A, B) "tcgen05.mma.cta_group::1.kind::f16 [%0], " A ", " B ", %3, q;\n\t"
#define LA_MMA_SS_NEXT(N) "add.s64 a, %1, " N ";\n\tadd.s64 b, %2, " N ";\n\t" LA_MMA_SS("a", "b")
template <int STEPS>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    static_assert(STEPS == 4 || STEPS == 8, "64 or 128 columns");
    if constexpr (STEPS == 4)
        asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, 0, 0;\n\tsetp.eq.u32 q, 0, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
                     LA_MMA_SS_NEXT("2") LA_MMA_SS_NEXT("4") LA_MMA_SS_NEXT("6") "}" ::"r"(d), "l"(a), "l"(b), "r"(idesc) : "memory");
    else
        asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, 0, 0;\n\tsetp.eq.u32 q, 0, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
                     LA_MMA_SS_NEXT("2") LA_MMA_SS_NEXT("4") LA_MMA_SS_NEXT("6") LA_MMA_SS_NEXT("1024") LA_MMA_SS_NEXT("1026")
                     LA_MMA_SS_NEXT("1028") LA_MMA_SS_NEXT("1030") "}" ::"r"(d), "l"(a), "l"(b), "r"(idesc) : "memory");
}
// O += P V over 128 keys: P from tensor memory (8 columns a step), V with keys along atoms of 2048 bytes.
#define LA_MMA_TS_NEXT(N, M) "add.s32 a, %1, " N ";\n\tadd.s64 b, %2, " M ";\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, q;\n\t"
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 q, 0, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
                 LA_MMA_TS_NEXT("8", "128") LA_MMA_TS_NEXT("16", "256") LA_MMA_TS_NEXT("24", "384") LA_MMA_TS_NEXT("32", "512")
                 LA_MMA_TS_NEXT("40", "640") LA_MMA_TS_NEXT("48", "768") LA_MMA_TS_NEXT("56", "896") "}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(add)
                 : "memory");
}

// A segment of the block's range as its roles need it, worked out by one warp for all of them.
struct Job {
    Segment g;                    // g.rows < 0: no further one
    int row, cached, end;         // the request's first row of T, positions before its tokens, room of its table
    int k0, first, last, lo, hi;  // the tile's first step, positions of its first and last row, positions that it sees
    // Of each subtile: steps [a, b) of the tile's in which it takes part, rows, positions of its first and last row.
    int a[2], b[2], n[2], from[2], to[2];
    __device__ __forceinline__ void set(const Args& p, const Request& q, const Segment& s) {
        const Keys<KT> k(p, q, s.m0, min(s.m0 + TM, s.rows));
        g = s, row = q.first, cached = q.cached, end = q.end;
        k0 = k.k0, first = k.first, last = k.last, lo = k.lo, hi = k.hi;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            n[w] = min(max(s.rows - s.m0 - 128 * w, 0), 128);
            const int m = n[w] ? s.m0 + 128 * w : s.m0;
            const Keys<KT> y(p, q, m, m + max(n[w], 1));
            from[w] = y.first, to[w] = y.last;
            a[w] = max(s.a, y.k0 - k0);
            b[w] = max(a[w], n[w] ? min(s.b, y.k1 - k0) : a[w]);
        }
    }
};
constexpr int kJobs = 8;
constexpr int kReaders = 15;  // warps that read a job

template <int D>
__global__ void __launch_bounds__(NT, 1)
prefill_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
               const __grid_constant__ CUtensorMap qmap, const bf16* __restrict__ q, const bf16* __restrict__ K,
               const bf16* __restrict__ V, bf16* __restrict__ out, const Args p, const int q_tma, const int kv_tma) {
    using Ly = Lay<D>;
    constexpr int DP = Ly::DP, ATOMS = Ly::ATOMS, STAGES = Ly::STAGES;
    using Plan = prefill::Planner<TM, KT, NT>;
    using Walk = prefill::Walk<TM, KT>;
    extern __shared__ uint8_t sm_raw[];
    __shared__ uint64_t s_full[STAGES], s_empty[STAGES], s_vready[STAGES];
    __shared__ Job s_jobs[kJobs];
    __shared__ uint64_t s_jfull[kJobs], s_jfree[kJobs];
    __shared__ uint64_t s_qfull, s_qempty, s_sfull[2], s_pfull[2], s_odone[2], s_end;
    __shared__ uint32_t s_mask[2][kMasks][4];  // positions of a step that are on a page, a bit each, as keys' and values' loader saw them
    // A value that was not finite was replaced, in this or an earlier segment, or in a later one: it stays set, as the
    // warps that replace may be segments ahead of a subtile's outputs.  So it only says whether to look.
    __shared__ volatile int s_odd;
    __shared__ volatile int s_abort;
    __shared__ volatile int s_issued[2];     // tiles of keys, of values that their loaders have begun
    __shared__ uint32_t s_tmem;
    __shared__ prefill::Range s_range;
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint8_t* ring = sm + Ly::Q;
    const int tid = threadIdx.x, lane = tid & 31, warp = (tid >> 5) ^ 8;  // by role
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) mbar_init(s_full + i, 1), mbar_init(s_empty + i, 1), mbar_init(s_vready + i, kAux / 32);
        for (int i = 0; i < kJobs; ++i) mbar_init(s_jfull + i, 1), mbar_init(s_jfree + i, kReaders);
        mbar_init(&s_qfull, kAux / 32);
        mbar_init(&s_qempty, 1);
        mbar_init(&s_end, 1);
        for (int w = 0; w < 2; ++w) mbar_init(s_sfull + w, 1), mbar_init(s_pfull + w, 4), mbar_init(s_odone + w, 1);
        s_abort = 0, s_odd = 0, s_issued[0] = 0, s_issued[1] = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&s_tmem, 512);
        tmem_relinquish();
    }
    if (tid < 2) p.desc[2 * blockIdx.x + tid] = make_int4(0, 0, 0, 0);
    Plan& plan = *reinterpret_cast<Plan*>(sm);  // before anything else is in there
    plan.run(p);
    if (tid == 0) s_range = plan.range;
    fence_before_sync();
    fence_proxy_async();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = s_tmem;
    const prefill::Range range = s_range;
    const auto fail = [&]() {
        s_abort = 1;
        atomicOr(p.status, tcf::kErrWait);
    };
    // Waits give up after kLimit polls, or once any of them has.
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
        const int e = mbar_wait_or(bar, parity & 1u, kLimit, const_cast<const volatile int*>(&s_abort));
        if (e == 2) fail();
        return e == 0;
    };
    const auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity & 1u))) return true;
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };

    // The role's next segment, copied; its place is free then.
    uint32_t n_job = 0;
    const auto next = [&](Job& x) {
        const uint32_t at = n_job % kJobs;
        if (!warp_wait(s_jfull + at, n_job / kJobs)) return false;
        x = s_jobs[at];
        __syncwarp();
        if (lane == 0) mbar_arrive(s_jfree + at);
        ++n_job;
        return x.g.rows >= 0;
    };

    // The launch's 128 registers a thread become 192 for the softmax and 64 for the rest.
    if (range.any) {
        if (warp < 8) {
            // ---------------------------------------------------------------- softmax
            asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
            const int w = warp >> 2, row = 32 * (warp & 3) + lane;
            const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // the warp's quarter of the lanes
            const uint32_t ts = tm + 128 * w + lanes, to = tm + Ly::T_O + DP * w + lanes;
            const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
            const float c = fabsf(p.s.scale) * 1.4426950408889634f;
            uint32_t n_s = 0, n_o = 0, step = 0;  // phases seen, steps of the block
            for (Job x; next(x);) {
                const Segment& g = x.g;
                const int k0 = x.k0, m = g.m0 + 128 * w + row;
                const int part_a = w ? x.a[1] : x.a[0], part_b = w ? x.b[1] : x.b[0];
                const int part_from = w ? x.from[1] : x.from[0], part_to = w ? x.to[1] : x.to[0];
                const bool live = row < (w ? x.n[1] : x.n[0]);
                const int pos = x.cached + token_of(p, m);             // of the row
                const int from = p.s.window ? pos - p.s.window : -1;  // it sees positions past this one
                float top = -INFINITY, sum = 0.f;
                bool ok = true;
                for (int j = g.a; j < g.b; ++j, ++step) {
                    if (j < part_a || j >= part_b) continue;
                    if (!(ok = warp_wait(s_sfull + w, n_s++))) break;
                    fence_after_sync();
                    float s[128];
#pragma unroll
                    for (int i = 0; i < 4; ++i) ld32(ts + 32 * i, s + 32 * i);
                    const int x0 = (k0 + j) * KT;
                    const uint32_t* mask = s_mask[0][step % kMasks];
                    const uint32_t m0 = mask[0], m1 = mask[1], m2 = mask[2], m3 = mask[3];
                    const bool all = x0 + KT - 1 <= part_from && (p.s.window == 0 || x0 > part_to - p.s.window) &&
                                     (m0 & m1 & m2 & m3) == 0xFFFFFFFFu;
                    ld_wait(s);
                    if (!all) {
                        const int c0 = from + 1 - x0, c1 = pos - x0;  // columns [c0, c1] of the tile are seen
                        const uint32_t bits[4] = {m0 & span(c0, c1), m1 & span(c0 - 32, c1 - 32), m2 & span(c0 - 64, c1 - 64),
                                                  m3 & span(c0 - 96, c1 - 96)};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (__all_sync(0xffffffffu, bits[i] == 0xFFFFFFFFu)) continue;
#pragma unroll
                            for (int x = 0; x < 32; ++x) s[32 * i + x] = bits[i] & (1u << x) ? s[32 * i + x] : -INFINITY;
                        }
                    }
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx[i] = fmaxf(s[i], s[4 + i]);
#pragma unroll
                    for (int i = 8; i < 128; i += 8)
#pragma unroll
                        for (int x = 0; x < 4; ++x) mx[x] = max3(mx[x], s[i + x], s[i + 4 + x]);
                    const float best = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * c;
                    const bool raise = best > top + kSlack;  // also from -infinity
                    if (__any_sync(0xffffffffu, raise)) {
                        const float f = raise ? (top == -INFINITY ? 0.f : ex2(top - best)) : 1.f;
                        if (raise) top = best;
                        sum *= f;
                        if (j > part_a) {  // the product before this one has finished: the scores came behind it
#pragma unroll 1
                            for (int i = 0; i < DP; i += 16) {
                                float o[16];
                                tmem_ld16(to + i, o);
#pragma unroll
                                for (int x = 0; x < 16; ++x) o[x] *= f;
                                tmem_st16(to + i, o);
                            }
                        }
                    }
                    const float base = top == -INFINITY ? 0.f : -top;
                    float2 t0 = make_float2(0.f, 0.f), t1 = t0;
#pragma unroll
                    for (int i = 0; i < 128; i += 32) {
                        uint32_t pk[16];
#pragma unroll
                        for (int x = 0; x < 16; x += 2) {
                            float2 a = fma2(s[i + 2 * x], s[i + 2 * x + 1], c, base);
                            float2 b = fma2(s[i + 2 * x + 2], s[i + 2 * x + 3], c, base);
                            a.x = ex2(a.x), a.y = ex2(a.y), b.x = ex2(b.x), b.y = ex2(b.y);
                            t0 = add2(t0, a);
                            t1 = add2(t1, b);
                            pk[x] = pack_bf16(a.x, a.y);
                            pk[x + 1] = pack_bf16(b.x, b.y);
                        }
                        st16(ts + i / 2, pk);
                    }
                    t0 = add2(t0, t1);
                    sum += t0.x + t0.y;
                    st_wait();
                    fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_pfull + w);
                }
                if (!ok) break;
                // ------------------------------------------------------------ the rows' outputs
                const bool some = part_b > part_a;
                if (some) {
                    if (!warp_wait(s_odone + w, n_o++)) break;
                    fence_after_sync();
                }
                const bool whole = g.whole();
                const int slot = 2 * blockIdx.x + (g.a == 0 ? 1 : 0);
                const bool good = sum > 0.f || sum != sum;
                const float inv = !whole ? 1.f : good ? 1.f / sum : 0.f;
                const int token = token_of(p, m);
                const int64_t at = (static_cast<int64_t>(x.row) + token) * p.s.Hq + static_cast<int64_t>(g.kh) * p.G + (m - token * p.G);
                float* part = p.part + (static_cast<int64_t>(slot) * TM + 128 * w + row) * D;
#pragma unroll 1
                for (int i = 0; i < D; i += 32) {
                    float o[32];
                    if (some) {
                        tmem_ld32(to + i, o);
                    } else {
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = 0.f;
                    }
                    if (s_odd) {  // rare: does this row see one of the replaced values?
                        uint32_t bits = 0;
                        for (int j = part_a; live && j < part_b; ++j)
                            bits |= prefill::odd_columns<bf16, D, KT, false>(p, V, g.r, g.kh, x.first, x.last, x.end, k0 + j, from, pos, i);
#pragma unroll
                        for (int x = 0; x < 32; ++x)
                            if (bits >> x & 1u) o[x] = __uint_as_float(0x7FFFFFFFu);
                    }
                    if (live) {
#pragma unroll
                        for (int x = 0; x < 32; x += 16) {
                            uint32_t v[8];
                            if (whole) {
#pragma unroll
                                for (int y = 0; y < 8; ++y) v[y] = pack_bf16(o[x + 2 * y] * inv, o[x + 2 * y + 1] * inv);
                                store32(out + at * D + i + x, v, wide);
                            } else {
#pragma unroll
                                for (int h = 0; h < 16; h += 8) {
#pragma unroll
                                    for (int y = 0; y < 8; ++y) v[y] = __float_as_uint(o[x + h + y]);
                                    store32(part + i + x + h, v, true);
                                }
                            }
                        }
                    }
                    __syncwarp();
                }
                if (live) {
                    if (!whole) p.ml[static_cast<int64_t>(slot) * TM + 128 * w + row] = make_float2(top, sum);
                    else if (p.lse) p.lse[at] = good ? (top + log2f(sum)) * 0.6931471805599453f : -INFINITY;
                }
                fence_before_sync();  // the outputs' columns are free with the next arrival
            }
        } else {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
            if (warp == 8) {
            // ---------------------------------------------------------------- products
            constexpr uint32_t ID_S = idesc_bf16(128, 128, false, false), ID_O = idesc_bf16(128, DP, false, true);
            const uint64_t dq = sdesc(smem_u32(sm), 16, 1024), dk = sdesc(smem_u32(ring), 16, 1024), dv = sdesc(smem_u32(ring), kAtom, 1024);
            constexpr uint32_t STEP = Ly::TILE >> 4;  // of a descriptor, from tile to tile
            uint32_t n_q = 0, n_p = 0, sk = 0, tk = 0, sv = 1, n_v = 0;  // stages of the next keys and values, turns of the ring, value tiles
            bool ok = true;
            for (Job x; ok && next(x);) {
                const Segment& g = x.g;
                if (!(ok = warp_wait(&s_qfull, n_q++) && warp_wait(s_full + sk, tk))) break;
                fence_after_sync();
                if (elect()) {
                    const uint64_t k = dk + sk * STEP;
#pragma unroll 1
                    for (int w = 0; w < 2; ++w)
                        if (g.a >= (w ? x.a[1] : x.a[0]) && g.a < (w ? x.b[1] : x.b[0])) {
                            mma_scores<DP / 16>(tm + 128 * w, dq + w * STEP, k, ID_S);
                            mma_commit(s_sfull + w);
                        }
                    mma_commit(s_empty + sk);
                    if (g.a + 1 == g.b) mma_commit(&s_qempty);
                }
                __syncwarp();
                if ((sk += 2) >= STAGES) sk -= STAGES, ++tk;
                for (int j = g.a; j < g.b; ++j, ++n_v) {
                    const bool more = j + 1 < g.b;
                    // the values of this step and the keys of the next, mostly here before the weights
                    if (!(ok = warp_wait(s_vready + sv, Ly::value_turn(2 * n_v + 1)))) break;
#pragma unroll Ly::COPIES
                    for (int w = 0; w < 2; ++w) {
                        const int part_a = w ? x.a[1] : x.a[0], part_b = w ? x.b[1] : x.b[0];
                        const bool on = j >= part_a && j < part_b, on_next = j + 1 >= part_a && j + 1 < part_b;
                        if (on && !(ok = warp_wait(s_pfull + w, n_p >> w & 1u))) break;
                        if (on) n_p ^= 1u << w;
                        fence_after_sync();
                        if (elect()) {
                            if (on) mma_values(tm + Ly::T_O + DP * w, tm + 128 * w, dv + sv * STEP, ID_O, j > part_a ? 1u : 0u);
                            if (more && on_next) {
                                mma_scores<DP / 16>(tm + 128 * w, dq + w * STEP, dk + sk * STEP, ID_S);
                                mma_commit(s_sfull + w);
                            }
                            if (on && j + 1 == part_b) mma_commit(s_odone + w);
                            if (w == 1) {
                                mma_commit(s_empty + sv);
                                if (more) mma_commit(s_empty + sk);
                                if (j + 2 == g.b) mma_commit(&s_qempty);
                            }
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    if ((sv += 2) >= STAGES) sv -= STAGES;
                    if (more && (sk += 2) >= STAGES) sk -= STAGES, ++tk;
                }
            }
            // nothing may be under way when the block ends
            if (elect()) mma_commit(&s_end);
            __syncwarp();
            if (!mbar_wait(&s_end, 0, kDrain)) fail();
        } else if (warp < 11) {
            // ---------------------------------------------------------------- keys (warp 9), values (warp 10)
            const int kv = warp - 9;
            const bf16* pool = kv ? V : K;
            const CUtensorMap* map = kv ? &vmap : &kmap;
            const int log2p = p.s.log2p, page = 1 << log2p, off_mask = page - 1;
            const int rows = min(page, KT);              // of a copy
            const int copies = KT / rows;                // of a tile
            uint32_t it = kv, step = 0;                  // the ring's tiles: K, V, K, V, ...
            bool ok = true, bad = false;
            // With an odd number of stages keys and values take turns in each.  A stage's phase then tells whether it
            // is free only once the other loader has begun its last turn there.
            const auto in_turn = [&](uint32_t tile) {
                if (STAGES % 2 == 0) return true;
                const int need = tile < STAGES ? 0 : static_cast<int>(tile - STAGES) / 2 + 1;
                uint32_t i = 0;
                while (s_issued[1 - kv] < need && !s_abort && ++i < kLimit) {}
                if (i == kLimit) fail();
                const bool there = s_issued[1 - kv] >= need;
                __threadfence_block();
                return __all_sync(0xffffffffu, there) != 0;
            };
            for (Job k; ok && next(k);) {
                const Segment& g = k.g;
                const int* table = p.table + static_cast<int64_t>(g.r) * p.s.max_pages;
                // Page i of the request; -1 if it is none of the pool, -2 if no row sees a position of it.
                const auto page_of = [&](int64_t i) {
                    if ((i << log2p) >= k.hi || ((i + 1) << log2p) <= k.lo) return -2;
                    const int id = table[i];
                    return static_cast<unsigned>(id) < static_cast<unsigned>(p.s.num_pages) ? id : -1;
                };
                // Page numbers are fetched 32 at a time, a group ahead.
                int group = ((k.k0 + g.a) * KT >> log2p) >> 5;
                int now = -2, next = -2;
                if (kv_tma) now = page_of(32ll * group + lane), next = page_of(32ll * group + 32 + lane);
                for (int j = g.a; j < g.b; ++j, ++step, it += 2) {
                    const int x0 = (k.k0 + j) * KT, first = x0 >> log2p;
                    const uint32_t sg = it % STAGES;
                    if (kv_tma) {
                        if (first >> 5 != group) {
                            group = first >> 5;
                            now = next;
                            next = page_of(32ll * group + 32 + lane);
                        }
                        const uint32_t in = ((1u << copies) - 1u) << (first & 31);
                        if (!(ok = in_turn(it))) break;
                        const uint32_t who = __ballot_sync(0xffffffffu, now >= 0) & in;
                        const uint32_t lost = (__ballot_sync(0xffffffffu, now == -1) & in) >> (first & 31);
                        bad |= lost != 0;
                        if (!(ok = warp_wait(s_empty + sg, it / STAGES + 1))) break;
                        if (lane < 4) {  // 32 positions a word: those on a lost page, or past the table, are off
                            uint32_t m = 0xFFFFFFFFu;
                            for (int i = 0; i < 32 && (lost || x0 + KT > k.end); ++i) {
                                const int y = 32 * lane + i;
                                if ((lost >> (y / rows) & 1u) || x0 + y >= k.end) m &= ~(1u << i);
                            }
                            s_mask[kv][step % kMasks][lane] = m;
                        }
                        __syncwarp();
                        const bool one = elect();
                        if (one) {
                            if (who) mbar_arrive_expect_tx(s_full + sg, __popc(who) * rows * ATOMS * 128);
                            else mbar_arrive(s_full + sg);
                        }
                        uint8_t* dst = ring + sg * Ly::TILE;
                        for (int c = 0; c < copies; ++c, dst += rows * 128) {
                            const int to = __shfl_sync(0xffffffffu, now, (first + c) & 31);
                            if (to >= 0 && one) {
#pragma unroll
                                for (int a = 0; a < ATOMS; ++a)
                                    tma_load_3d(dst + a * kAtom, map, s_full + sg, 64 * a, x0 & off_mask, to * p.s.Hkv + g.kh);
                            }
                        }
                    } else {
                        // pages of fewer than eight positions: four rows a lane, 16 bytes at a time
                        int ids[4];
                        uint32_t mask[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int y = x0 + 32 * i + lane;
                            ids[i] = page_of(y >> log2p);
                            bad |= ids[i] == -1;
                            mask[i] = __ballot_sync(0xffffffffu, ids[i] != -1 && y < k.end);
                        }
                        if (!(ok = in_turn(it))) break;
                        if (!(ok = warp_wait(s_empty + sg, it / STAGES + 1))) break;
                        const uint32_t dst = smem_u32(ring + sg * Ly::TILE);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int y = 32 * i + lane;
                            const int64_t src = ids[i] < 0 ? 0 : (((static_cast<int64_t>(ids[i]) * p.s.Hkv + g.kh) << log2p) + ((x0 + y) & off_mask)) * D;
                            for (int e = 0; e < DP / 8; ++e) {
                                const bool on = ids[i] >= 0 && e < D / 8;
                                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + (e >> 3) * kAtom + swz(y, e & 7)),
                                             "l"(on ? pool + src + e * 8 : q), "r"(on ? 16 : 0)
                                             : "memory");
                            }
                        }
                        asm volatile("cp.async.wait_all;" ::: "memory");
                        if (lane == 0)
                            for (int i = 0; i < 4; ++i) s_mask[kv][step % kMasks][i] = mask[i];
                        fence_proxy_async();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(s_full + sg);
                    }
                    if (STAGES % 2 && lane == 0) s_issued[kv] = static_cast<int>(it / 2) + 1;
                }
            }
            if (bad) atomicOr(p.status, kStatusBadIndex);
            // copies under way end before the block does: the last ones of each stage (it is the first tile not issued)
            for (uint32_t i = it > 2 * STAGES ? it - 2 * STAGES : kv; i < it; i += 2)
                if (i + STAGES >= it && !mbar_wait(s_full + i % STAGES, i / STAGES & 1u, kDrain)) fail();
        } else if (warp == 11) {
            // ---------------------------------------------------------------- the segments, for all
            Walk walk(p, range);
            Segment g;
            bool any = true;
            for (uint32_t i = 0; any; ++i) {
                const Request rq = walk.q;  // of the segment that comes (only the last can be without a step)
                any = walk.next(p, g);
                Job x;
                x.g.rows = -1;
                if (any) x.set(p, rq, g);
                if (!warp_wait(s_jfree + i % kJobs, i / kJobs + 1)) break;
                if (lane == 0) s_jobs[i % kJobs] = x;
                __syncwarp();
                if (lane == 0) mbar_arrive(s_jfull + i % kJobs);
            }
        } else {
            // ---------------------------------------------------------------- queries, values seen in part
            const int t = 32 * (warp - 12) + lane;
            uint32_t item = 0, n_q = 0, step = 0;
            bool ok = true;
            if (warp == 12 && static_cast<int>(blockIdx.x) == p.withhold) {
                // (test hook) no queries come: this wait for them gives up, and with it all the others
                if (!mbar_wait(&s_qfull, 0, p.limit)) fail();
                ok = false;
            }
            for (Job k; ok && next(k);) {
                const Segment& g = k.g;
                if (n_q && !(ok = warp_wait(&s_qempty, n_q - 1))) break;
                ++n_q;
                const int subs = g.rows - g.m0 > 128 ? 2 : 1;
                if (q_tma) {
                    if (t == 0) {
                        mbar_arrive_expect_tx(&s_qfull, subs * Ly::TILE);  // (one of the barrier's arrivals, the others are the other warps')
                        for (int w = 0; w < subs; ++w)
                            for (int a = 0; a < ATOMS; ++a)
                                tma_load_3d(sm + w * Ly::TILE + a * kAtom, &qmap, &s_qfull, 64 * a, g.kh * p.G, k.row + token_of(p, g.m0 + 128 * w));
                    } else if (lane == 0) {
                        mbar_arrive(&s_qfull);
                    }
                } else {
                    // any number of heads, or a negative scale: 16 bytes at a time, the sign turned here
                    const uint32_t flip = p.s.scale < 0.f ? 0x80008000u : 0u;
                    constexpr int CH = DP / 8;
                    for (int i0 = t; i0 < subs * 128 * CH; i0 += kAux * 4) {
                        uint4 x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = i0 + kAux * i, y = e / CH, ch = e % CH, m = g.m0 + y;
                            x[i] = make_uint4(0u, 0u, 0u, 0u);
                            const int token = token_of(p, m);
                            if (m < g.rows && ch < D / 8)
                                x[i] = *reinterpret_cast<const uint4*>(
                                    q + ((static_cast<int64_t>(k.row) + token) * p.s.Hq + static_cast<int64_t>(g.kh) * p.G + (m - token * p.G)) * D + ch * 8);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = i0 + kAux * i, y = e / CH, ch = e % CH;
                            x[i].x ^= flip, x[i].y ^= flip, x[i].z ^= flip, x[i].w ^= flip;
                            *reinterpret_cast<uint4*>(sm + (y >> 7) * Ly::TILE + (ch >> 3) * kAtom + swz(y & 127, ch & 7)) = x[i];
                        }
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_qfull);
                }
                if (!(ok = warp_wait(s_full + item % STAGES, item / STAGES))) break;  // every tile of the ring, so that no phase is missed
                for (int j = g.a; ok && j < g.b; ++j, ++step, item += 2) {
                    const uint32_t v = item + 1, sg = v % STAGES;
                    if (!(ok = warp_wait(s_full + sg, v / STAGES))) break;
                    const int x0 = (k.k0 + j) * KT;
                    const uint32_t* mask = s_mask[1][step % kMasks];
                    const bool all = x0 + KT - 1 <= k.first && (p.s.window == 0 || x0 > k.last - p.s.window) &&
                                     (mask[0] & mask[1] & mask[2] & mask[3]) == 0xFFFFFFFFu;
                    if (!all) {
                        uint8_t* tile = ring + sg * Ly::TILE;
                        bool odd = false;
                        // rows that every row sees, [in0, in1), stay as they are
                        const int in0 = p.s.window ? k.last - p.s.window + 1 - x0 : 0, in1 = k.first + 1 - x0;
#pragma unroll 1
                        for (int e = t; e < 128 * ATOMS; e += kAux) {  // 128 bytes of a row
                            const int y = e & 127, x = x0 + y;
                            const bool lost = x < k.lo || x >= k.hi || !(mask[y >> 5] >> (y & 31) & 1u);
                            if (!lost && y >= in0 && y < in1) continue;
                            uint4* at = reinterpret_cast<uint4*>(tile + e * 128);
                            if (lost) {
#pragma unroll
                                for (int i = 0; i < 8; ++i) at[i ^ (t & 7)] = make_uint4(0u, 0u, 0u, 0u);  // each lane another bank
                                continue;
                            }
                            uint4 u[8];
                            uint32_t z0 = 0, z1 = 0;  // 0, or NaN after a value that is not finite
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                u[i] = at[i ^ (t & 7)];
                                z0 = zero2(u[i].x, z0), z1 = zero2(u[i].y, z1), z0 = zero2(u[i].z, z0), z1 = zero2(u[i].w, z1);
                            }
                            if (!(not_finite2(z0) | not_finite2(z1))) continue;
                            odd = true;
#pragma unroll 1
                            for (int i = 0; i < 8; ++i) {
                                uint32_t* z = reinterpret_cast<uint32_t*>(at + i);
                                for (int w = 0; w < 4; ++w) {
                                    const uint32_t b = not_finite2(z[w]);
                                    z[w] &= ~((b & 0x8000u ? 0xFFFFu : 0u) | (b & 0x80000000u ? 0xFFFF0000u : 0u));
                                }
                            }
                        }
                        if (odd) s_odd = 1;
                        fence_proxy_async();
                    }
                    // and the next step's keys, so that the products wait once
                    if (j + 1 < g.b && !(ok = warp_wait(s_full + (v + 1) % STAGES, (v + 1) / STAGES))) break;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_vready + sg);
                }
            }
            if (q_tma && n_q && t == 0 && !mbar_wait(&s_qfull, (n_q - 1) & 1u, kDrain)) fail();
        }
        }
    }
    prefill::finish_range<bf16, D, TM, KT, NT>(p, range, !s_abort, out);
    fence_before_sync();
    __syncthreads();
    if (warp == 8) {
        fence_after_sync();
        tmem_dealloc(tm, 512);
    }
}

cudaError_t encode(CUtensorMap* m, const void* base, const cuuint64_t (&dims)[3], const cuuint32_t (&box)[3]) {
    tcf::EncodeTiled enc = tcf::encoder();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t strides[2] = {dims[0] * 2, dims[0] * dims[1] * 2};
    cuuint32_t es[3] = {1, 1, 1};
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

size_t paged_prefill_tc_scratch(int D, int num_sms) { return prefill::scratch_bytes(D, TM, num_sms); }

template <int D>
cudaError_t paged_prefill_tc(const LaunchCtx& c, const bf16* q, const bf16* K, const bf16* V, const int* table,
                             const int* lens, const int* starts, bf16* out, float* lse, const PrefillShape& s, int fill) {
    using Ly = Lay<D>;
    Args p = {};
    prefill::set_group(p, s.Hq / s.Hkv, TM);
    p.s = s, p.table = table, p.lens = lens, p.starts = starts, p.lse = lse, p.fill = fill;
    p.status = c.status_word;
    p.withhold = c.withhold_unit;
    p.limit = c.spin_limit;
    int per_sm = 1;
    cudaError_t e = resident_blocks<prefill_kernel<D>>(c.device, NT, Ly::SMEM, &per_sm);
    if (e != cudaSuccess) return e;
    CUtensorMap kmap = {}, vmap = {}, qmap = {};
    const int page = 1 << s.log2p;
    const int kv_tma = s.log2p >= 3 && s.num_pages > 0 && static_cast<int64_t>(s.num_pages) * s.Hkv < INT_MAX;
    if (kv_tma) {
        const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(page), static_cast<cuuint64_t>(s.num_pages) * s.Hkv};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(std::min(page, KT)), 1};
        if ((e = encode(&kmap, K, dims, box)) != cudaSuccess || (e = encode(&vmap, V, dims, box)) != cudaSuccess) return e;
    }
    const int q_tma = s.scale > 0.f && p.G <= 128 && 128 % p.G == 0;
    if (q_tma) {
        const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(s.Hq), static_cast<cuuint64_t>(s.T)};
        const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(128 / p.G)};
        if ((e = encode(&qmap, q, dims, box)) != cudaSuccess) return e;
    }
    uint8_t* base = nullptr;
    if ((e = scratch_alloc(c, reinterpret_cast<void**>(&base), paged_prefill_tc_scratch(D, c.num_sms))) != cudaSuccess) return e;
    prefill::set_scratch(p, base, D, TM, c.num_sms);
    prefill_kernel<D><<<c.num_sms, NT, Ly::SMEM, c.stream>>>(kmap, vmap, qmap, q, K, V, out, p, q_tma, kv_tma);
    note_launch();
    e = cudaGetLastError();
    if (e == cudaSuccess) e = prefill::launch_join<bf16, D, TM>(p, out, c.num_sms, c.stream);
    scratch_free(c, base);
    return e;
}

#define LA_INST_PT(D)                                                                                                   \
    template cudaError_t paged_prefill_tc<D>(const LaunchCtx&, const bf16*, const bf16*, const bf16*, const int*, \
                                             const int*, const int*, bf16*, float*, const PrefillShape&, int);
LA_INST_PT(32) LA_INST_PT(64) LA_INST_PT(128)

}  // namespace la
