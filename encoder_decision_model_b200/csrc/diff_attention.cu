// Differential attention over packed rows: D = softmax(Q0 K0^T) V - lambda softmax(Q1 K1^T) V, with
// each head's RMS norm and gain in the same launch.
//
// One pass over the keys with the running maximum and sum of both softmaxes.  A work item is 128
// queries of one row and head; its two maps run side by side, as two query tiles of an ordinary
// attention would, over the same 128-wide V tiles:
//
//   warp 0          TMA producer: the item's Q_0, Q_1 (two buffers), K_0 and K_1 tiles of 64 keys (a ring
//                   of 8 KB units, freed when their S product completes), V tiles (64 keys x 128, a
//                   ring of 16 KB stages)
//   warp 1, warp 3  one lane issues the tcgen05.mma of map 0 and of map 1 (warp 1 holds the TMEM):
//                     S_x = Q_x K_x^T  (M 128, N 64, K 64)
//                     O_x += P_x V     (M 128, N 128, K 64; P from TMEM, V read MN-major)
//   warp 2          zeroes the rows of an item's last V tile that lie past its keys: their
//                   probabilities are 0, but 0 times what another row holds there may be NaN
//   warps 4..7      softmax of map 0, warps 8..11 of map 1: one query row a thread
//   warps 12..15    read-out: D, its norm and the output row, while the others are at the next item
//
// TMEM is full: O_0 and O_1 take 256 columns, and each map has two S tiles of 64 columns in turn, so
// that its next scores are there while it works on these; P_x overwrites its S tile (the thread that
// stores a row's P has read all of its S).
//
// Measured: 16 rows of 8192 with three heads and FP16 values 3.74 to 3.79 ms one after another (660
// TFLOP/s, 0.40 of the measured burst rate), single runs 3.3 to 3.6 ms; 256 rows of 64 to 1024 with BF16
// values 433 us in a few calls, 468 to 483 after hundreds in a row, with FP16 values 483 to 503; with a
// window of 64 and FP16 values 218 to 231 us.  On the long rows a step of 64 keys takes a softmax warp 2,080 clocks:
// 1,130 to 1,180 of exponentials, their rounding and packing (two warps a scheduler share the units), 290 to 320 waiting
// for S, 350 for its read and the maximum, 260 for handing P over.  What did not pay, each against the
// kernel as it was then: one thread issuing the MMAs of both maps (5.7 ms), or not elected by elect.sync
// (603 against 511 us on the ragged rows); one S tile of 128 keys a map, whose next product waits for P V
// (852 against 636 us there); two threads a row (long rows the same, ragged ones 10 % slower); asking
// for the next S before P is handed over (3.1 against 3.0 ms); a quarter of the exponentials as
// polynomials on the FMA pipe (2 to 8 % slower: the warps are bound by instructions and their
// latencies, not by the exponential unit alone).
//
// Floor: 768 FLOP and two exponentials a visible (query, key) pair and head; at 8192 FLOP and 16
// exponentials a clock and SM, 0.094 and 0.125 clocks (0.156 for the 1,280 FLOP that a pair P costs).
//
// Rounding of P.  P enters the PV product as a pair of 16-bit numbers hi + lo (lo in the S tile's other 32
// columns), twice the MMAs of PV: 2^-22 of it is lost in FP16, 2^-16 in BF16.  One number alone would lose 2^-11 or
// 2^-8, and D is a difference: where the two maps are alike the norm makes that up to (1 + lambda) / (1 - lambda)
// times larger, 9 times at the lambda of 0.8 of deep layers and without bound towards 1, however long the row.
// Emulated in 64 bits with P as one FP16 number, nearly equal maps and FP16 values, elements of a BF16 result were off by up
// to 47 half steps at lambda 0.8 and 160 at 0.95 (rows of 2 to 512 keys); with the pair the sums' own error is what is left.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "diff_attention.h"
#include "kernels.h"

namespace jd {

namespace {

constexpr int TQ = 128, TK = 64, VD = 128;
constexpr int Q_BYTES = TQ * 128;            // one map's queries: 128 rows x 64 elements of 16 bits
constexpr int K_BYTES = TK * 128;            // one map's keys
constexpr int V_HALF = TK * 128;             // 64 columns of a V tile
constexpr int V_BYTES = 2 * V_HALF;
constexpr int NK = 8, NV = 4;                // ring depths
constexpr int OFF_Q = 0;                     // [item buffer][map]
constexpr int OFF_K = OFF_Q + 4 * Q_BYTES;
constexpr int OFF_V = OFF_K + NK * K_BYTES;
constexpr int OFF_BAR = OFF_V + NV * V_BYTES;
constexpr int NBAR = 2 + 2 + 2 * NK + 3 * NV + 3 * 4 + 2 + 2 + 1;
constexpr int OFF_F = OFF_BAR + ((NBAR * 8 + 15) / 16) * 16;
// floats: gain[128], row sums [item % 2][map][128]; then the TMEM slot and a status word
constexpr int DIFF_SMEM = OFF_F + (128 + 2 * 256) * 4 + 16 + 1024;
static_assert(DIFF_SMEM <= 227 * 1024, "differential attention shared memory");
constexpr uint32_t T_S = 0, T_O = 256;
constexpr float kLazy = 8.0f;                // log2 headroom before a running max is moved: P <= 2^8
constexpr int THREADS = 16 * 32;
// The launch gives every thread REGS registers (the compiled count, checked on the host before the first
// launch: a warp group asking for more than the launch holds would wait for ever); the warp groups of the
// roles and of the read-out give up some, which the softmax groups take.
constexpr int REGS = 128, REGS_ROLES = 72, REGS_READOUT = 104, REGS_SOFTMAX = 160;
// After an expired wait: how long a block stays, for its copies and products in flight (microseconds, if they come at all).
constexpr int LINGER_STEPS = 100'000;
constexpr uint64_t LINGER_NS = 20'000'000;
constexpr int BAR_GAIN = 1;  // named barrier of the read-out warps
static_assert(128 * (REGS_ROLES + REGS_READOUT) + 256 * REGS_SOFTMAX <= THREADS * REGS, "register split");

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mov.b64 rc, {%6, %7};\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ void tma_load_heads(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int head, int token) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(head), "r"(token)
        : "memory");
}

// Matrix descriptors, 128-byte swizzle, eight rows 1024 bytes apart (stride).  Q and K: K-major.  V:
// MN-major, the next 64 elements V_HALF further on (leading).  The upper words are the same; adding
// to the lower word moves the start, in units of 16 bytes.
constexpr uint32_t DESC_HI = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t leading) {
    return ((saddr & 0x3FFFFu) >> 4) | (leading << 16);
}

// S = Q K^T over 64 elements: four steps of 16 (32 bytes of a row each), issued back to back.
__device__ __forceinline__ void mma_s(uint32_t d_tmem, uint32_t q_lo, uint32_t k_lo, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred on, off;\n\t.reg .b64 a0, a1, a2, a3, b0, b1, b2, b3;\n\t"
        "setp.eq.u32 on, 0, 0;\n\tsetp.ne.u32 off, 0, 0;\n\t"
        "mov.b64 a0, {%1, %4};\n\tmov.b64 b0, {%2, %4};\n\t"
        "add.u64 a1, a0, 2;\n\tadd.u64 b1, b0, 2;\n\tadd.u64 a2, a0, 4;\n\tadd.u64 b2, b0, 4;\n\t"
        "add.u64 a3, a0, 6;\n\tadd.u64 b3, b0, 6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a0, b0, %3, off;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, on;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, on;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, on;\n\t}" ::"r"(d_tmem),
        "r"(q_lo), "r"(k_lo), "r"(idesc), "n"(DESC_HI)
        : "memory");
}
// O (+)= P V over 64 keys: four steps of 16 (8 columns of P, 16 rows of V).
__device__ __forceinline__ void mma_pv(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred on, acc;\n\t.reg .b64 b0, b1, b2, b3;\n\t.reg .b32 p1, p2, p3;\n\t"
        "setp.eq.u32 on, 0, 0;\n\tsetp.ne.u32 acc, %4, 0;\n\t"
        "mov.b64 b0, {%2, %5};\n\tadd.u64 b1, b0, 128;\n\tadd.u64 b2, b0, 256;\n\tadd.u64 b3, b0, 384;\n\t"
        "add.u32 p1, %1, 8;\n\tadd.u32 p2, %1, 16;\n\tadd.u32 p3, %1, 24;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b0, %3, acc;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [p1], b1, %3, on;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [p2], b2, %3, on;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [p3], b3, %3, on;\n\t}" ::"r"(d_tmem),
        "r"(p_tmem), "r"(v_lo), "r"(idesc), "r"(accumulate), "n"(DESC_HI)
        : "memory");
}
// One such step (the last keys of a row).
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t p_tmem, uint32_t v_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred acc;\n\t.reg .b64 b0;\n\tsetp.ne.u32 acc, %4, 0;\n\tmov.b64 b0, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b0, %3, acc;\n\t}" ::"r"(d_tmem),
        "r"(p_tmem), "r"(v_lo), "r"(idesc), "r"(accumulate), "n"(DESC_HI)
        : "memory");
}

// The bounded wait, with its slow half out of the way: the roles run through their loops once a tile,
// between warps whose unrolled loops fill the instruction cache, so every instruction here counts.
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, unsigned *status) {
    if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return;
    uint64_t t0 = 0;
    for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
        if (it & 255u) continue;
        if (*reinterpret_cast<volatile unsigned *>(status) & ST_WAIT_TIMEOUT) return;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        else if (now - t0 > 2000000000ull) {
            atomicOr(status, ST_WAIT_TIMEOUT);
            return;
        }
    }
}
// 32 lanes x 16 columns of 32-bit TMEM cells -> 16 registers a thread.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr));
}
// One lane of a converged warp; the compiler knows that only one thread goes on.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

struct Item {
    int h, cs, ce, q0;   // head, row, first query
    int k0, kend, nt;    // keys [k0, kend) in nt tiles
    bool on;
    __device__ int in_last() const { return kend - k0 - (nt - 1) * TK; }  // keys of the last tile
};

// Work item w: head w % heads of query tile w / heads.  Tile numbers are spread so that no table is
// needed: row r's tiles start at cu[r] / 128 + r, which leaves every row room for all of its tiles; a
// number past a row's last tile is an empty item.  A role's items ascend, so its search goes on from the
// last row, 31 rows a look (one load, and the row's ends by shuffle).  All lanes of a warp call this.
__device__ __forceinline__ Item find_item(const DiffOp &p, int w, int lane, int &lo) {
    Item t;
    const int b = w / p.heads;
    t.h = w - b * p.heads;
    for (;;) {
        const int at = lo + lane, v = p.cu[min(at, p.n_rows)];
        const unsigned below = __ballot_sync(0xffffffffu, at < p.n_rows && (v >> 7) + at <= b);
        if (below == 0xffffffffu) {  // lane 31 then lies before n_rows: after the step lane 0 does
            lo += 31;
            continue;
        }
        const int k = 31 - __clz(below | 1u);  // at most 30: lane k + 1 holds the row's end
        t.cs = max(__shfl_sync(0xffffffffu, v, k), 0);
        t.ce = min(__shfl_sync(0xffffffffu, v, k + 1), p.n_tokens);
        lo += k;
        break;
    }
    t.q0 = t.cs + (b - (t.cs >> 7) - lo) * TQ;
    t.on = t.q0 >= t.cs && t.q0 < t.ce;
    t.k0 = p.window < 0 ? t.cs : max(t.cs, t.q0 - p.window);
    t.kend = p.window < 0 ? t.ce : min(t.ce, min(t.q0 + TQ, t.ce) + p.window);
    t.nt = (t.kend - t.k0 + TK - 1) / TK;
    return t;
}

// The next item that is not empty, from w on; w moves past it.
__device__ __forceinline__ Item find_on(const DiffOp &p, int &w, int n_items, int lane, int &lo) {
    Item t;
    for (t.on = false; w < n_items && !t.on; w += gridDim.x) t = find_item(p, w, lane, lo);
    return t;
}

// Bits a .. b - 1 of a word.
__device__ __forceinline__ uint32_t bits(int a, int b) {
    const uint32_t from = a <= 0 ? 0xffffffffu : (a < 32 ? 0xffffffffu << a : 0u);
    const uint32_t to = b >= 32 ? 0xffffffffu : (b > 0 ? (1u << b) - 1u : 0u);
    return from & to;
}

template <bool V16>  // V16: FP16 values, else BF16
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
    return V16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}
template <bool V16>
__device__ __forceinline__ float2 unpack_p(uint32_t u) {
    if (V16) return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// V16: FP16 values, else BF16
template <bool V16>
__global__ void __launch_bounds__(THREADS, 1)
    k_diff_attention(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ DiffOp p, int n_items) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + OFF_BAR);
    uint64_t *qfull = bars, *qfree = qfull + 2, *kfull = qfree + 2, *kfree = kfull + NK, *vfull = kfree + NK,
             *vfree = vfull + NV, *vtail = vfree + NV, *sfull = vtail + NV, *pready = sfull + 4, *pvdone = pready + 4,
             *odone = pvdone + 4, *summed = odone + 2, *ofree = summed + 2;  // sfull, pready, pvdone: 2 map + tile % 2; odone: map
    float *gain = reinterpret_cast<float *>(smem + OFF_F), *sums = gain + 128;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sums + 512);
    unsigned *status = tmem_slot + 1;  // expired waits of this CTA: the caller's word may hold another call's
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&kfull[i], 1);
            mbar_init(&kfree[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&vfull[i], 1);
            mbar_init(&vfree[i], 2);
            mbar_init(&vtail[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qfull[i], 1);
            mbar_init(&qfree[i], 2);
            mbar_init(&odone[i], 1);
            mbar_init(&summed[i], 8);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pready[i], 4);
            mbar_init(&pvdone[i], 1);
        }
        mbar_init(ofree, 4);
        *status = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    int row = 0;  // where this warp's search for items has got to
    if (warp < 4) {  // warp group 0: producers, MMA issue, the tail of V
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_ROLES));
        if (warp == 0) {
            uint32_t c = 0, it = 0;  // tiles, items
            for (int w = blockIdx.x; w < n_items; w += gridDim.x) {
                const Item t = find_item(p, w, lane, row);
                if (!t.on) continue;
                if (lane == 0) {
                    const int vh = t.h / (p.heads / p.kv_heads);
                    const uint32_t buf = it & 1;
                    if (it >= 2) mbar_wait(&qfree[buf], ((it - 2) >> 1) & 1, status);
                    mbar_arrive_expect_tx(&qfull[buf], 2 * Q_BYTES);
                    for (int x = 0; x < 2; ++x)
                        tma_load_heads(smem + OFF_Q + (buf * 2 + x) * Q_BYTES, &tm_q, &qfull[buf], 0, 2 * t.h + x, t.q0);
                    for (int j = 0; j < t.nt; ++j, ++c) {
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t u = 2 * c + x, s = u % NK;
                            if (u >= NK) mbar_wait(&kfree[s], ((u - NK) / NK) & 1, status);
                            mbar_arrive_expect_tx(&kfull[s], K_BYTES);
                            tma_load_heads(smem + OFF_K + s * K_BYTES, &tm_k, &kfull[s], 0, 2 * vh + x, t.k0 + j * TK);
                        }
                        const uint32_t s = c % NV;
                        if (c >= NV) mbar_wait(&vfree[s], ((c - NV) / NV) & 1, status);
                        // a tile that warp 2 has to finish lands on a barrier of its own
                        uint64_t *bar = j == t.nt - 1 && (t.in_last() & 15) ? &vtail[s] : &vfull[s];
                        mbar_arrive_expect_tx(bar, V_BYTES);
                        for (int x = 0; x < 2; ++x)
                            tma_load_heads(smem + OFF_V + s * V_BYTES + x * V_HALF, &tm_v, bar, 64 * x, vh, t.k0 + j * TK);
                    }
                }
                ++it;
                __syncwarp();
            }
        } else if (warp == 2) {
            uint32_t c = 0, tails[NV] = {};
            for (int w = blockIdx.x; w < n_items; w += gridDim.x) {
                const Item t = find_item(p, w, lane, row);
                if (!t.on) continue;
                c += t.nt;
                const int valid = t.in_last();
                if ((valid & 15) == 0) continue;  // the MMAs stop at the last whole step of 16 keys
                const uint32_t s = (c - 1) % NV;
                mbar_wait(&vtail[s], tails[s]++ & 1, status);
                __syncwarp();
                const int pieces = (((valid + 15) & ~15) - valid) * 8;  // 16 bytes each, in both halves
                for (int i = lane; i < 2 * pieces; i += 32) {
                    uint8_t *half = smem + OFF_V + s * V_BYTES + (i >= pieces ? V_HALF : 0);
                    *reinterpret_cast<uint4 *>(half + valid * 128 + (i >= pieces ? i - pieces : i) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&vfull[s]);
            }
        } else {
            const int x = warp >> 1;  // warp 1: map 0, warp 3: map 1
            const uint32_t idesc_s = p.qk_dtype == JD_F16 ? idesc_f16_f32(TK) : idesc_bf16_f32(TK);
            constexpr uint32_t idesc_pv = (V16 ? idesc_f16_f32(VD) : idesc_bf16_f32(VD)) | (1u << 16);  // V is MN-major
            const uint32_t q_lo = desc_lo(smem_u32(smem + OFF_Q) + x * Q_BYTES, 1), k_lo = desc_lo(smem_u32(smem + OFF_K), 1),
                           v_lo = desc_lo(smem_u32(smem + OFF_V), V_HALF >> 4);
            const uint32_t b_sfull = smem_u32(sfull + 2 * x), b_pready = smem_u32(pready + 2 * x),
                           b_pvdone = smem_u32(pvdone + 2 * x), b_kfull = smem_u32(kfull), b_kfree = smem_u32(kfree),
                           b_vfull = smem_u32(vfull), b_vfree = smem_u32(vfree);
            uint32_t sc = 0, c = 0, it = 0;  // S and PV products issued, items
            // the next S product, of an item whose queries are in buffer buf
            auto issue_s = [&](uint32_t buf, bool last) {
                const uint32_t b = sc & 1, u = 2 * sc + x, s = u % NK;
                wait(b_kfull + 8 * s, (u / NK) & 1, status);
                if (sc >= 2) wait(b_pvdone + 8 * b, ((sc - 2) >> 1) & 1, status);  // its last P has been used
                tc_fence_after();
                mma_s(tmem + T_S + 2 * TK * x + TK * b, q_lo + buf * (2 * Q_BYTES >> 4), k_lo + s * (K_BYTES >> 4), idesc_s);
                commit(b_sfull + 8 * b);
                commit(b_kfree + 8 * s);
                if (last) commit(smem_u32(&qfree[buf]));
                ++sc;
            };
            // S products run up to two tiles ahead of the PV products, into the next item if it has come to that
            int w = blockIdx.x, ahead = 0;  // ahead: S products of the current item issued so far
            Item now = find_on(p, w, n_items, lane, row);
            while (now.on) {
                const Item next = find_on(p, w, n_items, lane, row);
                if (elect_one()) {
                    const uint32_t buf = it & 1;
                    if (ahead == 0) wait(smem_u32(&qfull[buf]), (it >> 1) & 1, status);
                    while (ahead < min(2, now.nt)) ++ahead, issue_s(buf, ahead == now.nt);
                    int nahead = 0;
                    for (int j = 0; j < now.nt; ++j, ++c) {
                        const uint32_t b = c & 1, s = c % NV;
                        wait(b_vfull + 8 * s, (c / NV) & 1, status);
                        wait(b_pready + 8 * b, (c >> 1) & 1, status);
                        if (j == 0 && it > 0) wait(smem_u32(ofree), (it - 1) & 1, status);  // the last O has been read
                        tc_fence_after();
                        const uint32_t o = tmem + T_O + VD * x, pt = tmem + T_S + 2 * TK * x + TK * b,
                                       v = v_lo + s * (V_BYTES >> 4);
                        const bool last = j == now.nt - 1;
                        const int steps = last ? (now.in_last() + 15) >> 4 : TK / 16;
                        if (steps == TK / 16) {
                            mma_pv(o, pt, v, idesc_pv, j);
                            mma_pv(o, pt + 32, v, idesc_pv, 1);
                        } else {
                            for (int ks = 0; ks < steps; ++ks) {
                                mma_ts(o, pt + 8 * ks, v + ks * (16 * 128 >> 4), idesc_pv, j | ks);
                                mma_ts(o, pt + 32 + 8 * ks, v + ks * (16 * 128 >> 4), idesc_pv, 1);
                            }
                        }
                        commit(b_pvdone + 8 * b);
                        commit(b_vfree + 8 * s);
                        if (last) commit(smem_u32(&odone[x]));
                        if (ahead < now.nt) {
                            ++ahead;
                            issue_s(buf, ahead == now.nt);
                        } else if (next.on && nahead < min(2, next.nt)) {
                            if (nahead == 0) wait(smem_u32(&qfull[buf ^ 1]), ((it + 1) >> 1) & 1, status);
                            ++nahead;
                            issue_s(buf ^ 1, nahead == next.nt);
                        }
                    }
                    ahead = nahead;
                    ++it;
                }
                __syncwarp();
                now = next;
            }
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
        const int x = (warp - 4) >> 2;         // this group's map
        const int r = (warp & 3) * 32 + lane;  // query row inside the tile = TMEM lane
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t to = tl + T_O, b_sfull = smem_u32(sfull + 2 * x), b_pready = smem_u32(pready + 2 * x);
        const float sl2 = p.scale * 1.4426950408889634f;
        uint32_t c = 0, it = 0;  // tiles of this map and items so far
        int w = blockIdx.x;
        Item next = find_on(p, w, n_items, lane, row);
        while (next.on) {
            const Item t = next;
            next = find_on(p, w, n_items, lane, row);
            const int qi = t.q0 + r;
            const bool dead = t.q0 + (warp & 3) * 32 >= t.ce;  // no row of this warp: it only keeps the order
            // keys this row sees, from the tile's first on: [a, b)
            int a = (p.window < 0 ? t.cs : max(t.cs, qi - p.window)) - t.k0;
            int b = (p.window < 0 ? t.ce : min(t.ce, qi + p.window + 1)) - t.k0;
            float m = -INFINITY, l = 0.f;
            for (int j = 0; j < t.nt; ++j, ++c, a -= TK, b -= TK) {
                const uint32_t ts = tl + T_S + 2 * TK * x + TK * (c & 1);
                wait(b_sfull + 8 * (c & 1), (c >> 1) & 1, status);
                __syncwarp();
                if (!dead && !__any_sync(0xffffffffu, a < TK && b > 0)) {
                    // none of this warp's rows sees any of these keys (the ends of a window)
                    tc_fence_after();
                    uint32_t zero[32] = {};
                    tmem_st32(ts, zero);
                    tmem_st32(ts + 32, zero);
                    tmem_st_wait();
                    tc_fence_before();
                } else if (!dead) {
                    tc_fence_after();
                    uint32_t sv[TK];
                    tmem_ld32(ts, *reinterpret_cast<uint32_t(*)[32]>(&sv[0]));
                    tmem_ld32(ts + 32, *reinterpret_cast<uint32_t(*)[32]>(&sv[32]));
                    tmem_ld_wait();
                    if (__any_sync(0xffffffffu, a > 0 || b < TK)) {
                        const uint32_t seen[2] = {bits(a, b), bits(a - 32, b - 32)};
#pragma unroll
                        for (int e = 0; e < TK; ++e)
                            if (!(seen[e >> 5] & (1u << (e & 31)))) sv[e] = __float_as_uint(-INFINITY);
                    }
                    float m4[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        m4[i] = fmaxf(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1]));
#pragma unroll
                    for (int e = 8; e < TK; e += 8)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            m4[i] = max3(m4[i], __uint_as_float(sv[e + 2 * i]), __uint_as_float(sv[e + 2 * i + 1]));
                    const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2;
                    // Rows move their maximum one by one, but TMEM is read and written by whole warps (the
                    // instructions are aligned): all rows of the warp go along, most with a factor of 1.
                    const bool grows = mx > m + kLazy, scaled = grows && m != -INFINITY;
                    if (__any_sync(0xffffffffu, scaled)) {
                        const float alpha = scaled ? exp2_fast(m - mx) : 1.0f;
                        l *= alpha;
                        mbar_wait(&pvdone[2 * x + ((c - 1) & 1)], ((c - 1) >> 1) & 1, status);  // O_x is at rest
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int hc = 0; hc < VD; hc += 32) {
                            uint32_t o[32];
                            tmem_ld32(to + VD * x + hc, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st32(to + VD * x + hc, o);
                        }
                    }
                    if (grows) m = mx;
                    __syncwarp();
                    const float mm = m == -INFINITY ? 0.f : m;  // nothing seen yet: every P is 0
                    float2 ls[2] = {{0.f, 0.f}, {0.f, 0.f}};
                    uint32_t pk[32], pl[32];  // hi, lo
#pragma unroll
                    for (int e = 0; e < TK; e += 2) {
                        const float2 xv =
                            fma_f32x2(make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])),
                                      make_float2(sl2, sl2), make_float2(-mm, -mm));
                        const float2 pv = make_float2(exp2_fast(xv.x), exp2_fast(xv.y));
                        ls[(e >> 1) & 1] = add_f32x2(ls[(e >> 1) & 1], pv);
                        pk[e >> 1] = pack_p<V16>(pv.x, pv.y);
                        const float2 h = unpack_p<V16>(pk[e >> 1]);
                        pl[e >> 1] = pack_p<V16>(pv.x - h.x, pv.y - h.y);
                    }
                    tmem_st32(ts, pk);
                    tmem_st32(ts + 32, pl);
                    l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
                    tmem_st_wait();
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) arrive(b_pready + 8 * (c & 1));
            }
            sums[256 * (it & 1) + 128 * x + r] = l;
            __syncwarp();
            if (lane == 0) arrive(smem_u32(&summed[it & 1]));
            ++it;
        }
    } else {
        // Read-out, one row a thread: D in two passes over both O (its norm, then its values: all of D would not
        // fit the registers), while the softmax groups are at the next item: they may finish it, so the sums of two
        // items are kept, but not the one behind it, whose S follow the next O, which waits for this read-out.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_READOUT));
        const int r = (warp & 3) * 32 + lane;
        const uint32_t to = tmem + ((uint32_t)((warp & 3) * 32) << 16) + T_O;
        const float la = warp_sum(p.lq1[lane] * p.lk1[lane] + p.lq1[lane + 32] * p.lk1[lane + 32]);
        const float lb = warp_sum(p.lq2[lane] * p.lk2[lane] + p.lq2[lane + 32] * p.lk2[lane + 32]);
        const float lam = expf(la) - expf(lb) + p.lambda_init;
        gain[r] = p.gain ? p.gain[r] * (1.0f - p.lambda_init) : 1.0f;
        named_bar_sync(BAR_GAIN, 128);
        const bool out16 = p.qk_dtype == JD_F16;
        // elements e, e + 1 of a O_0 + b O_1
        auto both = [](const uint32_t (&x)[16], const uint32_t (&y)[16], int e, float a, float b) {
            const float2 z = make_float2(__uint_as_float(x[e]) * a, __uint_as_float(x[e + 1]) * a);
            return fma_f32x2(make_float2(__uint_as_float(y[e]), __uint_as_float(y[e + 1])), make_float2(b, b), z);
        };
        uint32_t it = 0;
        int w = blockIdx.x;
        Item next = find_on(p, w, n_items, lane, row);
        while (next.on) {
            const Item t = next;
            next = find_on(p, w, n_items, lane, row);
            wait(smem_u32(&summed[it & 1]), (it >> 1) & 1, status);
            wait(smem_u32(&odone[0]), it & 1, status);
            wait(smem_u32(&odone[1]), it & 1, status);
            __syncwarp();
            const int qi = t.q0 + r;
            if (t.q0 + (warp & 3) * 32 < t.ce) {
                tc_fence_after();
                const float *sum = sums + 256 * (it & 1) + r;
                const float i0 = 1.0f / sum[0], i1 = -lam / sum[128];
                float f = 1.0f;
                // Sixteen columns of both O at a time, the next ones asked for before these are worked on.
                uint32_t o0[2][16], o1[2][16];
                auto ask = [&](int e0, int k) {
                    tmem_ld16(to + e0, o0[k]);
                    tmem_ld16(to + VD + e0, o1[k]);
                };
                ask(0, 0);
                if (p.gain) {
                    float2 sq = make_float2(0.f, 0.f);
#pragma unroll 1
                    for (int e0 = 0; e0 < VD; e0 += 32) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            tmem_ld_wait();
                            ask((e0 + 16 * k + 16) & (VD - 1), k ^ 1);  // (behind the last the first again)
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const float2 d = both(o0[k], o1[k], e, i0, i1);
                                sq = fma_f32x2(d, d, sq);
                            }
                        }
                    }
                    f = rsqrtf((sq.x + sq.y) * (1.0f / VD) + p.eps);
                }
                const float f0 = f * i0, f1 = f * i1;
                uint8_t *dst = static_cast<uint8_t *>(p.out) + 2 * (qi * p.out_token + t.h * p.out_head);
#pragma unroll 1
                for (int e0 = 0; e0 < VD; e0 += 32) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int at = e0 + 16 * k;
                        tmem_ld_wait();
                        if (at < VD - 16) {
                            ask(at + 16, k ^ 1);
                        } else {  // both O have been read
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) arrive(smem_u32(ofree));
                        }
                        uint32_t u[8];
#pragma unroll
                        for (int i = 0; i < 8; i += 2) {
                            const float4 g = *reinterpret_cast<const float4 *>(&gain[at + 2 * i]);
                            float2 v = both(o0[k], o1[k], 2 * i, f0, f1), v2 = both(o0[k], o1[k], 2 * i + 2, f0, f1);
                            u[i] = out16 ? pack_f16x2(v.x * g.x, v.y * g.y) : pack_bf16x2(v.x * g.x, v.y * g.y);
                            u[i + 1] = out16 ? pack_f16x2(v2.x * g.z, v2.y * g.w) : pack_bf16x2(v2.x * g.z, v2.y * g.w);
                        }
                        if (qi < t.ce) {
                            if (p.out32) {  // a row a thread: 32-byte stores fill whole sectors
                                st_global_v8(dst + 2 * at, u[0], u[1], u[2], u[3], u[4], u[5], u[6], u[7]);
                            } else {
                                *reinterpret_cast<uint4 *>(dst + 2 * at) = make_uint4(u[0], u[1], u[2], u[3]);
                                *reinterpret_cast<uint4 *>(dst + 2 * at + 16) = make_uint4(u[4], u[5], u[6], u[7]);
                            }
                        }
                        __syncwarp();  // whole warps read TMEM
                    }
                }
            } else if (lane == 0) {
                arrive(smem_u32(ofree));
            }
            __syncwarp();
            ++it;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && p.status && *status) atomicOr(p.status, *status);
    if (*status) {
        const uint64_t from = globaltimer_ns();
        for (int i = 0; i < LINGER_STEPS && globaltimer_ns() - from < LINGER_NS; ++i) __nanosleep(1000);
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ FP32

constexpr int FK = 64, QP = 68;  // keys of a tile; padded row of a transposed tile
constexpr int F32_THREADS = 128;
// floats: Q [map][64][QP] (at the end the second map's O [8 R][132]), K and then P [map][64][QP], V [FK][VD],
// gain, lambda
constexpr int F32_SMEM = (2 * 64 * QP + 2 * 64 * QP + FK * VD + 128 + 4) * 4;
static_assert(64 * 132 <= 2 * 64 * QP, "the second map's O lies over Q");

// 8 R queries of one row and head against its keys, 64 at a time; two warps a map.  A thread holds R x 8
// scores and R x 16 outputs of the same rows, so that a row's running maximum and sum stay with it and
// its seven neighbours.  Shared memory hands a lane one float a clock against four FMAs: with R = 8 the
// scores take 4 FMAs a float, the outputs 5.3; R = 4 is for calls too small to fill the SMs with that.
// Q, K and P lie transposed (element-major), whole vectors a step; P takes K's place.  Two CTAs an SM.
// Bound by FP32 arithmetic, 768 operations a visible pair and head, the FMA pipe active 52 % of the cycles:
// 24 rows of 64 to 512 with four heads 348 us, two rows of 8192 10.5 ms (39 TFLOP/s).  With 4 x 4 scores
// and 4 x 8 outputs of both maps in every thread these took 415 us and 14.1 ms.
template <int R>
__global__ void __launch_bounds__(F32_THREADS, 2) k_diff_attention_f32(const __grid_constant__ DiffOp p) {
    constexpr int FQ = 8 * R, SHIFT = R == 8 ? 6 : 5;
    extern __shared__ float fs[];
    float *Q = fs, *K = Q + 2 * 64 * QP, *V = K + 2 * 64 * QP, *gain = V + FK * VD, *lambda = gain + 128;
    const int tid = threadIdx.x, lane = tid & 31, x = tid >> 6, u = tid & 63;
    // the tiles' numbering of find_item, with FQ queries a tile
    const int b = blockIdx.x, h = blockIdx.y;
    int row = 0, n = p.n_rows;
    while (n > 1) {
        const int step = (n + 31) >> 5, at = lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, at < n && (p.cu[row + at] >> SHIFT) + row + at <= b);
        if (!(below & 1u)) return;
        const int k = 31 - __clz(below);
        row += k * step;
        n = min(step, n - k * step);
    }
    const int cs = max(p.cu[row], 0), ce = min(p.cu[row + 1], p.n_tokens);
    const int q0 = cs + (b - (cs >> SHIFT) - row) * FQ;
    if (q0 < cs || q0 >= ce) return;
    const int k0 = p.window < 0 ? cs : max(cs, q0 - p.window);
    const int kend = p.window < 0 ? ce : min(ce, min(q0 + FQ, ce) + p.window);
    const int g = h / (p.heads / p.kv_heads);
    const float *qp = static_cast<const float *>(p.q) + 2 * h * p.q_head;
    const float *kp = static_cast<const float *>(p.k) + 2 * g * p.k_head;
    const float *vp = static_cast<const float *>(p.v) + g * p.v_head;
    if (tid < 32) {
        const float a = warp_sum(p.lq1[lane] * p.lk1[lane] + p.lq1[lane + 32] * p.lk1[lane + 32]);
        const float c = warp_sum(p.lq2[lane] * p.lk2[lane] + p.lq2[lane + 32] * p.lk2[lane + 32]);
        if (lane == 0) *lambda = expf(a) - expf(c) + p.lambda_init;
    }
    gain[tid] = p.gain ? p.gain[tid] * (1.0f - p.lambda_init) : 1.0f;
    // Both maps of `rows` tokens, transposed: a warp takes 16 tokens by 32 bytes, whole sectors
    auto load_t = [&](float *dst, int rows, const float *src, int64_t token, int64_t head, int first, int end) {
        const int groups = rows >> 4;
#pragma unroll 4
        for (int i = tid; i < 2 * 16 * rows; i += F32_THREADS) {
            const int block = i >> 5, r = (i & 15) + 16 * (block & (groups - 1)),
                      v4 = ((i >> 4) & 1) + 2 * (block / groups & 7), m = block / groups >> 3;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            if (first + r < end) a = *reinterpret_cast<const float4 *>(src + (first + r) * token + m * head + 4 * v4);
            float *d = dst + (m * 64 + 4 * v4) * QP + r;
            d[0] = a.x, d[QP] = a.y, d[2 * QP] = a.z, d[3 * QP] = a.w;
        }
    };
    load_t(Q, FQ, qp, p.q_token, p.q_head, q0, ce);
    const int ty = u >> 3, tx = u & 7;  // rows R ty ..; keys 4 tx .., 32 + 4 tx ..; columns 4 tx + 32 i ..
    const float *Qm = Q + x * 64 * QP + R * ty;
    float *Km = K + x * 64 * QP;
    float2 o[R][8];
    float m[R], l[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[i][e] = make_float2(0.f, 0.f);
    }
    for (int kt = k0; kt < kend; kt += FK) {
        __syncthreads();  // the last tile's P and V have been used
        load_t(K, FK, kp, p.k_token, p.k_head, kt, kend);
#pragma unroll 4
        for (int i = tid; i < FK * VD / 4; i += F32_THREADS) {
            const int r = i >> 5, v4 = i & 31;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            if (kt + r < kend) a = *reinterpret_cast<const float4 *>(vp + (kt + r) * p.v_token + 4 * v4);
            *reinterpret_cast<float4 *>(V + r * VD + 4 * v4) = a;
        }
        __syncthreads();
        float2 s[R][4];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[i][e] = make_float2(0.f, 0.f);
#pragma unroll 2
        for (int d = 0; d < 64; ++d) {
            float av[R];
#pragma unroll
            for (int i = 0; i < R; i += 4) *reinterpret_cast<float4 *>(&av[i]) = *reinterpret_cast<const float4 *>(Qm + d * QP + i);
            const float4 c0 = *reinterpret_cast<const float4 *>(Km + d * QP + 4 * tx),
                         c1 = *reinterpret_cast<const float4 *>(Km + d * QP + 32 + 4 * tx);
            const float2 cv[4] = {{c0.x, c0.y}, {c0.z, c0.w}, {c1.x, c1.y}, {c1.z, c1.w}};
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][e] = fma_f32x2(make_float2(av[i], av[i]), cv[e], s[i][e]);
        }
        __syncthreads();  // K has been used: P takes its place
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int qi = q0 + R * ty + i;
            float v[8], mx = -INFINITY;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int kj = kt + 4 * tx + (e & 3) + (e >> 2) * 32;
                const bool seen = kj < kend && (p.window < 0 || (kj - qi <= p.window && qi - kj <= p.window));
                v[e] = seen ? (e & 1 ? s[i][e >> 1].y : s[i][e >> 1].x) * p.scale : -INFINITY;
                mx = fmaxf(mx, v[e]);
            }
            for (int w = 4; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float now = fmaxf(m[i], mx), mm = now == -INFINITY ? 0.f : now;  // nothing seen yet: every P is 0
            const float alpha = expf(m[i] - mm);
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] = expf(v[e] - mm);
                sum += v[e];
                s[i][e >> 1] = e & 1 ? make_float2(v[e - 1], v[e]) : s[i][e >> 1];
            }
            l[i] = l[i] * alpha + sum;
            m[i] = now;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[i][e] = make_float2(o[i][e].x * alpha, o[i][e].y * alpha);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float *dst = Km + (4 * tx + (e & 3) + (e >> 2) * 32) * QP + R * ty;
#pragma unroll
            for (int i = 0; i < R; i += 4)
                *reinterpret_cast<float4 *>(dst + i) =
                    e & 1 ? make_float4(s[i][e >> 1].y, s[i + 1][e >> 1].y, s[i + 2][e >> 1].y, s[i + 3][e >> 1].y)
                          : make_float4(s[i][e >> 1].x, s[i + 1][e >> 1].x, s[i + 2][e >> 1].x, s[i + 3][e >> 1].x);
        }
        __syncthreads();
        const int keys = min(FK, kend - kt);
#pragma unroll 2
        for (int k = 0; k < keys; ++k) {
            float pv[R];
#pragma unroll
            for (int i = 0; i < R; i += 4)
                *reinterpret_cast<float4 *>(&pv[i]) = *reinterpret_cast<const float4 *>(Km + k * QP + R * ty + i);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float4 v = *reinterpret_cast<const float4 *>(V + k * VD + 32 * c + 4 * tx);
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    o[i][2 * c] = fma_f32x2(make_float2(pv[i], pv[i]), make_float2(v.x, v.y), o[i][2 * c]);
                    o[i][2 * c + 1] = fma_f32x2(make_float2(pv[i], pv[i]), make_float2(v.z, v.w), o[i][2 * c + 1]);
                }
            }
        }
    }
    const float lam = *lambda;
    float *O1 = Q;  // [64][132]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) {
        for (int w = 4; w; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
        const float f = (x ? -lam : 1.0f) / l[i];
#pragma unroll
        for (int e = 0; e < 8; ++e) o[i][e] = make_float2(o[i][e].x * f, o[i][e].y * f);
        if (x)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                *reinterpret_cast<float4 *>(O1 + (R * ty + i) * 132 + 32 * c + 4 * tx) =
                    make_float4(o[i][2 * c].x, o[i][2 * c].y, o[i][2 * c + 1].x, o[i][2 * c + 1].y);
    }
    __syncthreads();
    if (x) return;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float sq = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float4 a = *reinterpret_cast<const float4 *>(O1 + (R * ty + i) * 132 + 32 * c + 4 * tx);
            o[i][2 * c] = make_float2(o[i][2 * c].x + a.x, o[i][2 * c].y + a.y);
            o[i][2 * c + 1] = make_float2(o[i][2 * c + 1].x + a.z, o[i][2 * c + 1].y + a.w);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(o[i][e].x, o[i][e].x, fmaf(o[i][e].y, o[i][e].y, sq));
        for (int w = 4; w; w >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, w);
        const float f = p.gain ? 1.0f / sqrtf(sq * (1.0f / VD) + p.eps) : 1.0f;
        const int qi = q0 + R * ty + i;
        if (qi < ce) {
            float *dst = static_cast<float *>(p.out) + qi * p.out_token + h * p.out_head;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int at = 32 * c + 4 * tx;
                *reinterpret_cast<float4 *>(dst + at) =
                    make_float4(o[i][2 * c].x * f * gain[at], o[i][2 * c].y * f * gain[at + 1],
                                o[i][2 * c + 1].x * f * gain[at + 2], o[i][2 * c + 1].y * f * gain[at + 3]);
            }
        }
    }
}

const void *tensor_kernel(const DiffOp &op) {
    return op.v_dtype == JD_F16 ? reinterpret_cast<const void *>(&k_diff_attention<true>)
                                : reinterpret_cast<const void *>(&k_diff_attention<false>);
}

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static EncodeTiled fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiled>(f);
    });
    return fn;
}

}  // namespace

jd_status make_diff_maps(const DiffOp &op, DiffMaps *maps) {
    EncodeTiled fn = encode_tiled();
    if (!fn) return fail(JD_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
    struct {
        CUtensorMap *m;
        const void *data;
        int width, heads, rows, dtype;
        int64_t token, head;
    } t[3] = {{&maps->q, op.q, 64, 2 * op.heads, TQ, op.qk_dtype, op.q_token, op.q_head},
              {&maps->k, op.k, 64, 2 * op.kv_heads, TK, op.qk_dtype, op.k_token, op.k_head},
              {&maps->v, op.v, 128, op.kv_heads, TK, op.v_dtype, op.v_token, op.v_head}};
    for (auto &a : t) {
        // an axis of one entry is never stepped along: any stride does
        const cuuint64_t dims[3] = {(cuuint64_t)a.width, (cuuint64_t)a.heads, (cuuint64_t)op.n_tokens};
        const cuuint64_t strides[2] = {2 * (cuuint64_t)(a.heads > 1 ? a.head : a.width),
                                       2 * (cuuint64_t)(op.n_tokens > 1 ? a.token : a.width)};
        const cuuint32_t box[3] = {64, 1, (cuuint32_t)a.rows}, es[3] = {1, 1, 1};
        const CUresult r =
            fn(a.m, a.dtype == JD_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<void *>(a.data), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) return fail(JD_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    }
    return JD_OK;
}

cudaError_t diff_attention_prepare(int device) {
    static std::atomic<bool> done[64];
    if (device >= 0 && device < 64 && done[device].load(std::memory_order_acquire)) return cudaSuccess;
    const void *kernels[2] = {reinterpret_cast<const void *>(&k_diff_attention<false>),
                              reinterpret_cast<const void *>(&k_diff_attention<true>)};
    for (const void *k : kernels) {
        // a group asking for more registers than the launch holds would wait for ever
        cudaFuncAttributes fa;
        cudaError_t e = cudaFuncGetAttributes(&fa, k);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != REGS) return cudaErrorInvalidKernelImage;
        e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, DIFF_SMEM);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = cudaFuncSetAttribute(k_diff_attention_f32<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, F32_SMEM);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_diff_attention_f32<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, F32_SMEM);
    if (e == cudaSuccess && device >= 0 && device < 64) done[device].store(true, std::memory_order_release);
    return e;
}

cudaError_t launch_diff_attention(const DiffOp &op, const DiffMaps *maps, int num_sms, cudaStream_t st) {
    if (op.n_tokens <= 0 || op.n_rows <= 0) return cudaSuccess;
    if (op.qk_dtype == JD_F32) {
        // 64 queries a CTA unless two an SM would not be had: then 32, on twice the CTAs (8 rows of 200 to 300 with
        // four heads, 157 CTAs: 73 against 118 us; 16 such rows, 314 CTAs: 132 against 127)
        const int64_t ctas = ((int64_t)op.n_tokens / 64 + op.n_rows) * op.heads;
        if (ctas > 2 * num_sms)
            k_diff_attention_f32<8><<<dim3(op.n_tokens / 64 + op.n_rows, op.heads), F32_THREADS, F32_SMEM, st>>>(op);
        else
            k_diff_attention_f32<4><<<dim3(op.n_tokens / 32 + op.n_rows, op.heads), F32_THREADS, F32_SMEM, st>>>(op);
        return cudaGetLastError();
    }
    const int64_t items = ((int64_t)op.n_tokens / TQ + op.n_rows) * op.heads;
    int n_items = (int)items;
    const int grid = n_items < num_sms ? n_items : num_sms;
    void *args[5] = {const_cast<CUtensorMap *>(&maps->q), const_cast<CUtensorMap *>(&maps->k),
                     const_cast<CUtensorMap *>(&maps->v), const_cast<DiffOp *>(&op), &n_items};
    return cudaLaunchKernel(tensor_kernel(op), dim3(grid), dim3(THREADS), args, DIFF_SMEM, st);
}

}  // namespace jd

using namespace jd;

extern "C" jd_status jd_diff_attention(const jd_diff_attention_args *a, void *stream) {
    clear_error();
    if (!a) return fail(JD_ERR_INVALID_ARG, "NULL argument");
    const bool f32 = a->qk_dtype == JD_F32;
    if (a->qk_dtype != JD_F32 && a->qk_dtype != JD_F16 && a->qk_dtype != JD_BF16)
        return fail(JD_ERR_INVALID_ARG, "unknown dtype %d", a->qk_dtype);
    if (f32 ? a->v_dtype != JD_F32 : (a->v_dtype != JD_F16 && a->v_dtype != JD_BF16))
        return fail(JD_ERR_INVALID_ARG, "v_dtype %d does not go with qk_dtype %d", a->v_dtype, a->qk_dtype);
    if (a->n_tokens < 0 || a->n_rows < 0) return fail(JD_ERR_INVALID_ARG, "negative n_tokens or n_rows");
    const int heads = a->out.n_heads, kv = a->kv_heads;
    if (heads < 1 || heads > 32767 || kv < 1 || heads % kv)
        return fail(JD_ERR_INVALID_ARG, "heads: out.n_heads 1..32767, a multiple of kv_heads");
    if (a->q.n_heads != 2 * heads || a->k.n_heads != 2 * kv || a->v.n_heads != kv)
        return fail(JD_ERR_INVALID_ARG, "heads: q has 2 heads, k 2 kv_heads, v kv_heads");
    // (a query tile of a row of 2^24 takes a quarter of a second, which the kernel's bounded waits of two allow for)
    if (a->n_tokens > (1 << 24) || ((int64_t)a->n_tokens / 32 + a->n_rows) * heads > INT32_MAX - 65536)
        return fail(JD_ERR_INVALID_ARG, "too many tokens, rows and heads");
    if (!std::isfinite(a->lambda_init) || !(a->norm_eps >= 0) || !std::isfinite(a->norm_eps) || !(a->scale >= 0) ||
        !std::isfinite(a->scale))
        return fail(JD_ERR_INVALID_ARG, "lambda_init, norm_eps or scale is not finite, or norm_eps or scale negative");
    const jd_heads *in[3] = {&a->q, &a->k, &a->v};
    const char *name[3] = {"q", "k", "v"};
    const size_t elem = f32 ? 4 : 2;
    for (int i = 0; i < 3; ++i) {
        const jd_heads &t = *in[i];
        const int64_t most = (int64_t)1 << 38;  // a tensor map's strides are below 2^40 bytes
        if ((t.token_stride < 1 && a->n_tokens > 1) || (t.head_stride < 1 && t.n_heads > 1) || t.token_stride > most ||
            t.head_stride > most)
            return fail(JD_ERR_INVALID_ARG, "%s: strides must be positive and at most 2^38", name[i]);
    }
    jd_status s = check_written(a->out, a->n_tokens, 128, "out");
    if (s != JD_OK) return s;
    if (a->n_tokens == 0 || a->n_rows == 0) return JD_OK;
    if (!a->q.data || !a->k.data || !a->v.data || !a->out.data || !a->cu_seqlens || !a->lambda_q1 || !a->lambda_k1 ||
        !a->lambda_q2 || !a->lambda_k2)
        return fail(JD_ERR_INVALID_ARG, "a tensor is NULL");
    for (const jd_heads *t : {&a->q, &a->k, &a->v, &a->out})
        if (!heads_aligned(*t, elem, 16)) return fail(JD_ERR_INVALID_ARG, "alignment: pointers and strides of 16 bytes required");
    for (const jd_heads *t : in)
        if (t->data == a->out.data) return fail(JD_ERR_INVALID_ARG, "out is an input");
    DiffOp op{};
    op.cu = a->cu_seqlens;
    op.n_rows = a->n_rows;
    op.n_tokens = a->n_tokens;
    op.window = a->window < 0 ? -1 : (a->window < a->n_tokens ? a->window : a->n_tokens);
    op.heads = heads;
    op.kv_heads = kv;
    op.qk_dtype = a->qk_dtype;
    op.v_dtype = a->v_dtype;
    op.q = a->q.data, op.q_token = a->q.token_stride, op.q_head = a->q.head_stride;
    op.k = a->k.data, op.k_token = a->k.token_stride, op.k_head = a->k.head_stride;
    op.v = a->v.data, op.v_token = a->v.token_stride, op.v_head = a->v.head_stride;
    op.out = a->out.data, op.out_token = a->out.token_stride, op.out_head = a->out.head_stride;
    op.out32 = heads_aligned(a->out, elem, 32);
    op.lq1 = a->lambda_q1, op.lk1 = a->lambda_k1, op.lq2 = a->lambda_q2, op.lk2 = a->lambda_k2;
    op.gain = a->norm_gain;
    op.lambda_init = a->lambda_init;
    op.eps = a->norm_eps;
    op.scale = a->scale != 0.f ? a->scale : 0.125f;
    op.status = a->status;
    OpDevice dev;
    s = dev.enter({op.q, op.k, op.v, op.out, op.cu, op.lq1, op.lk1, op.lq2, op.lk2, op.gain, op.status});
    if (s != JD_OK) return s;
    DiffMaps maps;
    if (!f32 && (s = make_diff_maps(op, &maps)) != JD_OK) return s;
    cudaError_t e = diff_attention_prepare(dev.device);
    if (e == cudaSuccess) e = launch_diff_attention(op, &maps, num_sms(), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(JD_ERR_CUDA, "differential attention: %s", cudaGetErrorString(e));
    return JD_OK;
}
