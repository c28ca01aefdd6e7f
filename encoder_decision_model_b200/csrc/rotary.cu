// Rotary positions, with or without a norm of every head in the same pass.
//
// All heads of a token turn by the same angles.  A token's threads (all in one warp) form its r/2
// sines and cosines once and share them through shared memory; each thread then turns the same
// eight pairs of one head after another, with the sines in registers.  Its sixteen elements, two runs
// of eight, never leave it: in the half layout runs r/2 apart hold eight pairs, in the interleaved
// one any run holds four.  A head's norm is a sum over the thread's elements and a few shuffles.  A
// thread's next three heads are always on their way into shared memory (cp.async), also across
// tokens: with them in registers the kernel took 114 of those and ran at 80 us where it now takes 68.
//
// Angles are formed, not read from a table: p * w_j is reduced to a fraction of a turn in 64 bits, exact
// for any position (in 32 bits the angle at position 10^5 is off by 4e-3); sine and cosine of the
// fraction are FP32.  The pass reads and writes each element once and is bound by HBM: 131,072 tokens
// of 12 heads of 64 in BF16 take 68 to 70 us (0.88 to 0.91 of the measured copy), 139,809 in FP16 with half
// of each head interleaved 72 to 78 us (0.84 to 0.91); 556,823 with RMS norms 296 us in a few calls and 320 to 343
// in a row (0.76 to 0.88), where the issue slots are two thirds full.
//
// Two kernels: k_rotary as above, where head_dim and the two runs fall on 16-byte vectors, and
// k_rotary_any for every other width, offset and stride (a thread holds eight elements and finds
// their partners where the other threads' are kept): 15,932 tokens of 8 heads of 80 in FP32, 20 elements
// turning, take 28 us (0.45), bound by issued instructions and their latencies.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <cmath>

#include "op_common.h"
#include "rotary.h"

namespace jd {

namespace {

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// Eight elements as they lie in memory, in registers.
template <typename T>
struct Vec8 {
    static constexpr int N = sizeof(T) / 2;
    uint4 v[N];
};

template <typename T>
__device__ __forceinline__ void unpack2(uint32_t u, float &lo, float &hi);
template <>
__device__ __forceinline__ void unpack2<__nv_bfloat16>(uint32_t u, float &lo, float &hi) {
    lo = __uint_as_float(u << 16);
    hi = __uint_as_float(u & 0xffff0000u);
}
template <>
__device__ __forceinline__ void unpack2<__half>(uint32_t u, float &lo, float &hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
    lo = f.x;
    hi = f.y;
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

template <typename T>
__device__ __forceinline__ void unpack8(const Vec8<T> &x, float *y) {
#pragma unroll
    for (int i = 0; i < Vec8<T>::N; ++i) {
        const uint32_t u[4] = {x.v[i].x, x.v[i].y, x.v[i].z, x.v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) y[4 * i + j] = __uint_as_float(u[j]);
            else unpack2<T>(u[j], y[2 * j], y[2 * j + 1]);
        }
    }
}
template <typename T>
__device__ __forceinline__ Vec8<T> pack8(const float *y) {
    Vec8<T> x;
#pragma unroll
    for (int i = 0; i < Vec8<T>::N; ++i) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) u[j] = __float_as_uint(y[4 * i + j]);
            else u[j] = pack2<T>(y[2 * j], y[2 * j + 1]);
        }
        x.v[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
    return x;
}
template <typename T>
__device__ __forceinline__ void put8(T *p, const Vec8<T> &x) {
#pragma unroll
    for (int i = 0; i < Vec8<T>::N; ++i) reinterpret_cast<uint4 *>(p)[i] = x.v[i];
}

// Row of token t: the last r with cu[r] <= t, found by 32 probes at a time; -1 for a token outside
// every row.
__device__ __forceinline__ int row_of(const int *cu, int n_rows, int t, int lane) {
    int lo = 0, n = n_rows;
    if (n < 1 || cu[n_rows] <= t) return -1;
    while (n > 1) {
        const int step = (n + 31) >> 5;
        const int at = lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, at < n && cu[lo + at] <= t);
        if (!(below & 1u)) return -1;
        const int k = 31 - __clz(below);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return cu[lo] <= t ? lo : -1;
}

__device__ __forceinline__ void load8f(const float *p, float *y) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    y[0] = a.x, y[1] = a.y, y[2] = a.z, y[3] = a.w, y[4] = b.x, y[5] = b.y, y[6] = b.z, y[7] = b.w;
}

// Two FP32 operations an instruction (sm_100 f32x2 forms).
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mov.b64 rc, {%6, %7};\n\tfma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ void copy_async16(void *shared, const void *global) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(shared))),
                 "l"(global)
                 : "memory");
}

// Sixteen elements of a thread (two runs of eight) as eight pairs, and back.
template <bool INTERLEAVED>
__device__ __forceinline__ void split_pairs(const float *y, float2 *a, float2 *b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        a[j] = INTERLEAVED ? make_float2(y[4 * j], y[4 * j + 2]) : make_float2(y[2 * j], y[2 * j + 1]);
        b[j] = INTERLEAVED ? make_float2(y[4 * j + 1], y[4 * j + 3]) : make_float2(y[8 + 2 * j], y[9 + 2 * j]);
    }
}
template <bool INTERLEAVED>
__device__ __forceinline__ void join_pairs(float *z, const float2 *a, const float2 *b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        z[INTERLEAVED ? 4 * j : 2 * j] = a[j].x;
        z[INTERLEAVED ? 4 * j + 2 : 2 * j + 1] = a[j].y;
        z[INTERLEAVED ? 4 * j + 1 : 8 + 2 * j] = b[j].x;
        z[INTERLEAVED ? 4 * j + 3 : 9 + 2 * j] = b[j].y;
    }
}

constexpr int VWARPS = 4;         // warps of a k_rotary CTA
constexpr int AHEAD = 3;          // heads on their way to each thread
constexpr int SMS = 148;
constexpr int CTAS_RESIDENT = 5;  // CTAs that an SM holds at once
constexpr int CTAS_PER_SM = 32;   // CTAs of a large launch, at most, for each SM

// NORM: 0 none, 1 RMS, 2 layer norm
template <typename T, bool INTERLEAVED, int NORM>
__global__ void __launch_bounds__(32 * VWARPS) k_rotary(const __grid_constant__ RotaryOp op) {
    // heads on their way, in 16-byte pieces: each thread reads only what it asked for.  One place
    // more than are on their way, so that none is overwritten in the turn that reads it.
    constexpr int PIECES = 2 * Vec8<T>::N;
    __shared__ uint4 ring[AHEAD + 1][PIECES][32 * VWARPS];
    // cosines, sines of the CTA's tokens: 32 * VWARPS threads of at most eight pairs each
    __shared__ __align__(16) float cosines[32 * VWARPS * 8], sines[32 * VWARPS * 8];
    __shared__ double turns[ROTARY_MAX_PAIRS];
    const int lane = threadIdx.x & 31;
    const int L = op.lanes_per_head, HS = op.heads_at_once, TPT = L * HS;  // powers of two, TPT <= 32
    const int in_token = threadIdx.x & (TPT - 1), unit = in_token & (L - 1), hs = in_token / L;
    const int r = op.dims, half = r >> 1, turning = r >> 4;  // half layout: threads of a head that turn
    const int n_heads = op.n_heads[0] + op.n_heads[1];
    // This thread's two runs of eight elements: half of what they divide apart, so that neighbouring
    // threads touch neighbouring 16 bytes (32-byte steps cost a third of the bandwidth).
    const int low = INTERLEAVED || unit < turning ? 0 : r, wide = INTERLEAVED ? op.head_dim : (low ? op.head_dim - r : r);
    const int e0 = low + 8 * (unit - (low >> 4)), e1 = e0 + (wide >> 1);
    const bool live = 16 * unit < op.head_dim;
    // its eight pairs' sines: the half layout's from 8 * unit on, the interleaved ones' with their runs
    const int pair0 = INTERLEAVED ? e0 >> 1 : 8 * unit, pair4 = INTERLEAVED ? e1 >> 1 : 8 * unit + 4;
    const int turns0 = live ? min(4, max(0, half - pair0)) : 0, turns4 = live ? min(4, max(0, half - pair4)) : 0;
    const bool on = live && !(NORM == 0 && op.in_place && turns0 + turns4 == 0);
    const float inv_n = 1.0f / (float)op.head_dim;
    const int slot = (threadIdx.x / TPT) * (8 * L);  // this token's sines
    for (int j = threadIdx.x; j < half; j += 32 * VWARPS) turns[j] = op.turns[j];
    __syncthreads();
    // a CTA walks consecutive tokens, each warp 32 / TPT at a time, and follows their rows
    const int at_once = 32 / TPT, step = VWARPS * at_once;
    const int begin = blockIdx.x * op.tokens_per_cta, last = min(op.n_tokens, begin + op.tokens_per_cta);
    const int first = begin + (threadIdx.x >> 5) * at_once;
    if (first >= last) return;

    // where head hs of a token lies among the queries, and where it would lie among the keys
    auto queries = [&](const void *base, int64_t token, int64_t head, int t) {
        return static_cast<const T *>(base) + t * token + hs * head + e0;
    };
    auto keys = [&](const void *base, int64_t token, int64_t head, int t) {
        return static_cast<const T *>(base) + t * token + (hs - op.n_heads[0]) * head + e0;
    };
    // the next head to ask for: an index, its token, and the two places
    int next_t = first + lane / TPT, next_h = hs, next_place = 0;
    const T *next_q = queries(op.src[0], op.src_token[0], op.src_head[0], next_t);
    const T *next_k = keys(op.src[1], op.src_token[1], op.src_head[1], next_t);
    auto ask = [&]() {
        if (on && next_t < last && next_h < n_heads) {
            const T *p = next_h < op.n_heads[0] ? next_q : next_k;
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
                copy_async16(&ring[next_place][i][threadIdx.x],
                             reinterpret_cast<const uint4 *>(i < PIECES / 2 ? p : p + (e1 - e0)) + i % (PIECES / 2));
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        next_place = next_place == AHEAD ? 0 : next_place + 1;
        next_h += HS;
        next_q += HS * op.src_head[0];
        next_k += HS * op.src_head[1];
        if (next_h - hs >= n_heads) {
            next_h = hs;
            next_t += step;
            next_q = queries(op.src[0], op.src_token[0], op.src_head[0], next_t);
            next_k = keys(op.src[1], op.src_token[1], op.src_head[1], next_t);
        }
    };
#pragma unroll 1
    for (int i = 0; i < AHEAD; ++i) ask();

    int row = -1, row_start = 0, row_end = op.n_tokens;
    if (!op.positions) {
        row = row_of(op.cu, op.n_rows, first, lane);
        row_start = row < 0 ? 0 : op.cu[row];
        row_end = row < 0 ? 0 : op.cu[row + 1];  // past every row: nothing to do, and nothing follows
    }
    int place = 0;
    for (int t0 = first; t0 < last; t0 += step) {
        const int t = t0 + lane / TPT;
        bool work = on && t < last;
        int pos = 0;
        if (op.positions) {
            if (t < last) pos = op.positions[t];
        } else {
            while (row >= 0 && t >= row_end && row + 1 < op.n_rows) {
                ++row;
                row_start = row_end;
                row_end = op.cu[row + 1];
            }
            work = work && t < row_end;
            pos = t - row_start;
        }
        __syncwarp();  // the last tokens' sines have been read
        for (int j = in_token; j < half; j += TPT) {
            double a = (double)pos * turns[j];
            a -= rint(a);
            float s, c;
            sincospif(2.0f * (float)a, &s, &c);
            cosines[slot + j] = op.amplitude * c;
            sines[slot + j] = op.amplitude * s;
        }
        __syncwarp();
        float2 c[4], s[4];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            const int at = slot + (j ? pair4 : pair0);
            const float4 c4 = *reinterpret_cast<const float4 *>(&cosines[at]), s4 = *reinterpret_cast<const float4 *>(&sines[at]);
            c[j] = make_float2(c4.x, c4.y), c[j + 1] = make_float2(c4.z, c4.w);
            s[j] = make_float2(s4.x, s4.y), s[j + 1] = make_float2(s4.z, s4.w);
        }

        T *out_q = const_cast<T *>(queries(op.dst[0], op.dst_token[0], op.dst_head[0], t));
        T *out_k = const_cast<T *>(keys(op.dst[1], op.dst_token[1], op.dst_head[1], t));
#pragma unroll 1
        for (int h = hs; h - hs < n_heads; h += HS, out_q += HS * op.dst_head[0], out_k += HS * op.dst_head[1]) {
            ask();
            asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD) : "memory");
            // eight pairs (a_j, b_j), two and two: the first elements in ya, the second in yb
            float2 ya[4], yb[4];
            {
                float y[16];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    Vec8<T> x;
#pragma unroll
                    for (int j = 0; j < PIECES / 2; ++j) x.v[j] = ring[place][i * (PIECES / 2) + j][threadIdx.x];
                    unpack8(x, y + 8 * i);
                }
                split_pairs<INTERLEAVED>(y, ya, yb);
            }
            place = place == AHEAD ? 0 : place + 1;
            const bool mine = work && h < n_heads;
            const int w = h < op.n_heads[0] ? 0 : 1;
            if (NORM) {
                if (!mine) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) ya[j] = yb[j] = make_float2(0.f, 0.f);
                }
                if (NORM == 2) {
                    float2 m2 = make_float2(0.f, 0.f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) m2 = add2(m2, add2(ya[j], yb[j]));
                    float m = m2.x + m2.y;
                    for (int o = L >> 1; o; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
                    m = live ? -m * inv_n : 0.f;
                    m2 = make_float2(m, m);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        ya[j] = add2(ya[j], m2);
                        yb[j] = add2(yb[j], m2);
                    }
                }
                float2 q2 = make_float2(0.f, 0.f), p2 = q2;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    q2 = fma2(ya[j], ya[j], q2);
                    p2 = fma2(yb[j], yb[j], p2);
                }
                float q = (q2.x + q2.y) + (p2.x + p2.y);
                for (int o = L >> 1; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
                const float f = rsqrtf(fmaf(q, inv_n, op.eps));
                const float2 f2 = make_float2(f, f);
                const float *g = op.gain[w];
                if (g && live) {
                    float ga[16];
                    load8f(g + e0, ga);
                    load8f(g + e1, ga + 8);
                    float2 g0[4], g1[4];
                    split_pairs<INTERLEAVED>(ga, g0, g1);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        ya[j] = mul2(ya[j], mul2(f2, g0[j]));
                        yb[j] = mul2(yb[j], mul2(f2, g1[j]));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        ya[j] = mul2(ya[j], f2);
                        yb[j] = mul2(yb[j], f2);
                    }
                }
            }
            if (!mine) continue;
            float2 za[4], zb[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 minus = make_float2(-yb[j].x, -yb[j].y);
                za[j] = fma2(ya[j], c[j], mul2(minus, s[j]));
                zb[j] = fma2(yb[j], c[j], mul2(ya[j], s[j]));
            }
            if (turns0 + turns4 < 8) {  // what does not turn passes through (0 * inf must not enter)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int some = j < 2 ? turns0 : turns4, first_of = (j & 1) * 2;
                    if (first_of >= some) za[j].x = ya[j].x, zb[j].x = yb[j].x;
                    if (first_of + 1 >= some) za[j].y = ya[j].y, zb[j].y = yb[j].y;
                }
            }
            float z[16];
            join_pairs<INTERLEAVED>(z, za, zb);
            T *p = w ? out_k : out_q;
            put8(p, pack8<T>(z));
            put8(p + (e1 - e0), pack8<T>(z + 8));
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Any head_dim, dims and strides.  A thread holds one run of eight elements; the half layout's partners
// lie in other threads' runs, wherever half = r/2 puts them, and are read from their place in the ring.
// VEC: head_dim, pointers and strides allow 16-byte pieces; else elements are loaded one by one.
template <typename T, bool INTERLEAVED, bool NORM, bool VEC>
__global__ void __launch_bounds__(32 * VWARPS) k_rotary_any(const __grid_constant__ RotaryOp op) {
    constexpr int PIECES = Vec8<T>::N, PER = 16 / sizeof(T);  // elements of a piece
    __shared__ uint4 ring[AHEAD + 1][PIECES][32 * VWARPS];
    __shared__ float2 angles[32 * VWARPS * 4];  // cosine, sine; at most four pairs a thread
    __shared__ double turns[ROTARY_MAX_PAIRS];
    const int lane = threadIdx.x & 31;
    const int L = op.lanes_per_head, HS = op.heads_at_once, TPT = L * HS;
    const int in_token = threadIdx.x & (TPT - 1), unit = in_token & (L - 1), hs = in_token / L;
    const int r = op.dims, half = r >> 1, e0 = 8 * unit, head_dim = op.head_dim;
    const int n_heads = op.n_heads[0] + op.n_heads[1];
    const bool live = e0 < head_dim;
    // in place and without a norm the runs past r keep their values where they are
    const bool on = live && (NORM || !op.in_place || e0 < r);
    const float inv_n = 1.0f / (float)head_dim;
    float2 *cs = angles + (threadIdx.x / TPT) * (4 * L);
    for (int j = threadIdx.x; j < half; j += 32 * VWARPS) turns[j] = op.turns[j];
    __syncthreads();
    const int at_once = 32 / TPT, step = VWARPS * at_once;
    const int begin = blockIdx.x * op.tokens_per_cta, last = min(op.n_tokens, begin + op.tokens_per_cta);
    const int first = begin + (threadIdx.x >> 5) * at_once;
    if (first >= last) return;

    int next_t = first + lane / TPT, next_h = hs, next_place = 0;  // the next head to ask for
    auto place_of = [&](const void *base, int64_t token, int64_t head, int t, int h) {
        return static_cast<const T *>(base) + t * token + h * head + e0;
    };
    auto ask = [&]() {
        if (on && next_t < last && next_h < n_heads) {
            const int w = next_h < op.n_heads[0] ? 0 : 1;
            const T *p = place_of(op.src[w], op.src_token[w], op.src_head[w], next_t, next_h - (w ? op.n_heads[0] : 0));
            if (VEC) {
#pragma unroll
                for (int i = 0; i < PIECES; ++i)
                    copy_async16(&ring[next_place][i][threadIdx.x], reinterpret_cast<const uint4 *>(p) + i);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    reinterpret_cast<T *>(&ring[next_place][j / PER][threadIdx.x])[j % PER] =
                        e0 + j < head_dim ? p[j] : from_f<T>(0.f);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        next_place = next_place == AHEAD ? 0 : next_place + 1;
        next_h += HS;
        if (next_h - hs >= n_heads) {
            next_h = hs;
            next_t += step;
        }
    };
#pragma unroll 1
    for (int i = 0; i < AHEAD; ++i) ask();

    int row = -1, row_start = 0, row_end = op.n_tokens;
    if (!op.positions) {
        row = row_of(op.cu, op.n_rows, first, lane);
        row_start = row < 0 ? 0 : op.cu[row];
        row_end = row < 0 ? 0 : op.cu[row + 1];  // past every row: nothing to do, and nothing follows
    }
    int place = 0;
    for (int t0 = first; t0 < last; t0 += step) {
        const int t = t0 + lane / TPT;
        bool work = on && t < last;
        int pos = 0;
        if (op.positions) {
            if (t < last) pos = op.positions[t];
        } else {
            while (row >= 0 && t >= row_end && row + 1 < op.n_rows) {
                ++row;
                row_start = row_end;
                row_end = op.cu[row + 1];
            }
            work = work && t < row_end;
            pos = t - row_start;
        }
        __syncwarp();  // the last tokens' sines have been read
        for (int j = in_token; j < half; j += TPT) {
            double a = (double)pos * turns[j];
            a -= rint(a);
            float s, c;
            sincospif(2.0f * (float)a, &s, &c);
            cs[j] = make_float2(op.amplitude * c, op.amplitude * s);
        }
        __syncwarp();
        float c[8], s[8];  // of this thread's elements; s carries the sign of the partner's share
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = e0 + j;
            const bool one = INTERLEAVED ? (e & 1) == 0 : e < half;  // a of its pair, or b
            const float2 v = e < r ? cs[INTERLEAVED ? e >> 1 : (one ? e : e - half)] : make_float2(1.f, 0.f);
            c[j] = v.x;
            s[j] = one ? -v.y : v.y;
        }

#pragma unroll 1
        for (int h = hs; h - hs < n_heads; h += HS) {
            ask();
            asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD) : "memory");
            if (!INTERLEAVED) __syncwarp();  // the other threads' runs are there too
            float y[8], q[8];
            const bool mine = work && h < n_heads;
            const int w = h < op.n_heads[0] ? 0 : 1;
            {
                Vec8<T> x;
#pragma unroll
                for (int i = 0; i < PIECES; ++i) x.v[i] = ring[place][i][threadIdx.x];
                unpack8(x, y);
            }
            int partner[8];
            if (!INTERLEAVED) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int e = e0 + j;
                    partner[j] = e < r ? (e < half ? e + half : e - half) : e;
                    const int in = partner[j] & 7;
                    q[j] = to_f(reinterpret_cast<const T *>(&ring[place][in / PER][threadIdx.x - unit + (partner[j] >> 3)])[in % PER]);
                }
                __syncwarp();  // read: the place may be asked for again
            }
            place = place == AHEAD ? 0 : place + 1;
            if (NORM) {
                if (!mine) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = 0.f;
                }
                float m = 0.f;
                if (op.layer_norm) {
                    m = ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
                    for (int o = L >> 1; o; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
                    m *= inv_n;
                }
                float sq = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    y[j] = e0 + j < head_dim ? y[j] - m : 0.f;
                    sq = fmaf(y[j], y[j], sq);
                }
                for (int o = L >> 1; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
                const float f = rsqrtf(fmaf(sq, inv_n, op.eps));
                const float *g = op.gain[w];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    y[j] *= g && e0 + j < head_dim ? f * __ldg(g + e0 + j) : f;
                    if (!INTERLEAVED) q[j] = (q[j] - m) * (g && partner[j] < head_dim ? f * __ldg(g + partner[j]) : f);
                }
            }
            if (INTERLEAVED) {
#pragma unroll
                for (int j = 0; j < 8; ++j) q[j] = y[j ^ 1];
            }
            if (!mine) continue;
            float z[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)  // past r nothing else may enter (0 * inf)
                z[j] = e0 + j < r ? fmaf(y[j], c[j], q[j] * s[j]) : y[j];
            T *p = const_cast<T *>(place_of(op.dst[w], op.dst_token[w], op.dst_head[w], t, h - (w ? op.n_heads[0] : 0)));
            if (VEC) {
                put8(p, pack8<T>(z));
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (e0 + j < head_dim) p[j] = from_f<T>(z[j]);
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T, bool INTERLEAVED>
void launch_typed(const RotaryOp &op, cudaStream_t st) {
    const dim3 g(op.ctas), b(32 * VWARPS);
    if (op.vec) {
        if (!op.norm) k_rotary<T, INTERLEAVED, 0><<<g, b, 0, st>>>(op);
        else if (!op.layer_norm) k_rotary<T, INTERLEAVED, 1><<<g, b, 0, st>>>(op);
        else k_rotary<T, INTERLEAVED, 2><<<g, b, 0, st>>>(op);
        return;
    }
    if (op.vec8) {
        if (op.norm) k_rotary_any<T, INTERLEAVED, true, true><<<g, b, 0, st>>>(op);
        else k_rotary_any<T, INTERLEAVED, false, true><<<g, b, 0, st>>>(op);
    } else {
        if (op.norm) k_rotary_any<T, INTERLEAVED, true, false><<<g, b, 0, st>>>(op);
        else k_rotary_any<T, INTERLEAVED, false, false><<<g, b, 0, st>>>(op);
    }
}

template <typename T>
void launch_layout(const RotaryOp &op, cudaStream_t st) {
    if (op.interleaved) launch_typed<T, true>(op, st);
    else launch_typed<T, false>(op, st);
}

}  // namespace

void rotary_plan(RotaryOp &op, bool aligned) {
    // vectors of eight elements throughout; in the half layout also the second run of eight
    op.vec8 = aligned && op.head_dim % 8 == 0;
    op.vec = aligned && op.head_dim % 16 == 0 && (op.interleaved || op.dims % 16 == 0);
    op.lanes_per_head = 1;
    while (op.lanes_per_head * (op.vec ? 16 : 8) < op.head_dim) op.lanes_per_head *= 2;
    // heads that a token's threads take at once: four, or as many as there are
    op.heads_at_once = 1;
    while (op.heads_at_once < 4 && op.heads_at_once * 2 <= op.n_heads[0] + op.n_heads[1] &&
           op.heads_at_once * 2 * op.lanes_per_head <= 32)
        op.heads_at_once *= 2;
    // Tokens of one step of a CTA, and how many steps a CTA takes.  Small calls: as many CTAs as are resident
    // at once, so that their start (a row search, the frequencies) is paid once: 14,268 tokens of 40 heads of 128,
    // five steps a CTA, take 67 us, and 71 on CTAs of one step.  From eight steps a CTA on more CTAs than
    // that even out the SMs' ends: 139,809 tokens of 12 heads of 64 take 72 us on 32 CTAs an SM, 85 on 5.
    const int per_step = VWARPS * 32 / (op.lanes_per_head * op.heads_at_once);
    const int steps = (op.n_tokens + per_step - 1) / per_step, resident = SMS * CTAS_RESIDENT;
    const int ctas = steps < 8 * resident ? resident : SMS * CTAS_PER_SM;
    op.tokens_per_cta = (steps + ctas - 1) / ctas * per_step;
    op.ctas = (op.n_tokens + op.tokens_per_cta - 1) / op.tokens_per_cta;
}

cudaError_t launch_rotary(const RotaryOp &op, cudaStream_t st) {
    if (op.n_tokens <= 0) return cudaSuccess;
    if (op.dtype == JD_F32) launch_layout<float>(op, st);
    else if (op.dtype == JD_F16) launch_layout<__half>(op, st);
    else launch_layout<__nv_bfloat16>(op, st);
    return cudaGetLastError();
}

jd_status rotary_turns(const jd_rotary_config &c, int head_dim, double *turns, float *amplitude) {
    if (c.layout != JD_ROTARY_HALF && c.layout != JD_ROTARY_INTERLEAVED)
        return fail(JD_ERR_INVALID_ARG, "unknown rotary layout %d", c.layout);
    if (c.dims < 2 || c.dims % 2 || c.dims > head_dim)
        return fail(JD_ERR_INVALID_ARG, "rotary dims %d: an even number in [2, %d] is required", c.dims, head_dim);
    if (c.scaling < JD_SCALING_NONE || c.scaling > JD_SCALING_YARN)
        return fail(JD_ERR_INVALID_ARG, "unknown rotary scaling %d", c.scaling);
    if (!(c.theta > 0) || !std::isfinite(c.theta)) return fail(JD_ERR_INVALID_ARG, "rotary theta must be positive");
    if (c.scaling != JD_SCALING_NONE && (!(c.factor > 0) || !std::isfinite(c.factor)))
        return fail(JD_ERR_INVALID_ARG, "rotary factor must be positive");
    const int r = c.dims;
    double theta = c.theta, low = 0, high = 0;
    *amplitude = 1.0f;
    // with a single pair the base does not enter (w_0 = 1), and the exponent r / (r - 2) has no value
    if (c.scaling == JD_SCALING_NTK && r > 2) theta *= std::pow(c.factor, r / (r - 2.0));
    const double two_pi = 6.283185307179586476925286766559;
    if (c.scaling == JD_SCALING_YARN) {
        if (c.original_length < 1 || !(c.theta > 1) || !(c.beta_slow > 0) || !(c.beta_fast > c.beta_slow) ||
            !std::isfinite(c.beta_fast))
            return fail(JD_ERR_INVALID_ARG, "yarn: original_length >= 1, theta > 1 and beta_fast > beta_slow > 0 required");
        auto pair_of = [&](double n) { return r * std::log(c.original_length / (n * two_pi)) / (2.0 * std::log(theta)); };
        low = std::fmax(std::floor(pair_of(c.beta_fast)), 0.0);
        high = std::fmin(std::ceil(pair_of(c.beta_slow)), r - 1.0);
        if (c.factor > 1) *amplitude = (float)(0.1 * std::log(c.factor) + 1.0);
    }
    for (int j = 0; j < r / 2; ++j) {
        double w = std::pow(theta, -2.0 * j / r);
        if (c.scaling == JD_SCALING_LINEAR) w /= c.factor;
        if (c.scaling == JD_SCALING_YARN) {
            const double g = std::fmin(std::fmax((j - low) / std::fmax(high - low, 1e-3), 0.0), 1.0);
            w = w * (1.0 - g) + w / c.factor * g;
        }
        turns[j] = w / two_pi;
    }
    return JD_OK;
}

jd_status OpDevice::enter(std::initializer_list<const void *> buffers) {
    for (const void *p : buffers) {
        if (!p) continue;
        cudaPointerAttributes at;
        const cudaError_t e = cudaPointerGetAttributes(&at, p);
        if (e != cudaSuccess) {
            cudaGetLastError();
            return fail(JD_ERR_CUDA, "cudaPointerGetAttributes: %s", cudaGetErrorString(e));
        }
        if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
            return fail(JD_ERR_INVALID_ARG, "a buffer is not device memory");
        if (device >= 0 && at.device != device) return fail(JD_ERR_INVALID_ARG, "buffers of two devices");
        device = at.device;
    }
    int major = 0;
    cudaError_t e = cudaGetDevice(&saved);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device);
    if (e == cudaSuccess && saved != device) e = cudaSetDevice(device);
    if (e != cudaSuccess) return fail(JD_ERR_CUDA, "device %d: %s", device, cudaGetErrorString(e));
    if (major != 10) return fail(JD_ERR_CUDA, "this library is built for sm_100a; device %d is not", device);
    return JD_OK;
}

jd_status check_written(const jd_heads &h, int n_tokens, int head_dim, const char *name) {
    const int64_t big = (int64_t)1 << 46;
    if (h.token_stride < 0 || h.head_stride < 0 || h.token_stride > big || h.head_stride > big)
        return fail(JD_ERR_INVALID_ARG, "%s: strides must lie in [0, 2^46]", name);
    // the nearer of the two axes must clear one head, the other all of the nearer one
    int64_t n0 = h.n_heads, s0 = h.head_stride, n1 = n_tokens, s1 = h.token_stride;
    if (n0 < 2 || (n1 >= 2 && s1 < s0)) {
        std::swap(n0, n1);
        std::swap(s0, s1);
    }
    int64_t span = head_dim;
    if (n0 >= 2) {
        if (s0 < span) return fail(JD_ERR_INVALID_ARG, "%s: strides make its elements overlap", name);
        if (s0 > (((int64_t)1 << 62) - span) / n0) return fail(JD_ERR_INVALID_ARG, "%s: strides too large", name);
        span += s0 * (n0 - 1);
    }
    if (n1 >= 2 && s1 < span) return fail(JD_ERR_INVALID_ARG, "%s: strides make its elements overlap", name);
    return JD_OK;
}

}  // namespace jd

using namespace jd;

namespace {

jd_status check_read(const jd_heads &h, const char *name) {
    const int64_t big = (int64_t)1 << 46;
    if (h.token_stride < 0 || h.head_stride < 0 || h.token_stride > big || h.head_stride > big)
        return fail(JD_ERR_INVALID_ARG, "%s: strides must lie in [0, 2^46]", name);
    return JD_OK;
}

jd_status rotary_call(const jd_rotary_args *a, const jd_head_norm *norm, void *stream) {
    if (a->dtype != JD_F32 && a->dtype != JD_F16 && a->dtype != JD_BF16)
        return fail(JD_ERR_INVALID_ARG, "unknown dtype %d", a->dtype);
    if (a->head_dim < 2 || a->head_dim > 2 * ROTARY_MAX_PAIRS)
        return fail(JD_ERR_INVALID_ARG, "head_dim %d: 2..256 is required", a->head_dim);
    if (a->n_tokens < 0 || a->n_rows < 0) return fail(JD_ERR_INVALID_ARG, "negative n_tokens or n_rows");
    if (a->n_tokens > (1 << 30)) return fail(JD_ERR_INVALID_ARG, "too many tokens: 2^30 at most");
    if (a->q.n_heads < 1 || a->k.n_heads < 0 || a->q.n_heads > 65536 || a->k.n_heads > 65536)
        return fail(JD_ERR_INVALID_ARG, "heads: q 1..65536, k 0..65536");
    if (a->q_out.n_heads != a->q.n_heads || a->k_out.n_heads != a->k.n_heads)
        return fail(JD_ERR_INVALID_ARG, "an output's n_heads differs from its input's");
    RotaryOp op{};
    jd_status s = rotary_turns(a->rotary, a->head_dim, op.turns, &op.amplitude);
    if (s != JD_OK) return s;
    if (norm) {
        if (norm->kind != JD_NORM_RMS && norm->kind != JD_NORM_LAYER)
            return fail(JD_ERR_INVALID_ARG, "unknown norm %d", norm->kind);
        if (!(norm->eps >= 0) || !std::isfinite(norm->eps)) return fail(JD_ERR_INVALID_ARG, "norm eps must be >= 0");
    }
    const bool keys = a->k.n_heads > 0;
    if ((s = check_read(a->q, "q")) != JD_OK || (s = check_written(a->q_out, a->n_tokens, a->head_dim, "q_out")) != JD_OK)
        return s;
    if (keys && ((s = check_read(a->k, "k")) != JD_OK ||
                 (s = check_written(a->k_out, a->n_tokens, a->head_dim, "k_out")) != JD_OK))
        return s;
    if (a->n_tokens == 0) return JD_OK;
    if (!a->q.data || !a->q_out.data || (keys && (!a->k.data || !a->k_out.data)))
        return fail(JD_ERR_INVALID_ARG, "a tensor is NULL");
    if (!a->positions && (!a->cu_seqlens || a->n_rows < 1))
        return fail(JD_ERR_INVALID_ARG, "positions or cu_seqlens is required");
    const jd_heads *in[2] = {&a->q, &a->k}, *out[2] = {&a->q_out, &a->k_out};
    const size_t elem = dtype_bytes(a->dtype);
    bool aligned = (((uintptr_t)(norm ? norm->q_gain : nullptr) | (uintptr_t)(norm ? norm->k_gain : nullptr)) & 15) == 0;
    op.in_place = true;
    for (int w = 0; w < 2; ++w) {
        op.n_heads[w] = in[w]->n_heads;
        if (w == 1 && !keys) break;
        const bool same = in[w]->data == out[w]->data;
        const bool strides = in[w]->token_stride == out[w]->token_stride && in[w]->head_stride == out[w]->head_stride;
        if (same && !strides)
            return fail(JD_ERR_INVALID_ARG, "%s_out is %s with other strides", w ? "k" : "q", w ? "k" : "q");
        op.in_place = op.in_place && same;
        op.src[w] = in[w]->data;
        op.dst[w] = out[w]->data;
        op.src_token[w] = in[w]->token_stride;
        op.src_head[w] = in[w]->head_stride;
        op.dst_token[w] = out[w]->token_stride;
        op.dst_head[w] = out[w]->head_stride;
        aligned = aligned && heads_aligned(*in[w], elem, 16) && heads_aligned(*out[w], elem, 16);
    }
    if (keys && (a->q_out.data == a->k_out.data || a->q_out.data == a->k.data || a->k_out.data == a->q.data))
        return fail(JD_ERR_INVALID_ARG, "an output is the other output or the other input");
    op.dtype = a->dtype;
    op.head_dim = a->head_dim;
    op.dims = a->rotary.dims;
    op.interleaved = a->rotary.layout == JD_ROTARY_INTERLEAVED;
    op.positions = a->positions;
    op.cu = a->cu_seqlens;
    op.n_rows = a->n_rows;
    op.n_tokens = a->n_tokens;
    rotary_plan(op, aligned);
    op.norm = norm != nullptr;
    if (norm) {
        op.layer_norm = norm->kind == JD_NORM_LAYER;
        op.eps = norm->eps;
        op.gain[0] = norm->q_gain;
        op.gain[1] = norm->k_gain;
    }
    OpDevice dev;
    s = dev.enter({op.src[0], op.dst[0], op.src[1], op.dst[1], a->positions ? a->positions : a->cu_seqlens,
                   op.gain[0], op.gain[1]});
    if (s != JD_OK) return s;
    const cudaError_t e = launch_rotary(op, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(JD_ERR_CUDA, "rotary: %s", cudaGetErrorString(e));
    return JD_OK;
}

}  // namespace

extern "C" jd_status jd_rotary(const jd_rotary_args *args, void *stream) {
    clear_error();
    if (!args) return fail(JD_ERR_INVALID_ARG, "NULL argument");
    return rotary_call(args, nullptr, stream);
}

extern "C" jd_status jd_qk_norm_rotary(const jd_rotary_args *args, const jd_head_norm *norm, void *stream) {
    clear_error();
    if (!args || !norm) return fail(JD_ERR_INVALID_ARG, "NULL argument");
    return rotary_call(args, norm, stream);
}
