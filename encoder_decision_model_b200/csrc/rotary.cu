// Rotary positions, with or without a norm of every head in the same pass.
//
// A warp takes one token: all its query and key heads turn by the same angles, so the warp forms
// the r/2 sines and cosines once (a lane per pair) and passes them on through shared memory.  The
// token's heads then go by in groups: head_dim / 8 lanes (up to the next power of two) hold one
// head, eight elements a lane, so that a head's norm is a few shuffles and a lane's loads and
// stores are 16 bytes.  Up to four groups are loaded before the first is worked on.
//
// The pass is bound by HBM: it reads and writes each element once.  Computing the angles instead
// of reading a table costs a fifth of the issue slots that the memory time leaves free and keeps
// any position exact: p * w_j is formed and reduced to a fraction of a turn in 64 bits (in 32 bits
// the angle of position 10^5 is off by 4e-3), sine and cosine of the fraction are then FP32.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <cmath>

#include "op_common.h"
#include "rotary.h"

namespace jd {

namespace {

constexpr int WARPS = 8;

enum Pairing { INTERLEAVED, HALF_LANES, HALF_SHARED };

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

template <typename T>
struct alignas(16) Vec8 {
    T v[8];
};

// Eight elements of a head from element e0 on; past head_dim zeros are read and nothing is written.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(Vec8<T> &x, const T *p, int e0, int head_dim) {
    if (VEC) {
        x = *reinterpret_cast<const Vec8<T> *>(p + e0);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x.v[j] = e0 + j < head_dim ? p[e0 + j] : from_f<T>(0.f);
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *p, const Vec8<T> &x, int e0, int head_dim) {
    if (VEC) {
        *reinterpret_cast<Vec8<T> *>(p + e0) = x;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (e0 + j < head_dim) p[e0 + j] = x.v[j];
    }
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

template <typename T, Pairing PAIR, bool NORM, bool VEC>
__global__ void __launch_bounds__(32 * WARPS) k_rotary(const __grid_constant__ RotaryOp op) {
    __shared__ float2 cs_all[WARPS][ROTARY_MAX_PAIRS];
    __shared__ float swap_all[PAIR == HALF_SHARED ? WARPS : 1][PAIR == HALF_SHARED ? 32 * 8 : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float2 *cs = cs_all[warp];
    float *swap = swap_all[PAIR == HALF_SHARED ? warp : 0];
    const int r = op.dims, half = r >> 1;

    double turns[ROTARY_MAX_PAIRS / 32];
#pragma unroll
    for (int i = 0; i < ROTARY_MAX_PAIRS / 32; ++i) {
        const int j = lane + 32 * i;
        turns[i] = j < half ? op.turns[j] : 0.0;
    }
    const int G = op.lanes_per_head;      // lanes of one head: a power of two
    const int e0 = (lane & (G - 1)) * 8;  // this lane's first element, the same in every head
    const int heads_at_once = 32 / G, sub = lane / G;
    const int n_heads = op.n_heads[0] + op.n_heads[1];
    const bool live = e0 < op.head_dim;
    // in place and without a norm the elements past r keep their values where they are
    const bool skip = !live || (!NORM && op.in_place && e0 >= r);
    const float inv_n = 1.0f / (float)op.head_dim;
    const int partner = PAIR == HALF_LANES ? (e0 < half ? lane + (half >> 3) : lane - (half >> 3)) : lane;

    for (int t = blockIdx.x * WARPS + warp; t < op.n_tokens; t += gridDim.x * WARPS) {
        int pos;
        if (op.positions) {
            pos = op.positions[t];
        } else {
            const int row = row_of(op.cu, op.n_rows, t, lane);
            if (row < 0) continue;
            pos = t - op.cu[row];
        }
#pragma unroll
        for (int i = 0; i < ROTARY_MAX_PAIRS / 32; ++i) {
            if (32 * i < half) {
                double a = (double)pos * turns[i];
                a -= rint(a);
                float s, c;
                sincospif(2.0f * (float)a, &s, &c);
                cs[lane + 32 * i] = make_float2(op.amplitude * c, op.amplitude * s);
            }
        }
        __syncwarp();
        float c[8], s[8];  // of this lane's elements; s carries the sign of the partner's share
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = e0 + j;
            const bool first = PAIR == INTERLEAVED ? (e & 1) == 0 : e < half;
            const int pair = PAIR == INTERLEAVED ? e >> 1 : (first ? e : e - half);
            const float2 v = e < r ? cs[pair] : make_float2(1.f, 0.f);
            c[j] = v.x;
            s[j] = first ? -v.y : v.y;
        }
        __syncwarp();

        for (int h0 = 0; h0 < n_heads; h0 += 4 * heads_at_once) {
            Vec8<T> x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int hh = h0 + u * heads_at_once + sub;
                if (hh < n_heads && !skip) {
                    const int w = hh < op.n_heads[0] ? 0 : 1;
                    const int h = w ? hh - op.n_heads[0] : hh;
                    load8<T, VEC>(x[u], static_cast<const T *>(op.src[w]) + t * op.src_token[w] + h * op.src_head[w], e0,
                                  op.head_dim);
                }
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (h0 + u * heads_at_once >= n_heads) break;  // the same for the whole warp
                const int hh = h0 + u * heads_at_once + sub;
                const bool on = hh < n_heads && !skip;
                const int w = hh < op.n_heads[0] ? 0 : 1;
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = on ? to_f(x[u].v[j]) : 0.f;
                if (NORM) {
                    if (op.layer_norm) {
                        float m = ((y[0] + y[1]) + (y[2] + y[3])) + ((y[4] + y[5]) + (y[6] + y[7]));
                        for (int o = G >> 1; o; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
                        m *= inv_n;
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = VEC || e0 + j < op.head_dim ? y[j] - m : 0.f;
                        if (!live) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) y[j] = 0.f;
                        }
                    }
                    float q = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) q = fmaf(y[j], y[j], q);
                    for (int o = G >> 1; o; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
                    const float f = 1.0f / sqrtf(fmaf(q, inv_n, op.eps));
                    const float *g = w ? op.gain[1] : op.gain[0];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        y[j] *= f;
                        if (g && e0 + j < op.head_dim) y[j] *= __ldg(g + e0 + j);
                    }
                }
                float p[8];
                if (PAIR == INTERLEAVED) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[j] = y[j ^ 1];
                } else if (PAIR == HALF_LANES) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[j] = __shfl_sync(0xffffffffu, y[j], partner);
                } else {
                    float *mine = swap + sub * G * 8;
#pragma unroll
                    for (int j = 0; j < 8; ++j) mine[e0 + j] = y[j];
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int e = e0 + j;
                        p[j] = e < r ? mine[e < half ? e + half : e - half] : 0.f;
                    }
                    __syncwarp();
                }
                Vec8<T> z;
#pragma unroll
                for (int j = 0; j < 8; ++j)  // past r the partner is another element: it must not enter (0 * inf)
                    z.v[j] = from_f<T>(e0 + j < r ? fmaf(p[j], s[j], y[j] * c[j]) : y[j]);
                if (on) {
                    const int h = w ? hh - op.n_heads[0] : hh;
                    store8<T, VEC>(static_cast<T *>(op.dst[w]) + t * op.dst_token[w] + h * op.dst_head[w], z, e0,
                                   op.head_dim);
                }
            }
        }
    }
}

template <typename T, bool NORM>
void launch_pairing(const RotaryOp &op, int grid, cudaStream_t st) {
    const dim3 g(grid), b(32 * WARPS);
    if (op.vec) {
        if (op.interleaved) k_rotary<T, INTERLEAVED, NORM, true><<<g, b, 0, st>>>(op);
        else if (op.dims % 16 == 0) k_rotary<T, HALF_LANES, NORM, true><<<g, b, 0, st>>>(op);
        else k_rotary<T, HALF_SHARED, NORM, true><<<g, b, 0, st>>>(op);
    } else {
        if (op.interleaved) k_rotary<T, INTERLEAVED, NORM, false><<<g, b, 0, st>>>(op);
        else k_rotary<T, HALF_SHARED, NORM, false><<<g, b, 0, st>>>(op);
    }
}

template <typename T>
void launch_norm(const RotaryOp &op, int grid, cudaStream_t st) {
    if (op.norm) launch_pairing<T, true>(op, grid, st);
    else launch_pairing<T, false>(op, grid, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryOp &op, cudaStream_t st) {
    if (op.n_tokens <= 0) return cudaSuccess;
    // enough CTAs to fill every SM several times over; beyond that warps walk the tokens
    const int want = (op.n_tokens + WARPS - 1) / WARPS;
    const int grid = want < 148 * 8 ? want : 148 * 8;
    if (op.dtype == JD_F32) launch_norm<float>(op, grid, st);
    else if (op.dtype == JD_F16) launch_norm<__half>(op, grid, st);
    else launch_norm<__nv_bfloat16>(op, grid, st);
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
    op.vec = a->head_dim % 8 == 0;
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
        op.vec = op.vec && heads_aligned(*in[w], elem, 16) && heads_aligned(*out[w], elem, 16);
    }
    if (keys && (a->q_out.data == a->k_out.data || a->q_out.data == a->k.data || a->k_out.data == a->q.data))
        return fail(JD_ERR_INVALID_ARG, "an output is the other output or the other input");
    op.dtype = a->dtype;
    op.head_dim = a->head_dim;
    op.dims = a->rotary.dims;
    op.interleaved = a->rotary.layout == JD_ROTARY_INTERLEAVED;
    op.lanes_per_head = 1;
    while (op.lanes_per_head * 8 < a->head_dim) op.lanes_per_head *= 2;
    op.positions = a->positions;
    op.cu = a->cu_seqlens;
    op.n_rows = a->n_rows;
    op.n_tokens = a->n_tokens;
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
