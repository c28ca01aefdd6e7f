// Host-side helpers of the stateless operator calls: where their buffers live, and the checks of
// jd_heads that they share.
#pragma once

#include <cuda_runtime.h>

#include <initializer_list>

#include "host_common.h"

namespace jd {

// Makes the device that holds the buffers current for one call and puts the caller's back.
struct OpDevice {
    int saved = -1, device = -1;
    jd_status enter(std::initializer_list<const void *> buffers);
    ~OpDevice() {
        if (saved >= 0 && saved != device) cudaSetDevice(saved);
    }
};

// A tensor that is written: strides that keep its elements apart.
jd_status check_written(const jd_heads &h, int n_tokens, int head_dim, const char *name);

inline size_t dtype_bytes(int dtype) { return dtype == JD_F32 ? 4 : 2; }

// Pointer and strides on multiples of `bytes`.
inline bool heads_aligned(const jd_heads &h, size_t elem, size_t bytes) {
    return ((uintptr_t)h.data | (uintptr_t)(h.token_stride * (int64_t)elem) |
            (uintptr_t)(h.head_stride * (int64_t)elem)) % bytes == 0;
}

// Angle per position of every rotated pair in turns (w_j / 2 pi), and the factor of cos and sin.
constexpr int ROTARY_MAX_PAIRS = 128;
jd_status rotary_turns(const jd_rotary_config &c, int head_dim, double *turns, float *amplitude);

}  // namespace jd
