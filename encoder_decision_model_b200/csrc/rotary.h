// Launcher of the rotary kernel (with or without head norms), for the operator calls and the model.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "op_common.h"

namespace jd {

// Index 0: queries, 1: keys (n_heads[1] may be 0).  Strides in elements.
struct RotaryOp {
    const void *src[2];
    void *dst[2];
    int64_t src_token[2], src_head[2], dst_token[2], dst_head[2];
    int n_heads[2];
    int dtype, head_dim, dims;
    bool interleaved;
    // set by rotary_plan: the kernel, and how a token's heads are laid over its threads
    bool vec, vec8;
    int lanes_per_head, heads_at_once;  // powers of two
    int tokens_per_cta, ctas;
    bool in_place;            // both outputs are their inputs
    bool norm, layer_norm;
    const int *positions, *cu;  // positions, or row offsets [n_rows + 1]
    int n_rows, n_tokens;
    const float *gain[2];
    float eps, amplitude;
    double turns[ROTARY_MAX_PAIRS];
};
// Choose the kernel; `aligned`: pointers and strides (gains included) on multiples of 16 bytes.
void rotary_plan(RotaryOp &op, bool aligned);
cudaError_t launch_rotary(const RotaryOp &op, cudaStream_t st);

}  // namespace jd
