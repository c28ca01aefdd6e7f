// Launchers of the differential attention, for the operator call and the model.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "op_common.h"

namespace jd {

struct DiffOp {
    const int *cu;
    int n_rows, n_tokens, window;  // window <= n_tokens; negative: none
    int heads, kv_heads;
    int qk_dtype, v_dtype;
    const void *q, *k, *v;         // FP32 path
    int64_t q_token, q_head, k_token, k_head, v_token, v_head;
    void *out;
    int64_t out_token, out_head;
    bool out32;                    // out and its strides on 32-byte multiples
    const float *lq1, *lk1, *lq2, *lk2, *gain;
    float lambda_init, eps, scale;
    unsigned *status;
};

// Maps of q, k and v for the tensor-core kernel: (element, head, token), boxes of 64
// elements of one head and 128 (q) or 64 tokens.
struct DiffMaps {
    CUtensorMap q, k, v;
};
jd_status make_diff_maps(const DiffOp &op, DiffMaps *maps);

// Once per device before the first launch there (cheap when done).
cudaError_t diff_attention_prepare(int device);
cudaError_t launch_diff_attention(const DiffOp &op, const DiffMaps *maps, int num_sms, cudaStream_t st);

}  // namespace jd
