// Interface between the C-ABI layer (api.hip) and the kernels that work on what
// dispatch wrote: the experts' products (experts.hip) and the gradients' norm and
// clipping (grads.hip). Not installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moonep.h"

namespace moonep {

// Shape of one product grouped by expert. Rank r's S*K rows are cut by seg_ptr[r]
// (n_seg + 1 offsets) into segments: j < G is home expert r*G + j, G + b is
// duplicate slot b of the rank.
struct ExpertShape {
    int32_t R, G, B;      // B: duplicate slots a segment can name, min(B, dcap)
    int32_t slots;        // duplicate slots per rank of the weight and gradient arrays
    int32_t n_seg, SK;
    int32_t n_in, n_out;  // columns of x and of y
    int32_t transposed;   // an expert's matrix is [n_in, n_out] (0) or [n_out, n_in] (1)
    int64_t block;        // elements from one expert's matrix to the next
    int64_t scale_block;  // the same for the 8-bit weights' scales
};

// Largest row of the products, in bytes: a tile of 256 rows is addressed with
// 32-bit byte offsets.
constexpr int64_t kMaxProductRow = (int64_t)1 << 22;
// Columns whose 8-bit products cannot overflow int32: 128 * 128 * n < 2^31.
constexpr int64_t kMaxQuantCols = 131071;

// Outputs of this size or more are stored past the caches: the last of them, which all
// XCDs share, holds as much, and what lies there when the next kernel reads it is worth
// more than the faster store.
constexpr int64_t kStreamBytes = (int64_t)256 << 20;

// One store, past the caches if `stream`. The empty statements keep the compiler from
// making one plain store of the two.
template <typename V>
__device__ __forceinline__ void store_streamed(V v, V *to, bool stream) {
    if (stream) {
        asm volatile("");
        __builtin_nontemporal_store(v, to);
        asm volatile("");
    } else {
        *to = v;
    }
}

hipError_t launch_expert_matmul(const ExpertShape &sh, const int32_t *seg_ptr, const void *x,
                                const void *w, const void *dup_w, void *y, int bf16,
                                hipStream_t st);

hipError_t launch_expert_wgrad(const ExpertShape &sh, const int32_t *seg_ptr, const void *x,
                               const void *g, float *home, float *dup, int bf16, hipStream_t st);

hipError_t launch_expert_matmul_quant(const ExpertShape &sh, const int32_t *seg_ptr,
                                      const int8_t *x, const float *x_scale, const int8_t *w,
                                      const float *w_scale, const int8_t *dup_w,
                                      const float *dup_scale, void *y, int y_bf16, hipStream_t st);

hipError_t launch_quantize_rows(int64_t n_rows, int32_t cols, const void *x, int bf16, int8_t *q,
                                float *scale, hipStream_t st);

// The host arrays of n tensors are read during the call only.
hipError_t launch_grad_sumsq(int32_t n, const void *const *grads, const int64_t *numel,
                             const int32_t *dtypes, double *acc, hipStream_t st);
hipError_t launch_grad_clip(int32_t n, const void *const *grads, void *const *outs,
                            const int64_t *numel, const int32_t *dtypes, const double *acc,
                            double max_norm, float *norm, hipStream_t st);

}  // namespace moonep
