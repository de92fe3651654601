// Interface between the C-ABI layer (api.hip) and the kernels of a layer that stand around
// the experts' products: the norm (norm.hip), the gated activation (activation.hip), 4-bit
// rows and products (mx.hip) and the whole layer for a few tokens (layer.hip). Not
// installed, not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "experts.h"
#include "moonep.h"

namespace moonep {

// Rows of a norm and where they go. out_kind: emit::Out.
struct NormRows {
    const void *x, *residual, *gamma;
    void *sum, *out, *scale;
    float *inv_rms;
    double eps;
    int64_t n_rows;
    int32_t cols, bf16, out_kind;
};
hipError_t launch_norm(const NormRows &n, hipStream_t st);

struct NormGrad {
    const void *grad_out, *grad_sum, *x, *gamma;
    const float *inv_rms;
    void *grad_x;
    float *grad_gamma, *work;
    int64_t n_rows;
    int32_t cols, bf16;
};
hipError_t launch_norm_backward(const NormGrad &n, hipStream_t st);

// gate and up: rows `ld` elements apart. out_kind: emit::Out.
struct GatedRows {
    const void *gate, *up;
    void *out, *scale;
    int64_t n_rows, ld;
    int32_t cols, bf16, out_kind;
};
hipError_t launch_swiglu(const GatedRows &g, hipStream_t st);

struct GatedGrad {
    const void *grad_out, *gate, *up;
    void *grad_gate, *grad_up;
    int64_t n_rows, ld, grad_ld;
    int32_t cols, bf16;
};
hipError_t launch_swiglu_backward(const GatedGrad &g, hipStream_t st);

hipError_t launch_quantize_rows_mx(int64_t n_rows, int32_t cols, const void *x, int bf16,
                                    uint8_t *q, uint8_t *scale, hipStream_t st);

// sh.n_in counts values; sh.block and sh.scale_block are in bytes.
hipError_t launch_expert_matmul_mx(const ExpertShape &sh, const int32_t *seg_ptr, const uint8_t *x,
                                    const uint8_t *x_scale, const uint8_t *w, const uint8_t *w_scale,
                                    const uint8_t *dup_w, const uint8_t *dup_scale, void *y,
                                    int y_bf16, hipStream_t st);

// The whole layer for a few tokens.
constexpr int kFewTokens = MOONEP_FEW_TOKENS;
struct FewLayer {
    const int32_t *ids;
    const float *topk_w;
    const void *x, *gate, *up, *down;
    const uint8_t *gate_scale, *up_scale, *down_scale;  // NULL: weights of the rows' type
    void *out, *work;
    int64_t in_block, out_block, in_scale_block, out_scale_block;  // elements (4 bits: bytes)
    int32_t T, E, K, H, F, bf16;
};
hipError_t launch_few_layer(const FewLayer &l, hipStream_t st);
int64_t few_layer_bytes(int32_t T, int32_t E, int32_t K, int32_t F);

}  // namespace moonep
