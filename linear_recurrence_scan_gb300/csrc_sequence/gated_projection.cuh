// gated_projection.cuh -- the gated feed-forward block's launchers, as the C
// entry points call them.
#pragma once

#include "sequence.cuh"

namespace rlscan {
namespace seq {

// act(z) and its slope
__device__ __forceinline__ float2 act_slope(float z, int act)
{
    if (act == RLSCAN_SILU) {
        const float g = sigmoid(z), a = z * g;
        return make_float2(a, fmaf(a, 1.f - g, g));
    }
    const float half = 0.5f * erfcf(-0.70710678118654752f * z);  // the normal distribution up to z
    return make_float2(z * half, fmaf(z * 0.3989422804014327f, exp2_fast(-0.5f * kLog2e * z * z), half));
}

// Few rows: read from the weights' rows as they are (no workspace).
bool projection_is_few(const rlscan_gated_projection_args &a);
rlscan_status launch_gated_projection_few(const rlscan_gated_projection_args &a, void *h, cudaStream_t s);

size_t gated_projection_workspace(const rlscan_gated_projection_args &a);
rlscan_status launch_gated_projection(const rlscan_gated_projection_args &a, void *h, void *ws, cudaStream_t s);
size_t gated_projection_backward_workspace(const rlscan_gated_projection_args &a);
rlscan_status launch_gated_projection_backward(const rlscan_gated_projection_args &a, const void *grad_h,
                                               int64_t grad_h_stride, void *grad_x, void *grad_gate, void *grad_up,
                                               void *ws, cudaStream_t s);
rlscan_status gated_projection_status(cudaStream_t s);

}  // namespace seq
}  // namespace rlscan
