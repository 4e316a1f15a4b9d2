// gated_projection.cuh -- the gated feed-forward block's launchers, as the C
// entry points call them.
#pragma once

#include "sequence.cuh"

namespace rlscan {
namespace seq {

size_t gated_projection_workspace(const rlscan_gated_projection_args &a);
rlscan_status launch_gated_projection(const rlscan_gated_projection_args &a, void *h, void *ws, cudaStream_t s);
size_t gated_projection_backward_workspace(const rlscan_gated_projection_args &a);
rlscan_status launch_gated_projection_backward(const rlscan_gated_projection_args &a, const void *grad_h,
                                               int64_t grad_h_stride, void *grad_x, void *grad_gate, void *grad_up,
                                               void *ws, cudaStream_t s);
rlscan_status gated_projection_status(cudaStream_t s);

}  // namespace seq
}  // namespace rlscan
