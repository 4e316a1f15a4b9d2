// gated_projection.cuh -- the gated feed-forward block's launchers, as the C
// entry points call them.
#pragma once

#include "sequence.cuh"

namespace rlscan {
namespace seq {

// act(z) and its slope
struct Activated {
    f2 value, slope;
};
__device__ __forceinline__ Activated silu(f2 z)
{
    const f2 g = sigmoid(z), a = mul2(z, g);
    return {a, fma2(a, fma2(g, both(-1.f), both(1.f)), g)};
}
// With the normal distribution up to -|z|, exp(-z^2 / 2) t Q(t), t = 1 / (1 + 0.44
// |z| / sqrt 2): Q is the polynomial of degree 7 whose largest relative error
// over |z| < 14 is least (1.8e-7, 5e-7 as evaluated here; found by reweighted
// least squares), and the exponential is the slope's too.  The forward pass of 5000 x
// 2560 x 6912 took 248 us with the error function of CUDA, and takes 221.
__device__ __forceinline__ Activated gelu(f2 z)
{
    const float2 h = halves(z);
    const f2 t = rcp_fast(fma2(pair(fabsf(h.x), fabsf(h.y)), both(0.311126984f), both(1.f)));
    const f2 e = exp2_fast(mul2(mul2(z, z), both(-0.5f * kLog2e)));
    f2 q = both(0.0356117043f);
    q = fma2(q, t, both(-0.138973894f));
    q = fma2(q, t, both(0.148343561f));
    q = fma2(q, t, both(-0.0100901891f));
    q = fma2(q, t, both(0.107906052f));
    q = fma2(q, t, both(0.108656792f));
    q = fma2(q, t, both(0.124435588f));
    q = fma2(q, t, both(0.124110477f));
    const float2 far = halves(mul2(mul2(e, t), q));
    const f2 up_to = pair(h.x < 0.f ? far.x : 1.f - far.x, h.y < 0.f ? far.y : 1.f - far.y);
    return {mul2(z, up_to), fma2(mul2(z, both(0.3989422804014327f)), e, up_to)};
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
