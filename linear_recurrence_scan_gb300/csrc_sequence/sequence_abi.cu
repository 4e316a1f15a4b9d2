// sequence_abi.cu -- the extern "C" entry points of the state-space layer:
// argument validation, then the launchers of k_selective_scan*.cu,
// k_causal_conv.cu and k_rms_norm.cu.
#include "abi_checks.cuh"

using namespace rlscan;
using namespace rlscan::seq;

namespace {

rlscan_status check_scan(const rlscan_selective_scan_args *a)
{
    if (a == nullptr) return RLSCAN_ERR_NULL;
    if (!sizes_ok({a->N, a->T, a->D, 8})) return RLSCAN_ERR_SHAPE;
    if (a->S < 1 || a->S > kMaxStates || !is_io_type(a->dtype) || (a->delta_softplus != 0 && a->delta_softplus != 1))
        return RLSCAN_ERR_ARG_VALUE;
    return RLSCAN_OK;
}

rlscan_status check_scan_inputs(const rlscan_selective_scan_args &a)
{
    if (a.A == nullptr || (a.T > 0 && (!a.x.data || !a.delta.data || !a.B.data || !a.C.data))) return RLSCAN_ERR_NULL;
    return RLSCAN_OK;
}

bool is_scan_input(const void *out, const rlscan_selective_scan_args &a)
{
    return equals_any(out, {a.x.data, a.delta.data, a.z.data, a.B.data, a.C.data, a.A, a.skip, a.delta_bias,
                            a.initial_state, a.resets, a.lengths});
}

bool scan_reachable(const rlscan_selective_scan_args &a)
{
    return reachable({a.x.data, a.delta.data, a.z.data, a.B.data, a.C.data, a.A, a.skip, a.delta_bias,
                      a.initial_state, a.resets, a.lengths});
}

rlscan_status check_conv(const rlscan_causal_conv_args *a)
{
    if (a == nullptr) return RLSCAN_ERR_NULL;
    if (!sizes_ok({a->N, a->T, a->D})) return RLSCAN_ERR_SHAPE;
    if (a->K < 1 || a->K > kMaxTaps || !is_io_type(a->dtype) || (a->silu != 0 && a->silu != 1))
        return RLSCAN_ERR_ARG_VALUE;
    return RLSCAN_OK;
}

bool is_conv_input(const void *out, const rlscan_causal_conv_args &a)
{
    return equals_any(out, {a.x.data, a.weight, a.bias, a.initial_state, a.resets, a.lengths});
}

bool conv_reachable(const rlscan_causal_conv_args &a)
{
    return reachable({a.x.data, a.weight, a.bias, a.initial_state, a.resets, a.lengths});
}

}  // namespace

extern "C" {

RLSCAN_API size_t rlscan_selective_scan_workspace_bytes(const rlscan_selective_scan_args *args)
{
    if (check_scan(args) != RLSCAN_OK) return 0;
    return selective_scan_workspace(*args);
}

RLSCAN_API rlscan_status rlscan_selective_scan(const rlscan_selective_scan_args *args, void *y, float *final_state,
                                               float *checkpoints, void *ws, size_t ws_bytes, rlscan_stream_t stream)
{
    RLSCAN_TRY(check_scan(args));
    const rlscan_selective_scan_args &a = *args;
    if (a.N == 0 || a.D == 0) return RLSCAN_OK;
    RLSCAN_TRY(check_scan_inputs(a));
    if (a.T > 0 && y == nullptr) return RLSCAN_ERR_NULL;
    for (const void *o : {static_cast<const void *>(y), static_cast<const void *>(final_state),
                          static_cast<const void *>(checkpoints)})
        if (o != nullptr && is_scan_input(o, a)) return RLSCAN_ERR_ARG_CONFLICT;
    if (!workspace_ok(ws, ws_bytes, selective_scan_workspace(a))) return RLSCAN_ERR_WORKSPACE;
    if (!scan_reachable(a) || !reachable({y, final_state, checkpoints})) return RLSCAN_ERR_MEMORY;
    return launch_selective_scan(a, y, final_state, checkpoints, ws, cs(stream));
}

RLSCAN_API size_t rlscan_selective_scan_backward_workspace_bytes(const rlscan_selective_scan_args *args)
{
    if (check_scan(args) != RLSCAN_OK) return 0;
    return selective_scan_backward_workspace(*args);
}

RLSCAN_API rlscan_status rlscan_selective_scan_backward(const rlscan_selective_scan_args *args,
                                                        const rlscan_array3 *grad_y, const float *grad_final_state,
                                                        const float *checkpoints,
                                                        const rlscan_selective_scan_grads *grads, void *ws,
                                                        size_t ws_bytes, rlscan_stream_t stream)
{
    RLSCAN_TRY(check_scan(args));
    if (grad_y == nullptr || grads == nullptr) return RLSCAN_ERR_NULL;
    const rlscan_selective_scan_args &a = *args;
    const rlscan_selective_scan_grads &g = *grads;
    if (a.N > 0 && a.D > 0) {  // without channels the gradients of B and C are zeros, and read nothing
        RLSCAN_TRY(check_scan_inputs(a));
        if (a.T > 0 && (!grad_y->data || !checkpoints || !g.x)) return RLSCAN_ERR_NULL;
    }
    if ((g.z && !a.z.data) || (g.skip && !a.skip) || (g.delta_bias && !a.delta_bias)) return RLSCAN_ERR_ARG_CONFLICT;
    for (const void *o : {static_cast<const void *>(g.x), static_cast<const void *>(g.delta), static_cast<const void *>(g.z),
                          static_cast<const void *>(g.B), static_cast<const void *>(g.C), static_cast<const void *>(g.A),
                          static_cast<const void *>(g.skip), static_cast<const void *>(g.delta_bias),
                          static_cast<const void *>(g.initial_state)})
        if (o != nullptr && (is_scan_input(o, a) || equals_any(o, {grad_y->data, grad_final_state, checkpoints})))
            return RLSCAN_ERR_ARG_CONFLICT;
    if (!workspace_ok(ws, ws_bytes, selective_scan_backward_workspace(a))) return RLSCAN_ERR_WORKSPACE;
    if (!scan_reachable(a) || !reachable({grad_y->data, grad_final_state, checkpoints, g.x, g.delta, g.z, g.B, g.C, g.A,
                                          g.skip, g.delta_bias, g.initial_state}))
        return RLSCAN_ERR_MEMORY;
    return launch_selective_scan_backward(a, *grad_y, grad_final_state, checkpoints, g, ws, cs(stream));
}

RLSCAN_API rlscan_status rlscan_selective_scan_step(const rlscan_selective_scan_args *args, float *state, int64_t P,
                                                    const int32_t *slots, void *y, rlscan_stream_t stream)
{
    RLSCAN_TRY(check_scan(args));
    const rlscan_selective_scan_args &a = *args;
    if (a.T != 1 || P < 0 || (slots == nullptr && P < a.N)) return RLSCAN_ERR_SHAPE;
    if (a.N == 0 || a.D == 0) return RLSCAN_OK;
    RLSCAN_TRY(check_scan_inputs(a));
    if ((P > 0 && state == nullptr) || y == nullptr) return RLSCAN_ERR_NULL;
    for (const void *o : {static_cast<const void *>(y), static_cast<const void *>(state)})
        if (o != nullptr && (is_scan_input(o, a) || o == slots)) return RLSCAN_ERR_ARG_CONFLICT;
    if (y == state) return RLSCAN_ERR_ARG_CONFLICT;
    if (!scan_reachable(a) || !reachable({state, slots, y})) return RLSCAN_ERR_MEMORY;
    return launch_selective_scan_step(a, state, P, slots, y, cs(stream));
}

RLSCAN_API rlscan_status rlscan_causal_conv(const rlscan_causal_conv_args *args, void *y, void *final_state,
                                            rlscan_stream_t stream)
{
    RLSCAN_TRY(check_conv(args));
    const rlscan_causal_conv_args &a = *args;
    if (a.N == 0 || a.D == 0) return RLSCAN_OK;
    if (!a.weight || (a.T > 0 && (!a.x.data || !y))) return RLSCAN_ERR_NULL;
    for (const void *o : {static_cast<const void *>(y), static_cast<const void *>(final_state)})
        if (o != nullptr && is_conv_input(o, a)) return RLSCAN_ERR_ARG_CONFLICT;
    if (!conv_reachable(a) || !reachable({y, final_state})) return RLSCAN_ERR_MEMORY;
    return launch_causal_conv(a, y, final_state, cs(stream));
}

RLSCAN_API size_t rlscan_causal_conv_backward_workspace_bytes(const rlscan_causal_conv_args *args)
{
    if (check_conv(args) != RLSCAN_OK) return 0;
    return causal_conv_backward_workspace(*args);
}

RLSCAN_API rlscan_status rlscan_causal_conv_backward(const rlscan_causal_conv_args *args, const rlscan_array3 *grad_y,
                                                     const void *grad_final_state, void *grad_x, float *grad_weight,
                                                     float *grad_bias, void *grad_initial_state, void *ws,
                                                     size_t ws_bytes, rlscan_stream_t stream)
{
    RLSCAN_TRY(check_conv(args));
    if (grad_y == nullptr) return RLSCAN_ERR_NULL;
    const rlscan_causal_conv_args &a = *args;
    if (a.D == 0) return RLSCAN_OK;
    if (a.N > 0 && (!a.weight || (a.T > 0 && (!a.x.data || !grad_y->data || !grad_x)))) return RLSCAN_ERR_NULL;
    for (const void *o : {static_cast<const void *>(grad_x), static_cast<const void *>(grad_weight),
                          static_cast<const void *>(grad_bias), static_cast<const void *>(grad_initial_state)})
        if (o != nullptr && (is_conv_input(o, a) || equals_any(o, {grad_y->data, grad_final_state})))
            return RLSCAN_ERR_ARG_CONFLICT;
    if ((grad_weight || grad_bias) && !workspace_ok(ws, ws_bytes, causal_conv_backward_workspace(a)))
        return RLSCAN_ERR_WORKSPACE;
    if (!conv_reachable(a) ||
        !reachable({grad_y->data, grad_final_state, grad_x, grad_weight, grad_bias, grad_initial_state}))
        return RLSCAN_ERR_MEMORY;
    return launch_causal_conv_backward(a, *grad_y, grad_final_state, grad_x, grad_weight, grad_bias,
                                       grad_initial_state, ws, cs(stream));
}

RLSCAN_API rlscan_status rlscan_causal_conv_step(const rlscan_causal_conv_args *args, void *state, int64_t P,
                                                 const int32_t *slots, void *y, rlscan_stream_t stream)
{
    RLSCAN_TRY(check_conv(args));
    const rlscan_causal_conv_args &a = *args;
    if (a.T != 1 || P < 0 || (slots == nullptr && P < a.N)) return RLSCAN_ERR_SHAPE;
    if (a.N == 0 || a.D == 0) return RLSCAN_OK;
    if (!a.weight || !a.x.data || !y || (P > 0 && a.K > 1 && !state)) return RLSCAN_ERR_NULL;
    for (const void *o : {static_cast<const void *>(y), static_cast<const void *>(state)})
        if (o != nullptr && (is_conv_input(o, a) || o == slots)) return RLSCAN_ERR_ARG_CONFLICT;
    if (y == state) return RLSCAN_ERR_ARG_CONFLICT;
    if (!conv_reachable(a) || !reachable({state, slots, y})) return RLSCAN_ERR_MEMORY;
    return launch_causal_conv_step(a, state, P, slots, y, cs(stream));
}

RLSCAN_API rlscan_status rlscan_add_rms_norm(const void *x, int64_t x_stride, const void *residual,
                                             int64_t residual_stride, const float *weight, int64_t M, int64_t D,
                                             float eps, rlscan_dtype dtype, rlscan_dtype residual_dtype, void *y,
                                             float *scales, void *residual_out, rlscan_stream_t stream)
{
    if (!sizes_ok({M, D})) return RLSCAN_ERR_SHAPE;
    if (!is_io_type(dtype) || (residual != nullptr && residual_dtype != RLSCAN_F32 && residual_dtype != dtype) ||
        !(eps >= 0.f))
        return RLSCAN_ERR_ARG_VALUE;
    if (M == 0 || D == 0) return RLSCAN_OK;
    if (!x || !weight || !y || (residual && !residual_out)) return RLSCAN_ERR_NULL;
    for (const void *o : {static_cast<const void *>(y), static_cast<const void *>(scales),
                          static_cast<const void *>(residual_out)})
        if (o != nullptr && equals_any(o, {x, residual, weight})) return RLSCAN_ERR_ARG_CONFLICT;
    if (y == residual_out || y == scales || (scales && scales == residual_out)) return RLSCAN_ERR_ARG_CONFLICT;
    if (!reachable({x, residual, weight, y, scales, residual_out})) return RLSCAN_ERR_MEMORY;
    const NormArgs a{x, residual, x_stride, residual_stride, weight, M, D, eps, y, scales, residual_out};
    return launch_add_rms_norm(a, dtype == RLSCAN_BF16,
                               residual == nullptr ? dtype == RLSCAN_BF16 : residual_dtype == RLSCAN_BF16, cs(stream));
}

RLSCAN_API size_t rlscan_add_rms_norm_backward_workspace_bytes(int64_t M, int64_t D)
{
    return sizes_ok({M, D}) ? add_rms_norm_backward_workspace(M, D) : 0;
}

RLSCAN_API rlscan_status rlscan_add_rms_norm_backward(const void *grad_y, int64_t grad_y_stride, const void *h,
                                                      int64_t h_stride, const void *grad_residual,
                                                      int64_t grad_residual_stride, const float *weight, int64_t M,
                                                      int64_t D, float eps, rlscan_dtype dtype, rlscan_dtype h_dtype,
                                                      void *grad_x, void *grad_h, float *grad_weight, void *ws,
                                                      size_t ws_bytes, rlscan_stream_t stream)
{
    if (!sizes_ok({M, D})) return RLSCAN_ERR_SHAPE;
    if (!is_io_type(dtype) || (h_dtype != RLSCAN_F32 && h_dtype != dtype) || !(eps >= 0.f)) return RLSCAN_ERR_ARG_VALUE;
    if (D == 0) return RLSCAN_OK;
    if (M > 0 && (!grad_y || !h || !weight || !grad_x)) return RLSCAN_ERR_NULL;
    for (const void *o : {static_cast<const void *>(grad_x), static_cast<const void *>(grad_h),
                          static_cast<const void *>(grad_weight)})
        if (o != nullptr && equals_any(o, {grad_y, h, grad_residual, weight})) return RLSCAN_ERR_ARG_CONFLICT;
    if (M > 0 && (grad_x == grad_h || grad_x == grad_weight)) return RLSCAN_ERR_ARG_CONFLICT;
    if (grad_weight && !workspace_ok(ws, ws_bytes, add_rms_norm_backward_workspace(M, D))) return RLSCAN_ERR_WORKSPACE;
    if (!reachable({grad_y, h, grad_residual, weight, grad_x, grad_h, grad_weight})) return RLSCAN_ERR_MEMORY;
    const NormGradArgs a{grad_y, h, grad_residual, grad_y_stride, h_stride, grad_residual_stride, weight, M, D, eps,
                         grad_x, grad_h, grad_weight};
    return launch_add_rms_norm_backward(a, dtype == RLSCAN_BF16, h_dtype == RLSCAN_BF16, ws, cs(stream));
}

}  // extern "C"
