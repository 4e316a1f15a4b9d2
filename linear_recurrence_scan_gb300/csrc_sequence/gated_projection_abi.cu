// gated_projection_abi.cu -- the extern "C" entry points of the gated
// feed-forward block: argument validation, then its launchers.
#include "abi_checks.cuh"
#include "gated_projection.cuh"

using namespace rlscan;
using namespace rlscan::seq;

namespace {

rlscan_status check_projection(const rlscan_gated_projection_args *a)
{
    if (a == nullptr) return RLSCAN_ERR_NULL;
    constexpr int64_t kMost = 0x7fffffff - 256;  // coordinates of copies are 32-bit
    if (!sizes_ok({a->M, a->D, 8}) || !sizes_ok({a->M, a->F, 8}) || !sizes_ok({a->F, a->D, 8}) || a->M > kMost || a->D > kMost || a->F > kMost)
        return RLSCAN_ERR_SHAPE;
    return a->activation == RLSCAN_SILU || a->activation == RLSCAN_GELU ? RLSCAN_OK : RLSCAN_ERR_ARG_VALUE;
}

bool inputs_given(const rlscan_gated_projection_args &a)
{
    return a.D == 0 || ((a.M == 0 || a.x) && (a.F == 0 || (a.gate_weight && a.up_weight)));
}

}  // namespace

extern "C" {

RLSCAN_API size_t rlscan_gated_projection_workspace_bytes(const rlscan_gated_projection_args *args)
{
    return check_projection(args) == RLSCAN_OK ? gated_projection_workspace(*args) : 0;
}

RLSCAN_API rlscan_status rlscan_gated_projection(const rlscan_gated_projection_args *args, void *h, void *ws,
                                                 size_t ws_bytes, rlscan_stream_t stream)
{
    RLSCAN_TRY(check_projection(args));
    const rlscan_gated_projection_args &a = *args;
    if (a.M == 0 || a.F == 0) return RLSCAN_OK;
    if (!inputs_given(a) || h == nullptr) return RLSCAN_ERR_NULL;
    if (equals_any(h, {a.x, a.gate_weight, a.up_weight})) return RLSCAN_ERR_ARG_CONFLICT;
    if (!workspace_ok(ws, ws_bytes, gated_projection_workspace(a))) return RLSCAN_ERR_WORKSPACE;
    if (!on_device({a.x, a.gate_weight, a.up_weight, h})) return RLSCAN_ERR_MEMORY;
    return launch_gated_projection(a, h, ws, cs(stream));
}

RLSCAN_API size_t rlscan_gated_projection_backward_workspace_bytes(const rlscan_gated_projection_args *args)
{
    return check_projection(args) == RLSCAN_OK ? gated_projection_backward_workspace(*args) : 0;
}

RLSCAN_API rlscan_status rlscan_gated_projection_backward(const rlscan_gated_projection_args *args, const void *grad_h,
                                                          int64_t grad_h_stride, void *grad_x, void *grad_gate,
                                                          void *grad_up, void *ws, size_t ws_bytes, rlscan_stream_t stream)
{
    RLSCAN_TRY(check_projection(args));
    const rlscan_gated_projection_args &a = *args;
    if (!inputs_given(a) || (a.M > 0 && a.F > 0 && a.D > 0 && grad_h == nullptr) || (grad_gate == nullptr) != (grad_up == nullptr))
        return RLSCAN_ERR_NULL;
    for (const void *o : {grad_x, grad_gate, grad_up})
        if (equals_any(o, {a.x, a.gate_weight, a.up_weight, grad_h})) return RLSCAN_ERR_ARG_CONFLICT;
    if ((grad_x && (grad_x == grad_gate || grad_x == grad_up)) || (grad_gate && grad_gate == grad_up)) return RLSCAN_ERR_ARG_CONFLICT;
    if (!workspace_ok(ws, ws_bytes, gated_projection_backward_workspace(a))) return RLSCAN_ERR_WORKSPACE;
    if (!on_device({a.x, a.gate_weight, a.up_weight, grad_h, grad_x, grad_gate, grad_up})) return RLSCAN_ERR_MEMORY;
    return launch_gated_projection_backward(a, grad_h, grad_h_stride, grad_x, grad_gate, grad_up, ws, cs(stream));
}

}  // extern "C"
