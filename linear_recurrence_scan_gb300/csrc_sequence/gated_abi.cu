// gated_abi.cu -- the extern "C" entry points of the gated recurrence: argument
// validation, then the launchers of k_gated_scan*.cu.
#include "abi_checks.cuh"
#include "distill.cuh"
#include "gated_projection.cuh"

using namespace rlscan;
using namespace rlscan::seq;

namespace {

rlscan_status check_gated(const rlscan_gated_scan_args *a)
{
    if (a == nullptr) return RLSCAN_ERR_NULL;
    if (!sizes_ok({a->N, a->T, a->D, 8})) return RLSCAN_ERR_SHAPE;
    return is_io_type(a->dtype) ? RLSCAN_OK : RLSCAN_ERR_ARG_VALUE;
}

bool inputs_given(const rlscan_gated_scan_args &a)
{
    return a.log_decay != nullptr && (a.T == 0 || (a.x.data && a.gate.data && a.input_gate.data));
}

bool is_gated_input(const void *out, const rlscan_gated_scan_args &a)
{
    return equals_any(out, {a.x.data, a.gate.data, a.input_gate.data, a.log_decay, a.initial_state, a.resets, a.lengths});
}

bool gated_reachable(const rlscan_gated_scan_args &a)
{
    return reachable({a.log_decay, a.initial_state, a.resets, a.lengths});
}

// outputs that are one another or an input
bool conflict(const rlscan_gated_scan_args &a, std::initializer_list<const void *> outs, std::initializer_list<const void *> more)
{
    for (auto i = outs.begin(); i != outs.end(); ++i) {
        if (*i == nullptr) continue;
        if (is_gated_input(*i, a) || equals_any(*i, more)) return true;
        for (auto j = outs.begin(); j != i; ++j)
            if (*j == *i) return true;
    }
    return false;
}

}  // namespace

extern "C" {

RLSCAN_API rlscan_status rlscan_gated_scan(const rlscan_gated_scan_args *args, void *y, float *final_state,
                                           float *checkpoints, rlscan_stream_t stream)
{
    RLSCAN_TRY(check_gated(args));
    const rlscan_gated_scan_args &a = *args;
    if (a.N == 0 || a.D == 0) return RLSCAN_OK;
    if (!inputs_given(a) || (a.T > 0 && y == nullptr)) return RLSCAN_ERR_NULL;
    if (conflict(a, {y, final_state, checkpoints}, {})) return RLSCAN_ERR_ARG_CONFLICT;
    const Residency tokens = residency_of({a.x.data, a.gate.data, a.input_gate.data, y});
    if (tokens == Residency::Unreachable || !gated_reachable(a) || !reachable({final_state, checkpoints})) return RLSCAN_ERR_MEMORY;
    return launch_gated_scan(a, y, final_state, checkpoints, tokens == Residency::Device, cs(stream));
}

RLSCAN_API size_t rlscan_gated_scan_backward_workspace_bytes(const rlscan_gated_scan_args *args)
{
    return check_gated(args) == RLSCAN_OK ? gated_scan_backward_workspace(*args) : 0;
}

RLSCAN_API rlscan_status rlscan_gated_scan_backward(const rlscan_gated_scan_args *args, const rlscan_array3 *grad_y,
                                                    const float *grad_final_state, const float *checkpoints,
                                                    const rlscan_gated_scan_grads *grads, void *ws, size_t ws_bytes,
                                                    rlscan_stream_t stream)
{
    RLSCAN_TRY(check_gated(args));
    if (grad_y == nullptr || grads == nullptr) return RLSCAN_ERR_NULL;
    const rlscan_gated_scan_args &a = *args;
    const rlscan_gated_scan_grads &g = *grads;
    if (a.D == 0) return RLSCAN_OK;
    if (a.N > 0 && (!inputs_given(a) || (a.T > 0 && (!grad_y->data || !checkpoints || !g.x || !g.gate || !g.input_gate))))
        return RLSCAN_ERR_NULL;
    if (conflict(a, {g.x, g.gate, g.input_gate, g.log_decay, g.initial_state}, {grad_y->data, grad_final_state, checkpoints}))
        return RLSCAN_ERR_ARG_CONFLICT;
    if (g.log_decay && !workspace_ok(ws, ws_bytes, gated_scan_backward_workspace(a))) return RLSCAN_ERR_WORKSPACE;
    const Residency tokens = residency_of({a.x.data, a.gate.data, a.input_gate.data, grad_y->data, g.x, g.gate, g.input_gate});
    if (tokens == Residency::Unreachable || !gated_reachable(a) || !reachable({grad_final_state, checkpoints, g.log_decay, g.initial_state}))
        return RLSCAN_ERR_MEMORY;
    return launch_gated_scan_backward(a, *grad_y, grad_final_state, checkpoints, g, ws, tokens == Residency::Device, cs(stream));
}

RLSCAN_API rlscan_status rlscan_gated_scan_step(const rlscan_gated_scan_args *args, float *state, int64_t P,
                                                const int32_t *slots, void *y, rlscan_stream_t stream)
{
    RLSCAN_TRY(check_gated(args));
    const rlscan_gated_scan_args &a = *args;
    if (a.T != 1 || P < 0 || (slots == nullptr && P < a.N)) return RLSCAN_ERR_SHAPE;
    if (a.N == 0 || a.D == 0) return RLSCAN_OK;
    if (!inputs_given(a) || (P > 0 && state == nullptr) || y == nullptr) return RLSCAN_ERR_NULL;
    if (conflict(a, {y, state}, {slots})) return RLSCAN_ERR_ARG_CONFLICT;
    if (!gated_reachable(a) || !reachable({a.x.data, a.gate.data, a.input_gate.data, state, slots, y})) return RLSCAN_ERR_MEMORY;
    return launch_gated_scan_step(a, state, P, slots, y, cs(stream));
}

RLSCAN_API rlscan_status rlscan_wait_status(rlscan_stream_t stream)
{
    const rlscan_status all[] = {gated_scan_status(cs(stream)), gated_scan_backward_status(cs(stream)), gated_projection_status(cs(stream)),
                                 distill_status(cs(stream))};
    for (const rlscan_status st : all) RLSCAN_TRY(st);
    return RLSCAN_OK;
}

}  // extern "C"
