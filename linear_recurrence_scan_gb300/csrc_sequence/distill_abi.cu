// distill_abi.cu -- the extern "C" entry points of the distillation loss:
// argument validation, then the launchers of k_distill.cu.
#include "abi_checks.cuh"
#include "distill.cuh"

using namespace rlscan;
using namespace rlscan::seq;

namespace {

rlscan_status check_distill(const rlscan_distill_args *a)
{
    if (a == nullptr) return RLSCAN_ERR_NULL;
    if (!sizes_ok({a->N, a->T, a->V, 8}) || a->V > 0x7fffffff) return RLSCAN_ERR_SHAPE;
    if (a->K < 1 || a->K > kMostTeacher || !is_io_type(a->dtype) || !is_io_type(a->teacher_dtype) ||
        (a->token_bytes != 4 && a->token_bytes != 8) || !(a->temperature > 0 && a->temperature <= 1e6 && a->temperature >= 1e-6))
        return RLSCAN_ERR_ARG_VALUE;
    return RLSCAN_OK;
}

rlscan_status check_distill_call(const rlscan_distill_args &a, std::initializer_list<const void *> outs,
                                 std::initializer_list<const void *> more)
{
    if (!a.logits.data || !a.teacher_logits || !a.teacher_tokens) return RLSCAN_ERR_NULL;
    for (auto i = outs.begin(); i != outs.end(); ++i) {
        if (*i == nullptr) continue;
        if (equals_any(*i, {a.logits.data, a.teacher_logits, a.teacher_tokens, a.mask}) || equals_any(*i, more))
            return RLSCAN_ERR_ARG_CONFLICT;
        for (auto j = outs.begin(); j != i; ++j)
            if (*j == *i) return RLSCAN_ERR_ARG_CONFLICT;
    }
    return on_device({a.logits.data}) && reachable({a.teacher_logits, a.teacher_tokens, a.mask}) && reachable(outs) && reachable(more)
               ? RLSCAN_OK
               : RLSCAN_ERR_MEMORY;
}

}  // namespace

extern "C" {

RLSCAN_API rlscan_status rlscan_distill_loss(const rlscan_distill_args *args, float *loss, float *normalizers,
                                             rlscan_stream_t stream)
{
    RLSCAN_TRY(check_distill(args));
    const rlscan_distill_args &a = *args;
    if (a.N == 0 || a.T == 0) return RLSCAN_OK;
    if (a.V == 0) return RLSCAN_ERR_SHAPE;  // a token without a vocabulary has no distribution
    if (loss == nullptr) return RLSCAN_ERR_NULL;
    RLSCAN_TRY(check_distill_call(a, {loss, normalizers}, {}));
    return launch_distill(a, DistillOut{loss, normalizers, nullptr, nullptr}, cs(stream));
}

RLSCAN_API rlscan_status rlscan_distill_loss_backward(const rlscan_distill_args *args, const float *grad_loss,
                                                      const float *normalizers, void *grad_logits, rlscan_stream_t stream)
{
    RLSCAN_TRY(check_distill(args));
    const rlscan_distill_args &a = *args;
    if (a.N == 0 || a.T == 0) return RLSCAN_OK;
    if (a.V == 0) return RLSCAN_ERR_SHAPE;
    if (!grad_loss || !normalizers || !grad_logits) return RLSCAN_ERR_NULL;
    RLSCAN_TRY(check_distill_call(a, {grad_logits}, {grad_loss, normalizers}));
    return launch_distill_backward(a, DistillOut{nullptr, const_cast<float *>(normalizers), grad_loss, grad_logits}, cs(stream));
}

RLSCAN_API rlscan_status rlscan_distill_loss_and_grad(const rlscan_distill_args *args, const float *grad_loss, float *loss,
                                                      float *normalizers, void *grad_logits, rlscan_stream_t stream)
{
    RLSCAN_TRY(check_distill(args));
    const rlscan_distill_args &a = *args;
    if (a.N == 0 || a.T == 0) return RLSCAN_OK;
    if (a.V == 0) return RLSCAN_ERR_SHAPE;
    if (!grad_loss || !loss || !normalizers || !grad_logits) return RLSCAN_ERR_NULL;
    RLSCAN_TRY(check_distill_call(a, {loss, normalizers, grad_logits}, {grad_loss}));
    const DistillOut o{loss, normalizers, grad_loss, grad_logits};
    if (distill_fits(a)) return launch_distill_both(a, o, cs(stream));
    RLSCAN_TRY(launch_distill(a, o, cs(stream)));
    return launch_distill_backward(a, o, cs(stream));
}

}  // extern "C"
