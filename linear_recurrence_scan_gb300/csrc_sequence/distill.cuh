// distill.cuh -- the distillation loss's launchers, as the C entry points call them.
#pragma once

#include "sequence.cuh"

namespace rlscan {
namespace seq {

constexpr int kMostTeacher = RLSCAN_DISTILL_MOST;  // teacher's tokens of a row

struct DistillOut {
    float *loss;               // [N,T]
    float *normalizers;        // [N,T,2]: written with the loss, read by the gradient alone
    const float *grad_loss;    // [N,T]
    void *grad;                // [N,T,V]
};

enum class Part { Loss, Grad, Both };

// Rows of at most kShortUnits units of 16 bytes
constexpr int64_t kShortUnits = 256;
rlscan_status launch_distill_short(const rlscan_distill_args &a, Part part, const DistillOut &o, cudaStream_t s);

rlscan_status launch_distill(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s);
rlscan_status launch_distill_backward(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s);
// Loss and gradient; false: the rows do not fit on chip (the two calls above do the same).
bool distill_fits(const rlscan_distill_args &a);
rlscan_status distill_status(cudaStream_t s);  // whether a wait ran out
rlscan_status launch_distill_both(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s);

}  // namespace seq
}  // namespace rlscan
