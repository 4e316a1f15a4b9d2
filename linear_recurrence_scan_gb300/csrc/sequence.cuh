// sequence.cuh -- what the state-space layer's kernels share: loads and
// stores of the two activation types, the scalar functions of the gates and
// the time steps, and the internal launchers the C entry points call.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "rlscan.h"

namespace rlscan {
namespace seq {

constexpr int kCheckpoint = RLSCAN_SELECTIVE_SCAN_CHECKPOINT;
constexpr int kMaxStates = 128;
constexpr int kMaxTaps = 8;
constexpr int kScaleBlock = 128;      // columns that share one scale of an 8-bit output
constexpr float kE4m3Max = 448.f;
constexpr float kScaleFloor = 0x1p-100f;  // smallest block maximum a scale is made from

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16 from_f<bf16>(float v) { return __float2bfloat16_rn(v); }

// 2^v and 1/v to within 2 units in the last place (PTX ex2.approx, rcp.approx)
__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rcp_fast(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + exp(-v)); 2^x is infinite below v = -88, whose reciprocal is 0
__device__ __forceinline__ float sigmoid(float v) { return rcp_fast(1.f + exp2_fast(-kLog2e * v)); }

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1], with
// log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3, by atanh's power series
// s (1 + s^2/3 + s^4/5 + ...): its first omitted term, s^14/15, is below
// 1.4e-8 of the sum.  (log(1 + e) itself would lose the small time steps,
// which are e for large negative v, to the rounding of 1 + e.)
__device__ __forceinline__ float softplus(float v)
{
    const float e = exp2_fast(-kLog2e * fabsf(v));
    const float s = e * rcp_fast(2.f + e);
    const float q = s * s;
    float p = 1.f / 13.f;
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return fmaf(2.f * s, p, fmaxf(v, 0.f));
}

// tokens of row n, clamped to the array
__device__ __forceinline__ int64_t row_length(const int32_t *lengths, int64_t n, int64_t T)
{
    if (lengths == nullptr) return T;
    const int64_t len = lengths[n];
    return len < 0 ? 0 : (len < T ? len : T);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Lanes of a channel's states, four states each: 1, 2, 4, ... 32.
inline int state_lanes(int64_t S)
{
    int lanes = 1;
    while (4 * lanes < S) lanes *= 2;
    return lanes;
}

rlscan_status launch_selective_scan(const rlscan_selective_scan_args &a, void *y, float *final_state,
                                    float *checkpoints, void *ws, cudaStream_t s);
size_t selective_scan_workspace(const rlscan_selective_scan_args &a);
rlscan_status launch_selective_scan_step(const rlscan_selective_scan_args &a, float *state, int64_t P,
                                         const int32_t *slots, void *y, cudaStream_t s);
rlscan_status launch_selective_scan_backward(const rlscan_selective_scan_args &a, const rlscan_array3 &grad_y,
                                             const float *grad_final_state, const float *checkpoints,
                                             const rlscan_selective_scan_grads &g, void *ws, cudaStream_t s);
size_t selective_scan_backward_workspace(const rlscan_selective_scan_args &a);
rlscan_status launch_causal_conv(const rlscan_causal_conv_args &a, void *y, void *final_state, cudaStream_t s);
rlscan_status launch_causal_conv_step(const rlscan_causal_conv_args &a, void *state, int64_t P, const int32_t *slots,
                                      void *y, cudaStream_t s);
rlscan_status launch_causal_conv_backward(const rlscan_causal_conv_args &a, const rlscan_array3 &grad_y,
                                          const void *grad_final_state, void *grad_x, float *grad_weight,
                                          float *grad_bias, void *grad_initial_state, void *ws, cudaStream_t s);
size_t causal_conv_backward_workspace(const rlscan_causal_conv_args &a);

struct NormArgs {
    const void *x, *residual;
    int64_t x_stride, residual_stride;
    const float *weight;
    int64_t M, D;
    float eps;
    void *y;
    float *scales;
    void *residual_out;
};
rlscan_status launch_add_rms_norm(const NormArgs &a, bool bf16_io, bool bf16_residual, cudaStream_t s);

struct NormGradArgs {
    const void *grad_y, *h, *grad_residual;
    int64_t grad_y_stride, h_stride, grad_residual_stride;
    const float *weight;
    int64_t M, D;
    float eps;
    void *grad_x, *grad_h;
    float *grad_weight;
};
rlscan_status launch_add_rms_norm_backward(const NormGradArgs &a, bool bf16_io, bool bf16_h, void *ws, cudaStream_t s);
size_t add_rms_norm_backward_workspace(int64_t M, int64_t D);

// out[i] = sum over w in order of part[w * pitch + i], i < m, rounded to `bf16_out`'s type
rlscan_status launch_sum_parts(const float *part, int64_t parts, int64_t pitch, int64_t m, void *out, bool bf16_out,
                               cudaStream_t s);

inline rlscan_status launched()
{
    return cudaGetLastError() == cudaSuccess ? RLSCAN_OK : RLSCAN_ERR_CUDA;
}

}  // namespace seq
}  // namespace rlscan
