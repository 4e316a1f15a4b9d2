// k_rms_norm.cu -- root-mean-square norm with the residual's addition, its
// 8-bit output with a scale for each 128 columns, and its gradients.
// A block of threads takes a row.
#include <cuda_fp8.h>

#include "sequence.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kThreads = 128;

// the block's sum, the same bits in every thread
__device__ __forceinline__ float block_sum(float v, float *scratch)
{
#pragma unroll
    for (int m = 16; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
    __syncthreads();  // scratch is free again
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += scratch[w];
    return s;
}

template <class T, class R>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float scratch[kThreads / 32];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
    const R *r = a.residual != nullptr ? static_cast<const R *>(a.residual) + row * a.residual_stride : nullptr;
    auto sum_at = [&](int64_t c) { return to_f(x[c]) + (r != nullptr ? to_f(r[c]) : 0.f); };
    float ss = 0.f;
    for (int64_t c = threadIdx.x; c < a.D; c += kThreads) {
        const float h = sum_at(c);
        ss = fmaf(h, h, ss);
        if (r != nullptr) static_cast<R *>(a.residual_out)[row * a.D + c] = from_f<R>(h);
    }
    const float inv = rsqrtf(block_sum(ss, scratch) / static_cast<float>(a.D) + a.eps);
    if (a.scales == nullptr) {
        for (int64_t c = threadIdx.x; c < a.D; c += kThreads)
            static_cast<T *>(a.y)[row * a.D + c] = from_f<T>(sum_at(c) * inv * a.weight[c]);
        return;
    }
    // 8 bits: a warp takes a block of columns
    const int64_t blocks = (a.D + kScaleBlock - 1) / kScaleBlock;
    const int lane = threadIdx.x & 31;
    for (int64_t b = threadIdx.x / 32; b < blocks; b += kThreads / 32) {
        float v[kScaleBlock / 32], top = 0.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kScaleBlock / 32; ++i) {
            const int64_t c = b * kScaleBlock + i * 32 + lane;
            v[i] = c < a.D ? sum_at(c) * inv * a.weight[c] : 0.f;
            top = fmaxf(top, fabsf(v[i]));
            bad = bad || !(fabsf(v[i]) <= 3.402823466e38f);
        }
#pragma unroll
        for (int m = 16; m > 0; m /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        bad = __any_sync(0xffffffffu, bad);
        const float scale = bad ? __int_as_float(0x7fffffff) : fmaxf(top, kScaleFloor) / kE4m3Max;
#pragma unroll
        for (int i = 0; i < kScaleBlock / 32; ++i) {
            const int64_t c = b * kScaleBlock + i * 32 + lane;
            if (c < a.D)
                static_cast<__nv_fp8_storage_t *>(a.y)[row * a.D + c] =
                    __nv_cvt_float_to_fp8(v[i] / scale, __NV_SATFINITE, __NV_E4M3);
        }
        if (lane == 0) a.scales[row * blocks + b] = scale;
    }
}

// Rows are taken in strides of the grid; a block's sums of dy n over its
// rows go to its own row of `part`.
template <class T, class R>
__global__ void __launch_bounds__(kThreads)
    norm_grad_kernel(const __grid_constant__ NormGradArgs a, float *part)
{
    __shared__ float scratch[kThreads / 32];
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const T *gy = static_cast<const T *>(a.grad_y) + row * a.grad_y_stride;
        const R *h = static_cast<const R *>(a.h) + row * a.h_stride;
        const R *gr = a.grad_residual != nullptr ? static_cast<const R *>(a.grad_residual) + row * a.grad_residual_stride
                                                 : nullptr;
        float ss = 0.f, dot = 0.f;
        for (int64_t c = threadIdx.x; c < a.D; c += kThreads) {
            const float hv = to_f(h[c]);
            ss = fmaf(hv, hv, ss);
            dot = fmaf(to_f(gy[c]) * a.weight[c], hv, dot);
        }
        const float inv = rsqrtf(block_sum(ss, scratch) / static_cast<float>(a.D) + a.eps);
        const float mean = block_sum(dot, scratch) * inv / static_cast<float>(a.D);
        for (int64_t c = threadIdx.x; c < a.D; c += kThreads) {
            const float nv = to_f(h[c]) * inv, gv = to_f(gy[c]);
            const float gh = inv * fmaf(-nv, mean, gv * a.weight[c]) + (gr != nullptr ? to_f(gr[c]) : 0.f);
            static_cast<T *>(a.grad_x)[row * a.D + c] = from_f<T>(gh);
            if (a.grad_h != nullptr) static_cast<R *>(a.grad_h)[row * a.D + c] = from_f<R>(gh);
            if (part != nullptr) {
                float *p = part + blockIdx.x * a.D + c;
                *p = (row == blockIdx.x ? 0.f : *p) + gv * nv;
            }
        }
    }
}

constexpr int64_t kGradBlocks = 1024;
int64_t grad_blocks(int64_t M) { return M < kGradBlocks ? M : kGradBlocks; }

}  // namespace

rlscan_status launch_add_rms_norm(const NormArgs &a, bool bf16_io, bool bf16_residual, cudaStream_t s)
{
    const unsigned grid = static_cast<unsigned>(a.M);
    if (!bf16_io)
        norm_kernel<float, float><<<grid, kThreads, 0, s>>>(a);
    else if (bf16_residual)
        norm_kernel<bf16, bf16><<<grid, kThreads, 0, s>>>(a);
    else
        norm_kernel<bf16, float><<<grid, kThreads, 0, s>>>(a);
    return launched();
}

size_t add_rms_norm_backward_workspace(int64_t M, int64_t D)
{
    return sizeof(float) * static_cast<size_t>(grad_blocks(M)) * D;
}

rlscan_status launch_add_rms_norm_backward(const NormGradArgs &a, bool bf16_io, bool bf16_h, void *ws, cudaStream_t s)
{
    float *part = a.grad_weight != nullptr ? static_cast<float *>(ws) : nullptr;
    const unsigned grid = static_cast<unsigned>(grad_blocks(a.M));
    if (a.M > 0) {
        if (!bf16_io)
            norm_grad_kernel<float, float><<<grid, kThreads, 0, s>>>(a, part);
        else if (bf16_h)
            norm_grad_kernel<bf16, bf16><<<grid, kThreads, 0, s>>>(a, part);
        else
            norm_grad_kernel<bf16, float><<<grid, kThreads, 0, s>>>(a, part);
        const rlscan_status st = launched();
        if (st != RLSCAN_OK) return st;
    }
    if (a.grad_weight == nullptr) return RLSCAN_OK;
    return launch_sum_parts(part, grad_blocks(a.M), a.D, a.D, a.grad_weight, false, s);
}

}  // namespace seq
}  // namespace rlscan
