// k_rms_norm.cu -- root-mean-square norm with the residual's addition, its
// 8-bit output with a scale for each 128 columns, and its gradients.
//
// One pass: TPR threads take a row and keep it in registers (two chunks of
// 16 bytes of x each) between the sum of squares and the outputs.
#include <cuda_fp8.h>

#include "sequence.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kChunks = 2;  // chunks of a thread

template <class T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

// the smallest power of two of threads that holds a row, 0 if 1024 do not
template <class T>
int row_threads(int64_t D)
{
    for (int t = 32; t <= 1024; t *= 2)
        if (D <= static_cast<int64_t>(t) * kChunks * kVec<T>) return t;
    return 0;
}

// a chunk of V values of type R, wide where `vec`, else those inside the row (the others 0)
template <class R, int V>
__device__ __forceinline__ void load_chunk(float *v, const R *p, int64_t c, int64_t D, bool vec)
{
    if (vec) {
        constexpr int B = V * static_cast<int>(sizeof(R));
        alignas(16) R raw[V];
        if (c < D) {
            if constexpr (B >= 16) {
#pragma unroll
                for (int i = 0; i < B / 16; ++i)
                    reinterpret_cast<uint4 *>(raw)[i] = __ldg(reinterpret_cast<const uint4 *>(p + c) + i);
            } else {
                *reinterpret_cast<uint2 *>(raw) = __ldg(reinterpret_cast<const uint2 *>(p + c));
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = c < D ? to_f(raw[i]) : 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = c + i < D ? to_f(p[c + i]) : 0.f;
    }
}

template <class R, int V>
__device__ __forceinline__ void store_chunk(R *p, const float *v, int64_t c, int64_t D, bool vec)
{
    if (vec) {
        constexpr int B = V * static_cast<int>(sizeof(R));
        alignas(16) R raw[V];
#pragma unroll
        for (int i = 0; i < V; ++i) raw[i] = from_f<R>(v[i]);
        if (c < D) {
            if constexpr (B >= 16) {
#pragma unroll
                for (int i = 0; i < B / 16; ++i) reinterpret_cast<uint4 *>(p + c)[i] = reinterpret_cast<uint4 *>(raw)[i];
            } else {
                *reinterpret_cast<uint2 *>(p + c) = *reinterpret_cast<uint2 *>(raw);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c + i < D) p[c + i] = from_f<R>(v[i]);
    }
}

// Sums of v[0..N) over a row's TPR threads, the same bits in each.
template <int TPR, int N>
__device__ __forceinline__ void row_sums(float *v, float (*scratch)[N])
{
#pragma unroll
    for (int m = 16; m > 0; m /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x / 32;
        __syncthreads();  // scratch is free again
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) scratch[warp][i] = v[i];
        __syncthreads();
        const int first = warp / (TPR / 32) * (TPR / 32);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.f;
#pragma unroll
            for (int w = 0; w < TPR / 32; ++w) v[i] += scratch[first + w][i];
        }
    }
}

template <int TPR>
constexpr int kBlock = TPR > 128 ? TPR : 128;

template <class T, class R, int TPR>
__global__ void __launch_bounds__(kBlock<TPR>) norm_kernel(const __grid_constant__ NormArgs a)
{
    constexpr int V = kVec<T>, ROWS = kBlock<TPR> / TPR;
    __shared__ float scratch[kBlock<TPR> / 32][1];
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int64_t row = blockIdx.x * static_cast<int64_t>(ROWS) + threadIdx.x / TPR;
    const bool on = row < a.M;
    const int64_t D = on ? a.D : 0;
    const int64_t rr = on ? row : 0;
    const int tid = threadIdx.x % TPR;
    const T *x = static_cast<const T *>(a.x) + rr * a.x_stride;
    const R *r = static_cast<const R *>(a.residual) + (a.residual != nullptr ? rr * a.residual_stride : 0);
    float h[kChunks][V];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) load_chunk<T, V>(h[j], x, (j * TPR + tid) * V, D, a.vec);
    if (a.residual != nullptr) {
        float q[kChunks][V];
#pragma unroll
        for (int j = 0; j < kChunks; ++j) load_chunk<R, V>(q[j], r, (j * TPR + tid) * V, D, a.vec);
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
#pragma unroll
            for (int i = 0; i < V; ++i) h[j][i] += q[j][i];
            store_chunk<R, V>(static_cast<R *>(a.residual_out) + rr * a.D, h[j], (j * TPR + tid) * V, D, a.vec);
        }
    }
    float ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) ss[0] = fmaf(h[j][i], h[j][i], ss[0]);
    row_sums<TPR, 1>(ss, scratch);
    const float inv = rsqrtf(ss[0] / static_cast<float>(a.D) + a.eps);
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        const int64_t c = (j * TPR + tid) * V;
        if (TPR * V * j >= a.D) break;
        float w[V];
        load_chunk<float, V>(w, a.weight, c, D, a.vec);
#pragma unroll
        for (int i = 0; i < V; ++i) h[j][i] = h[j][i] * inv * w[i];
        if (a.scales == nullptr) {
            store_chunk<T, V>(static_cast<T *>(a.y) + rr * a.D, h[j], c, D, a.vec);
            continue;
        }
        // kScaleBlock / V neighbouring lanes hold a block of columns
        float top = 0.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            top = fmaxf(top, fabsf(h[j][i]));
            bad = bad || !(fabsf(h[j][i]) <= 3.402823466e38f);
        }
        top = bad ? __int_as_float(0x7f800000) : top;
#pragma unroll
        for (int m = kScaleBlock / V / 2; m > 0; m /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        const float scale = top <= 3.402823466e38f ? fmaxf(top, kScaleFloor) / kE4m3Max : __int_as_float(0x7fffffff);
        uint32_t q[V / 4];
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(h[j][i] / scale, h[j][i + 1] / scale),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(h[j][i + 2] / scale, h[j][i + 3] / scale),
                                                         __NV_SATFINITE, __NV_E4M3);
            q[i / 4] = lo | hi << 16;
        }
        uint8_t *y = static_cast<uint8_t *>(a.y) + rr * a.D;
        if (a.vec) {
            if (c < D) {
#pragma unroll
                for (int i = 0; i < V / 4; ++i) reinterpret_cast<uint32_t *>(y + c)[i] = q[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c + i < D) y[c + i] = static_cast<uint8_t>(q[i / 4] >> (i % 4 * 8));
        }
        if (c < D && c % kScaleBlock == 0)
            a.scales[rr * ((a.D + kScaleBlock - 1) / kScaleBlock) + c / kScaleBlock] = scale;
    }
}

// Rows of any length: a block of 1024 threads walks the row twice.
constexpr int kLongThreads = 1024;

template <class T, class R>
__global__ void __launch_bounds__(kLongThreads) long_norm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float scratch[kLongThreads / 32][1];
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
    const R *r = a.residual != nullptr ? static_cast<const R *>(a.residual) + row * a.residual_stride : nullptr;
    auto sum_at = [&](int64_t c) { return to_f(x[c]) + (r != nullptr ? to_f(r[c]) : 0.f); };
    float ss[1] = {0.f};
    for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) {
        const float h = sum_at(c);
        ss[0] = fmaf(h, h, ss[0]);
        if (r != nullptr) static_cast<R *>(a.residual_out)[row * a.D + c] = from_f<R>(h);
    }
    row_sums<kLongThreads, 1>(ss, scratch);
    const float inv = rsqrtf(ss[0] / static_cast<float>(a.D) + a.eps);
    if (a.scales == nullptr) {
        for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads)
            static_cast<T *>(a.y)[row * a.D + c] = from_f<T>(sum_at(c) * inv * a.weight[c]);
        return;
    }
    const int64_t blocks = (a.D + kScaleBlock - 1) / kScaleBlock;
    const int lane = threadIdx.x & 31;
    for (int64_t b = threadIdx.x / 32; b < blocks; b += kLongThreads / 32) {
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

// Gradients: dh = r (gn - n mean(gn n)) + grad_residual.  A block takes rows
// in strides of the grid, the next row's loads ahead of this row's sums, and
// keeps its sums of dy n in registers: one row of `part` for each row it
// works on at a time.
template <class T, class R, int TPR>
__global__ void __launch_bounds__(kBlock<TPR>)
    norm_grad_kernel(const __grid_constant__ NormGradArgs a, float *part)
{
    constexpr int V = kVec<T>, ROWS = kBlock<TPR> / TPR;
    __shared__ float scratch[kBlock<TPR> / 32][2];
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int tid = threadIdx.x % TPR;
    const int64_t slot = blockIdx.x * static_cast<int64_t>(ROWS) + threadIdx.x / TPR;
    const int64_t step = static_cast<int64_t>(gridDim.x) * ROWS;
    float w[kChunks][V], dw[kChunks][V];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) {
        load_chunk<float, V>(w[j], a.weight, (j * TPR + tid) * V, a.D, a.vec);
#pragma unroll
        for (int i = 0; i < V; ++i) dw[j][i] = 0.f;
    }
    const float over = 1.f / static_cast<float>(a.D);
    for (int64_t base = blockIdx.x * static_cast<int64_t>(ROWS); base < a.M; base += step) {
        const int64_t row = base + threadIdx.x / TPR;
        const bool on = row < a.M;
        const int64_t rr = on ? row : 0, D = on ? a.D : 0;
        const T *gy = static_cast<const T *>(a.grad_y) + rr * a.grad_y_stride;
        const R *h = static_cast<const R *>(a.h) + rr * a.h_stride;
        float hv[kChunks][V], gv[kChunks][V], gr[kChunks][V];
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            load_chunk<R, V>(hv[j], h, (j * TPR + tid) * V, D, a.vec);
            load_chunk<T, V>(gv[j], gy, (j * TPR + tid) * V, D, a.vec);
            if (a.grad_residual != nullptr) {
                load_chunk<R, V>(gr[j], static_cast<const R *>(a.grad_residual) + rr * a.grad_residual_stride,
                                 (j * TPR + tid) * V, D, a.vec);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) gr[j][i] = 0.f;
            }
        }
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kChunks; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s[0] = fmaf(hv[j][i], hv[j][i], s[0]);
                s[1] = fmaf(gv[j][i] * w[j][i], hv[j][i], s[1]);
            }
        row_sums<TPR, 2>(s, scratch);
        const float inv = rsqrtf(fmaf(s[0], over, a.eps)), mean = s[1] * inv * over;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            const int64_t c = (j * TPR + tid) * V;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float nv = hv[j][i] * inv;
                dw[j][i] = fmaf(gv[j][i], nv, dw[j][i]);
                gr[j][i] = fmaf(inv, fmaf(-nv, mean, gv[j][i] * w[j][i]), gr[j][i]);
            }
            store_chunk<T, V>(static_cast<T *>(a.grad_x) + rr * a.D, gr[j], c, D, a.vec);
            if (a.grad_h != nullptr) store_chunk<R, V>(static_cast<R *>(a.grad_h) + rr * a.D, gr[j], c, D, a.vec);
        }
    }
    if (part != nullptr) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j)
            store_chunk<float, V>(part + slot * a.D, dw[j], (j * TPR + tid) * V, a.D, a.vec);
    }
}

template <class T, class R>
__global__ void __launch_bounds__(kLongThreads) long_norm_grad_kernel(const __grid_constant__ NormGradArgs a, float *part)
{
    __shared__ float scratch[kLongThreads / 32][2];
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const T *gy = static_cast<const T *>(a.grad_y) + row * a.grad_y_stride;
        const R *h = static_cast<const R *>(a.h) + row * a.h_stride;
        const R *gr = a.grad_residual != nullptr ? static_cast<const R *>(a.grad_residual) + row * a.grad_residual_stride
                                                 : nullptr;
        float s[2] = {0.f, 0.f};
        for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) {
            const float hv = to_f(h[c]);
            s[0] = fmaf(hv, hv, s[0]);
            s[1] = fmaf(to_f(gy[c]) * a.weight[c], hv, s[1]);
        }
        row_sums<kLongThreads, 2>(s, scratch);
        const float inv = rsqrtf(s[0] / static_cast<float>(a.D) + a.eps), mean = s[1] * inv / static_cast<float>(a.D);
        for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) {
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

template <class T, class R>
rlscan_status forward(const NormArgs &a, cudaStream_t s)
{
    auto go = [&](auto tpr) {
        constexpr int TPR = decltype(tpr)::value;
        return launch_overlapped(norm_kernel<T, R, TPR>, ceil_div(a.M, kBlock<TPR> / TPR), kBlock<TPR>, 0, s, a);
    };
    switch (row_threads<T>(a.D)) {
    case 32: return go(std::integral_constant<int, 32>());
    case 64: return go(std::integral_constant<int, 64>());
    case 128: return go(std::integral_constant<int, 128>());
    case 256: return go(std::integral_constant<int, 256>());
    case 512: return go(std::integral_constant<int, 512>());
    case 1024: return go(std::integral_constant<int, 1024>());
    default: return launch_overlapped(long_norm_kernel<T, R>, a.M, kLongThreads, 0, s, a);
    }
}

// Rows of partial sums of the weight's gradient: a wave of blocks' worth.
constexpr int64_t kParts = 152 * 8;

template <class T>
int64_t grad_grid(int64_t M, int64_t D)
{
    const int tpr = row_threads<T>(D);
    const int64_t rows = tpr > 0 && tpr < 128 ? 128 / tpr : 1;   // a block works on at a time
    const int64_t most = tpr > 256 || tpr == 0 ? kParts / 4 : kParts / rows;
    const int64_t need = ceil_div(M, rows);
    return need < most ? need : most;
}

template <class T, class R>
rlscan_status backward(const NormGradArgs &a, float *part, cudaStream_t s)
{
    const int64_t grid = grad_grid<T>(a.M, a.D);
    auto go = [&](auto tpr) {
        constexpr int TPR = decltype(tpr)::value;
        return launch_overlapped(norm_grad_kernel<T, R, TPR>, grid, kBlock<TPR>, 0, s, a, part);
    };
    switch (row_threads<T>(a.D)) {
    case 32: return go(std::integral_constant<int, 32>());
    case 64: return go(std::integral_constant<int, 64>());
    case 128: return go(std::integral_constant<int, 128>());
    case 256: return go(std::integral_constant<int, 256>());
    case 512: return go(std::integral_constant<int, 512>());
    case 1024: return go(std::integral_constant<int, 1024>());
    default: return launch_overlapped(long_norm_grad_kernel<T, R>, grid, kLongThreads, 0, s, a, part);
    }
}

// rows of `part` that a call fills
template <class T>
int64_t parts_of(int64_t M, int64_t D)
{
    const int tpr = row_threads<T>(D);
    return grad_grid<T>(M, D) * (tpr > 0 && tpr < 128 ? 128 / tpr : 1);
}

uint64_t low_bits(const void *p) { return reinterpret_cast<uintptr_t>(p); }

}  // namespace

rlscan_status launch_add_rms_norm(const NormArgs &args, bool bf16_io, bool bf16_residual, cudaStream_t s)
{
    NormArgs a = args;
    const int ts = bf16_io ? 2 : 4, rs = bf16_residual ? 2 : 4;
    // wide accesses: whole chunks in every row, 16-byte aligned rows
    uint64_t bits = low_bits(a.x) | a.x_stride * ts | a.D * ts | low_bits(a.y) | low_bits(a.weight);
    if (a.residual != nullptr) bits |= low_bits(a.residual) | a.residual_stride * rs | low_bits(a.residual_out);
    a.vec = bits % 16 == 0;
    if (!bf16_io) return forward<float, float>(a, s);
    return bf16_residual ? forward<bf16, bf16>(a, s) : forward<bf16, float>(a, s);
}

size_t add_rms_norm_backward_workspace(int64_t M, int64_t D)
{
    const int64_t f = parts_of<float>(M, D), b = parts_of<bf16>(M, D);
    return sizeof(float) * static_cast<size_t>(f > b ? f : b) * D;
}

rlscan_status launch_add_rms_norm_backward(const NormGradArgs &args, bool bf16_io, bool bf16_h, void *ws, cudaStream_t s)
{
    NormGradArgs a = args;
    const int ts = bf16_io ? 2 : 4, hs = bf16_h ? 2 : 4;
    uint64_t bits = low_bits(a.grad_y) | a.grad_y_stride * ts | a.D * ts | low_bits(a.h) | a.h_stride * hs |
                    low_bits(a.grad_x) | low_bits(a.grad_h) | low_bits(a.weight);
    if (a.grad_residual != nullptr) bits |= low_bits(a.grad_residual) | a.grad_residual_stride * hs;
    a.vec = bits % 16 == 0;
    float *part = a.grad_weight != nullptr ? static_cast<float *>(ws) : nullptr;
    if (a.M > 0) {
        const rlscan_status st = !bf16_io ? backward<float, float>(a, part, s)
                                          : (bf16_h ? backward<bf16, bf16>(a, part, s) : backward<bf16, float>(a, part, s));
        if (st != RLSCAN_OK) return st;
    }
    if (a.grad_weight == nullptr) return RLSCAN_OK;
    const int64_t parts = a.M == 0 ? 0 : (bf16_io ? parts_of<bf16>(a.M, a.D) : parts_of<float>(a.M, a.D));
    SumJobs jobs;
    jobs.add(part, parts, a.D, a.D, a.grad_weight, false);
    return launch_sums(jobs, s);
}

}  // namespace seq
}  // namespace rlscan
