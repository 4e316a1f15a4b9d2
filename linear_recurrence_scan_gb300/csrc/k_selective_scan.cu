// k_selective_scan.cu -- the selective scan over prompts and for one token.
//
//   h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,   y_t = (C_t h_t + skip x_t) silu(z_t)
//
// A lane holds four states of one channel in registers and walks the tokens
// in order; the lanes of a channel add their parts of C h with shuffles.
#include "sequence.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kThreads = 128;

struct ScanOut {
    void *y;
    float *final_state, *checkpoints;
};

template <class T, int LANES>
__global__ void __launch_bounds__(kThreads)
    scan_kernel(const __grid_constant__ rlscan_selective_scan_args a, const __grid_constant__ ScanOut o)
{
    constexpr int CH = 32 / LANES;  // channels of a warp
    const int lane = threadIdx.x & 31, sl = lane % LANES;
    const int64_t blocks = (a.D + CH - 1) / CH;
    const int64_t warp = blockIdx.x * static_cast<int64_t>(kThreads / 32) + threadIdx.x / 32;
    if (warp >= a.N * blocks) return;
    const int64_t n = warp / blocks, d = (warp % blocks) * CH + lane / LANES;
    const bool live = d < a.D;
    const int64_t dd = live ? d : a.D - 1;
    const int s0 = 4 * sl, S = static_cast<int>(a.S);
    float A2[4], h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        A2[i] = s0 + i < S ? a.A[dd * S + s0 + i] * kLog2e : 0.f;
        h[i] = s0 + i < S && a.initial_state != nullptr ? a.initial_state[(n * a.D + dd) * S + s0 + i] : 0.f;
    }
    const float bias = a.delta_bias != nullptr ? a.delta_bias[dd] : 0.f;
    const float skip = a.skip != nullptr ? a.skip[dd] : 0.f;
    const T *x = static_cast<const T *>(a.x.data) + n * a.x.row_stride + dd;
    const T *delta = static_cast<const T *>(a.delta.data) + n * a.delta.row_stride + dd;
    const T *z = a.z.data != nullptr ? static_cast<const T *>(a.z.data) + n * a.z.row_stride + dd : nullptr;
    const T *B = static_cast<const T *>(a.B.data) + n * a.B.row_stride;
    const T *C = static_cast<const T *>(a.C.data) + n * a.C.row_stride;
    T *y = static_cast<T *>(o.y) + n * a.T * a.D + dd;
    const int64_t len = row_length(a.lengths, n, a.T);
    const int64_t marks = (a.T + kCheckpoint - 1) / kCheckpoint;
    for (int64_t t = 0; t < len; ++t) {
        if (o.checkpoints != nullptr && t % kCheckpoint == 0 && live)
            for (int i = 0; i < 4; ++i)
                if (s0 + i < S) o.checkpoints[((n * marks + t / kCheckpoint) * a.D + d) * S + s0 + i] = h[i];
        if (a.resets != nullptr && a.resets[n * a.T + t] != 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = 0.f;
        }
        const float xv = to_f(x[t * a.x.token_stride]);
        float dt = to_f(delta[t * a.delta.token_stride]) + bias;
        if (a.delta_softplus) dt = softplus(dt);
        const float dtx = dt * xv;
        float acc = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (s0 + i < S) {
                h[i] = fmaf(exp2_fast(dt * A2[i]), h[i], dtx * to_f(B[t * a.B.token_stride + s0 + i]));
                acc = fmaf(to_f(C[t * a.C.token_stride + s0 + i]), h[i], acc);
            }
        }
#pragma unroll
        for (int m = LANES / 2; m > 0; m /= 2) acc += __shfl_xor_sync(0xffffffffu, acc, m);
        acc = fmaf(skip, xv, acc);
        if (z != nullptr) {
            const float zv = to_f(z[t * a.z.token_stride]);
            acc *= zv * sigmoid(zv);
        }
        if (live && sl == 0) y[t * a.D] = from_f<T>(acc);
    }
    if (live && sl == 0)
        for (int64_t t = len; t < a.T; ++t) y[t * a.D] = from_f<T>(0.f);
    if (live)
        for (int i = 0; i < 4; ++i) {
            if (s0 + i >= S) break;
            // checkpoints past the last token: the final state
            if (o.checkpoints != nullptr)
                for (int64_t m = (len + kCheckpoint - 1) / kCheckpoint; m < marks; ++m)
                    o.checkpoints[((n * marks + m) * a.D + d) * S + s0 + i] = h[i];
            if (o.final_state != nullptr) o.final_state[(n * a.D + d) * S + s0 + i] = h[i];
        }
}

template <class T>
__global__ void __launch_bounds__(kThreads)
    step_kernel(const __grid_constant__ rlscan_selective_scan_args a, float *state, int64_t P, const int32_t *slots, T *y)
{
    const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    if (i >= a.N * a.D) return;
    const int64_t n = i / a.D, d = i % a.D, slot = slots != nullptr ? slots[n] : n;
    if (slot < 0 || slot >= P) {
        y[i] = from_f<T>(0.f);
        return;
    }
    const int S = static_cast<int>(a.S);
    const float xv = to_f(static_cast<const T *>(a.x.data)[n * a.x.row_stride + d]);
    float dt = to_f(static_cast<const T *>(a.delta.data)[n * a.delta.row_stride + d]);
    if (a.delta_bias != nullptr) dt += a.delta_bias[d];
    if (a.delta_softplus) dt = softplus(dt);
    const T *B = static_cast<const T *>(a.B.data) + n * a.B.row_stride;
    const T *C = static_cast<const T *>(a.C.data) + n * a.C.row_stride;
    float *h = state + (slot * a.D + d) * S;
    float acc = a.skip != nullptr ? a.skip[d] * xv : 0.f;
    for (int s = 0; s < S; ++s) {
        const float v = fmaf(exp2_fast(dt * (a.A[d * S + s] * kLog2e)), h[s], dt * xv * to_f(B[s]));
        h[s] = v;
        acc = fmaf(to_f(C[s]), v, acc);
    }
    if (a.z.data != nullptr) {
        const float zv = to_f(static_cast<const T *>(a.z.data)[n * a.z.row_stride + d]);
        acc *= zv * sigmoid(zv);
    }
    y[i] = from_f<T>(acc);
}

template <class T>
rlscan_status launch_typed(const rlscan_selective_scan_args &a, const ScanOut &o, cudaStream_t s)
{
    const int lanes = state_lanes(a.S);
    const int64_t warps = a.N * ceil_div(a.D, 32 / lanes);
    const unsigned grid = static_cast<unsigned>(ceil_div(warps, kThreads / 32));
    switch (lanes) {
    case 1: scan_kernel<T, 1><<<grid, kThreads, 0, s>>>(a, o); break;
    case 2: scan_kernel<T, 2><<<grid, kThreads, 0, s>>>(a, o); break;
    case 4: scan_kernel<T, 4><<<grid, kThreads, 0, s>>>(a, o); break;
    case 8: scan_kernel<T, 8><<<grid, kThreads, 0, s>>>(a, o); break;
    case 16: scan_kernel<T, 16><<<grid, kThreads, 0, s>>>(a, o); break;
    default: scan_kernel<T, 32><<<grid, kThreads, 0, s>>>(a, o); break;
    }
    return launched();
}

}  // namespace

size_t selective_scan_workspace(const rlscan_selective_scan_args &) { return 0; }

rlscan_status launch_selective_scan(const rlscan_selective_scan_args &a, void *y, float *final_state,
                                    float *checkpoints, void *, cudaStream_t s)
{
    const ScanOut o{y, final_state, checkpoints};
    return a.dtype == RLSCAN_BF16 ? launch_typed<bf16>(a, o, s) : launch_typed<float>(a, o, s);
}

rlscan_status launch_selective_scan_step(const rlscan_selective_scan_args &a, float *state, int64_t P,
                                         const int32_t *slots, void *y, cudaStream_t s)
{
    const unsigned grid = static_cast<unsigned>(ceil_div(a.N * a.D, kThreads));
    if (a.dtype == RLSCAN_BF16)
        step_kernel<bf16><<<grid, kThreads, 0, s>>>(a, state, P, slots, static_cast<bf16 *>(y));
    else
        step_kernel<float><<<grid, kThreads, 0, s>>>(a, state, P, slots, static_cast<float *>(y));
    return launched();
}

}  // namespace seq
}  // namespace rlscan
