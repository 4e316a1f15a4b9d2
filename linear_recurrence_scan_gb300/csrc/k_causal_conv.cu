// k_causal_conv.cu -- the short causal convolution of each channel, its
// gradients and its form for one token.
//
// A thread walks a run of tokens of one channel with the K-1 inputs before
// the token in registers.  A reset clears that window, so that taps never
// reach into the episode before; a run starts by walking the K-1 tokens in
// front of it (or the initial state).
#include "sequence.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kThreads = 128;
constexpr int kRun = 32;  // tokens of a thread

struct ConvOut {
    void *y, *final_state;
};

// One tap window of a channel: the K-1 last inputs, oldest first.
template <class T, int K>
struct Window {
    float v[K];  // v[K-1] is the current token's place
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = 0.f;
    }
    __device__ __forceinline__ void push(float x)
    {
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) v[k] = v[k + 1];
        v[K - 1] = x;
    }
};

// The window in front of token t0 of row n.
template <class T, int K>
__device__ __forceinline__ void fill(Window<T, K> &w, const rlscan_causal_conv_args &a, const T *x, int64_t n, int64_t d,
                                     int64_t t0)
{
    w.clear();
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
        const int64_t t = t0 - (K - 1) + k;
        float v = 0.f;
        if (t >= 0) {
            if (a.resets != nullptr && a.resets[n * a.T + t] != 0) w.clear();
            v = to_f(x[t * a.x.token_stride]);
        } else if (a.initial_state != nullptr) {
            v = to_f(static_cast<const T *>(a.initial_state)[(n * (K - 1) + t + K - 1) * a.D + d]);
        }
        w.push(v);
    }
}

template <class T, int K>
__global__ void __launch_bounds__(kThreads)
    conv_kernel(const __grid_constant__ rlscan_causal_conv_args a, const __grid_constant__ ConvOut o, int64_t runs)
{
    const int64_t blocks = (a.D + kThreads - 1) / kThreads;
    const int64_t d = blockIdx.x % blocks * kThreads + threadIdx.x, run = blockIdx.x / blocks % runs,
                  n = blockIdx.x / blocks / runs;
    if (d >= a.D) return;
    const T *x = static_cast<const T *>(a.x.data) + n * a.x.row_stride + d;
    T *y = static_cast<T *>(o.y) + n * a.T * a.D + d;
    const int64_t len = row_length(a.lengths, n, a.T), t0 = run * kRun;
    const int64_t t1 = t0 + kRun < a.T ? t0 + kRun : a.T;
    float wt[K];
#pragma unroll
    for (int k = 0; k < K; ++k) wt[k] = a.weight[d * K + k];
    const float bias = a.bias != nullptr ? a.bias[d] : 0.f;
    Window<T, K> w;
    fill<T, K>(w, a, x, n, d, t0 < len ? t0 : len);
    for (int64_t t = t0; t < t1; ++t) {
        if (t >= len) {
            y[t * a.D] = from_f<T>(0.f);
            continue;
        }
        if (a.resets != nullptr && a.resets[n * a.T + t] != 0) w.clear();
        w.push(to_f(x[t * a.x.token_stride]));
        float acc = bias;
#pragma unroll
        for (int k = 0; k < K; ++k) acc = fmaf(wt[k], w.v[k], acc);
        if (a.silu) acc *= sigmoid(acc);
        y[t * a.D] = from_f<T>(acc);
    }
    // the run that holds the last token writes the final state (run 0 of an empty row)
    if (o.final_state != nullptr && (len > t0 ? len <= t0 + kRun : len == 0 && run == 0)) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
            static_cast<T *>(o.final_state)[(n * (K - 1) + k) * a.D + d] = from_f<T>(w.v[k + 1]);
    }
}

template <class T, int K>
__global__ void __launch_bounds__(kThreads)
    conv_step_kernel(const __grid_constant__ rlscan_causal_conv_args a, T *state, int64_t P, const int32_t *slots, T *y)
{
    const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    if (i >= a.N * a.D) return;
    const int64_t n = i / a.D, d = i % a.D, slot = slots != nullptr ? slots[n] : n;
    if (slot < 0 || slot >= P) {
        y[i] = from_f<T>(0.f);
        return;
    }
    const T xv = static_cast<const T *>(a.x.data)[n * a.x.row_stride + d];
    T *w = state + slot * (K - 1) * a.D + d;
    T v[K];
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) v[k] = w[k * a.D];
    v[K - 1] = xv;
    float acc = a.bias != nullptr ? a.bias[d] : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) acc = fmaf(a.weight[d * K + k], to_f(v[k]), acc);
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) w[k * a.D] = v[k + 1];
    if (a.silu) acc *= sigmoid(acc);
    y[i] = from_f<T>(acc);
}

struct ConvGrad {
    rlscan_array3 grad_y;
    const void *grad_final;
    void *grad_x, *grad_initial;
    float *part;  // [N runs][K+1][D]: taps, bias
};

// dx_u is complete once the K-1 tokens after u have been seen: the run walks
// them too and adds only what they give to its own tokens.
template <class T, int K>
__global__ void __launch_bounds__(kThreads)
    conv_grad_kernel(const __grid_constant__ rlscan_causal_conv_args a, const __grid_constant__ ConvGrad g, int64_t runs)
{
    const int64_t blocks = (a.D + kThreads - 1) / kThreads;
    const int64_t d = blockIdx.x % blocks * kThreads + threadIdx.x, run = blockIdx.x / blocks % runs,
                  n = blockIdx.x / blocks / runs;
    if (d >= a.D) return;
    const T *x = static_cast<const T *>(a.x.data) + n * a.x.row_stride + d;
    const T *gy = static_cast<const T *>(g.grad_y.data) + n * g.grad_y.row_stride + d;
    const int64_t len = row_length(a.lengths, n, a.T), t0 = run * kRun;
    const int64_t t1 = t0 + kRun < a.T ? t0 + kRun : a.T;
    const int64_t first = run == 0 ? -(K - 1) : t0;  // the tokens whose dx this run writes: first <= u < t1
    float wt[K], acc_x[K], dw[K], db = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        wt[k] = a.weight[d * K + k];
        acc_x[k] = dw[k] = 0.f;
    }
    const float bias = a.bias != nullptr ? a.bias[d] : 0.f;
    Window<T, K> w;
    fill<T, K>(w, a, x, n, d, t0 < len ? t0 : len);
    int since = K;  // tokens of the episode before t, up to K: further back than a tap reaches where unknown
    const int64_t stop = t1 + K - 1;
    for (int64_t t = t0; t < stop; ++t) {
        // acc_x[k] belongs to token t-K+1+k
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) acc_x[k] = acc_x[k + 1];
        acc_x[K - 1] = 0.f;
        if (t < len) {
            if (a.resets != nullptr && a.resets[n * a.T + t] != 0) {
                w.clear();
                since = 0;
            }
            w.push(to_f(x[t * a.x.token_stride]));
            float gv = to_f(gy[t * g.grad_y.token_stride]);
            if (a.silu) {
                float pre = bias;
#pragma unroll
                for (int k = 0; k < K; ++k) pre = fmaf(wt[k], w.v[k], pre);
                const float sg = sigmoid(pre);
                gv *= sg * fmaf(pre, 1.f - sg, 1.f);
            }
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (K - 1 - k <= since) acc_x[k] = fmaf(wt[k], gv, acc_x[k]);
            if (t < t1) {
                db += gv;
#pragma unroll
                for (int k = 0; k < K; ++k) dw[k] = fmaf(gv, w.v[k], dw[k]);
            }
            since = since < K ? since + 1 : K;
        }
        const int64_t u = t - (K - 1);
        if (u >= first && u < t1) {
            float v = acc_x[0];
            if (g.grad_final != nullptr && u < len && u >= len - (K - 1)) {
                bool mine = true;  // of the last token's episode
                for (int64_t r = u + 1 > 0 ? u + 1 : 0; r < len; ++r)
                    mine = mine && !(a.resets != nullptr && a.resets[n * a.T + r] != 0);
                if (mine) v += to_f(static_cast<const T *>(g.grad_final)[(n * (K - 1) + u - len + K - 1) * a.D + d]);
            }
            if (u >= 0)
                static_cast<T *>(g.grad_x)[(n * a.T + u) * a.D + d] = from_f<T>(v);
            else if (g.grad_initial != nullptr)
                static_cast<T *>(g.grad_initial)[(n * (K - 1) + u + K - 1) * a.D + d] = from_f<T>(v);
        }
    }
    if (g.part != nullptr) {
        float *p = g.part + (n * runs + run) * (K + 1) * a.D + d;
#pragma unroll
        for (int k = 0; k < K; ++k) p[k * a.D] = dw[k];
        p[K * a.D] = db;
    }
}

// grad_weight[d][k], grad_bias[d] from the runs' parts
__global__ void conv_parts_kernel(const float *part, int64_t parts, int64_t D, int K, float *grad_weight,
                                  float *grad_bias)
{
    const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
    if (i >= (K + 1) * D) return;
    float acc = 0.f;
    for (int64_t w = 0; w < parts; ++w) acc += part[w * (K + 1) * D + i];
    const int64_t k = i / D, d = i % D;
    if (k < K) {
        if (grad_weight != nullptr) grad_weight[d * K + k] = acc;
    } else if (grad_bias != nullptr) {
        grad_bias[d] = acc;
    }
}

int64_t runs_of(int64_t T) { return T > 0 ? ceil_div(T, kRun) : 1; }

template <class T, class F>
rlscan_status by_taps(int64_t K, F f)
{
    switch (K) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    default: return f(std::integral_constant<int, 8>());
    }
}

template <class T>
rlscan_status forward(const rlscan_causal_conv_args &a, const ConvOut &o, cudaStream_t s)
{
    const int64_t runs = runs_of(a.T);
    const unsigned grid = static_cast<unsigned>(ceil_div(a.D, kThreads) * runs * a.N);
    return by_taps<T>(a.K, [&](auto k) {
        conv_kernel<T, decltype(k)::value><<<grid, kThreads, 0, s>>>(a, o, runs);
        return launched();
    });
}

template <class T>
rlscan_status step(const rlscan_causal_conv_args &a, void *state, int64_t P, const int32_t *slots, void *y,
                   cudaStream_t s)
{
    const unsigned grid = static_cast<unsigned>(ceil_div(a.N * a.D, kThreads));
    return by_taps<T>(a.K, [&](auto k) {
        conv_step_kernel<T, decltype(k)::value>
            <<<grid, kThreads, 0, s>>>(a, static_cast<T *>(state), P, slots, static_cast<T *>(y));
        return launched();
    });
}

template <class T>
rlscan_status backward(const rlscan_causal_conv_args &a, const ConvGrad &g, cudaStream_t s)
{
    const int64_t runs = runs_of(a.T);
    const unsigned grid = static_cast<unsigned>(ceil_div(a.D, kThreads) * runs * a.N);
    return by_taps<T>(a.K, [&](auto k) {
        conv_grad_kernel<T, decltype(k)::value><<<grid, kThreads, 0, s>>>(a, g, runs);
        return launched();
    });
}

}  // namespace

rlscan_status launch_causal_conv(const rlscan_causal_conv_args &a, void *y, void *final_state, cudaStream_t s)
{
    const ConvOut o{y, final_state};
    return a.dtype == RLSCAN_BF16 ? forward<bf16>(a, o, s) : forward<float>(a, o, s);
}

rlscan_status launch_causal_conv_step(const rlscan_causal_conv_args &a, void *state, int64_t P, const int32_t *slots,
                                      void *y, cudaStream_t s)
{
    return a.dtype == RLSCAN_BF16 ? step<bf16>(a, state, P, slots, y, s) : step<float>(a, state, P, slots, y, s);
}

size_t causal_conv_backward_workspace(const rlscan_causal_conv_args &a)
{
    return sizeof(float) * static_cast<size_t>(a.N) * runs_of(a.T) * (a.K + 1) * a.D;
}

rlscan_status launch_causal_conv_backward(const rlscan_causal_conv_args &a, const rlscan_array3 &grad_y,
                                          const void *grad_final_state, void *grad_x, float *grad_weight,
                                          float *grad_bias, void *grad_initial_state, void *ws, cudaStream_t s)
{
    ConvGrad g;
    g.grad_y = grad_y;
    g.grad_final = grad_final_state;
    g.grad_x = grad_x;
    g.grad_initial = grad_initial_state;
    g.part = grad_weight != nullptr || grad_bias != nullptr ? static_cast<float *>(ws) : nullptr;
    if (a.N > 0) {
        const rlscan_status st = a.dtype == RLSCAN_BF16 ? backward<bf16>(a, g, s) : backward<float>(a, g, s);
        if (st != RLSCAN_OK) return st;
    }
    if (grad_weight == nullptr && grad_bias == nullptr) return RLSCAN_OK;
    const int64_t m = (a.K + 1) * a.D;
    conv_parts_kernel<<<static_cast<unsigned>(ceil_div(m, 256)), 256, 0, s>>>(
        g.part, a.N * runs_of(a.T), a.D, static_cast<int>(a.K), grad_weight, grad_bias);
    return launched();
}

}  // namespace seq
}  // namespace rlscan
