// k_causal_conv.cu -- the short causal convolution of each channel, its
// gradients and its form for one token.
//
// A thread walks a run of tokens of V neighbouring channels with the K-1
// inputs before the token in registers, in pairs of channels.  A reset clears
// that window, so that taps never reach into the episode before; a run starts
// by reading the K-1 tokens in front of it (or the initial state).
#include "sequence.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 4;  // tokens whose loads are in flight together

struct ConvOut {
    void *y, *final_state;
    int64_t run, runs;  // tokens of a thread, runs of a row
};

// V channels (an even number of them, or one) as pairs
template <int V>
constexpr int kPairs = (V + 1) / 2;

template <class T, int V>
struct Raw {  // V values as they are stored
    alignas(V * sizeof(T)) T v[V];
};

template <class T, int V>
__device__ __forceinline__ Raw<T, V> load_raw(const T *p)
{
    return *reinterpret_cast<const Raw<T, V> *>(p);
}

template <class T, int V>
__device__ __forceinline__ void widen(f2 *to, const Raw<T, V> &r)
{
#pragma unroll
    for (int i = 0; i < V; i += 2) to[i / 2] = pair(to_f(r.v[i]), i + 1 < V ? to_f(r.v[i + 1 < V ? i + 1 : i]) : 0.f);
}

template <class T, int V>
__device__ __forceinline__ void store(T *p, const f2 *v)
{
    Raw<T, V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float2 h = halves(v[i / 2]);
        r.v[i] = from_f<T>(i % 2 == 0 ? h.x : h.y);
    }
    *reinterpret_cast<Raw<T, V> *>(p) = r;
}

// a channel's values of a [D, K] array, for V channels: to[k][pair]
template <int K, int V>
__device__ __forceinline__ void load_taps(f2 (*to)[kPairs<V>], const float *w)
{
    float v[V * K];
    if (V % 4 == 0 && (reinterpret_cast<uintptr_t>(w) & 15u) == 0) {
#pragma unroll
        for (int i = 0; i + 3 < V * K; i += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(w + i);
            v[i] = q.x;
            v[i + 1] = q.y;
            v[i + 2] = q.z;
            v[i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * K; ++i) v[i] = w[i];
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; i += 2) to[k][i / 2] = pair(v[i * K + k], i + 1 < V ? v[(i + 1 < V ? i + 1 : i) * K + k] : 0.f);
}

// The K-1 last inputs of V channels, oldest first, and the current one behind them.
template <class T, int K, int V>
struct Window {
    f2 v[K][kPairs<V>];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i) v[k][i] = 0ull;
    }
    __device__ __forceinline__ void push(const Raw<T, V> &x)
    {
#pragma unroll
        for (int k = 0; k + 1 < K; ++k)
#pragma unroll
            for (int i = 0; i < kPairs<V>; ++i) v[k][i] = v[k + 1][i];
        widen<T, V>(v[K - 1], x);
    }
    // the window in front of token t0 of row n
    __device__ __forceinline__ void fill(const rlscan_causal_conv_args &a, const T *x, int64_t n, int64_t d, int64_t t0)
    {
        clear();
#pragma unroll
        for (int k = 0; k < K - 1; ++k) {
            const int64_t t = t0 - (K - 1) + k;
            Raw<T, V> r;
#pragma unroll
            for (int i = 0; i < V; ++i) r.v[i] = from_f<T>(0.f);
            if (t >= 0) {
                if (a.resets != nullptr && a.resets[n * a.T + t] != 0) clear();
                r = load_raw<T, V>(x + t * a.x.token_stride);
            } else if (a.initial_state != nullptr) {
                r = load_raw<T, V>(static_cast<const T *>(a.initial_state) + (n * (K - 1) + t + K - 1) * a.D + d);
            }
            push(r);
        }
    }
    __device__ __forceinline__ void dot(f2 *acc, const f2 (*w)[kPairs<V>], const f2 *bias) const
    {
#pragma unroll
        for (int i = 0; i < kPairs<V>; ++i) {
            f2 s = bias[i];
#pragma unroll
            for (int k = 0; k < K; ++k) s = fma2(w[k][i], v[k][i], s);
            acc[i] = s;
        }
    }
};

template <int V>
__device__ __forceinline__ void load_bias(f2 *bias, const float *b, int64_t d)
{
#pragma unroll
    for (int i = 0; i < V; i += 2)
        bias[i / 2] = b != nullptr ? pair(b[d + i], i + 1 < V ? b[d + i + 1] : 0.f) : 0ull;
}

template <class T, int K, int V>
__global__ void __launch_bounds__(kThreads)
    conv_kernel(const __grid_constant__ rlscan_causal_conv_args a, const __grid_constant__ ConvOut o)
{
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int64_t vecs = a.D / V, i0 = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    const int64_t d = i0 % vecs * V, run = i0 / vecs % o.runs, n = i0 / vecs / o.runs;
    if (n >= a.N) return;
    const T *x = static_cast<const T *>(a.x.data) + n * a.x.row_stride + d;
    T *y = static_cast<T *>(o.y) + n * a.T * a.D + d;
    const int64_t len = row_length(a.lengths, n, a.T), t0 = run * o.run;
    const int64_t t1 = t0 + o.run < a.T ? t0 + o.run : a.T, stop = len < t1 ? len : t1;
    f2 w[K][kPairs<V>], bias[kPairs<V>];
    load_taps<K, V>(w, a.weight + d * K);
    load_bias<V>(bias, a.bias, d);
    Window<T, K, V> win;
    win.fill(a, x, n, d, t0 < len ? t0 : len);
    for (int64_t t = t0; t < stop; t += kAhead) {
        Raw<T, V> r[kAhead];
        uint8_t starts[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (t + u < stop) {
                r[u] = load_raw<T, V>(x + (t + u) * a.x.token_stride);
                starts[u] = a.resets != nullptr ? a.resets[n * a.T + t + u] : 0;
            }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (t + u < stop) {
                if (starts[u] != 0) win.clear();
                win.push(r[u]);
                f2 acc[kPairs<V>];
                win.dot(acc, w, bias);
                if (a.silu) {
#pragma unroll
                    for (int i = 0; i < kPairs<V>; ++i) acc[i] = mul2(acc[i], sigmoid(acc[i]));
                }
                store<T, V>(y + (t + u) * a.D, acc);
            }
    }
    const f2 zero[kPairs<V>] = {};
    for (int64_t t = stop > t0 ? stop : t0; t < t1; ++t) store<T, V>(y + t * a.D, zero);
    // the run that holds the last token writes the final state (run 0 of an empty row)
    if (o.final_state != nullptr && (len > t0 ? len <= t0 + o.run : len == 0 && run == 0)) {
#pragma unroll
        for (int k = 0; k < K - 1; ++k)
            store<T, V>(static_cast<T *>(o.final_state) + (n * (K - 1) + k) * a.D + d, win.v[k + 1]);
    }
}

template <class T, int K, int V>
__global__ void __launch_bounds__(kThreads)
    conv_step_kernel(const __grid_constant__ rlscan_causal_conv_args a, T *state, int64_t P, const int32_t *slots, T *y)
{
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int64_t vecs = a.D / V, i0 = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    const int64_t n = i0 / vecs, d = i0 % vecs * V;
    if (n >= a.N) return;
    const int64_t slot = slots != nullptr ? slots[n] : n;
    const Raw<T, V> xv = load_raw<T, V>(static_cast<const T *>(a.x.data) + n * a.x.row_stride + d);
    f2 w[K][kPairs<V>], bias[kPairs<V>];
    load_taps<K, V>(w, a.weight + d * K);
    load_bias<V>(bias, a.bias, d);
    const bool idle = slot < 0 || slot >= P;
    Window<T, K, V> win;
    win.clear();
    T *st = state + (idle ? 0 : slot) * (K - 1) * a.D + d;
    if (!idle) {
        Raw<T, V> r[K];
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) r[k] = load_raw<T, V>(st + k * a.D);
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) win.push(r[k]);
        win.push(xv);
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) *reinterpret_cast<Raw<T, V> *>(st + k * a.D) = k + 2 < K ? r[k + 1] : xv;
    }
    f2 acc[kPairs<V>];
    win.dot(acc, w, bias);
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) {
        if (a.silu) acc[i] = mul2(acc[i], sigmoid(acc[i]));
        if (idle) acc[i] = 0ull;
    }
    store<T, V>(y + n * a.D + d, acc);
}

struct ConvGrad {
    rlscan_array3 grad_y;
    const void *grad_final;
    void *grad_x, *grad_initial;
    float *part;  // [N runs][D K | D]: taps, bias
    int64_t run, runs;
};

// dx_u is complete once the K-1 tokens after u have been seen: a run walks
// them too and adds only what they give to its own tokens.
template <class T, int K, int V>
__global__ void __launch_bounds__(kThreads)
    conv_grad_kernel(const __grid_constant__ rlscan_causal_conv_args a, const __grid_constant__ ConvGrad g)
{
    constexpr int H = kPairs<V>;
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int64_t vecs = a.D / V, i0 = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    const int64_t d = i0 % vecs * V, run = i0 / vecs % g.runs, n = i0 / vecs / g.runs;
    if (n >= a.N) return;
    const T *x = static_cast<const T *>(a.x.data) + n * a.x.row_stride + d;
    const T *gy = static_cast<const T *>(g.grad_y.data) + n * g.grad_y.row_stride + d;
    const int64_t len = row_length(a.lengths, n, a.T), t0 = run * g.run;
    const int64_t t1 = t0 + g.run < a.T ? t0 + g.run : a.T;
    const int64_t first = run == 0 ? -(K - 1) : t0;  // the tokens whose dx this run writes: first <= u < t1
    const int64_t stop = t1 + K - 1;
    f2 w[K][H], acc_x[K][H], dw[K][H], db[H], bias[H];
    load_taps<K, V>(w, a.weight + d * K);
    load_bias<V>(bias, a.bias, d);
#pragma unroll
    for (int i = 0; i < H; ++i) {
        db[i] = 0ull;
#pragma unroll
        for (int k = 0; k < K; ++k) acc_x[k][i] = dw[k][i] = 0ull;
    }
    Window<T, K, V> win;
    win.fill(a, x, n, d, t0 < len ? t0 : len);
    int since = K;  // tokens of the episode in front of t, as far as a tap of this run's tokens can see
    for (int64_t t = t0; t < stop; t += kAhead) {
        Raw<T, V> rx[kAhead], rg[kAhead];
        uint8_t starts[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (t + u < stop && t + u < len) {
                rx[u] = load_raw<T, V>(x + (t + u) * a.x.token_stride);
                rg[u] = load_raw<T, V>(gy + (t + u) * g.grad_y.token_stride);
                starts[u] = a.resets != nullptr ? a.resets[n * a.T + t + u] : 0;
            }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t at = t + u;
            if (at >= stop) break;
            // acc_x[k] belongs to token at-K+1+k
#pragma unroll
            for (int i = 0; i < H; ++i) {
#pragma unroll
                for (int k = 0; k + 1 < K; ++k) acc_x[k][i] = acc_x[k + 1][i];
                acc_x[K - 1][i] = 0ull;
            }
            if (at < len) {
                if (starts[u] != 0) {
                    win.clear();
                    since = 0;
                }
                win.push(rx[u]);
                f2 gv[H];
                widen<T, V>(gv, rg[u]);
                if (a.silu) {
                    f2 pre[H];
                    win.dot(pre, w, bias);
#pragma unroll
                    for (int i = 0; i < H; ++i) {  // silu' = s (1 + v (1 - s))
                        const f2 s = sigmoid(pre[i]);
                        const f2 rest = fma2(s, both(-1.f), both(1.f));
                        gv[i] = mul2(gv[i], mul2(s, fma2(pre[i], rest, both(1.f))));
                    }
                }
                if (since >= K - 1) {
#pragma unroll
                    for (int k = 0; k < K; ++k)
#pragma unroll
                        for (int i = 0; i < H; ++i) acc_x[k][i] = fma2(w[k][i], gv[i], acc_x[k][i]);
                } else {
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (K - 1 - k <= since)
#pragma unroll
                            for (int i = 0; i < H; ++i) acc_x[k][i] = fma2(w[k][i], gv[i], acc_x[k][i]);
                }
                if (at < t1) {
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        db[i] = add2(db[i], gv[i]);
#pragma unroll
                        for (int k = 0; k < K; ++k) dw[k][i] = fma2(gv[i], win.v[k][i], dw[k][i]);
                    }
                }
                since = since < K ? since + 1 : K;
            }
            const int64_t to = at - (K - 1);
            if (to >= first && to < t1) {
                f2 v[H];
#pragma unroll
                for (int i = 0; i < H; ++i) v[i] = acc_x[0][i];
                if (g.grad_final != nullptr && to < len && to >= len - (K - 1)) {
                    bool mine = true;  // of the last token's episode
                    for (int64_t r = to + 1 > 0 ? to + 1 : 0; r < len; ++r)
                        mine = mine && !(a.resets != nullptr && a.resets[n * a.T + r] != 0);
                    if (mine) {
                        f2 f[H];
                        widen<T, V>(f, load_raw<T, V>(static_cast<const T *>(g.grad_final) +
                                                      (n * (K - 1) + to - len + K - 1) * a.D + d));
#pragma unroll
                        for (int i = 0; i < H; ++i) v[i] = add2(v[i], f[i]);
                    }
                }
                if (to >= 0)
                    store<T, V>(static_cast<T *>(g.grad_x) + (n * a.T + to) * a.D + d, v);
                else if (g.grad_initial != nullptr)
                    store<T, V>(static_cast<T *>(g.grad_initial) + (n * (K - 1) + to + K - 1) * a.D + d, v);
            }
        }
    }
    if (g.part != nullptr) {
        float *p = g.part + (n * g.runs + run) * (K + 1) * a.D;
        float flat[V * K];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float2 h = halves(dw[k][i / 2]);
                flat[i * K + k] = i % 2 == 0 ? h.x : h.y;
            }
        if constexpr (V % 4 == 0) {  // D is a multiple of V, the workspace aligned
#pragma unroll
            for (int i = 0; i < V * K; i += 4)
                *reinterpret_cast<float4 *>(p + d * K + i) = make_float4(flat[i], flat[i + 1], flat[i + 2], flat[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < V * K; ++i) p[d * K + i] = flat[i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 h = halves(db[i / 2]);
            p[K * a.D + d + i] = i % 2 == 0 ? h.x : h.y;
        }
    }
}

// Tokens of a thread: as many as leave enough threads to keep loads in
// flight, since each run reads K-1 tokens of its neighbours again.
int64_t run_length(const rlscan_causal_conv_args &a, int v, int64_t most)
{
    const int sms = sm_count() > 0 ? sm_count() : 152;
    int64_t run = most;
    while (run > 8 && a.N * ceil_div(a.T, run) * (a.D / v) < sms * 768ll) run /= 2;
    return run;
}

constexpr int64_t kMostRun = 64, kMostGradRun = 128;

template <class F>
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

template <class T, int V>
rlscan_status forward(const rlscan_causal_conv_args &a, ConvOut o, cudaStream_t s)
{
    o.run = run_length(a, V, kMostRun);
    o.runs = a.T > 0 ? ceil_div(a.T, o.run) : 1;
    return by_taps(a.K, [&](auto k) {
        return launch_overlapped(conv_kernel<T, decltype(k)::value, V>, ceil_div(a.N * o.runs * (a.D / V), kThreads), kThreads,
                                 0, s, a, o);
    });
}

template <class T, int V>
rlscan_status step(const rlscan_causal_conv_args &a, void *state, int64_t P, const int32_t *slots, void *y,
                   cudaStream_t s)
{
    return by_taps(a.K, [&](auto k) {
        return launch_overlapped(conv_step_kernel<T, decltype(k)::value, V>, ceil_div(a.N * (a.D / V), kThreads), kThreads, 0, s,
                                 a, static_cast<T *>(state), P, slots, static_cast<T *>(y));
    });
}

template <class T, int V>
rlscan_status backward(const rlscan_causal_conv_args &a, const ConvGrad &g, cudaStream_t s)
{
    return by_taps(a.K, [&](auto k) {
        return launch_overlapped(conv_grad_kernel<T, decltype(k)::value, V>, ceil_div(a.N * g.runs * (a.D / V), kThreads),
                                 kThreads, 0, s, a, g);
    });
}

// Whether the rows of all arrays are whole, aligned units of `v` values.
bool wide(const rlscan_causal_conv_args &a, int v, std::initializer_list<const void *> dense)
{
    const int size = a.dtype == RLSCAN_BF16 ? 2 : 4;
    uint64_t bits = static_cast<uint64_t>(a.D) * size | reinterpret_cast<uintptr_t>(a.x.data) |
                    static_cast<uint64_t>(a.x.row_stride) * size | static_cast<uint64_t>(a.x.token_stride) * size;
    for (const void *p : dense) bits |= reinterpret_cast<uintptr_t>(p);
    return bits % (v * size) == 0;
}

// channels of a thread of the gradients' kernel, by the shape alone (the
// workspace has to suffice for either)
constexpr int kGradVec = 4;

int64_t grad_runs(const rlscan_causal_conv_args &a, int v)
{
    return a.T > 0 ? ceil_div(a.T, run_length(a, v, kMostGradRun)) : 1;
}

}  // namespace

rlscan_status launch_causal_conv(const rlscan_causal_conv_args &a, void *y, void *final_state, cudaStream_t s)
{
    const ConvOut o{y, final_state, 0, 0};
    const bool b16 = a.dtype == RLSCAN_BF16;
    if (wide(a, b16 ? 8 : 4, {y, final_state, a.initial_state}))
        return b16 ? forward<bf16, 8>(a, o, s) : forward<float, 4>(a, o, s);
    return b16 ? forward<bf16, 1>(a, o, s) : forward<float, 1>(a, o, s);
}

rlscan_status launch_causal_conv_step(const rlscan_causal_conv_args &a, void *state, int64_t P, const int32_t *slots,
                                      void *y, cudaStream_t s)
{
    const bool b16 = a.dtype == RLSCAN_BF16;
    if (wide(a, 4, {state, y})) return b16 ? step<bf16, 4>(a, state, P, slots, y, s) : step<float, 4>(a, state, P, slots, y, s);
    return b16 ? step<bf16, 1>(a, state, P, slots, y, s) : step<float, 1>(a, state, P, slots, y, s);
}

size_t causal_conv_backward_workspace(const rlscan_causal_conv_args &a)
{
    const int64_t one = grad_runs(a, 1), four = grad_runs(a, kGradVec);
    return sizeof(float) * static_cast<size_t>(a.N) * (one > four ? one : four) * (a.K + 1) * a.D;
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
    const bool b16 = a.dtype == RLSCAN_BF16;
    const int size = b16 ? 2 : 4;
    const bool four = wide(a, kGradVec, {grad_y.data, grad_x, grad_final_state, a.initial_state, grad_initial_state}) &&
                      grad_y.row_stride * size % (kGradVec * size) == 0 && grad_y.token_stride % kGradVec == 0;
    const int v = four ? kGradVec : 1;
    g.runs = grad_runs(a, v);
    g.run = run_length(a, v, kMostGradRun);
    if (a.N > 0) {
        const rlscan_status st = four ? (b16 ? backward<bf16, kGradVec>(a, g, s) : backward<float, kGradVec>(a, g, s))
                                      : (b16 ? backward<bf16, 1>(a, g, s) : backward<float, 1>(a, g, s));
        if (st != RLSCAN_OK) return st;
    }
    SumJobs jobs;
    const int64_t pitch = (a.K + 1) * a.D, parts = a.N * g.runs;
    if (grad_weight != nullptr) jobs.add(g.part, parts, pitch, a.K * a.D, grad_weight, false);
    if (grad_bias != nullptr) jobs.add(g.part + a.K * a.D, parts, pitch, a.D, grad_bias, false);
    return launch_sums(jobs, s);
}

}  // namespace seq
}  // namespace rlscan
