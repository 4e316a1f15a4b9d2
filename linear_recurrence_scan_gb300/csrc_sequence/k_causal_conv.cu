// k_causal_conv.cu -- the short causal convolution of each channel, its
// gradients and its form for one token.
//
// A thread walks a run of tokens of V neighbouring channels with the K-1
// inputs before the token in registers, in pairs of channels.  A reset clears
// that window, so that taps never reach into the episode before; a run starts
// by reading the K-1 tokens in front of it (or the initial state).
// Bytes bound it: 8 x 4096 x 4096 bf16 97 us forward (5.5 TB/s), 289 us with
// gradients (4.6 TB/s, 60 % of the issue slots).
#include "sequence.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 4;   // tokens of a block
// Blocks on their way to a thread.  Measured (8 x 4096 x 4096 bf16, forward
// and with gradients): in registers, one block ahead, 121 and 327 us; through
// shared memory with 3, 4, 6, 8 blocks 99, 97, 97, 101 and 303, 296, 303, 315.
constexpr int kBlocks = 4;

struct ConvOut {
    void *y, *final_state;
    int64_t run, runs;  // tokens of a thread, runs of a row
};

// V channels (an even number of them, or one) as pairs
template <int V>
constexpr int kPairs = (V + 1) / 2;

template <class T, int V>
__device__ __forceinline__ void widen(f2 *to, const Words<T, V> &r)
{
#pragma unroll
    for (int i = 0; i < V; i += 2) to[i / 2] = pair(r[i], i + 1 < V ? r[i + 1 < V ? i + 1 : i] : 0.f);
}

template <class T, int V>
__device__ __forceinline__ void store(T *p, const f2 *v)
{
    Words<T, V> r;
#pragma unroll
    for (int i = 0; i < kPairs<V>; ++i) {
        const float2 h = halves(v[i]);
        r.set(i, h.x, h.y);
    }
    r.store(p);
}

// a channel's values of a [D, K] array, for V channels: to[k][pair]
template <int K, int V>
__device__ __forceinline__ void load_taps(f2 (*to)[kPairs<V>], const float *w)
{
    float v[V * K];
    if (V % 2 == 0 && (reinterpret_cast<uintptr_t>(w) & 7u) == 0) {
#pragma unroll
        for (int i = 0; i + 1 < V * K; i += 2) {
            const float2 q = *reinterpret_cast<const float2 *>(w + i);
            v[i] = q.x;
            v[i + 1] = q.y;
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
    __device__ __forceinline__ void push(const Words<T, V> &x)
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
            Words<T, V> r;
            r.zero();
            if (t >= 0) {
                if (a.resets != nullptr && a.resets[n * a.T + t] != 0) clear();
                r.load(x + t * a.x.token_stride);
            } else if (a.initial_state != nullptr) {
                r.load(static_cast<const T *>(a.initial_state) + (n * (K - 1) + t + K - 1) * a.D + d);
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

// A thread's next values of ARRAYS arrays, kBlocks blocks of kAhead tokens on
// their way: through its own place in shared memory by asynchronous copies,
// which hold no registers while in flight, or, for single 16-bit values,
// which these cannot copy, in registers and one block ahead.
template <class T, int V, int ARRAYS>
struct Feed {
    static constexpr int BYTES = V * static_cast<int>(sizeof(T));
    static constexpr bool RING = BYTES >= 4;
    static constexpr int DEPTH = RING ? kBlocks : 2;
    static constexpr size_t SMEM = RING ? static_cast<size_t>(DEPTH) * kAhead * ARRAYS * kThreads * BYTES : 0;
    char *ring;
    Words<T, V> next[RING ? 1 : ARRAYS][RING ? 1 : kAhead], held[RING ? 1 : ARRAYS][RING ? 1 : kAhead];
    uint32_t next_flag[kAhead], flag[kAhead];

    __device__ __forceinline__ char *place(int block, int u, int array)
    {
        return ring + (((block % DEPTH) * kAhead + u) * ARRAYS + array) * (kThreads * BYTES) + threadIdx.x * BYTES;
    }
    // token u of block `block`, `from` its address, if it is there
    __device__ __forceinline__ void take(int block, int u, int array, const T *from, const T *safe, bool there)
    {
        if constexpr (RING) {
            void *to = place(block, u, array);
            const T *at = there ? from : safe;
            const int bytes = there ? BYTES : 0;
            if constexpr (BYTES == 16)
                copy16(to, at, bytes);
            else if constexpr (BYTES == 8)
                copy8(to, at, bytes);
            else
                copy4(to, at, bytes);
        } else if (there) {
            next[array][u].load(from);
        }
    }
    // block `block`'s turn: its values are here
    __device__ __forceinline__ void turn()
    {
        if constexpr (RING) {
            copies_wait<DEPTH - 1>();
        } else {
#pragma unroll
            for (int i = 0; i < ARRAYS; ++i)
#pragma unroll
                for (int u = 0; u < kAhead; ++u) held[i][u] = next[i][u];
        }
    }
    __device__ __forceinline__ Words<T, V> get(int block, int u, int array)
    {
        if constexpr (RING) {
            Words<T, V> r;
            r.load(reinterpret_cast<const T *>(place(block, u, array)));
            return r;
        } else {
            return held[array][u];
        }
    }
};

// a bit for each token that starts an episode
__device__ __forceinline__ uint32_t bits(const uint32_t (&flag)[kAhead])
{
    uint32_t b = 0;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) b |= (flag[u] != 0 ? 1u : 0u) << u;
    return b;
}

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
    const Division at = divide(blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x, a.D / V);
    const Division at_row = divide(at.q, o.runs);
    const int64_t d = at.r * V, run = at_row.r, n = at_row.q;
    if (n >= a.N) return;
    const T *x = static_cast<const T *>(a.x.data) + n * a.x.row_stride + d;
    T *y = static_cast<T *>(o.y) + n * a.T * a.D + d;
    const int64_t len = row_length(a.lengths, n, a.T), t0 = run * o.run;
    const int64_t t1 = t0 + o.run < a.T ? t0 + o.run : a.T, stop = len < t1 ? len : t1;
    f2 w[K][kPairs<V>], bias[kPairs<V>];
    load_taps<K, V>(w, a.weight + d * K);
    load_bias<V>(bias, a.bias, d);
    const uint32_t silu = a.silu ? ~0u : 0u;
    Window<T, K, V> win;
    win.fill(a, x, n, d, t0 < len ? t0 : len);
    using F = Feed<T, V, 1>;
    extern __shared__ __align__(16) char ring[];
    F feed;
    feed.ring = ring;
    const int count = static_cast<int>(stop > t0 ? stop - t0 : 0), blocks = (count + kAhead - 1) / kAhead;
    const T *xt = x + t0 * a.x.token_stride;
    const uint8_t *resets = a.resets != nullptr ? a.resets + n * a.T + t0 : nullptr;
    T *yt = y + t0 * a.D;
    auto issue = [&](int block) {
        if (block * kAhead < count)
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int t = block * kAhead + u;
                feed.take(block, u, 0, xt + t * a.x.token_stride, x, t < count);
            }
        copies_commit();
    };
    auto flags_of = [&](int block) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int t = block * kAhead + u;
            feed.next_flag[u] = resets != nullptr && t < count ? load_byte(resets + t) : 0u;
        }
    };
#pragma unroll
    for (int b = 0; b < F::DEPTH - 1; ++b) issue(b);
    flags_of(0);
    for (int b = 0; b < blocks; ++b) {
        if (F::RING) issue(b + F::DEPTH - 1);
        feed.turn();
        if (!F::RING) issue(b + 1);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) feed.flag[u] = feed.next_flag[u];
        flags_of(b + 1);
        const uint32_t starts = bits(feed.flag);
        const int t = b * kAhead;
        auto walk = [&](auto fast) {
            constexpr bool FAST = decltype(fast)::value;
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (!FAST && t + u >= count) break;
                if (!FAST && (starts >> u & 1u) != 0) win.clear();
                win.push(feed.get(b, u, 0));
                f2 acc[kPairs<V>];
                win.dot(acc, w, bias);
#pragma unroll
                for (int i = 0; i < kPairs<V>; ++i) {
                    const float2 v = halves(acc[i]), g = halves(mul2(acc[i], sigmoid(acc[i])));
                    acc[i] = pair(choose(silu, g.x, v.x), choose(silu, g.y, v.y));
                }
                store<T, V>(yt + (t + u) * a.D, acc);
            }
        };
        if (starts == 0 && t + kAhead <= count)
            walk(std::true_type());
        else
            walk(std::false_type());
    }
    copies_wait<0>();
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
    const Division at = divide(blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x, a.D / V);
    const int64_t n = at.q, d = at.r * V;
    if (n >= a.N) return;
    const int64_t slot = slots != nullptr ? slots[n] : n;
    Words<T, V> xv;
    xv.load(static_cast<const T *>(a.x.data) + n * a.x.row_stride + d);
    f2 w[K][kPairs<V>], bias[kPairs<V>];
    load_taps<K, V>(w, a.weight + d * K);
    load_bias<V>(bias, a.bias, d);
    const bool idle = slot < 0 || slot >= P;
    Window<T, K, V> win;
    win.clear();
    T *st = state + (idle ? 0 : slot) * (K - 1) * a.D + d;
    if (!idle) {
        Words<T, V> r[K];
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) r[k].load(st + k * a.D);
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) win.push(r[k]);
        win.push(xv);
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) (k + 2 < K ? r[k + 1] : xv).store(st + k * a.D);
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
    const Division at = divide(blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x, a.D / V);
    const Division at_row = divide(at.q, g.runs);
    const int64_t d = at.r * V, run = at_row.r, n = at_row.q;
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
    // in tokens behind t0: the run's own, those with a dL/dy, all it walks
    const int own = static_cast<int>(t1 - t0), all = static_cast<int>(stop - t0);
    const int64_t rest = len - t0;
    const int live = static_cast<int>(rest < 0 ? 0 : (rest < all ? rest : all));
    const T *xt = x + t0 * a.x.token_stride, *gt = gy + t0 * g.grad_y.token_stride;
    const uint8_t *resets = a.resets != nullptr ? a.resets + n * a.T + t0 : nullptr;
    T *dx = static_cast<T *>(g.grad_x) + (n * a.T + t0) * a.D + d;
    const uint32_t silu = a.silu ? ~0u : 0u;
    using F = Feed<T, V, 2>;
    extern __shared__ __align__(16) char ring[];
    F feed;
    feed.ring = ring;
    auto issue = [&](int block) {
        if (block * kAhead < live)
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const int t = block * kAhead + u;
                feed.take(block, u, 0, xt + t * a.x.token_stride, x, t < live);
                feed.take(block, u, 1, gt + t * g.grad_y.token_stride, gy, t < live);
            }
        copies_commit();
    };
    auto flags_of = [&](int block) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int t = block * kAhead + u;
            feed.next_flag[u] = resets != nullptr && t < live ? load_byte(resets + t) : 0u;
        }
    };
    auto slope = [&](f2 *gv) {  // dL/dpre from dL/dy: silu' = s (1 + v (1 - s))
        f2 pre[H];
        win.dot(pre, w, bias);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const f2 s = sigmoid(pre[i]);
            const float2 v = halves(mul2(s, fma2(pre[i], fma2(s, both(-1.f), both(1.f)), both(1.f))));
            gv[i] = mul2(gv[i], pair(choose(silu, v.x, 1.f), choose(silu, v.y, 1.f)));
        }
    };
    // acc_x[k] belongs to the token K-1-k before the current one
    auto shift = [&] {
#pragma unroll
        for (int i = 0; i < H; ++i) {
#pragma unroll
            for (int k = 0; k + 1 < K; ++k) acc_x[k][i] = acc_x[k + 1][i];
            acc_x[K - 1][i] = 0ull;
        }
    };
    auto params = [&](const f2 *gv) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            db[i] = add2(db[i], gv[i]);
#pragma unroll
            for (int k = 0; k < K; ++k) dw[k][i] = fma2(gv[i], win.v[k][i], dw[k][i]);
        }
    };
#pragma unroll
    for (int b = 0; b < F::DEPTH - 1; ++b) issue(b);
    flags_of(0);
    for (int b = 0; b * kAhead < all; ++b) {
        if (F::RING) issue(b + F::DEPTH - 1);
        feed.turn();
        if (!F::RING) issue(b + 1);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) feed.flag[u] = feed.next_flag[u];
        flags_of(b + 1);
        const uint32_t starts = bits(feed.flag);
        const int t = b * kAhead;
        const int safe = g.grad_final == nullptr ? live : live - (K - 1);
        if (starts == 0 && since >= K - 1 && t >= K - 1 && t + kAhead <= own && t + kAhead <= safe) {
            // tokens of one episode inside the run, without a branch
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                shift();
                win.push(feed.get(b, u, 0));
                f2 gv[H];
                widen<T, V>(gv, feed.get(b, u, 1));
                slope(gv);
#pragma unroll
                for (int k = 0; k < K; ++k)
#pragma unroll
                    for (int i = 0; i < H; ++i) acc_x[k][i] = fma2(w[k][i], gv[i], acc_x[k][i]);
                params(gv);
                store<T, V>(dx + (t + u - (K - 1)) * a.D, acc_x[0]);
            }
            since = K;
        } else {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (t + u >= all) break;
                shift();
                if (t + u < live) {
                    if ((starts >> u & 1u) != 0) {
                        win.clear();
                        since = 0;
                    }
                    win.push(feed.get(b, u, 0));
                    f2 gv[H];
                    widen<T, V>(gv, feed.get(b, u, 1));
                    slope(gv);
#pragma unroll
                    for (int k = 0; k < K; ++k)
                        if (K - 1 - k <= since)
#pragma unroll
                            for (int i = 0; i < H; ++i) acc_x[k][i] = fma2(w[k][i], gv[i], acc_x[k][i]);
                    if (t + u < own) params(gv);
                    since = since < K ? since + 1 : K;
                }
                const int64_t to = t0 + t + u - (K - 1);
                if (to < first || to >= t1) continue;
                f2 v[H];
#pragma unroll
                for (int i = 0; i < H; ++i) v[i] = acc_x[0][i];
                if (g.grad_final != nullptr && to < len && to >= len - (K - 1)) {
                    bool mine = true;  // of the last token's episode
                    for (int64_t r = to + 1 > 0 ? to + 1 : 0; r < len; ++r)
                        mine = mine && !(a.resets != nullptr && a.resets[n * a.T + r] != 0);
                    if (mine) {
                        f2 f[H];
                        Words<T, V> gf;
                        gf.load(static_cast<const T *>(g.grad_final) + (n * (K - 1) + to - len + K - 1) * a.D + d);
                        widen<T, V>(f, gf);
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
    copies_wait<0>();
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
        if constexpr (V % 2 == 0) {  // D is a multiple of V, the workspace aligned
#pragma unroll
            for (int i = 0; i < V * K; i += 2)
                *reinterpret_cast<float2 *>(p + d * K + i) = make_float2(flat[i], flat[i + 1]);
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

// Channels of a thread: four (measured, 8 x 4096 x 4096 bf16 forward and
// backward, next block in registers: 328 us, with two 398, with eight 336), two where four do
// not fit the rows or leave too few threads even in runs of 8 tokens
// (1 x 509 x 1536 forward: 8.8 us with two, 10.9 us with four), else one.
constexpr int64_t kFullThreads = 768;  // threads an SM that keep enough loads in flight

int channels(const rlscan_causal_conv_args &a, uint64_t bits)
{
    const int size = a.dtype == RLSCAN_BF16 ? 2 : 4;
    const int64_t sms = sm_count() > 0 ? sm_count() : 152;
    if (bits % (4 * size) == 0 && a.N * ceil_div(a.T, 8) * (a.D / 4) >= sms * kFullThreads / 4) return 4;
    return bits % (2 * size) == 0 ? 2 : 1;
}

// Tokens of a thread: as many as leave enough threads, since each run reads
// K-1 tokens of its neighbours again.
int64_t run_length(const rlscan_causal_conv_args &a, int v, int64_t most)
{
    const int64_t sms = sm_count() > 0 ? sm_count() : 152;
    int64_t run = most;
    while (run > 8 && a.N * ceil_div(a.T, run) * (a.D / v) < sms * kFullThreads) run /= 2;
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
        auto kernel = conv_kernel<T, decltype(k)::value, V>;
        constexpr size_t SMEM = Feed<T, V, 1>::SMEM;
        static PerDevice raised;
        if (!raise_smem(raised, kernel, SMEM)) return RLSCAN_ERR_CUDA;
        return launch_overlapped(kernel, ceil_div(a.N * o.runs * (a.D / V), kThreads), kThreads, SMEM, s, a, o);
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
        auto kernel = conv_grad_kernel<T, decltype(k)::value, V>;
        constexpr size_t SMEM = Feed<T, V, 2>::SMEM;
        static PerDevice raised;
        if (!raise_smem(raised, kernel, SMEM)) return RLSCAN_ERR_CUDA;
        return launch_overlapped(kernel, ceil_div(a.N * g.runs * (a.D / V), kThreads), kThreads, SMEM, s, a, g);
    });
}

// The bits that are 0 in all addresses and strides, in bytes.
uint64_t low_bits(const rlscan_causal_conv_args &a, std::initializer_list<const void *> dense)
{
    const int size = a.dtype == RLSCAN_BF16 ? 2 : 4;
    uint64_t bits = static_cast<uint64_t>(a.D) * size | reinterpret_cast<uintptr_t>(a.x.data) |
                    static_cast<uint64_t>(a.x.row_stride) * size | static_cast<uint64_t>(a.x.token_stride) * size;
    for (const void *p : dense) bits |= reinterpret_cast<uintptr_t>(p);
    return bits;
}

int64_t grad_runs(const rlscan_causal_conv_args &a, int v)
{
    return a.T > 0 ? ceil_div(a.T, run_length(a, v, kMostGradRun)) : 1;
}

}  // namespace

rlscan_status launch_causal_conv(const rlscan_causal_conv_args &a, void *y, void *final_state, cudaStream_t s)
{
    const ConvOut o{y, final_state, 0, 0};
    const bool b16 = a.dtype == RLSCAN_BF16;
    switch (channels(a, low_bits(a, {y, final_state, a.initial_state}))) {
    case 4: return b16 ? forward<bf16, 4>(a, o, s) : forward<float, 4>(a, o, s);
    case 2: return b16 ? forward<bf16, 2>(a, o, s) : forward<float, 2>(a, o, s);
    default: return b16 ? forward<bf16, 1>(a, o, s) : forward<float, 1>(a, o, s);
    }
}

rlscan_status launch_causal_conv_step(const rlscan_causal_conv_args &a, void *state, int64_t P, const int32_t *slots,
                                      void *y, cudaStream_t s)
{
    const bool b16 = a.dtype == RLSCAN_BF16;
    if (low_bits(a, {state, y}) % (b16 ? 4 : 8) == 0)
        return b16 ? step<bf16, 2>(a, state, P, slots, y, s) : step<float, 2>(a, state, P, slots, y, s);
    return b16 ? step<bf16, 1>(a, state, P, slots, y, s) : step<float, 1>(a, state, P, slots, y, s);
}

size_t causal_conv_backward_workspace(const rlscan_causal_conv_args &a)
{
    int64_t most = 0;
    for (int v : {1, 2, 4}) {
        const int64_t runs = grad_runs(a, v);
        most = runs > most ? runs : most;
    }
    return sizeof(float) * static_cast<size_t>(a.N) * most * (a.K + 1) * a.D;
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
    const int v = channels(a, low_bits(a, {grad_y.data, grad_x, grad_final_state, a.initial_state, grad_initial_state}) |
                                  static_cast<uint64_t>(grad_y.row_stride) * size |
                                  static_cast<uint64_t>(grad_y.token_stride) * size);
    g.runs = grad_runs(a, v);
    g.run = run_length(a, v, kMostGradRun);
    if (a.N > 0) {
        const rlscan_status st = v == 4   ? (b16 ? backward<bf16, 4>(a, g, s) : backward<float, 4>(a, g, s))
                                 : v == 2 ? (b16 ? backward<bf16, 2>(a, g, s) : backward<float, 2>(a, g, s))
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
