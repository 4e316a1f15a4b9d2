// k_gated_scan.cu -- the gated recurrence over prompts and for single tokens:
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t,  a_t = exp(log_decay r_t),
// r and i the sigmoids of the two gates, one state a channel.
#include "gated_scan.cuh"

namespace rlscan {
namespace seq {
namespace {

struct ForwardArgs {
    void *y;
    float *final_state, *checkpoints;
};

// A block walks 64 channels of a row in steps of 64 tokens: a warp has eight
// tokens of each step, a lane two channels of them.  Every warp folds its
// tokens into one affine map (A, B) of the state before them; the maps of the
// warps before it, in order, give its first state, and its tokens follow.  The
// coefficients are made once and stay in registers, so the inputs are read
// once; the next step's inputs are in flight meanwhile.  CLUSTER: the blocks of
// a cluster take neighbouring steps and hand their maps round through shared
// memory.
template <class T, bool VEC, bool CLUSTER>
__global__ void __launch_bounds__(32 * kGatedWarps, sizeof(T) == 2 && VEC ? 3 : 2)
    forward_kernel(const __grid_constant__ rlscan_gated_scan_args a, const __grid_constant__ ForwardArgs o, int ranks)
{
    constexpr int TOK = kGatedTile / kGatedWarps;
    __shared__ float4 of_warp[2][kGatedWarps][32];
    __shared__ float4 of_rank[2][CLUSTER ? kGatedCluster : 1][32];
    __shared__ float2 last[2][32];  // the state after the step's last token
    ptx::pdl_trigger_dependents();
    if constexpr (CLUSTER) cluster_arrive();  // no block writes to one that has not begun
    ptx::pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int rank = CLUSTER ? static_cast<int>(blockIdx.x % static_cast<unsigned>(ranks)) : 0;
    const Division at = divide(CLUSTER ? blockIdx.x / static_cast<unsigned>(ranks) : blockIdx.x, (a.D + kGatedWidth - 1) / kGatedWidth);
    const int64_t n = at.q;
    const Lane<VEC> l(at.r, lane, a.D);
    const int64_t len = row_length(a.lengths, n, a.T), tiles = (a.T + kGatedTile - 1) / kGatedTile;
    const int64_t span = static_cast<int64_t>(ranks) * kGatedTile, steps = (len + span - 1) / span;
    const f2 log_decay = load_two<VEC>(a.log_decay + l.d, l.on0, l.on1), log2_decay = mul2(log_decay, both(kLog2e));
    f2 carry = a.initial_state != nullptr ? load_two<VEC>(a.initial_state + n * a.D + l.d, l.on0, l.on1) : both(0.f);
    Two<T, VEC> x[TOK], g[TOK], ig[TOK];
    uint32_t reset = 0;
    auto fetch = [&](int64_t t0) {
        fetch_tokens(g, a.gate, n, t0, len, l);
        fetch_tokens(ig, a.input_gate, n, t0, len, l);
        fetch_tokens(x, a.x, n, t0, len, l);
        reset = fetch_resets<TOK>(a.resets, n * a.T, t0, len, lane);
    };
    if (steps > 0) fetch(static_cast<int64_t>(rank) * kGatedTile + w * TOK);
    if constexpr (CLUSTER) cluster_wait();
    auto apply = [](f2 h, const float4 &m) { return fma2(pair(m.x, m.y), h, pair(m.z, m.w)); };
    for (int64_t s = 0; s < steps; ++s) {
        const int p = static_cast<int>(s & 1);
        const int64_t tile = s * ranks + rank, t0 = tile * kGatedTile + w * TOK;
        f2 keep[TOK], b[TOK];
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            const Gates v = gates(g[k].get(), ig[k].get(), log_decay, log2_decay);
            keep[k] = v.a;
            b[k] = mul2(mul2(v.root, v.i), x[k].get());
        }
        if (reset != 0) {
#pragma unroll
            for (int k = 0; k < TOK; ++k)
                if ((reset >> k & 1u) != 0u) keep[k] = both(0.f);
        }
        if (t0 + TOK > len) {  // padding hands the state on
#pragma unroll
            for (int k = 0; k < TOK; ++k)
                if (t0 + k >= len) keep[k] = both(1.f), b[k] = both(0.f);
        }
        if (s + 1 < steps) fetch(t0 + span);
        f2 A = keep[0], B = b[0];
#pragma unroll
        for (int k = 1; k < TOK; ++k) {
            A = mul2(A, keep[k]);
            B = fma2(keep[k], B, b[k]);
        }
        const float2 fa = halves(A), fb = halves(B);
        of_warp[p][w][lane] = make_float4(fa.x, fa.y, fb.x, fb.y);
        __syncthreads();
        f2 h = carry;
        if constexpr (CLUSTER) {
            f2 BA = both(1.f), BB = both(0.f);  // the block's map
#pragma unroll
            for (int q = 0; q < kGatedWarps; ++q) {
                const float4 m = of_warp[p][q][lane];
                BA = mul2(BA, pair(m.x, m.y));
                BB = apply(BB, m);
            }
            const float2 ga = halves(BA), gb = halves(BB);
            for (int q = w; q < ranks; q += kGatedWarps)
                store_to_rank(&of_rank[p][rank][lane], q, make_float4(ga.x, ga.y, gb.x, gb.y));
            cluster_arrive();
            cluster_wait();
            for (int q = 0; q < ranks; ++q) {
                if (q == rank) h = carry;
                carry = apply(carry, of_rank[p][q][lane]);
            }
        } else if (s > 0) {
            const float2 f = last[p ^ 1][lane];
            h = pair(f.x, f.y);
        }
#pragma unroll 1
        for (int q = 0; q < w; ++q) h = apply(h, of_warp[p][q][lane]);
        if (o.checkpoints != nullptr && w % (RLSCAN_GATED_SCAN_CHECKPOINT / TOK) == 0 && t0 < a.T) {
            float *to = o.checkpoints + (n * gated_marks(a.T) + t0 / RLSCAN_GATED_SCAN_CHECKPOINT) * a.D + l.d;
            store_two<float, VEC>(to, h, l.on0, l.on1);
        }
        T *to = static_cast<T *>(o.y) + (n * a.T + t0) * a.D + l.d;
        if (t0 + TOK <= len) {
#pragma unroll
            for (int k = 0; k < TOK; ++k, to += a.D) {
                h = fma2(keep[k], h, b[k]);
                store_two<T, VEC>(to, h, l.on0, l.on1);
            }
        } else {
#pragma unroll
            for (int k = 0; k < TOK; ++k) {
                h = fma2(keep[k], h, b[k]);
                const bool in = t0 + k < a.T;
                store_two<T, VEC>(to + k * a.D, t0 + k < len ? h : both(0.f), in && l.on0, in && l.on1);
            }
        }
        if constexpr (!CLUSTER) {
            if (w == kGatedWarps - 1) {
                last[p][lane] = halves(h);
                carry = h;
            }
        }
    }
    for (int64_t tile = steps * ranks + rank; tile < tiles; tile += ranks) {  // padding alone
        const int64_t t0 = tile * kGatedTile + w * TOK;
        T *to = static_cast<T *>(o.y) + (n * a.T + t0) * a.D + l.d;
        for (int k = 0; k < TOK; ++k)
            if (t0 + k < a.T) store_two<T, VEC>(to + k * a.D, both(0.f), l.on0, l.on1);
    }
    if (rank == 0 && w == kGatedWarps - 1) {  // has the last state
        if (o.final_state != nullptr) store_two<float, VEC>(o.final_state + n * a.D + l.d, carry, l.on0, l.on1);
        const int64_t marks = gated_marks(a.T);
        if (o.checkpoints != nullptr)
            for (int64_t i = steps * span / RLSCAN_GATED_SCAN_CHECKPOINT; i < marks; ++i)
                store_two<float, VEC>(o.checkpoints + (n * marks + i) * a.D + l.d, carry, l.on0, l.on1);
    }
}

// One token: a lane has two channels of one sequence.
struct StepArgs {
    float *state;
    int64_t P;
    const int32_t *slots;
    void *y;
};
constexpr int kStepWarps = 4;

template <class T, bool VEC>
__global__ void __launch_bounds__(32 * kStepWarps)
    step_kernel(const __grid_constant__ rlscan_gated_scan_args a, const __grid_constant__ StepArgs q)
{
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31;
    const int64_t warp = static_cast<int64_t>(blockIdx.x) * kStepWarps + (threadIdx.x >> 5);
    const Division at = divide(warp, (a.D + kGatedWidth - 1) / kGatedWidth);
    const int64_t n = at.q;
    if (n >= a.N) return;
    const Lane<VEC> l(at.r, lane, a.D);
    const int64_t d = l.d;
    const bool on0 = l.on0, on1 = l.on1;
    const int64_t slot = q.slots != nullptr ? q.slots[n] : n;
    const bool busy = slot >= 0 && slot < q.P;
    float *state = q.state + (busy ? slot * a.D : 0) + d;
    Two<T, VEC> x, g, ig;
    g.load(static_cast<const T *>(a.gate.data) + n * a.gate.row_stride + l.from, l.apart);
    ig.load(static_cast<const T *>(a.input_gate.data) + n * a.input_gate.row_stride + l.from, l.apart);
    x.load(static_cast<const T *>(a.x.data) + n * a.x.row_stride + l.from, l.apart);
    const f2 log_decay = load_two<VEC>(a.log_decay + d, on0, on1);
    f2 h = load_two<VEC>(state, busy && on0, busy && on1);
    const Gates v = gates(g.get(), ig.get(), log_decay, mul2(log_decay, both(kLog2e)));
    h = fma2(v.a, h, mul2(mul2(v.root, v.i), x.get()));
    store_two<float, VEC>(state, h, busy && on0, busy && on1);
    store_two<T, VEC>(static_cast<T *>(q.y) + n * a.D + d, busy ? h : both(0.f), on0, on1);
}

template <class T>
Chunk chunk_of(const rlscan_gated_scan_args &a)
{
    Chunk c;
    for (const rlscan_array3 *v : {&a.x, &a.gate, &a.input_gate}) c.add(v->data, v->row_stride, v->token_stride, sizeof(T));
    return c;
}

bool pairs_of_floats(std::initializer_list<const void *> ptrs)
{
    uintptr_t bits = 0;
    for (const void *p : ptrs) bits |= reinterpret_cast<uintptr_t>(p);
    return (bits & 7u) == 0;
}

template <class T>
rlscan_status forward_typed(const rlscan_gated_scan_args &a, const ForwardArgs &o, cudaStream_t s)
{
    Chunk c = chunk_of<T>(a);
    c.add(o.y, 0, 0, sizeof(T));
    const bool vec = gated_pairs<T>(c, a.D) && pairs_of_floats({o.final_state, o.checkpoints});
    const int64_t chains = a.N * ceil_div(a.D, kGatedWidth);
    const int threads = 32 * kGatedWarps;
    auto go = [&](auto pairs) {
        constexpr bool VEC = decltype(pairs)::value;
        const int ranks = gated_cluster<T, VEC>(forward_kernel<T, VEC, true>, chains, a.T, kGatedTile);
        return ranks > 1 ? launch_cluster(forward_kernel<T, VEC, true>, chains * ranks, threads, ranks, s, a, o, ranks)
                         : launch_cluster(forward_kernel<T, VEC, false>, chains, threads, 1, s, a, o, 1);
    };
    return vec ? go(std::true_type()) : go(std::false_type());
}

template <class T>
rlscan_status step_typed(const rlscan_gated_scan_args &a, const StepArgs &q, cudaStream_t s)
{
    Chunk c;
    for (const rlscan_array3 *v : {&a.x, &a.gate, &a.input_gate}) c.add(v->data, v->row_stride, 0, sizeof(T));
    c.add(q.y, 0, 0, sizeof(T));
    const bool vec = gated_pairs<T>(c, a.D) && pairs_of_floats({q.state});
    const int64_t grid = ceil_div(a.N * ceil_div(a.D, kGatedWidth), kStepWarps);
    return vec ? launch_overlapped(step_kernel<T, true>, grid, 32 * kStepWarps, 0, s, a, q)
               : launch_overlapped(step_kernel<T, false>, grid, 32 * kStepWarps, 0, s, a, q);
}

}  // namespace

rlscan_status launch_gated_scan(const rlscan_gated_scan_args &a, void *y, float *final_state, float *checkpoints,
                                cudaStream_t s)
{
    const ForwardArgs o{y, final_state, checkpoints};
    return a.dtype == RLSCAN_BF16 ? forward_typed<bf16>(a, o, s) : forward_typed<float>(a, o, s);
}

rlscan_status launch_gated_scan_step(const rlscan_gated_scan_args &a, float *state, int64_t P, const int32_t *slots,
                                     void *y, cudaStream_t s)
{
    const StepArgs q{state, P, slots, y};
    return a.dtype == RLSCAN_BF16 ? step_typed<bf16>(a, q, s) : step_typed<float>(a, q, s);
}

}  // namespace seq
}  // namespace rlscan
