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

// A block walks 64 channels of a row in steps of 64 tokens: a warp has TOK
// tokens of each step, a lane two channels of them.  Every warp folds its
// tokens into one affine map (A, B) of the state before them; the maps before
// a warp's own, in order, give its first state, and its tokens follow.  The
// coefficients are made once and stay in registers, so the inputs are read
// once.  CLUSTER: the blocks of a cluster take neighbouring steps and hand
// their maps round through shared memory; each applies the same maps in the
// same order, so states do not depend on how rows are split between blocks
// beyond the grouping of products that the split itself fixes.
template <class T, bool VEC, int TOK, bool CLUSTER>
__global__ void __launch_bounds__(32 * (kGatedTile / TOK), 2)
    forward_kernel(const __grid_constant__ rlscan_gated_scan_args a, const __grid_constant__ ForwardArgs o, int ranks)
{
    constexpr int WARPS = kGatedTile / TOK;
    __shared__ float4 of_warp[2][WARPS][32];
    __shared__ float4 of_rank[2][CLUSTER ? kGatedCluster : 1][32];
    ptx::pdl_trigger_dependents();
    if constexpr (CLUSTER) cluster_arrive();  // no block writes to one that has not begun
    ptx::pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int rank = CLUSTER ? static_cast<int>(blockIdx.x % static_cast<unsigned>(ranks)) : 0;
    const Division at = divide(CLUSTER ? blockIdx.x / static_cast<unsigned>(ranks) : blockIdx.x, (a.D + kGatedWidth - 1) / kGatedWidth);
    const int64_t n = at.q, d = at.r * kGatedWidth + (VEC ? 2 * lane : lane);
    const bool on0 = d < a.D, on1 = VEC ? on0 : d + 32 < a.D;
    const int64_t len = row_length(a.lengths, n, a.T), tiles = (a.T + kGatedTile - 1) / kGatedTile;
    const int64_t span = static_cast<int64_t>(ranks) * kGatedTile, steps = (len + span - 1) / span;
    const f2 log_decay = load_two<VEC>(a.log_decay + d, on0, on1), log2_decay = mul2(log_decay, both(kLog2e));
    f2 carry = a.initial_state != nullptr ? load_two<VEC>(a.initial_state + n * a.D + d, on0, on1) : both(0.f);
    Two<T, VEC> x[TOK], g[TOK], ig[TOK];
    uint32_t reset = 0;  // bit k: a new episode starts at the warp's token k
    auto fetch = [&](int64_t t0) {
        const T *px = static_cast<const T *>(a.x.data) + n * a.x.row_stride + t0 * a.x.token_stride + d;
        const T *pg = static_cast<const T *>(a.gate.data) + n * a.gate.row_stride + t0 * a.gate.token_stride + d;
        const T *pi = static_cast<const T *>(a.input_gate.data) + n * a.input_gate.row_stride + t0 * a.input_gate.token_stride + d;
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            const bool on = t0 + k < len;
            g[k].load(pg + k * a.gate.token_stride, on && on0, on && on1);
            ig[k].load(pi + k * a.input_gate.token_stride, on && on0, on && on1);
            x[k].load(px + k * a.x.token_stride, on && on0, on && on1);
        }
        uint32_t flag = 0;
        if (a.resets != nullptr && lane < TOK && t0 + lane < len) flag = a.resets[n * a.T + t0 + lane];
        reset = __ballot_sync(0xffffffffu, flag != 0);
    };
    if (steps > 0) fetch(static_cast<int64_t>(rank) * kGatedTile + w * TOK);
    if constexpr (CLUSTER) cluster_wait();
    for (int64_t s = 0; s < steps; ++s) {
        const int p = static_cast<int>(s & 1);
        const int64_t tile = s * ranks + rank, t0 = tile * kGatedTile + w * TOK;
        f2 keep[TOK], b[TOK], A = both(1.f), B = both(0.f);
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            const Gates v = gates(g[k].get(), ig[k].get(), log_decay, log2_decay);
            keep[k] = t0 + k < len ? ((reset >> k & 1u) != 0u ? both(0.f) : v.a) : both(1.f);
            b[k] = t0 + k < len ? mul2(mul2(v.root, v.i), x[k].get()) : both(0.f);
            A = mul2(A, keep[k]);
            B = fma2(keep[k], B, b[k]);
        }
        {
            const float2 fa = halves(A), fb = halves(B);
            of_warp[p][w][lane] = make_float4(fa.x, fa.y, fb.x, fb.y);
        }
        if (s + 1 < steps) fetch(t0 + span);
        __syncthreads();
        auto apply = [&](f2 h, const float4 &m) { return fma2(pair(m.x, m.y), h, pair(m.z, m.w)); };
        f2 h = carry;
        if constexpr (CLUSTER) {
            f2 BA = both(1.f), BB = both(0.f);  // the block's map
#pragma unroll
            for (int q = 0; q < WARPS; ++q) {
                const float4 m = of_warp[p][q][lane];
                BA = mul2(BA, pair(m.x, m.y));
                BB = apply(BB, m);
            }
            const float2 fa = halves(BA), fb = halves(BB);
            for (int q = w; q < ranks; q += WARPS)
                store_to_rank(&of_rank[p][rank][lane], q, make_float4(fa.x, fa.y, fb.x, fb.y));
            cluster_arrive();
            cluster_wait();
            for (int q = 0; q < ranks; ++q) {
                if (q == rank) h = carry;
                carry = apply(carry, of_rank[p][q][lane]);
            }
        }
        if (w == 0 && o.checkpoints != nullptr && tile < tiles) {
            float *to = o.checkpoints + (n * tiles + tile) * a.D + d;
            store_two<float, VEC>(to, h, on0, on1);
        }
#pragma unroll
        for (int q = 0; q < WARPS; ++q) {
            const float4 m = of_warp[p][q][lane];
            if (CLUSTER) {
                if (q < w) h = apply(h, m);
            } else {
                if (q == w) h = carry;
                carry = apply(carry, m);
            }
        }
        T *to = static_cast<T *>(o.y) + (n * a.T + t0) * a.D + d;
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            h = fma2(keep[k], h, b[k]);
            const bool in = t0 + k < a.T;
            store_two<T, VEC>(to + k * a.D, t0 + k < len ? h : both(0.f), in && on0, in && on1);
        }
    }
    for (int64_t tile = steps * ranks + rank; tile < tiles; tile += ranks) {  // padding alone
        const int64_t t0 = tile * kGatedTile + w * TOK;
        T *to = static_cast<T *>(o.y) + (n * a.T + t0) * a.D + d;
        for (int k = 0; k < TOK; ++k)
            if (t0 + k < a.T) store_two<T, VEC>(to + k * a.D, both(0.f), on0, on1);
        if (w == 0 && o.checkpoints != nullptr) store_two<float, VEC>(o.checkpoints + (n * tiles + tile) * a.D + d, carry, on0, on1);
    }
    if (rank == 0 && w == 0 && o.final_state != nullptr) store_two<float, VEC>(o.final_state + n * a.D + d, carry, on0, on1);
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
    const int64_t n = at.q, d = at.r * kGatedWidth + (VEC ? 2 * lane : lane);
    if (n >= a.N) return;
    const bool on0 = d < a.D, on1 = VEC ? on0 : d + 32 < a.D;
    const int64_t slot = q.slots != nullptr ? q.slots[n] : n;
    const bool busy = slot >= 0 && slot < q.P;
    float *state = q.state + (busy ? slot * a.D : 0) + d;
    Two<T, VEC> x, g, ig;
    g.load(static_cast<const T *>(a.gate.data) + n * a.gate.row_stride + d, on0, on1);
    ig.load(static_cast<const T *>(a.input_gate.data) + n * a.input_gate.row_stride + d, on0, on1);
    x.load(static_cast<const T *>(a.x.data) + n * a.x.row_stride + d, on0, on1);
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
    constexpr int TOK = 8;
    Chunk c = chunk_of<T>(a);
    c.add(o.y, 0, 0, sizeof(T));
    const bool vec = gated_pairs<T>(c, a.D) && pairs_of_floats({o.final_state, o.checkpoints});
    const int64_t chains = a.N * ceil_div(a.D, kGatedWidth);
    const int ranks = gated_cluster(chains, a.T), threads = 32 * (kGatedTile / TOK);
    if (ranks > 1)
        return vec ? launch_cluster(forward_kernel<T, true, TOK, true>, chains * ranks, threads, ranks, s, a, o, ranks)
                   : launch_cluster(forward_kernel<T, false, TOK, true>, chains * ranks, threads, ranks, s, a, o, ranks);
    return vec ? launch_cluster(forward_kernel<T, true, TOK, false>, chains, threads, 1, s, a, o, 1)
               : launch_cluster(forward_kernel<T, false, TOK, false>, chains, threads, 1, s, a, o, 1);
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
