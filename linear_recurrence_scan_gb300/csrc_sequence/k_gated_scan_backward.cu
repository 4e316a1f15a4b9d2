// k_gated_scan_backward.cu -- gradients of the gated recurrence.  With G_t the
// gradient of h_t and m_t the message that reaches it from the token behind:
//   G_t = grad_y_t + m_t,  m_{t-1} = a_t G_t  (0 over a reset)
//   dx = G root i,  dinput_gate = G root x i (1 - i),
//   dL = G (a h_{t-1} - i x a^2 / root),  dgate = dL log_decay r (1 - r),
//   dlog_decay = sum dL r.
#include "gated_scan.cuh"

namespace rlscan {
namespace seq {
namespace {

struct BackwardArgs {
    rlscan_array3 grad_y;
    const float *grad_final, *checkpoints;
    rlscan_gated_scan_grads g;
    float *parts;  // [N * ranks][D]: each block's share of dlog_decay
};

// The forward kernel's walk from the last step to the first, with two affine
// maps of a warp's tokens: of the state before them and of the message behind
// them (both have the same factor, the product of the decays).  The states
// start again from the checkpoint in front of the step, so only the messages
// are handed between steps.
template <class T, bool VEC, int TOK, bool CLUSTER>
__global__ void __launch_bounds__(32 * (kGatedTile / TOK), 1)
    backward_kernel(const __grid_constant__ rlscan_gated_scan_args a, const __grid_constant__ BackwardArgs o, int ranks)
{
    constexpr int WARPS = kGatedTile / TOK;
    __shared__ float2 factor[2][WARPS][32];
    __shared__ float4 rest[2][WARPS][32];  // (of the state, of the message)
    __shared__ float4 of_rank[2][CLUSTER ? kGatedCluster : 1][32];
    ptx::pdl_trigger_dependents();
    if constexpr (CLUSTER) cluster_arrive();
    ptx::pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int rank = CLUSTER ? static_cast<int>(blockIdx.x % static_cast<unsigned>(ranks)) : 0;
    const Division at = divide(CLUSTER ? blockIdx.x / static_cast<unsigned>(ranks) : blockIdx.x, (a.D + kGatedWidth - 1) / kGatedWidth);
    const int64_t n = at.q, d = at.r * kGatedWidth + (VEC ? 2 * lane : lane);
    const bool on0 = d < a.D, on1 = VEC ? on0 : d + 32 < a.D;
    const int64_t len = row_length(a.lengths, n, a.T), tiles = (a.T + kGatedTile - 1) / kGatedTile;
    const int64_t span = static_cast<int64_t>(ranks) * kGatedTile, steps = (len + span - 1) / span;
    const f2 log_decay = load_two<VEC>(a.log_decay + d, on0, on1), log2_decay = mul2(log_decay, both(kLog2e));
    f2 carry = o.grad_final != nullptr ? load_two<VEC>(o.grad_final + n * a.D + d, on0, on1) : both(0.f);
    f2 sum = both(0.f);  // the lane's share of dlog_decay
    Two<T, VEC> x[TOK], g[TOK], ig[TOK], gy[TOK];
    f2 mark;
    uint32_t reset = 0;
    auto fetch = [&](int64_t tile) {
        const int64_t t0 = tile * kGatedTile + w * TOK;
        const T *px = static_cast<const T *>(a.x.data) + n * a.x.row_stride + t0 * a.x.token_stride + d;
        const T *pg = static_cast<const T *>(a.gate.data) + n * a.gate.row_stride + t0 * a.gate.token_stride + d;
        const T *pi = static_cast<const T *>(a.input_gate.data) + n * a.input_gate.row_stride + t0 * a.input_gate.token_stride + d;
        const T *py = static_cast<const T *>(o.grad_y.data) + n * o.grad_y.row_stride + t0 * o.grad_y.token_stride + d;
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            const bool on = t0 + k < len;
            g[k].load(pg + k * a.gate.token_stride, on && on0, on && on1);
            ig[k].load(pi + k * a.input_gate.token_stride, on && on0, on && on1);
            x[k].load(px + k * a.x.token_stride, on && on0, on && on1);
            gy[k].load(py + k * o.grad_y.token_stride, on && on0, on && on1);
        }
        uint32_t flag = 0;
        if (a.resets != nullptr && lane < TOK && t0 + lane < len) flag = a.resets[n * a.T + t0 + lane];
        reset = __ballot_sync(0xffffffffu, flag != 0);
        const bool in = tile < tiles;
        mark = load_two<VEC>(o.checkpoints + (n * tiles + tile) * a.D + d, in && on0, in && on1);
    };
    if (steps > 0) fetch((steps - 1) * ranks + rank);
    if constexpr (CLUSTER) cluster_wait();
    T *gx = static_cast<T *>(o.g.x), *gg = static_cast<T *>(o.g.gate), *gi = static_cast<T *>(o.g.input_gate);
    for (int64_t s = steps - 1; s >= 0; --s) {
        const int p = static_cast<int>(s & 1);
        const int64_t tile = s * ranks + rank, t0 = tile * kGatedTile + w * TOK;
        Gates v[TOK];
        f2 xs[TOK], gs[TOK], A = both(1.f), B = both(0.f), M = both(0.f);
        const uint32_t cut = reset;
        f2 state = mark;
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            v[k] = gates(g[k].get(), ig[k].get(), log_decay, log2_decay);
            xs[k] = x[k].get();
            gs[k] = gy[k].get();
            if (t0 + k >= len) v[k].a = both(1.f), v[k].root = both(0.f);  // padding hands state and message on
            const f2 keep = (cut >> k & 1u) != 0u ? both(0.f) : v[k].a;
            A = mul2(A, keep);
            B = fma2(keep, B, mul2(mul2(v[k].root, v[k].i), xs[k]));
        }
#pragma unroll
        for (int k = TOK - 1; k >= 0; --k) {
            const f2 keep = (cut >> k & 1u) != 0u ? both(0.f) : v[k].a;
            M = mul2(keep, add2(gs[k], M));
        }
        {
            const float2 fb = halves(B), fm = halves(M);
            factor[p][w][lane] = halves(A);
            rest[p][w][lane] = make_float4(fb.x, fb.y, fm.x, fm.y);
        }
        if (s > 0) fetch(tile - ranks);
        __syncthreads();
        auto product = [&](int q) { const float2 f = factor[p][q][lane]; return pair(f.x, f.y); };
        auto of_state = [&](int q) { const float4 m = rest[p][q][lane]; return pair(m.x, m.y); };
        auto of_message = [&](int q) { const float4 m = rest[p][q][lane]; return pair(m.z, m.w); };
        f2 m = carry;
        if constexpr (CLUSTER) {
            f2 BA = both(1.f), BM = both(0.f);
#pragma unroll
            for (int q = WARPS - 1; q >= 0; --q) {
                const f2 f = product(q);
                BA = mul2(BA, f);
                BM = fma2(f, BM, of_message(q));
            }
            const float2 fa = halves(BA), fm = halves(BM);
            for (int q = w; q < ranks; q += WARPS)
                store_to_rank(&of_rank[p][rank][lane], q, make_float4(fa.x, fa.y, fm.x, fm.y));
            cluster_arrive();
            cluster_wait();
            for (int q = ranks - 1; q >= 0; --q) {
                if (q == rank) m = carry;
                const float4 r = of_rank[p][q][lane];
                carry = fma2(pair(r.x, r.y), carry, pair(r.z, r.w));
            }
        }
#pragma unroll
        for (int q = WARPS - 1; q >= 0; --q) {
            if (CLUSTER) {
                if (q > w) m = fma2(product(q), m, of_message(q));
            } else {
                if (q == w) m = carry;
                carry = fma2(product(q), carry, of_message(q));
            }
        }
#pragma unroll
        for (int q = 0; q < WARPS; ++q)
            if (q < w) state = fma2(product(q), state, of_state(q));
        f2 before[TOK];  // the state before each token, 0 behind a reset
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            before[k] = (cut >> k & 1u) != 0u ? both(0.f) : state;
            state = fma2(v[k].a, before[k], mul2(mul2(v[k].root, v[k].i), xs[k]));
        }
#pragma unroll
        for (int k = TOK - 1; k >= 0; --k) {
            const bool live = t0 + k < len, in = t0 + k < a.T;
            const int64_t at_token = (n * a.T + t0 + k) * a.D + d;
            const f2 G = add2(gs[k], m), hold = v[k].i, one = both(1.f);
            const f2 gain = mul2(v[k].root, hold), moved = mul2(hold, xs[k]);
            const float2 rt = halves(v[k].root);
            const f2 inverse = pair(rcp_fast(rt.x), rcp_fast(rt.y));
            f2 dL = fma2(v[k].a, before[k], neg2(mul2(mul2(moved, mul2(v[k].a, v[k].a)), inverse)));
            dL = live ? mul2(mul2(G, dL), v[k].r) : both(0.f);  // times r: log_decay's share
            sum = add2(sum, dL);
            const f2 dx = live ? mul2(G, gain) : both(0.f);
            const f2 dg = mul2(mul2(dL, log_decay), fma2(neg2(v[k].r), one, one));
            const f2 di = mul2(mul2(dx, xs[k]), fma2(neg2(hold), one, one));
            store_two<T, VEC>(gx + at_token, dx, in && on0, in && on1);
            store_two<T, VEC>(gg + at_token, dg, in && on0, in && on1);
            store_two<T, VEC>(gi + at_token, live ? di : both(0.f), in && on0, in && on1);
            m = (cut >> k & 1u) != 0u ? both(0.f) : mul2(v[k].a, G);
        }
    }
    for (int64_t tile = steps * ranks + rank; tile < tiles; tile += ranks) {  // padding alone
        const int64_t t0 = tile * kGatedTile + w * TOK;
        for (int k = 0; k < TOK; ++k) {
            if (t0 + k >= a.T) break;
            const int64_t at_token = (n * a.T + t0 + k) * a.D + d;
            store_two<T, VEC>(gx + at_token, both(0.f), on0, on1);
            store_two<T, VEC>(gg + at_token, both(0.f), on0, on1);
            store_two<T, VEC>(gi + at_token, both(0.f), on0, on1);
        }
    }
    if (rank == 0 && w == 0 && o.g.initial_state != nullptr) store_two<float, VEC>(o.g.initial_state + n * a.D + d, carry, on0, on1);
    if (o.parts != nullptr) {  // the warps' shares in order
        __syncthreads();
        factor[0][w][lane] = halves(sum);
        __syncthreads();
        if (w == 0) {
            f2 all = both(0.f);
#pragma unroll
            for (int q = 0; q < WARPS; ++q) {
                const float2 f = factor[0][q][lane];
                all = add2(all, pair(f.x, f.y));
            }
            store_two<float, VEC>(o.parts + (n * ranks + rank) * a.D + d, all, on0, on1);
        }
    }
}

template <class T>
rlscan_status backward_typed(const rlscan_gated_scan_args &a, const BackwardArgs &o, int ranks, cudaStream_t s)
{
    constexpr int TOK = 4;
    Chunk c;
    for (const rlscan_array3 *v : {&a.x, &a.gate, &a.input_gate, &o.grad_y}) c.add(v->data, v->row_stride, v->token_stride, sizeof(T));
    for (const void *p : {o.g.x, o.g.gate, o.g.input_gate}) c.add(p, 0, 0, sizeof(T));
    const bool vec = gated_pairs<T>(c, a.D) &&
                     ((reinterpret_cast<uintptr_t>(o.g.initial_state) | reinterpret_cast<uintptr_t>(o.parts)) & 7u) == 0;
    const int64_t chains = a.N * ceil_div(a.D, kGatedWidth);
    const int threads = 32 * (kGatedTile / TOK);
    if (ranks > 1)
        return vec ? launch_cluster(backward_kernel<T, true, TOK, true>, chains * ranks, threads, ranks, s, a, o, ranks)
                   : launch_cluster(backward_kernel<T, false, TOK, true>, chains * ranks, threads, ranks, s, a, o, ranks);
    return vec ? launch_cluster(backward_kernel<T, true, TOK, false>, chains, threads, 1, s, a, o, 1)
               : launch_cluster(backward_kernel<T, false, TOK, false>, chains, threads, 1, s, a, o, 1);
}

int ranks_of(const rlscan_gated_scan_args &a) { return gated_cluster(a.N * ceil_div(a.D, kGatedWidth), a.T); }

}  // namespace

size_t gated_scan_backward_workspace(const rlscan_gated_scan_args &a)
{
    if (a.N == 0 || a.D == 0) return 0;
    return static_cast<size_t>(a.N) * ranks_of(a) * a.D * sizeof(float);
}

rlscan_status launch_gated_scan_backward(const rlscan_gated_scan_args &a, const rlscan_array3 &grad_y,
                                         const float *grad_final_state, const float *checkpoints,
                                         const rlscan_gated_scan_grads &g, void *ws, cudaStream_t s)
{
    float *parts = g.log_decay != nullptr ? static_cast<float *>(ws) : nullptr;
    const int ranks = a.N > 0 ? ranks_of(a) : 1;
    if (a.N > 0) {
        const BackwardArgs o{grad_y, grad_final_state, checkpoints, g, parts};
        const rlscan_status st = a.dtype == RLSCAN_BF16 ? backward_typed<bf16>(a, o, ranks, s) : backward_typed<float>(a, o, ranks, s);
        if (st != RLSCAN_OK) return st;
    }
    if (g.log_decay == nullptr) return RLSCAN_OK;
    SumJobs jobs;  // without rows the sums have no parts, and are 0
    jobs.add(parts, a.N * ranks, a.D, a.D, g.log_decay, false);
    return launch_sums(jobs, s);
}

}  // namespace seq
}  // namespace rlscan
