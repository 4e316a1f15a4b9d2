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

constexpr int kBackTile = RLSCAN_GATED_SCAN_CHECKPOINT;  // tokens of a step

// The forward kernel's walk from the last step to the first, in steps of 32
// tokens, four of a warp, with two affine maps of a warp's tokens: of the
// state before them and of the message behind them (both have the same factor,
// the product of the decays).  The states start again from the checkpoint in
// front of the step, so only the messages are handed between steps.
template <class T, bool VEC, bool CLUSTER>
__global__ void __launch_bounds__(32 * kGatedWarps, 2)
    backward_kernel(const __grid_constant__ rlscan_gated_scan_args a, const __grid_constant__ BackwardArgs o, int ranks)
{
    constexpr int TOK = kBackTile / kGatedWarps;
    __shared__ float4 state_map[2][kGatedWarps][32], message_map[2][kGatedWarps][32];
    __shared__ float4 of_rank[2][CLUSTER ? kGatedCluster : 1][32];
    __shared__ float2 last[2][32];  // the message out of the step
    ptx::pdl_trigger_dependents();
    if constexpr (CLUSTER) cluster_arrive();
    ptx::pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int rank = CLUSTER ? static_cast<int>(blockIdx.x % static_cast<unsigned>(ranks)) : 0;
    const Division at = divide(CLUSTER ? blockIdx.x / static_cast<unsigned>(ranks) : blockIdx.x, (a.D + kGatedWidth - 1) / kGatedWidth);
    const int64_t n = at.q;
    const Lane<VEC> l(at.r, lane, a.D);
    const int64_t len = row_length(a.lengths, n, a.T), tiles = gated_marks(a.T);
    const int64_t span = static_cast<int64_t>(ranks) * kBackTile, steps = (len + span - 1) / span;
    const f2 log_decay = load_two<VEC>(a.log_decay + l.d, l.on0, l.on1), log2_decay = mul2(log_decay, both(kLog2e));
    f2 carry = o.grad_final != nullptr ? load_two<VEC>(o.grad_final + n * a.D + l.d, l.on0, l.on1) : both(0.f);
    f2 sum = both(0.f);  // the lane's share of dlog_decay
    Two<T, VEC> x[TOK], g[TOK], ig[TOK], gy[TOK];
    Two<float, VEC> mark;
    uint32_t reset = 0;
    auto fetch = [&](int64_t tile) {
        const int64_t t0 = tile * kBackTile + w * TOK;
        fetch_tokens(g, a.gate, n, t0, len, l);
        fetch_tokens(ig, a.input_gate, n, t0, len, l);
        fetch_tokens(x, a.x, n, t0, len, l);
        fetch_tokens(gy, o.grad_y, n, t0, len, l);
        reset = fetch_resets<TOK>(a.resets, n * a.T, t0, len, lane);
        mark.zero();
        if (tile < tiles) mark.load(o.checkpoints + (n * tiles + tile) * a.D + l.from, l.apart);
    };
    if (steps > 0) fetch((steps - 1) * ranks + rank);
    if constexpr (CLUSTER) cluster_wait();
    auto factor = [](const float4 &m) { return pair(m.x, m.y); };
    auto apply = [](f2 h, const float4 &m) { return fma2(pair(m.x, m.y), h, pair(m.z, m.w)); };
    T *gx = static_cast<T *>(o.g.x), *gg = static_cast<T *>(o.g.gate), *gi = static_cast<T *>(o.g.input_gate);
    for (int64_t s = steps - 1; s >= 0; --s) {
        const int p = static_cast<int>(s & 1);
        const int64_t tile = s * ranks + rank, t0 = tile * kBackTile + w * TOK;
        Gates v[TOK];
        f2 xs[TOK], gs[TOK], keep[TOK], b[TOK];
        const uint32_t cut = reset;
        f2 state = mark.get();
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            v[k] = gates(g[k].get(), ig[k].get(), log_decay, log2_decay);
            xs[k] = x[k].get();
            gs[k] = gy[k].get();
            b[k] = mul2(mul2(v[k].root, v[k].i), xs[k]);
            keep[k] = v[k].a;
        }
        if (cut != 0) {
#pragma unroll
            for (int k = 0; k < TOK; ++k)
                if ((cut >> k & 1u) != 0u) keep[k] = both(0.f);
        }
        const bool pad = t0 + TOK > len;
        if (pad) {  // padding hands state and message on
#pragma unroll
            for (int k = 0; k < TOK; ++k)
                if (t0 + k >= len) keep[k] = both(1.f), b[k] = gs[k] = xs[k] = both(0.f);
        }
        if (s > 0) fetch(tile - ranks);
        f2 A = keep[0], B = b[0], M = mul2(keep[TOK - 1], gs[TOK - 1]);
#pragma unroll
        for (int k = 1; k < TOK; ++k) {
            A = mul2(A, keep[k]);
            B = fma2(keep[k], B, b[k]);
            M = mul2(keep[TOK - 1 - k], add2(gs[TOK - 1 - k], M));
        }
        {
            const float2 fa = halves(A), fb = halves(B), fm = halves(M);
            state_map[p][w][lane] = make_float4(fa.x, fa.y, fb.x, fb.y);
            message_map[p][w][lane] = make_float4(fa.x, fa.y, fm.x, fm.y);
        }
        __syncthreads();
        f2 m = carry;
        if constexpr (CLUSTER) {
            f2 BA = both(1.f), BM = both(0.f);
#pragma unroll
            for (int q = kGatedWarps - 1; q >= 0; --q) {
                const float4 f = message_map[p][q][lane];
                BA = mul2(BA, factor(f));
                BM = apply(BM, f);
            }
            const float2 fa = halves(BA), fm = halves(BM);
            for (int q = w; q < ranks; q += kGatedWarps)
                store_to_rank(&of_rank[p][rank][lane], q, make_float4(fa.x, fa.y, fm.x, fm.y));
            cluster_arrive();
            cluster_wait();
            for (int q = ranks - 1; q >= 0; --q) {
                if (q == rank) m = carry;
                carry = apply(carry, of_rank[p][q][lane]);
            }
        } else if (s + 1 < steps) {
            const float2 f = last[p ^ 1][lane];
            m = pair(f.x, f.y);
        }
#pragma unroll 1
        for (int q = kGatedWarps - 1; q > w; --q) m = apply(m, message_map[p][q][lane]);
#pragma unroll 1
        for (int q = 0; q < w; ++q) state = apply(state, state_map[p][q][lane]);
        f2 before[TOK];  // the state before each token
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            before[k] = state;
            state = fma2(keep[k], state, b[k]);
        }
        const int64_t at_last = (n * a.T + t0 + TOK - 1) * a.D + l.d;
        T *px = gx + at_last, *pg = gg + at_last, *pi = gi + at_last;
#pragma unroll
        for (int k = TOK - 1; k >= 0; --k, px -= a.D, pg -= a.D, pi -= a.D) {
            const f2 G = add2(gs[k], m), one = both(1.f);
            m = mul2(keep[k], G);
            const f2 moved = mul2(v[k].i, xs[k]);
            const float2 rt = halves(v[k].root);
            const f2 slope = mul2(mul2(v[k].a, v[k].a), pair(rcp_fast(rt.x), rcp_fast(rt.y)));  // of the root, negated
            f2 dL = mul2(mul2(G, fma2(keep[k], before[k], neg2(mul2(moved, slope)))), v[k].r);  // times r: log_decay's share
            f2 dx = mul2(G, mul2(v[k].root, v[k].i));
            f2 dg = mul2(mul2(dL, log_decay), fma2(neg2(v[k].r), one, one));
            f2 di = mul2(mul2(dx, xs[k]), fma2(neg2(v[k].i), one, one));
            bool on0 = l.on0, on1 = l.on1;
            if (pad) {
                if (t0 + k >= len) dL = dx = dg = di = both(0.f);
                on0 = on0 && t0 + k < a.T, on1 = on1 && t0 + k < a.T;
            }
            sum = add2(sum, dL);
            store_two<T, VEC>(px, dx, on0, on1);
            store_two<T, VEC>(pg, dg, on0, on1);
            store_two<T, VEC>(pi, di, on0, on1);
        }
        if constexpr (!CLUSTER) {
            if (w == 0) {
                last[p][lane] = halves(m);
                carry = m;
            }
        }
    }
    for (int64_t tile = steps * ranks + rank; tile < tiles; tile += ranks) {  // padding alone
        const int64_t t0 = tile * kBackTile + w * TOK;
        for (int k = 0; k < TOK; ++k) {
            if (t0 + k >= a.T) break;
            const int64_t at_token = (n * a.T + t0 + k) * a.D + l.d;
            store_two<T, VEC>(gx + at_token, both(0.f), l.on0, l.on1);
            store_two<T, VEC>(gg + at_token, both(0.f), l.on0, l.on1);
            store_two<T, VEC>(gi + at_token, both(0.f), l.on0, l.on1);
        }
    }
    if (rank == 0 && w == 0 && o.g.initial_state != nullptr)
        store_two<float, VEC>(o.g.initial_state + n * a.D + l.d, carry, l.on0, l.on1);
    if (o.parts != nullptr) {  // the warps' shares in order
        __syncthreads();
        state_map[0][w][lane].x = halves(sum).x;
        state_map[0][w][lane].y = halves(sum).y;
        __syncthreads();
        if (w == 0) {
            f2 all = both(0.f);
#pragma unroll
            for (int q = 0; q < kGatedWarps; ++q) all = add2(all, factor(state_map[0][q][lane]));
            store_two<float, VEC>(o.parts + (n * ranks + rank) * a.D + l.d, all, l.on0, l.on1);
        }
    }
}

template <class T, bool VEC>
int back_ranks(const rlscan_gated_scan_args &a)
{
    return gated_cluster<T, VEC>(backward_kernel<T, VEC, true>, a.N * ceil_div(a.D, kGatedWidth), a.T, kBackTile);
}

template <class T, bool VEC>
rlscan_status backward_as(const rlscan_gated_scan_args &a, const BackwardArgs &o, int ranks, cudaStream_t s)
{
    const int64_t chains = a.N * ceil_div(a.D, kGatedWidth);
    const int threads = 32 * kGatedWarps;
    return ranks > 1 ? launch_cluster(backward_kernel<T, VEC, true>, chains * ranks, threads, ranks, s, a, o, ranks)
                     : launch_cluster(backward_kernel<T, VEC, false>, chains, threads, 1, s, a, o, 1);
}

template <class T>
rlscan_status backward_typed(const rlscan_gated_scan_args &a, BackwardArgs &o, int64_t &parts, cudaStream_t s)
{
    const rlscan_array3 &grad_y = o.grad_y;
    Chunk c;
    for (const rlscan_array3 *v : {&a.x, &a.gate, &a.input_gate, &grad_y}) c.add(v->data, v->row_stride, v->token_stride, sizeof(T));
    for (void *p : {o.g.x, o.g.gate, o.g.input_gate}) c.add(p, 0, 0, sizeof(T));
    const bool vec = gated_pairs<T>(c, a.D) && ((reinterpret_cast<uintptr_t>(o.g.initial_state) | reinterpret_cast<uintptr_t>(o.parts) |
                                                 reinterpret_cast<uintptr_t>(o.checkpoints)) & 7u) == 0;
    const int ranks = vec ? back_ranks<T, true>(a) : back_ranks<T, false>(a);
    parts = a.N * ranks;
    return vec ? backward_as<T, true>(a, o, ranks, s) : backward_as<T, false>(a, o, ranks, s);
}

}  // namespace

// for rows split over as many blocks as a cluster may have
size_t gated_scan_backward_workspace(const rlscan_gated_scan_args &a)
{
    if (a.N == 0 || a.D == 0) return 0;
    const int64_t tiles = ceil_div(a.T, kBackTile), most = tiles < 1 ? 1 : tiles < kGatedCluster ? tiles : kGatedCluster;
    return static_cast<size_t>(a.N) * most * a.D * sizeof(float);
}

rlscan_status launch_gated_scan_backward(const rlscan_gated_scan_args &a, const rlscan_array3 &grad_y,
                                         const float *grad_final_state, const float *checkpoints,
                                         const rlscan_gated_scan_grads &g, void *ws, cudaStream_t s)
{
    float *shares = g.log_decay != nullptr ? static_cast<float *>(ws) : nullptr;
    int64_t parts = 0;
    if (a.N > 0) {
        BackwardArgs o{grad_y, grad_final_state, checkpoints, g, shares};
        const rlscan_status st = a.dtype == RLSCAN_BF16 ? backward_typed<bf16>(a, o, parts, s) : backward_typed<float>(a, o, parts, s);
        if (st != RLSCAN_OK) return st;
    }
    if (g.log_decay == nullptr) return RLSCAN_OK;
    SumJobs jobs;  // without rows the sums have no parts, and are 0
    jobs.add(shares, parts, a.D, a.D, g.log_decay, false);
    return launch_sums(jobs, s);
}

}  // namespace seq
}  // namespace rlscan
