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

__device__ unsigned int g_timed_out;  // a wait ran out on this device

struct BackwardArgs {
    rlscan_array3 grad_y;
    const float *grad_final, *checkpoints;
    rlscan_gated_scan_grads g;
    float *parts;  // [N * ranks][D]: each block's share of dlog_decay
};

constexpr int kBackTile = RLSCAN_GATED_SCAN_CHECKPOINT;  // tokens of a step of the untiled kernel

// The forward kernel's walk from the last step to the first, with two affine
// maps of a warp's tokens: of the state before them and of the message behind
// them (both have the same factor, the product of the decays).  The states
// start again from the checkpoint in front of the step, so only the messages
// are handed between steps.

// What a token adds: dx, the gates' gradients, log_decay's share; and the
// message to the token in front of it.
struct TokenGrads {
    f2 x, gate, input_gate, share;
};
__device__ __forceinline__ TokenGrads token_grads(const Gates &v, f2 keep, f2 x, f2 gy, f2 before, f2 log_decay, f2 &m)
{
    const f2 one = both(1.f), minus = both(-1.f), G = add2(gy, m);
    m = mul2(keep, G);
    // i x a^2 / root: what the decay takes from the input
    const f2 taken = mul2(mul2(mul2(v.i, x), rcp2(v.root)), mul2(v.a, v.a));
    TokenGrads t;
    t.share = mul2(mul2(G, v.r), fma2(taken, minus, mul2(keep, before)));
    t.x = mul2(G, mul2(v.root, v.i));
    t.gate = mul2(mul2(t.share, log_decay), fma2(v.r, minus, one));
    t.input_gate = mul2(mul2(t.x, x), fma2(v.i, minus, one));
    return t;
}

// Behind the last step: zeros for tiles of padding, the initial state's
// gradient, the block's share of dlog_decay (its warps' in order).
template <class T, bool VEC, int TILE, bool CLUSTER>
__device__ __forceinline__ void finish(const rlscan_gated_scan_args &a, const BackwardArgs &o, const Walk &k, int ranks, const Lane<VEC> &l,
                                       f2 carry, f2 sum, TwoChains &chain)
{
    constexpr int TOK = TILE / kGatedWarps;
    for (int64_t tile = k.steps * ranks + k.rank; tile < k.tiles; tile += ranks) {
        const int64_t t0 = tile * TILE + k.w * TOK;
        for (int i = 0; i < TOK; ++i) {
            if (t0 + i >= a.T) break;
            const int64_t at_token = (k.n * a.T + t0 + i) * a.D + l.block + l.d;
            store_two<T, VEC>(static_cast<T *>(o.g.x) + at_token, both(0.f), l.on0, l.on1);
            store_two<T, VEC>(static_cast<T *>(o.g.gate) + at_token, both(0.f), l.on0, l.on1);
            store_two<T, VEC>(static_cast<T *>(o.g.input_gate) + at_token, both(0.f), l.on0, l.on1);
        }
    }
    if (k.rank == 0 && k.w == 0 && o.g.initial_state != nullptr)
        store_two<float, VEC>(o.g.initial_state + k.n * a.D + l.block + l.d, carry, l.on0, l.on1);
    if (o.parts == nullptr) return;
    __syncthreads();
    chain.put(0, k.w, k.lane, sum, sum, sum);
    __syncthreads();
    if (k.w == 0) {
        f2 all = both(0.f);
#pragma unroll
        for (int q = 0; q < kGatedWarps; ++q) all = add2(all, pair(chain.map[0][q][k.lane].x, chain.map[0][q][k.lane].y));
        store_two<float, VEC>(o.parts + (k.n * ranks + k.rank) * a.D + l.block + l.d, all, l.on0, l.on1);
    }
}

// The state in front of the warp's tokens, from the step's checkpoint (the
// selects cost less than a second loop: 8 x 2048 x 4096 238 us and 241)
__device__ __forceinline__ f2 state_in_front(const TwoChains &c, int p, int w, int lane, f2 mark)
{
    f2 h = mark;
#pragma unroll 1
    for (int q = 0; q < w; ++q) h = apply_cut(h, c.map[p][q][lane]);
    return h;
}

// Arrays of any alignment: the next step's values are loaded into registers
// while this one's are worked on.
template <class T, bool VEC, bool CLUSTER>
__global__ void __launch_bounds__(32 * kGatedWarps, 2)
    backward_kernel(const __grid_constant__ rlscan_gated_scan_args a, const __grid_constant__ BackwardArgs o, int ranks)
{
    constexpr int TILE = kBackTile, TOK = TILE / kGatedWarps;
    __shared__ TwoChains chain;
    __shared__ std::conditional_t<CLUSTER, Exchange<kGatedCluster>, char> exchange;
    __shared__ int gave_up;
    ptx::pdl_trigger_dependents();
    if (threadIdx.x == 0) {
        gave_up = 0;
        if constexpr (CLUSTER) exchange.init(), ptx::fence_mbar_init();
    }
    __syncthreads();
    if constexpr (CLUSTER) cluster_arrive();
    ptx::pdl_wait_prerequisites();
    int64_t block;
    const Walk k = walk<TILE, CLUSTER>(a, ranks, block);
    const Lane<VEC> l(block, k.lane, a.D);
    const f2 log_decay = load_two<VEC>(a.log_decay + l.block + l.d, l.on0, l.on1);
    const Decay decays(log_decay);
    f2 carry = o.grad_final != nullptr ? load_two<VEC>(o.grad_final + k.n * a.D + l.block + l.d, l.on0, l.on1) : both(0.f);
    f2 sum = both(0.f);  // the lane's share of dlog_decay
    Two<T, VEC> x[TOK], g[TOK], ig[TOK], gy[TOK];
    Two<float, VEC> mark;
    uint32_t flag = 0;
    auto fetch = [&](int64_t tile) {
        const int64_t t0 = tile * TILE + k.w * TOK;
        fetch_tokens(g, a.gate, k.n, t0, k.len, l);
        fetch_tokens(ig, a.input_gate, k.n, t0, k.len, l);
        fetch_tokens(x, a.x, k.n, t0, k.len, l);
        fetch_tokens(gy, o.grad_y, k.n, t0, k.len, l);
        flag = fetch_flag<TOK>(a.resets, k.n * a.T, t0, k.len, k.lane);
        mark.zero();
        if (tile < k.tiles) mark.load(o.checkpoints + (k.n * k.tiles + tile) * a.D + l.block + l.from, l.apart);
    };
    if (k.steps > 0) fetch((k.steps - 1) * ranks + k.rank);
    if constexpr (CLUSTER) cluster_wait();
    for (int64_t s = k.steps - 1; s >= 0; --s) {
        const int64_t turn = k.steps - 1 - s, tile = s * ranks + k.rank, t0 = tile * TILE + k.w * TOK;
        const int p = static_cast<int>(turn & 1);
        Gates v[TOK];
        f2 xs[TOK], gs[TOK], keep[TOK], b[TOK];
        const uint32_t cut = starts(flag);
        f2 state = mark.get();
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
            v[i] = gates(g[i].get(), ig[i].get(), decays);
            xs[i] = x[i].get();
            gs[i] = gy[i].get();
            b[i] = mul2(mul2(v[i].root, v[i].i), xs[i]);
            keep[i] = v[i].a;
        }
        const bool pad = t0 + TOK > k.len;
        if (pad) {  // padding hands state and message on
#pragma unroll
            for (int i = 0; i < TOK; ++i)
                if (t0 + i >= k.len) keep[i] = both(1.f), b[i] = gs[i] = xs[i] = both(0.f);
        }
        if (s > 0) fetch(tile - ranks);
        auto cuts = [&](int i) { return (cut >> i & 1u) != 0u; };
        f2 A = both(1.f), B = both(0.f), M = both(0.f);
        if (cut == 0) {
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                A = mul2(A, keep[i]);
                B = fma2(keep[i], B, b[i]);
                M = mul2(keep[TOK - 1 - i], add2(gs[TOK - 1 - i], M));
            }
        } else {  // a reset is a select, not a product with 0
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                A = cuts(i) ? both(kCut) : mul2(A, keep[i]);
                B = cuts(i) ? b[i] : fma2(keep[i], B, b[i]);
                M = cuts(TOK - 1 - i) ? both(0.f) : mul2(keep[TOK - 1 - i], add2(gs[TOK - 1 - i], M));
            }
        }
        chain.put(p, k.w, k.lane, A, B, M);
        __syncthreads();
        Exchange<kGatedCluster> *ex = nullptr;
        if constexpr (CLUSTER) ex = &exchange;
        f2 m = in_front<CLUSTER, false>(chain, ex, turn, k.w, k.lane, k.rank, ranks, carry, &gave_up);
        state = state_in_front(chain, p, k.w, k.lane, state);
        f2 before[TOK];  // the state before each token, 0 at a reset
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
            before[i] = cuts(i) ? both(0.f) : state;
            state = fma2(keep[i], before[i], b[i]);
        }
        const int64_t at_last = (k.n * a.T + t0 + TOK - 1) * a.D + l.block;
        T *px = static_cast<T *>(o.g.x) + at_last, *pg = static_cast<T *>(o.g.gate) + at_last, *pi = static_cast<T *>(o.g.input_gate) + at_last;
#pragma unroll
        for (int i = TOK - 1; i >= 0; --i, px -= a.D, pg -= a.D, pi -= a.D) {
            TokenGrads t = token_grads(v[i], keep[i], xs[i], gs[i], before[i], log_decay, m);
            if (cuts(i)) m = both(0.f);
            bool on0 = l.on0, on1 = l.on1;
            if (pad) {
                if (t0 + i >= k.len) t.x = t.gate = t.input_gate = t.share = both(0.f);
                on0 = on0 && t0 + i < a.T, on1 = on1 && t0 + i < a.T;
            }
            sum = add2(sum, t.share);
            store_two<T, VEC>(px + l.d, t.x, on0, on1);
            store_two<T, VEC>(pg + l.d, t.gate, on0, on1);
            store_two<T, VEC>(pi + l.d, t.input_gate, on0, on1);
        }
        if constexpr (!CLUSTER) {
            if (k.w == 0) {
                chain.last[p][k.lane] = halves(m);
                carry = m;
            }
        }
    }
    finish<T, VEC, TILE, CLUSTER>(a, o, k, ranks, l, carry, sum, chain);
    leave(&gave_up, &g_timed_out);
}

// Arrays that tensor maps take: two steps' inputs are on their way into shared
// memory while a third's are worked on; what the gradients need again (x,
// grad_y) is read again from there, and each gradient leaves from its input's
// place, which the same lane has read.  With two steps in shared memory, one of
// them on its way, the bytes in flight bound the kernel (a tenth slower).  Two
// blocks an SM leave 17 KB for the maps, which is why at most four blocks share
// a row here.  Measured: 8 x 2048 x 4096 bfloat16 238 us (its bytes' time 139), 4
// x 4096 x 4096 float32 297 us (277), 2 x 16384 x 2048 bfloat16 in clusters of
// four 299 us (139).  Float32 is bound by its bytes; bfloat16 by instructions (issue
// slots 58% busy at two blocks an SM; 8 x 2048 x 4096 has 512 blocks' work for
// 304 places).
constexpr int kBackCluster = 4, kBackStages = 3;
struct BackwardMaps {
    CUtensorMap x, gate, input_gate, grad_y, dx, dgate, dinput_gate;
};
template <class T>
struct BackwardTile {
    static constexpr int TOK = 16 / static_cast<int>(sizeof(T)), TOKENS = TOK * kGatedWarps;
    static constexpr uint32_t BYTES = TOKENS * kGatedWidth * sizeof(T);  // of one array
    static constexpr size_t SMEM = kBackStages * 4 * BYTES + 128;
};

template <class T, bool CLUSTER>
__global__ void __launch_bounds__(32 * kGatedWarps, 2)
    tiled_backward_kernel(const __grid_constant__ rlscan_gated_scan_args a, const __grid_constant__ BackwardArgs o,
                          const __grid_constant__ BackwardMaps maps, int ranks)
{
    constexpr int TOK = BackwardTile<T>::TOK, TILE = BackwardTile<T>::TOKENS, STEP = kGatedWidth * sizeof(T);
    constexpr uint32_t BYTES = BackwardTile<T>::BYTES;
    extern __shared__ char raw[];
    __shared__ TwoChains chain;
    __shared__ std::conditional_t<CLUSTER, Exchange<kBackCluster>, char> exchange;
    __shared__ uint64_t full[kBackStages];
    __shared__ int gave_up;
    ptx::pdl_trigger_dependents();
    char *stages = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw) + 127) & ~static_cast<uintptr_t>(127));
    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < kBackStages; ++i) ptx::mbar_init(&full[i], 1);
        if constexpr (CLUSTER) exchange.init();
        ptx::fence_mbar_init();
    }
    __syncthreads();
    if constexpr (CLUSTER) cluster_arrive();
    ptx::pdl_wait_prerequisites();
    int64_t block;
    const Walk k = walk<TILE, CLUSTER>(a, ranks, block);
    const Lane<true> l(block, k.lane, a.D);
    const int x0 = static_cast<int>(l.block), row = static_cast<int>(k.n);
    auto fetch = [&](int64_t turn, int st) {  // by one thread
        const int t = static_cast<int>(((k.steps - 1 - turn) * ranks + k.rank) * TILE);
        const uint32_t at = ptx::smem_u32(stages) + st * 4 * BYTES, bar = ptx::smem_u32(&full[st]);
        ptx::mbar_arrive_expect_tx(&full[st], 4 * BYTES);
        load_box3(at, &maps.gate, x0, t, row, bar);
        load_box3(at + BYTES, &maps.input_gate, x0, t, row, bar);
        load_box3(at + 2 * BYTES, &maps.x, x0, t, row, bar);
        load_box3(at + 3 * BYTES, &maps.grad_y, x0, t, row, bar);
    };
    const int64_t marks = gated_marks(a.T);
    f2 mark = both(0.f);
    uint32_t flag = 0;
    auto look = [&](int64_t turn) {  // the step's checkpoint and resets
        const int64_t t = ((k.steps - 1 - turn) * ranks + k.rank) * TILE;
        flag = fetch_flag<TOK>(a.resets, k.n * a.T, t + k.w * TOK, k.len, k.lane);
        const int64_t i = t / RLSCAN_GATED_SCAN_CHECKPOINT;
        mark = load_two<true>(o.checkpoints + (k.n * marks + i) * a.D + l.block + l.d, i < marks && l.on0, i < marks && l.on1);
    };
    const f2 log_decay = load_two<true>(a.log_decay + l.block + l.d, l.on0, l.on1);
    const Decay decays(log_decay);
    f2 carry = o.grad_final != nullptr ? load_two<true>(o.grad_final + k.n * a.D + l.block + l.d, l.on0, l.on1) : both(0.f);
    f2 sum = both(0.f);  // the lane's share of dlog_decay
    if (k.steps > 0) {
        if (threadIdx.x == 0) {
            fetch(0, 0);
            if (k.steps > 1) fetch(1, 1);
        }
        look(0);
    }
    if constexpr (CLUSTER) cluster_wait();
    const uint32_t mine = k.w * TOK * STEP + l.d * sizeof(T);  // of the lane, in a tile
    int stage = 0;
    uint32_t parity = 0;
    for (int64_t turn = 0; turn < k.steps; ++turn) {
        const int64_t t0 = ((k.steps - 1 - turn) * ranks + k.rank) * TILE + k.w * TOK;
        const int p = static_cast<int>(turn & 1);
        wait(ptx::smem_u32(&full[stage]), parity, &gave_up);
        char *in = stages + stage * 4 * BYTES + mine;
        const bool pad = t0 + TOK > k.len;
        if (pad) {  // x and grad_y of padding count 0
#pragma unroll 1
            for (int i = 0; i < TOK; ++i)
                if (t0 + i >= k.len) {
                    write_two<T>(in + 2 * BYTES + i * STEP, both(0.f));
                    write_two<T>(in + 3 * BYTES + i * STEP, both(0.f));
                }
            fence_async();  // in front of the copy that takes the stage next
        }
        Gates v[TOK];
#pragma unroll
        for (int i = 0; i < TOK; ++i) v[i] = gates(read_two<T>(in + i * STEP), read_two<T>(in + BYTES + i * STEP), decays);
        const uint32_t cut = starts(flag);
        f2 state = mark, A = both(1.f), B = both(0.f), M = both(0.f);
        if (pad) {  // and hands state and message on
#pragma unroll
            for (int i = 0; i < TOK; ++i)
                if (t0 + i >= k.len) v[i].a = both(1.f), v[i].root = both(0.f);
        }
        // A reset is a select, not a product with 0.  Steps without one, which are
        // most, take a path of their own.
        auto fold = [&](auto cutting) {
            auto cuts = [&](int i) { return decltype(cutting)::value && (cut >> i & 1u) != 0u; };
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                const f2 b = mul2(mul2(v[i].root, v[i].i), read_two<T>(in + 2 * BYTES + i * STEP));
                A = cuts(i) ? both(kCut) : mul2(A, v[i].a);
                B = cuts(i) ? b : fma2(v[i].a, B, b);
            }
#pragma unroll
            for (int i = TOK - 1; i >= 0; --i) M = cuts(i) ? both(0.f) : mul2(v[i].a, add2(read_two<T>(in + 3 * BYTES + i * STEP), M));
        };
        if (cut == 0) fold(std::false_type());
        else fold(std::true_type());
        chain.put(p, k.w, k.lane, A, B, M);
        if (k.lane == 0) stores_read();  // the step behind has left its stage,
        __syncthreads();                 // all of it: the stage takes the step after next
        const int behind = stage == 0 ? kBackStages - 1 : stage - 1;
        if (threadIdx.x == 0 && turn + 2 < k.steps && !has_given_up(&gave_up)) fetch(turn + 2, behind);
        Exchange<kBackCluster> *ex = nullptr;
        if constexpr (CLUSTER) ex = &exchange;
        f2 m = in_front<CLUSTER, false>(chain, ex, turn, k.w, k.lane, k.rank, ranks, carry, &gave_up);
        state = state_in_front(chain, p, k.w, k.lane, state);
        auto gradients = [&](auto cutting) {
            auto cuts = [&](int i) { return decltype(cutting)::value && (cut >> i & 1u) != 0u; };
            f2 before[TOK];  // the state before each token, 0 at a reset
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                before[i] = cuts(i) ? both(0.f) : state;
                state = fma2(v[i].a, before[i], mul2(mul2(v[i].root, v[i].i), read_two<T>(in + 2 * BYTES + i * STEP)));
            }
#pragma unroll
            for (int i = TOK - 1; i >= 0; --i) {
                TokenGrads t = token_grads(v[i], v[i].a, read_two<T>(in + 2 * BYTES + i * STEP), read_two<T>(in + 3 * BYTES + i * STEP),
                                           before[i], log_decay, m);
                if (cuts(i)) m = both(0.f);
                if (pad && t0 + i >= k.len) t.x = t.gate = t.input_gate = t.share = both(0.f);
                sum = add2(sum, t.share);
                write_two<T>(in + i * STEP, t.gate);
                write_two<T>(in + BYTES + i * STEP, t.input_gate);
                write_two<T>(in + 2 * BYTES + i * STEP, t.x);
                asm volatile("" ::: "memory");  // the next token's loads behind this: all at once they spill
            }
        };
        if (cut == 0) gradients(std::false_type());
        else gradients(std::true_type());
        fence_async();
        __syncwarp();
        if (k.lane == 0 && t0 < a.T) {
            const uint32_t from = ptx::smem_u32(stages) + stage * 4 * BYTES + k.w * TOK * STEP;
            store_box3(&maps.dgate, x0, static_cast<int>(t0), row, from);
            store_box3(&maps.dinput_gate, x0, static_cast<int>(t0), row, from + BYTES);
            store_box3(&maps.dx, x0, static_cast<int>(t0), row, from + 2 * BYTES);
            stores_commit();
        }
        if constexpr (!CLUSTER) {
            if (k.w == 0) {
                chain.last[p][k.lane] = halves(m);
                carry = m;
            }
        }
        if (turn + 1 < k.steps) look(turn + 1);  // here, where registers are free; looked at behind the gates
        if (++stage == kBackStages) stage = 0, parity ^= 1u;
    }
    finish<T, true, TILE, CLUSTER>(a, o, k, ranks, l, carry, sum, chain);
    if (k.lane == 0) stores_read();
    leave(&gave_up, &g_timed_out);
}

template <class T>
rlscan_status backward_typed(const rlscan_gated_scan_args &a, const BackwardArgs &o, int64_t &parts, bool on_device, cudaStream_t s)
{
    const int64_t chains = a.N * ceil_div(a.D, kGatedWidth);
    const int threads = 32 * kGatedWarps;
    const Access access = gated_access<T>({&a.x, &a.gate, &a.input_gate, &o.grad_y}, {o.g.x, o.g.gate, o.g.input_gate},
                                          {o.g.initial_state, o.parts, o.checkpoints}, a.N, a.T, a.D, on_device);
    if (access == Access::Tiles) {
        using Tile = BackwardTile<T>;
        static PerDevice alone, shared;
        if (!raise_smem(alone, tiled_backward_kernel<T, false>, Tile::SMEM) || !raise_smem(shared, tiled_backward_kernel<T, true>, Tile::SMEM))
            return RLSCAN_ERR_CUDA;
        BackwardMaps m;
        auto in = [&](CUtensorMap *map, const rlscan_array3 &v) {
            return gated_map<T>(map, v.data, v.row_stride, v.token_stride, a.N, a.T, a.D, Tile::TOKENS);
        };
        auto out = [&](CUtensorMap *map, void *p) { return gated_map<T>(map, p, a.T * a.D, a.D, a.N, a.T, a.D, Tile::TOK); };
        if (!in(&m.x, a.x) || !in(&m.gate, a.gate) || !in(&m.input_gate, a.input_gate) || !in(&m.grad_y, o.grad_y) ||
            !out(&m.dx, o.g.x) || !out(&m.dgate, o.g.gate) || !out(&m.dinput_gate, o.g.input_gate))
            return RLSCAN_ERR_CUDA;
        const int ranks = gated_cluster<T, 2>(tiled_backward_kernel<T, true>, chains, a.T, Tile::TOKENS, Tile::SMEM, kBackCluster);
        parts = a.N * ranks;
        return ranks > 1 ? launch_cluster(chains * ranks <= sm_count(), tiled_backward_kernel<T, true>, chains * ranks, threads, Tile::SMEM, ranks, s, a, o, m, ranks)
                         : launch_cluster(chains <= sm_count(), tiled_backward_kernel<T, false>, chains, threads, Tile::SMEM, 1, s, a, o, m, 1);
    }
    auto go = [&](auto pairs) {
        constexpr bool VEC = decltype(pairs)::value;
        const int ranks = gated_cluster<T, VEC>(backward_kernel<T, VEC, true>, chains, a.T, kBackTile, 0);
        parts = a.N * ranks;
        return ranks > 1 ? launch_cluster(chains * ranks <= sm_count(), backward_kernel<T, VEC, true>, chains * ranks, threads, 0, ranks, s, a, o, ranks)
                         : launch_cluster(chains <= sm_count(), backward_kernel<T, VEC, false>, chains, threads, 0, 1, s, a, o, 1);
    };
    return access != Access::Values ? go(std::true_type()) : go(std::false_type());
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
                                         const rlscan_gated_scan_grads &g, void *ws, bool on_device, cudaStream_t s)
{
    float *shares = g.log_decay != nullptr ? static_cast<float *>(ws) : nullptr;
    int64_t parts = 0;
    if (a.N > 0) {
        const BackwardArgs o{grad_y, grad_final_state, checkpoints, g, shares};
        const rlscan_status st = a.dtype == RLSCAN_BF16 ? backward_typed<bf16>(a, o, parts, on_device, s)
                                                        : backward_typed<float>(a, o, parts, on_device, s);
        if (st != RLSCAN_OK) return st;
    }
    if (g.log_decay == nullptr) return RLSCAN_OK;
    SumJobs jobs;  // without rows the sums have no parts, and are 0
    jobs.add(shares, parts, a.D, a.D, g.log_decay, false);
    return launch_sums(jobs, s);
}

rlscan_status gated_scan_backward_status(cudaStream_t s) { return take_flag(g_timed_out, s); }

}  // namespace seq
}  // namespace rlscan
