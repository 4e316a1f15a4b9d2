// k_gated_scan.cu -- the gated recurrence over prompts and for single tokens:
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) i_t x_t,  a_t = exp(log_decay r_t),
// r and i the sigmoids of the two gates, one state a channel.
#include "gated_scan.cuh"

namespace rlscan {
namespace seq {
namespace {

__device__ unsigned int g_timed_out;  // a wait ran out on this device

struct ForwardArgs {
    void *y;
    float *final_state, *checkpoints;
};

// A block walks 64 channels of a row in steps: a warp has TOK tokens of each
// step, a lane two channels of them.  Every warp folds its tokens into one
// affine map (A, B) of the state before them; the maps of the warps before it,
// in order, give its first state, and its tokens follow.  The coefficients are
// made once and stay in registers, so the inputs are read once.  CLUSTER: the
// blocks of a cluster take neighbouring steps and hand their maps round.

// Past the last token the state is handed on.
template <int TOK>
__device__ __forceinline__ void pad(f2 (&keep)[TOK], f2 (&b)[TOK], int64_t t0, int64_t len)
{
    if (t0 + TOK > len) {
#pragma unroll
        for (int k = 0; k < TOK; ++k)
            if (t0 + k >= len) keep[k] = both(1.f), b[k] = both(0.f);
    }
}

// A step's state from the one before.  A reset (bit k of `cut`) is a select,
// not a product with 0; steps without one, which are most, take no time for it.
template <bool CUTTING>
__device__ __forceinline__ f2 step_state(f2 h, f2 keep, f2 b, uint32_t cut, int k)
{
    const f2 v = fma2(keep, h, b);
    return CUTTING && (cut >> k & 1u) != 0u ? b : v;
}

template <bool CUTTING, int TOK>
__device__ __forceinline__ void fold(const f2 (&keep)[TOK], const f2 (&b)[TOK], uint32_t cut, f2 &A, f2 &B)
{
    A = CUTTING && (cut & 1u) != 0u ? both(kCut) : keep[0], B = b[0];
#pragma unroll
    for (int k = 1; k < TOK; ++k) {
        A = CUTTING && (cut >> k & 1u) != 0u ? both(kCut) : mul2(A, keep[k]);
        B = step_state<CUTTING>(B, keep[k], b[k], cut, k);
    }
}

// Behind the last step: zeros for tiles of padding, the final state, the
// checkpoints past the last step (all the state after the last token).
template <class T, bool VEC, int TILE, bool CLUSTER>
__device__ __forceinline__ void finish(const rlscan_gated_scan_args &a, const ForwardArgs &o, const Walk &k, int ranks, const Lane<VEC> &l, f2 carry)
{
    constexpr int TOK = TILE / kGatedWarps;
    for (int64_t tile = k.steps * ranks + k.rank; tile < k.tiles; tile += ranks) {
        const int64_t t0 = tile * TILE + k.w * TOK;
        T *to = static_cast<T *>(o.y) + (k.n * a.T + t0) * a.D + l.block;
        for (int i = 0; i < TOK; ++i)
            if (t0 + i < a.T) store_two<T, VEC>(to + i * a.D + l.d, both(0.f), l.on0, l.on1);
    }
    if (k.rank == 0 && k.w == kGatedWarps - 1) {
        if (o.final_state != nullptr) store_two<float, VEC>(o.final_state + k.n * a.D + l.block + l.d, carry, l.on0, l.on1);
        const int64_t marks = gated_marks(a.T);
        if (o.checkpoints != nullptr)
            for (int64_t i = k.steps * k.span / RLSCAN_GATED_SCAN_CHECKPOINT; i < marks; ++i)
                store_two<float, VEC>(o.checkpoints + (k.n * marks + i) * a.D + l.block + l.d, carry, l.on0, l.on1);
    }
}

// Arrays of any alignment: the next step's values are loaded into registers
// while this one's are worked on.  Measured, 3 x 1001 x 1111 float32 (13 MB a
// tensor, one value a load): 23 us, its bytes' time 8.
template <class T, bool VEC, bool CLUSTER>
__global__ void __launch_bounds__(32 * kGatedWarps, sizeof(T) == 2 && VEC ? 3 : 2)
    forward_kernel(const __grid_constant__ rlscan_gated_scan_args a, const __grid_constant__ ForwardArgs o, int ranks)
{
    constexpr int TILE = kGatedTile, TOK = TILE / kGatedWarps;
    __shared__ Chain chain;
    __shared__ std::conditional_t<CLUSTER, Exchange<kGatedCluster>, char> exchange;
    __shared__ int gave_up;
    ptx::pdl_trigger_dependents();
    if (threadIdx.x == 0) {
        gave_up = 0;
        if constexpr (CLUSTER) exchange.init(), ptx::fence_mbar_init();
    }
    __syncthreads();
    if constexpr (CLUSTER) cluster_arrive();  // no block sends to one that has not begun
    ptx::pdl_wait_prerequisites();
    int64_t block;
    const Walk k = walk<TILE, CLUSTER>(a, ranks, block);
    const Lane<VEC> l(block, k.lane, a.D);
    const Decay decays(load_two<VEC>(a.log_decay + l.block + l.d, l.on0, l.on1));
    f2 carry = a.initial_state != nullptr ? load_two<VEC>(a.initial_state + k.n * a.D + l.block + l.d, l.on0, l.on1) : both(0.f);
    Two<T, VEC> x[TOK], g[TOK], ig[TOK];
    uint32_t flag = 0;
    auto fetch = [&](int64_t t0) {
        fetch_tokens(g, a.gate, k.n, t0, k.len, l);
        fetch_tokens(ig, a.input_gate, k.n, t0, k.len, l);
        fetch_tokens(x, a.x, k.n, t0, k.len, l);
        flag = fetch_flag<TOK>(a.resets, k.n * a.T, t0, k.len, k.lane);
    };
    if (k.steps > 0) fetch(static_cast<int64_t>(k.rank) * TILE + k.w * TOK);
    if constexpr (CLUSTER) cluster_wait();
    for (int64_t s = 0; s < k.steps; ++s) {
        const int p = static_cast<int>(s & 1);
        const int64_t t0 = (s * ranks + k.rank) * TILE + k.w * TOK;
        f2 keep[TOK], b[TOK], A, B;
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
            const Gates v = gates(g[i].get(), ig[i].get(), decays);
            keep[i] = v.a;
            b[i] = mul2(mul2(v.root, v.i), x[i].get());
        }
        const uint32_t cut = starts(flag);
        pad(keep, b, t0, k.len);
        if (s + 1 < k.steps) fetch(t0 + k.span);
        if (cut == 0) fold<false>(keep, b, cut, A, B);
        else fold<true>(keep, b, cut, A, B);
        chain.put(p, k.w, k.lane, A, B);
        __syncthreads();
        Exchange<kGatedCluster> *ex = nullptr;
        if constexpr (CLUSTER) ex = &exchange;
        f2 h = in_front<CLUSTER, true>(chain, ex, s, k.w, k.lane, k.rank, ranks, carry, &gave_up);
        if (o.checkpoints != nullptr && k.w % (RLSCAN_GATED_SCAN_CHECKPOINT / TOK) == 0 && t0 < a.T) {
            float *to = o.checkpoints + (k.n * gated_marks(a.T) + t0 / RLSCAN_GATED_SCAN_CHECKPOINT) * a.D + l.block;
            store_two<float, VEC>(to + l.d, h, l.on0, l.on1);
        }
        T *to = static_cast<T *>(o.y) + (k.n * a.T + t0) * a.D + l.block;
        if (t0 + TOK <= k.len && cut == 0) {
#pragma unroll
            for (int i = 0; i < TOK; ++i, to += a.D) {
                h = fma2(keep[i], h, b[i]);
                store_two<T, VEC>(to + l.d, h, l.on0, l.on1);
            }
        } else {
#pragma unroll
            for (int i = 0; i < TOK; ++i, to += a.D) {
                h = step_state<true>(h, keep[i], b[i], cut, i);
                const bool in = t0 + i < a.T;
                store_two<T, VEC>(to + l.d, t0 + i < k.len ? h : both(0.f), in && l.on0, in && l.on1);
            }
        }
        if constexpr (!CLUSTER) {
            if (k.w == kGatedWarps - 1) {
                chain.last[p][k.lane] = halves(h);
                carry = h;
            }
        }
    }
    finish<T, VEC, TILE, CLUSTER>(a, o, k, ranks, l, carry);
    leave(&gave_up, &g_timed_out);
}

// Arrays that tensor maps take: two steps' inputs are on their way into shared
// memory, so registers hold coefficients alone and a warp takes twice the
// tokens of 16-bit values; y leaves through shared memory too.  Three blocks an
// SM are what 78 registers and 57 KB allow.  Measured: 8 x 2048 x 4096 bfloat16
// 120 us (its bytes' time 79), 4 x 4096 x 4096 float32 170 us (158), 2 x 16384 x
// 2048 bfloat16 in clusters of six 152 us (79).  Float32 is bound by its bytes;
// bfloat16 by instructions and by the steps' chain of waits: issue slots 63%
// busy, exponential units (three exponentials, two reciprocals and a reciprocal
// root a value) 42%, and of 512 blocks' work 456 at once leave a second round.
struct ForwardMaps {
    CUtensorMap x, gate, input_gate, y;
};
template <class T>
struct ForwardTile {
    static constexpr int TOK = 16 / static_cast<int>(sizeof(T)), TOKENS = TOK * kGatedWarps;
    static constexpr uint32_t BYTES = TOKENS * kGatedWidth * sizeof(T);          // of one array
    static constexpr size_t SMEM = 2 * 3 * BYTES + BYTES + 128;                  // two stages, y
};

template <class T, bool CLUSTER>
__global__ void __launch_bounds__(32 * kGatedWarps, 3)
    tiled_forward_kernel(const __grid_constant__ rlscan_gated_scan_args a, const __grid_constant__ ForwardArgs o,
                         const __grid_constant__ ForwardMaps maps, int ranks)
{
    constexpr int TOK = ForwardTile<T>::TOK, TILE = ForwardTile<T>::TOKENS;
    constexpr uint32_t BYTES = ForwardTile<T>::BYTES;
    extern __shared__ char raw[];
    __shared__ Chain chain;
    __shared__ std::conditional_t<CLUSTER, Exchange<kGatedCluster>, char> exchange;
    __shared__ uint64_t full[2];
    __shared__ int gave_up;
    ptx::pdl_trigger_dependents();
    char *stages = reinterpret_cast<char *>((reinterpret_cast<uintptr_t>(raw) + 127) & ~static_cast<uintptr_t>(127));
    if (threadIdx.x == 0) {
        gave_up = 0;
        ptx::mbar_init(&full[0], 1);
        ptx::mbar_init(&full[1], 1);
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
    auto fetch = [&](int64_t s) {  // by one thread
        const int st = static_cast<int>(s & 1), t = static_cast<int>((s * ranks + k.rank) * TILE);
        const uint32_t at = ptx::smem_u32(stages) + st * 3 * BYTES, bar = ptx::smem_u32(&full[st]);
        ptx::mbar_arrive_expect_tx(&full[st], 3 * BYTES);
        load_box3(at, &maps.gate, x0, t, row, bar);
        load_box3(at + BYTES, &maps.input_gate, x0, t, row, bar);
        load_box3(at + 2 * BYTES, &maps.x, x0, t, row, bar);
    };
    if (threadIdx.x == 0) {
        if (k.steps > 0) fetch(0);
        if (k.steps > 1) fetch(1);
    }
    const Decay decays(load_two<true>(a.log_decay + l.block + l.d, l.on0, l.on1));
    f2 carry = a.initial_state != nullptr ? load_two<true>(a.initial_state + k.n * a.D + l.block + l.d, l.on0, l.on1) : both(0.f);
    uint32_t flag = fetch_flag<TOK>(a.resets, k.n * a.T, static_cast<int64_t>(k.rank) * TILE + k.w * TOK, k.len, k.lane);
    if constexpr (CLUSTER) cluster_wait();
    const uint32_t mine = k.w * TOK * kGatedWidth * sizeof(T) + l.d * sizeof(T);  // of the lane, in a tile
    char *out = stages + 2 * 3 * BYTES;
    for (int64_t s = 0; s < k.steps; ++s) {
        const int p = static_cast<int>(s & 1);
        const int64_t t0 = (s * ranks + k.rank) * TILE + k.w * TOK;
        wait(ptx::smem_u32(&full[p]), static_cast<uint32_t>(s >> 1) & 1u, &gave_up);
        const char *in = stages + p * 3 * BYTES + mine;
        f2 keep[TOK], b[TOK], A, B;
#pragma unroll
        for (int i = 0; i < TOK; ++i) {
            constexpr int STEP = kGatedWidth * sizeof(T);
            const Gates v = gates(read_two<T>(in + i * STEP), read_two<T>(in + BYTES + i * STEP), decays);
            keep[i] = v.a;
            b[i] = mul2(mul2(v.root, v.i), read_two<T>(in + 2 * BYTES + i * STEP));
        }
        const uint32_t cut = starts(flag);
        pad(keep, b, t0, k.len);
        if (s + 1 < k.steps) flag = fetch_flag<TOK>(a.resets, k.n * a.T, t0 + k.span, k.len, k.lane);
        if (cut == 0) fold<false>(keep, b, cut, A, B);
        else fold<true>(keep, b, cut, A, B);
        chain.put(p, k.w, k.lane, A, B);
        __syncthreads();  // all have taken the stage's values
        if (threadIdx.x == 0 && s + 2 < k.steps && !has_given_up(&gave_up)) fetch(s + 2);
        Exchange<kGatedCluster> *ex = nullptr;
        if constexpr (CLUSTER) ex = &exchange;
        f2 h = in_front<CLUSTER, true>(chain, ex, s, k.w, k.lane, k.rank, ranks, carry, &gave_up);
        if (o.checkpoints != nullptr && k.w % (RLSCAN_GATED_SCAN_CHECKPOINT / TOK) == 0 && t0 < a.T) {
            float *to = o.checkpoints + (k.n * gated_marks(a.T) + t0 / RLSCAN_GATED_SCAN_CHECKPOINT) * a.D + l.block;
            store_two<float, true>(to + l.d, h, l.on0, l.on1);
        }
        if (k.lane == 0) stores_read();  // the step before has left the warp's part
        __syncwarp();
        if (cut == 0) {
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                h = fma2(keep[i], h, b[i]);
                write_two<T>(out + mine + i * kGatedWidth * sizeof(T), h);
            }
        } else {
#pragma unroll
            for (int i = 0; i < TOK; ++i) {
                h = step_state<true>(h, keep[i], b[i], cut, i);
                write_two<T>(out + mine + i * kGatedWidth * sizeof(T), h);
            }
        }
        if (t0 + TOK > k.len) {  // y of padding is 0
#pragma unroll
            for (int i = 0; i < TOK; ++i)
                if (t0 + i >= k.len) write_two<T>(out + mine + i * kGatedWidth * sizeof(T), both(0.f));
        }
        fence_async();
        __syncwarp();
        if (k.lane == 0 && t0 < a.T) {
            store_box3(&maps.y, x0, static_cast<int>(t0), row, ptx::smem_u32(out) + k.w * TOK * kGatedWidth * sizeof(T));
            stores_commit();
        }
        if constexpr (!CLUSTER) {
            if (k.w == kGatedWarps - 1) {
                chain.last[p][k.lane] = halves(h);
                carry = h;
            }
        }
    }
    finish<T, true, TILE, CLUSTER>(a, o, k, ranks, l, carry);
    if (k.lane == 0) stores_read();
    leave(&gave_up, &g_timed_out);
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
    const int64_t slot = q.slots != nullptr ? q.slots[n] : n;
    const bool busy = slot >= 0 && slot < q.P, on0 = busy && l.on0, on1 = busy && l.on1;
    float *state = q.state + (busy ? slot * a.D : 0) + l.block + l.d;
    Two<T, VEC> x, g, ig;
    g.load(static_cast<const T *>(a.gate.data) + n * a.gate.row_stride + l.block + l.from, l.apart);
    ig.load(static_cast<const T *>(a.input_gate.data) + n * a.input_gate.row_stride + l.block + l.from, l.apart);
    x.load(static_cast<const T *>(a.x.data) + n * a.x.row_stride + l.block + l.from, l.apart);
    const Decay decays(load_two<VEC>(a.log_decay + l.block + l.d, l.on0, l.on1));
    f2 h = load_two<VEC>(state, on0, on1);
    const Gates v = gates(g.get(), ig.get(), decays);
    h = fma2(v.a, h, mul2(mul2(v.root, v.i), x.get()));
    store_two<float, VEC>(state, h, on0, on1);
    store_two<T, VEC>(static_cast<T *>(q.y) + n * a.D + l.block + l.d, busy ? h : both(0.f), l.on0, l.on1);
}

template <class T>
rlscan_status forward_typed(const rlscan_gated_scan_args &a, const ForwardArgs &o, bool on_device, cudaStream_t s)
{
    const int64_t chains = a.N * ceil_div(a.D, kGatedWidth);
    const int threads = 32 * kGatedWarps;
    const Access access = gated_access<T>({&a.x, &a.gate, &a.input_gate}, {o.y}, {o.final_state, o.checkpoints}, a.N, a.T, a.D, on_device);
    if (access == Access::Tiles) {
        using Tile = ForwardTile<T>;
        static PerDevice alone, shared;
        if (!raise_smem(alone, tiled_forward_kernel<T, false>, Tile::SMEM) || !raise_smem(shared, tiled_forward_kernel<T, true>, Tile::SMEM))
            return RLSCAN_ERR_CUDA;
        ForwardMaps m;
        if (!gated_map<T>(&m.x, a.x.data, a.x.row_stride, a.x.token_stride, a.N, a.T, a.D, Tile::TOKENS) ||
            !gated_map<T>(&m.gate, a.gate.data, a.gate.row_stride, a.gate.token_stride, a.N, a.T, a.D, Tile::TOKENS) ||
            !gated_map<T>(&m.input_gate, a.input_gate.data, a.input_gate.row_stride, a.input_gate.token_stride, a.N, a.T, a.D, Tile::TOKENS) ||
            !gated_map<T>(&m.y, o.y, a.T * a.D, a.D, a.N, a.T, a.D, Tile::TOK))
            return RLSCAN_ERR_CUDA;
        const int ranks = gated_cluster<T, 2>(tiled_forward_kernel<T, true>, chains, a.T, Tile::TOKENS, Tile::SMEM);
        return ranks > 1 ? launch_cluster(chains * ranks <= sm_count(), tiled_forward_kernel<T, true>, chains * ranks, threads, Tile::SMEM, ranks, s, a, o, m, ranks)
                         : launch_cluster(chains <= sm_count(), tiled_forward_kernel<T, false>, chains, threads, Tile::SMEM, 1, s, a, o, m, 1);
    }
    auto go = [&](auto pairs) {
        constexpr bool VEC = decltype(pairs)::value;
        const int ranks = gated_cluster<T, VEC>(forward_kernel<T, VEC, true>, chains, a.T, kGatedTile, 0);
        return ranks > 1 ? launch_cluster(chains * ranks <= sm_count(), forward_kernel<T, VEC, true>, chains * ranks, threads, 0, ranks, s, a, o, ranks)
                         : launch_cluster(chains <= sm_count(), forward_kernel<T, VEC, false>, chains, threads, 0, 1, s, a, o, 1);
    };
    return access != Access::Values ? go(std::true_type()) : go(std::false_type());
}

template <class T>
rlscan_status step_typed(const rlscan_gated_scan_args &a, const StepArgs &q, cudaStream_t s)
{
    const bool pairs = gated_access<T>({&a.x, &a.gate, &a.input_gate}, {q.y}, {q.state}, a.N, 1, a.D, false) != Access::Values;
    const int64_t grid = ceil_div(a.N * ceil_div(a.D, kGatedWidth), kStepWarps);
    return pairs ? launch_overlapped(step_kernel<T, true>, grid, 32 * kStepWarps, 0, s, a, q)
                 : launch_overlapped(step_kernel<T, false>, grid, 32 * kStepWarps, 0, s, a, q);
}

}  // namespace

rlscan_status launch_gated_scan(const rlscan_gated_scan_args &a, void *y, float *final_state, float *checkpoints,
                                bool on_device, cudaStream_t s)
{
    const ForwardArgs o{y, final_state, checkpoints};
    return a.dtype == RLSCAN_BF16 ? forward_typed<bf16>(a, o, on_device, s) : forward_typed<float>(a, o, on_device, s);
}

rlscan_status launch_gated_scan_step(const rlscan_gated_scan_args &a, float *state, int64_t P, const int32_t *slots,
                                     void *y, cudaStream_t s)
{
    const StepArgs q{state, P, slots, y};
    return a.dtype == RLSCAN_BF16 ? step_typed<bf16>(a, q, s) : step_typed<float>(a, q, s);
}

rlscan_status gated_scan_status(cudaStream_t s) { return take_flag(g_timed_out, s); }

}  // namespace seq
}  // namespace rlscan
