// gated_scan.cuh -- what the gated recurrence's kernels share: two channels of
// a token in one register pair, the gates' arithmetic, and the exchange of the
// blocks of a cluster that walk one row together.
#pragma once

#include "async_copy.cuh"

namespace rlscan {
namespace seq {

constexpr int kGatedTile = 64;     // tokens of a block's step
constexpr int kGatedWarps = 8;     // of a block
constexpr int kGatedWidth = 64;    // channels of a block: two a lane
constexpr int kGatedCluster = 8;   // blocks that share a row, at most
constexpr float kSquareFloor = 0x1p-100f;

// NaN stays NaN
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float rsqrt_fast(float v)
{
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Two channels of one token as they are stored.  VEC: neighbours, one aligned
// load; otherwise `apart` values apart (32, less at the array's edge), so that
// a warp still reads whole sectors.  A load stays in flight until its value is
// looked at.
template <class T, bool VEC>
struct Two {
    static constexpr int N = VEC && sizeof(T) == 2 ? 1 : 2;
    uint32_t w[N];
    __device__ __forceinline__ void zero()
    {
        w[0] = 0u;
        if constexpr (N == 2) w[1] = 0u;
    }
    __device__ __forceinline__ void load(const T *p, int apart)
    {
        if constexpr (VEC) {
            if constexpr (N == 1)
                asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
            else
                asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
        } else if constexpr (sizeof(T) == 2) {
            asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(w[0]) : "l"(p));
            asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(w[1]) : "l"(p + apart));
        } else {
            asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
            asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(w[1]) : "l"(p + apart));
        }
    }
    __device__ __forceinline__ f2 get() const
    {
        if constexpr (N == 1) {
            return pair(__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u));
        } else if constexpr (sizeof(T) == 2) {
            return pair(__uint_as_float(w[0] << 16), __uint_as_float(w[1] << 16));
        } else {
            return pair(__uint_as_float(w[0]), __uint_as_float(w[1]));
        }
    }
};

// A lane's two channels of a block of 64: the block's first, the lane's first
// in it, whether both are the array's, and the one it reads from (a lane past
// the last channel reads the last ones, and writes nothing).
template <bool VEC>
struct Lane {
    int64_t block;
    uint32_t d, from;
    bool on0, on1;
    int apart;
    __device__ __forceinline__ Lane(int64_t number, int lane, int64_t D) : block(number * kGatedWidth)
    {
        const uint32_t left = D - block < kGatedWidth ? static_cast<uint32_t>(D - block) : kGatedWidth;
        d = VEC ? 2 * lane : lane;
        on0 = d < left;
        on1 = VEC ? on0 : d + 32 < left;
        from = on0 ? d : left - (VEC ? 2 : 1);
        apart = on1 ? 32 : 0;
    }
};

// The warp's number, the same for all lanes to the compiler too: addresses are
// then a uniform base and the lane's 32-bit offset.
__device__ __forceinline__ int warp_number() { return static_cast<int>(__reduce_max_sync(0xffffffffu, threadIdx.x >> 5)); }

// A block's row, its rank among those that share it, and their steps.
struct Walk {
    int lane, w, rank;
    int64_t n, len, tiles, span, steps;
};
template <int TILE, bool CLUSTER>
__device__ __forceinline__ Walk walk(const rlscan_gated_scan_args &a, int ranks, int64_t &block)
{
    Walk k;
    k.lane = threadIdx.x & 31;
    k.w = warp_number();
    k.rank = CLUSTER ? static_cast<int>(blockIdx.x % static_cast<unsigned>(ranks)) : 0;
    const Division at = divide(CLUSTER ? blockIdx.x / static_cast<unsigned>(ranks) : blockIdx.x, (a.D + kGatedWidth - 1) / kGatedWidth);
    k.n = at.q;
    block = at.r;
    k.len = row_length(a.lengths, k.n, a.T);
    k.tiles = (a.T + TILE - 1) / TILE;
    k.span = static_cast<int64_t>(ranks) * TILE;
    k.steps = (k.len + k.span - 1) / k.span;
    return k;
}

// TOK tokens from t0 on of one array; past `len` (the row's tokens) zeros
template <class T, bool VEC, int TOK>
__device__ __forceinline__ void fetch_tokens(Two<T, VEC> (&v)[TOK], const rlscan_array3 &a, int64_t n, int64_t t0, int64_t len, const Lane<VEC> &l)
{
    const T *p = static_cast<const T *>(a.data) + n * a.row_stride + t0 * a.token_stride + l.block;
    const int64_t step = a.token_stride;
    if (t0 + TOK <= len) {
#pragma unroll
        for (int k = 0; k < TOK; ++k, p += step) v[k].load(p + l.from, l.apart);
    } else {
#pragma unroll
        for (int k = 0; k < TOK; ++k, p += step) {
            v[k].zero();
            if (t0 + k < len) v[k].load(p + l.from, l.apart);
        }
    }
}

// The lane's flag of a warp's TOK tokens from t0 on.  The load stays in flight
// until `starts` looks at it: bit k, a new episode starts at token k.
template <int TOK>
__device__ __forceinline__ uint32_t fetch_flag(const uint8_t *resets, int64_t row, int64_t t0, int64_t len, int lane)
{
    uint32_t flag = 0;
    if (resets != nullptr && lane < TOK && t0 + lane < len) flag = load_byte(resets + row + t0 + lane);
    return flag;
}
__device__ __forceinline__ uint32_t starts(uint32_t flag) { return __ballot_sync(0xffffffffu, flag != 0); }

template <class T, bool VEC>
__device__ __forceinline__ void store_two(T *p, f2 v, bool on0, bool on1)
{
    const float2 h = halves(v);
    if constexpr (VEC) {
        if (on0) {
            if constexpr (sizeof(T) == 2) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(h.x, h.y);
                *reinterpret_cast<uint32_t *>(p) = *reinterpret_cast<const uint32_t *>(&b);
            } else {
                *reinterpret_cast<float2 *>(p) = h;
            }
        }
    } else {
        if (on0) p[0] = from_f<T>(h.x);
        if (on1) p[32] = from_f<T>(h.y);
    }
}

// Two neighbouring channels in shared memory
template <class T>
__device__ __forceinline__ f2 read_two(const char *p)
{
    if constexpr (sizeof(T) == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
        return pair(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        const float2 h = *reinterpret_cast<const float2 *>(p);
        return pair(h.x, h.y);
    }
}
template <class T>
__device__ __forceinline__ void write_two(char *p, f2 v)
{
    store_two<T, true>(reinterpret_cast<T *>(p), v, true, true);
}

// The lane's two channels of a [D] array of float32
template <bool VEC>
__device__ __forceinline__ f2 load_two(const float *p, bool on0, bool on1)
{
    return pair(on0 ? p[0] : 0.f, on1 ? p[VEC ? 1 : 32] : 0.f);
}

// reciprocals
__device__ __forceinline__ f2 rcp2(f2 v)
{
    const float2 h = halves(v);
    return pair(rcp_fast(h.x), rcp_fast(h.y));
}

// What a channel's tokens share: log_decay times log2 e, and times -2.
struct Decay {
    f2 log2, twice;
    __device__ __forceinline__ explicit Decay(f2 log_decay) : log2(mul2(log_decay, both(kLog2e))), twice(mul2(log_decay, both(-2.f))) {}
};

// What a token's gates give.  a = exp(L) with L = log_decay r.  The square of
// the root is 1 - a^2 = -2 a sinh(L) = a Y (1 + Y^2 / 24 + Y^4 / 1920 + ...)
// with Y = -2 L: where Y < 1/2 the first omitted term is below 5e-8 of the sum,
// and beyond, where a^2 < 0.61, 1 - a a is right to 5e-7 by a's own rounding.
// The square stays above 2^-100, so that a closed gate (a = 1) gives a finite
// gradient: the slope of the root grows without bound there, but the gate's
// slope vanishes faster.
struct Gates {
    f2 r, i, a, root;
};
__device__ __forceinline__ Gates gates(f2 gate, f2 input_gate, const Decay &d)
{
    Gates g;
    g.r = sigmoid(gate);
    g.i = sigmoid(input_gate);
    g.a = decay(g.r, d.log2);
    const f2 y = mul2(g.r, d.twice), q = mul2(y, y);
    const f2 p = fma2(fma2(q, both(1.f / 1920.f), both(1.f / 24.f)), q, both(1.f));
    const float2 near = halves(mul2(mul2(g.a, y), p)), a = halves(g.a), yy = halves(y);
    const float s0 = max_nan(yy.x < 0.5f ? near.x : fmaf(-a.x, a.x, 1.f), kSquareFloor);
    const float s1 = max_nan(yy.y < 0.5f ? near.y : fmaf(-a.y, a.y, 1.f), kSquareFloor);
    g.root = mul2(pair(s0, s1), pair(rsqrt_fast(s0), rsqrt_fast(s1)));
    return g;
}

// ---- the blocks of a cluster -------------------------------------------------
// (what the blocks tell each other so is that they have begun: what they write
// for each other has barriers of its own, and a release would wait for it)
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The maps of a cluster's blocks, handed round once a step: every block sends
// its own to all (stores that count on the receiver's barrier, so nobody waits
// for more than the values) and waits for all.  Two buffers take turns: who
// has all maps of a step knows that all have read those of the step before.
template <int RANKS>
struct Exchange {
    float4 map[2][RANKS][32];
    uint64_t bar[2];

    __device__ __forceinline__ void init()  // one thread; the blocks meet before the first send
    {
        ptx::mbar_init(&bar[0], 1);
        ptx::mbar_init(&bar[1], 1);
    }
    __device__ __forceinline__ void send(int p, int mine, int to, int lane, f2 factor, f2 rest)
    {
        const float2 a = halves(factor), b = halves(rest);
        uint32_t at, signal;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(&map[p][mine][lane])), "r"(to));
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(signal) : "r"(ptx::smem_u32(&bar[p])), "r"(to));
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
                     "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "r"(signal)
                     : "memory");
    }
    __device__ __forceinline__ void expect(int p, int ranks)  // one thread, once a step
    {
        ptx::mbar_arrive_expect_tx(&bar[p], static_cast<uint32_t>(ranks) * sizeof map[0][0]);
    }
    __device__ __forceinline__ void receive(int p, uint32_t parity, int *gave_up) { wait(ptx::smem_u32(&bar[p]), parity, gave_up); }
};

__device__ __forceinline__ f2 apply(f2 h, const float4 &m) { return fma2(pair(m.x, m.y), h, pair(m.z, m.w)); }

// A map with a reset cuts off what is in front of it whatever its value, which
// 0 times infinity would not: its factor is -0, which stays -0 in products with
// decays.  (A product of decays that is too small for 32 bits is +0, and cuts
// nothing off: a NaN stays, an infinity becomes one.)  Values that are not
// finite are rare, so the short form goes first and this one where it gave such.
constexpr float kCut = -0.f;
__device__ __forceinline__ bool is_cut(float factor) { return __float_as_uint(factor) == 0x80000000u; }
__device__ __forceinline__ f2 apply_cut(f2 h, const float4 &m)
{
    const float2 v = halves(apply(h, m));
    return pair(is_cut(m.x) ? m.z : v.x, is_cut(m.y) ? m.w : v.y);
}
__device__ __forceinline__ f2 multiply_cut(f2 f, const float4 &m)
{
    const float2 v = halves(mul2(f, pair(m.x, m.y))), g = halves(f);
    return pair(is_cut(m.x) || is_cut(g.x) ? kCut : v.x, is_cut(m.y) || is_cut(g.y) ? kCut : v.y);
}
// whether all lanes' values are finite
__device__ __forceinline__ bool all_finite(f2 v)
{
    const float2 h = halves(v);
    return __all_sync(0xffffffffu, fabsf(h.x) <= 3.4028234e38f && fabsf(h.y) <= 3.4028234e38f) != 0;
}

// What a step's warps share of one chain (states forwards, messages backwards).
struct Chain {
    float4 map[2][kGatedWarps][32];  // (factor, rest) of each warp's tokens
    float2 last[2][32];              // the value behind a step, of a block that walks alone
    __device__ __forceinline__ void put(int p, int w, int lane, f2 factor, f2 rest)
    {
        const float2 a = halves(factor), b = halves(rest);
        map[p][w][lane] = make_float4(a.x, a.y, b.x, b.y);
    }
    __device__ __forceinline__ float4 get(int p, int w, int lane) const { return map[p][w][lane]; }
};

// The same of states and messages together, whose maps share the factor.
struct TwoChains {
    float4 map[2][kGatedWarps][32];     // (factor, rest of the states)
    float2 message[2][kGatedWarps][32], last[2][32];
    __device__ __forceinline__ void put(int p, int w, int lane, f2 factor, f2 state, f2 m)
    {
        const float2 a = halves(factor), b = halves(state);
        map[p][w][lane] = make_float4(a.x, a.y, b.x, b.y);
        message[p][w][lane] = halves(m);
    }
    __device__ __forceinline__ float4 get(int p, int w, int lane) const
    {
        const float2 f = *reinterpret_cast<const float2 *>(&map[p][w][lane]), m = message[p][w][lane];
        return make_float4(f.x, f.y, m.x, m.y);
    }
};

// Behind the barrier that follows `put`: the value in front of the warp's
// tokens, from the one in front of the step, `carry` (kept current by every
// warp in a cluster, by the last warp alone otherwise).  turn: steps done.
template <bool CLUSTER, bool FORWARD, class C, class E>
__device__ __forceinline__ f2 in_front(C &c, E *ex, int64_t turn, int w, int lane, int rank, int ranks, f2 &carry,
                                       int *gave_up)
{
    const int p = static_cast<int>(turn & 1);
    f2 from = carry;  // in front of the block's tokens
    if constexpr (CLUSTER) {
        f2 factor = both(1.f), rest = both(0.f), signs = 0;  // the block's map
#pragma unroll
        for (int i = 0; i < kGatedWarps; ++i) {
            const float4 m = c.get(p, FORWARD ? i : kGatedWarps - 1 - i, lane);
            factor = mul2(factor, pair(m.x, m.y));
            signs |= pair(m.x, m.y);
            rest = apply(rest, m);
        }
        factor |= signs & both(kCut);  // -0 also where an even number of them are
        if (!all_finite(rest) || !all_finite(factor)) {
            factor = both(1.f), rest = both(0.f);
#pragma unroll 1
            for (int i = 0; i < kGatedWarps; ++i) {
                const float4 m = c.get(p, FORWARD ? i : kGatedWarps - 1 - i, lane);
                factor = multiply_cut(factor, m);
                rest = apply_cut(rest, m);
            }
        }
        if (!has_given_up(gave_up)) {
            if (w < ranks) ex->send(p, rank, w, lane, factor, rest);
            if (threadIdx.x == 0) ex->expect(p, ranks);
        }
        ex->receive(p, static_cast<uint32_t>(turn >> 1) & 1u, gave_up);
        const f2 first = carry;
#pragma unroll 2
        for (int i = 0; i < ranks; ++i) {
            const int q = FORWARD ? i : ranks - 1 - i;
            if (q == rank) from = carry;
            carry = apply(carry, ex->map[p][q][lane]);
        }
        if (!all_finite(carry) || !all_finite(from)) {
            carry = first;
#pragma unroll 1
            for (int i = 0; i < ranks; ++i) {
                const int q = FORWARD ? i : ranks - 1 - i;
                if (q == rank) from = carry;
                carry = apply_cut(carry, ex->map[p][q][lane]);
            }
        }
    } else if (turn > 0) {
        const float2 f = c.last[p ^ 1][lane];
        from = pair(f.x, f.y);
    }
    f2 h = from;
    const int earlier = FORWARD ? w : kGatedWarps - 1 - w;
#pragma unroll 1
    for (int i = 0; i < earlier; ++i) h = apply(h, c.get(p, FORWARD ? i : kGatedWarps - 1 - i, lane));
    if (!all_finite(h)) {
        h = from;
#pragma unroll 1
        for (int i = 0; i < earlier; ++i) h = apply_cut(h, c.get(p, FORWARD ? i : kGatedWarps - 1 - i, lane));
    }
    return h;
}
static_assert(kGatedWarps >= kGatedCluster);  // a warp sends to one block

__host__ __device__ inline int64_t gated_marks(int64_t T) { return (T + RLSCAN_GATED_SCAN_CHECKPOINT - 1) / RLSCAN_GATED_SCAN_CHECKPOINT; }

// Blocks of a cluster that share a row: as many as make the fewest steps one
// after the other, counting the rounds in which clusters of that size become
// resident.  A row split over blocks costs each step an exchange, taken as
// three quarters of a step.  Measured, bfloat16, forward / gradients, us, alone and
// in twos, threes, fours, sixes, eights (gradients at most fours), the rule's in
// brackets:
//   2 x 16384 x 2048, 64 chains    353/874  348/429  216/396  165/[301]  [150]  180
//   2 x 4096 x 4096, 128 chains    148/230  82/[152]  [78]/175  82/157  81  85
//   8 x 2048 x 2048, 256 chains    [67]/[125]  80/153  78/162  72/146  83  83
//   16 x 1024 x 2048, 512 chains   [64]/[126]  68/142  81/167  73/149  85  89
// and of 14 such calls in both types, with 16 to 512 chains, by tiles and by value,
// the rule's size was the fastest or, within 3 us, next to it.
template <class T, int KIND, class K>
inline int gated_cluster(K kernel, int64_t chains, int64_t tokens, int tile, size_t smem, int most = kGatedCluster)
{
    static PerDevice resident[kGatedCluster + 1];
    const int64_t tiles = ceil_div(tokens, tile);
    int best = 1;
    double least = 0;
    for (int c = 1; c <= most; ++c) {
        if (c > 1 && c > tiles) break;
        const int64_t fit = resident[c].get(current_device(), [&] {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(c));
            cfg.blockDim = dim3(32 * kGatedWarps);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = static_cast<unsigned>(c);
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            return ok(cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) ? n : 0;
        });
        if (fit <= 0) continue;
        const double time = static_cast<double>(ceil_div(chains, fit)) * static_cast<double>(ceil_div(tiles, c)) * (c > 1 ? 1.75 : 1.0);
        if (c == 1 || time < least) best = c, least = time;
    }
    return best;
}

// `overlapped`: whether the grid may start while the kernel before it still
// runs.  A grid of several blocks an SM would then go to the SMs that are done
// first, several at once, and end unevenly (4 x 4096 x 4096 float32 forward 194
// us back to back, started behind 170), so only grids of a block an SM do.
template <class K, class... Args>
inline rlscan_status launch_cluster(bool overlapped, K kernel, int64_t grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                                    Args... args)
{
    if (grid > 0x7fffffff) return RLSCAN_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = overlapped && pdl_enabled() ? 1 : 0;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return RLSCAN_ERR_CUDA;
    }
    return RLSCAN_OK;
}

// The kernel for a call's arrays: Tiles where all are device memory (`tiles`)
// and addresses and strides multiples of 16 bytes (tensor maps), Pairs where
// they are multiples of two channels, else Values.
enum class Access { Values, Pairs, Tiles };
template <class T>
inline Access gated_access(std::initializer_list<const rlscan_array3 *> in, std::initializer_list<const void *> out,
                           std::initializer_list<const void *> floats, int64_t N, int64_t T_, int64_t D, bool tiles)
{
    uint64_t bits = 0, wide = 0;
    // coordinates are 32-bit, those of a last block's end too (a negative one would read 0 and write nothing)
    bool plain = tiles && T_ > 0 && T_ < 0x7fffffff - 1024 && N < 0x7fffffff && D < 0x7fffffff - kGatedWidth;
    for (const rlscan_array3 *a : in) {
        const int64_t row = N > 1 ? a->row_stride : 0, token = T_ > 1 ? a->token_stride : 0;
        bits |= reinterpret_cast<uintptr_t>(a->data) | static_cast<uint64_t>(row * sizeof(T)) | static_cast<uint64_t>(token * sizeof(T));
        plain = plain && (N <= 1 || (row > 0 && row < (int64_t{1} << 36))) && (T_ <= 1 || (token > 0 && token < (int64_t{1} << 36)));
    }
    for (const void *p : out) bits |= reinterpret_cast<uintptr_t>(p);
    for (const void *p : floats) wide |= reinterpret_cast<uintptr_t>(p);
    if (D % 2 != 0 || bits % (2 * sizeof(T)) != 0 || wide % 8 != 0) return Access::Values;
    return plain && bits % 16 == 0 && D * sizeof(T) % 16 == 0 ? Access::Tiles : Access::Pairs;
}

// A map of [N,T,D] for boxes of 64 channels x `tokens`
template <class T>
inline bool gated_map(CUtensorMap *m, const void *p, int64_t row_stride, int64_t token_stride, int64_t N, int64_t T_, int64_t D, uint32_t tokens)
{
    constexpr int64_t e = sizeof(T);
    const int64_t token = T_ > 1 ? token_stride * e : D * e, row = N > 1 ? row_stride * e : token * T_;
    const int64_t extents[3] = {D, T_, N}, strides[2] = {token, row};
    const uint32_t box[3] = {kGatedWidth, tokens, 1};
    return encode_map(m, p, sizeof(T) == 2, 3, extents, strides, box, false);
}

}  // namespace seq
}  // namespace rlscan
