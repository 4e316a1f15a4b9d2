// gated_scan.cuh -- what the gated recurrence's kernels share: two channels of
// a token in one register pair, the gates' arithmetic, and the exchange of the
// blocks of a cluster that walk one row together.
#pragma once

#include "sequence.cuh"

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

// A lane's two channels: the first one, whether both are the array's, and the
// ones it reads (a lane past the last channel reads the last ones, and writes
// nothing).
template <bool VEC>
struct Lane {
    int64_t d, from;
    bool on0, on1;
    int apart;
    __device__ __forceinline__ Lane(int64_t block, int lane, int64_t D)
    {
        d = block * kGatedWidth + (VEC ? 2 * lane : lane);
        on0 = d < D;
        on1 = VEC ? on0 : d + 32 < D;
        from = on0 ? d : D - (VEC ? 2 : 1);
        apart = on1 ? 32 : 0;
    }
};

// TOK tokens from t0 on of one array; past `len` (the row's tokens) zeros
template <class T, bool VEC, int TOK>
__device__ __forceinline__ void fetch_tokens(Two<T, VEC> (&v)[TOK], const rlscan_array3 &a, int64_t n, int64_t t0, int64_t len, const Lane<VEC> &l)
{
    const T *p = static_cast<const T *>(a.data) + n * a.row_stride + t0 * a.token_stride + l.from;
    const int64_t step = a.token_stride;
    if (t0 + TOK <= len) {
#pragma unroll
        for (int k = 0; k < TOK; ++k, p += step) v[k].load(p, l.apart);
    } else {
#pragma unroll
        for (int k = 0; k < TOK; ++k) {
            v[k].zero();
            if (t0 + k < len) v[k].load(p + k * step, l.apart);
        }
    }
}

// bit k: a new episode starts at token t0 + k
template <int TOK>
__device__ __forceinline__ uint32_t fetch_resets(const uint8_t *resets, int64_t row, int64_t t0, int64_t len, int lane)
{
    if (resets == nullptr) return 0u;
    uint32_t flag = 0;
    if (lane < TOK && t0 + lane < len) flag = resets[row + t0 + lane];
    return __ballot_sync(0xffffffffu, flag != 0);
}

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

// The lane's two channels of a [D] array of float32
template <bool VEC>
__device__ __forceinline__ f2 load_two(const float *p, bool on0, bool on1)
{
    return pair(on0 ? p[0] : 0.f, on1 ? p[VEC ? 1 : 32] : 0.f);
}

__device__ __forceinline__ f2 neg2(f2 v) { return v ^ 0x8000000080000000ull; }

// What a token's gates give.  a = exp(L) with L = log_decay r; the square of
// the root, 1 - a^2 = -expm1(2 L), is its power series up to the sixth term
// where |2 L| < 1/4 (the first omitted is below 5e-8 of the sum) and 1 - a a
// beyond, where a's own rounding is below 5e-7 of it.  The square stays above
// 2^-100, so that a closed gate (a = 1) gives a finite gradient: the slope of
// the root grows without bound there, but the gate's slope vanishes faster.
struct Gates {
    f2 r, i, a, root;
};
__device__ __forceinline__ Gates gates(f2 gate, f2 input_gate, f2 log_decay, f2 log2_decay, f2 *inverse_root = nullptr)
{
    Gates g;
    g.r = sigmoid(gate);
    g.i = sigmoid(input_gate);
    g.a = decay(g.r, log2_decay);
    const f2 y = mul2(mul2(g.r, log_decay), both(2.f));
    f2 p = fma2(y, both(1.f / 720.f), both(1.f / 120.f));
    p = fma2(p, y, both(1.f / 24.f));
    p = fma2(p, y, both(1.f / 6.f));
    p = fma2(p, y, both(0.5f));
    p = fma2(p, y, both(1.f));
    const float2 near = halves(mul2(p, neg2(y))), far = halves(fma2(neg2(g.a), g.a, both(1.f))), yy = halves(y);
    const float s0 = max_nan(yy.x > -0.25f ? near.x : far.x, kSquareFloor);
    const float s1 = max_nan(yy.y > -0.25f ? near.y : far.y, kSquareFloor);
    const f2 inv = pair(rsqrt_fast(s0), rsqrt_fast(s1));
    g.root = mul2(pair(s0, s1), inv);
    if (inverse_root != nullptr) *inverse_root = inv;
    return g;
}

// ---- the blocks of a cluster -------------------------------------------------
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// a value into the same place of block `rank`'s shared memory
__device__ __forceinline__ void store_to_rank(const void *mine, int rank, float4 v)
{
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(mine)), "r"(rank));
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

__host__ __device__ inline int64_t gated_marks(int64_t T) { return (T + RLSCAN_GATED_SCAN_CHECKPOINT - 1) / RLSCAN_GATED_SCAN_CHECKPOINT; }

// Blocks of a cluster that share a row: as many as make the fewest steps one
// after the other, counting the rounds in which clusters of that size become
// resident.  A row split over blocks costs each step an exchange, taken as a
// quarter of a step.
template <class T, bool VEC, class K>
inline int gated_cluster(K kernel, int64_t chains, int64_t tokens, int tile)
{
    static PerDevice resident[kGatedCluster + 1];
    const int64_t tiles = ceil_div(tokens, tile);
    int best = 1;
    double least = 0;
    for (int c = 1; c <= kGatedCluster; ++c) {
        if (c > 1 && c > tiles) break;
        const int64_t fit = resident[c].get(current_device(), [&] {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(static_cast<unsigned>(c));
            cfg.blockDim = dim3(32 * kGatedWarps);
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
        const double time = static_cast<double>(ceil_div(chains, fit)) * static_cast<double>(ceil_div(tiles, c)) * (c > 1 ? 1.25 : 1.0);
        if (c == 1 || time < least) best = c, least = time;
    }
    return best;
}

template <class K, class... Args>
inline rlscan_status launch_cluster(K kernel, int64_t grid, int threads, int cluster, cudaStream_t stream, Args... args)
{
    if (grid > 0x7fffffff) return RLSCAN_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
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

// Whether pairs of channels are aligned in every array added to the chunk
template <class T>
inline bool gated_pairs(const Chunk &c, int64_t D)
{
    return D % 2 == 0 && c.bits % (2 * sizeof(T)) == 0;
}

}  // namespace seq
}  // namespace rlscan
