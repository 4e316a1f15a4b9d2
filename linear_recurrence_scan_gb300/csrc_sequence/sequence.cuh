// sequence.cuh -- what the state-space layer's kernels share: loads and
// stores of the two activation types, the scalar functions of the gates and
// the time steps, and the internal launchers the C entry points call.
#pragma once

#include <cstddef>
#include <cstdint>

#include <initializer_list>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "params.cuh"
#include "per_device.cuh"
#include "ptx.cuh"
#include "rlscan.h"

namespace rlscan {
namespace seq {

constexpr int kCheckpoint = RLSCAN_SELECTIVE_SCAN_CHECKPOINT;
constexpr int kMaxStates = 128;
constexpr int kMaxTaps = 8;
constexpr int kScaleBlock = 128;      // columns that share one scale of an 8-bit output
constexpr float kE4m3Max = 448.f;
constexpr float kScaleFloor = 0x1p-100f;  // smallest block maximum a scale is made from

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16 from_f<bf16>(float v) { return __float2bfloat16_rn(v); }

// 2^v and 1/v to within 2 units in the last place (PTX ex2.approx, rcp.approx)
__device__ __forceinline__ float exp2_fast(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rcp_fast(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

constexpr float kLog2e = 1.4426950408889634f;

// exp(dt A) from A log2 e.  A state multiplies thousands of these, so their mean
// error counts more than a single one's: ex2.approx lies 0.1 to 0.44 units of
// 2^-24 below the exact value on average for dt A in (-1, 0) (measured against
// 64 bits), which the small constant in the exponent takes back: the gradient
// of A over 8 x 2048 tokens is 0.7e-6 off with it, 1.6e-6 without.
constexpr float kDecayShift = 2.5e-8f;

// 1 / (1 + exp(-v)); 2^x is infinite below v = -88, whose reciprocal is 0
__device__ __forceinline__ float sigmoid(float v) { return rcp_fast(1.f + exp2_fast(-kLog2e * v)); }

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1], with
// log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3, by atanh's power series
// s (1 + s^2/3 + s^4/5 + ...): its first omitted term, s^14/15, is below
// 1.4e-8 of the sum.  (log(1 + e) itself would lose the small time steps,
// which are e for large negative v, to the rounding of 1 + e.)
__device__ __forceinline__ float softplus(float v)
{
    const float e = exp2_fast(-kLog2e * fabsf(v));
    const float s = e * rcp_fast(2.f + e);
    const float q = s * s;
    float p = 1.f / 13.f;
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return fmaf(2.f * s, p, fmaxf(v, 0.f));
}

// V neighbouring values as they are stored, in whole registers: a load into
// them can stay in flight until a value is looked at.
template <class T, int V>
struct Words {
    static constexpr int BYTES = V * static_cast<int>(sizeof(T)), N = (BYTES + 3) / 4;
    uint32_t w[N];
    __device__ __forceinline__ float operator[](int i) const
    {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        return __uint_as_float(i % 2 == 0 ? w[i / 2] << 16 : w[i / 2] & 0xffff0000u);
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ void load(const T *p)  // aligned to BYTES (or 16)
    {
        if constexpr (BYTES % 16 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const uint4 q = reinterpret_cast<const uint4 *>(p)[i / 4];
                w[i] = q.x;
                w[i + 1] = q.y;
                w[i + 2] = q.z;
                w[i + 3] = q.w;
            }
        } else if constexpr (BYTES == 8) {
            const uint2 q = *reinterpret_cast<const uint2 *>(p);
            w[0] = q.x;
            w[1] = q.y;
        } else if constexpr (BYTES == 4) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            static_assert(BYTES == 2);
            asm volatile("ld.u16 %0, [%1];" : "=r"(w[0]) : "l"(p) : "memory");
        }
    }
    __device__ __forceinline__ void store(T *p) const
    {
        if constexpr (BYTES % 16 == 0) {
#pragma unroll
            for (int i = 0; i < N; i += 4)
                reinterpret_cast<uint4 *>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        } else if constexpr (BYTES == 8) {
            *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else if constexpr (BYTES == 4) {
            *reinterpret_cast<uint32_t *>(p) = w[0];
        } else {
            *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(w[0]);
        }
    }
    // rounds values 2 i and 2 i + 1 (one value: 2 i alone) into their words
    __device__ __forceinline__ void set(int i, float lo, float hi)
    {
        if constexpr (sizeof(T) == 4) {
            w[2 * i] = __float_as_uint(lo);
            if (2 * i + 1 < V) w[2 * i + 1 < N ? 2 * i + 1 : 0] = __float_as_uint(hi);
        } else {
            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
};

// a byte in a whole register
__device__ __forceinline__ uint32_t load_byte(const uint8_t *p)
{
    uint32_t v;
    asm volatile("ld.u8 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// `a` where the mask is all ones, `b` where it is 0.  Bit by bit: a ternary
// around an expensive `a` becomes a branch, which would keep the work of
// neighbouring tokens from overlapping.
__device__ __forceinline__ float choose(uint32_t mask, float a, float b)
{
    return __uint_as_float((__float_as_uint(a) & mask) | (__float_as_uint(b) & ~mask));
}

// Sums of v[0..N) over the lanes that differ in the bits HI .. LO of their
// number, shared out: while values are left, each bit halves them (a lane
// keeps one half), after that lanes hold the same sums.  Returns the index of
// the first value kept.
template <int N, int HI, int LO>
__device__ __forceinline__ int scatter_sums(float *v, int lane)
{
    if constexpr (HI < LO || HI == 0) {
        return 0;
    } else if constexpr (N == 1) {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], HI);
        return scatter_sums<1, HI / 2, LO>(v, lane);
    } else {
        constexpr int H = N / 2;
        const bool upper = (lane & HI) != 0;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float give = upper ? v[i] : v[i + H], keep = upper ? v[i + H] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, HI);
        }
        return scatter_sums<H, HI / 2, LO>(v, lane) + (upper ? H : 0);
    }
}

// quotient and remainder; in 32 bits where the numbers fit (a 64-bit division
// is over a hundred instructions, more than all else a token's call needs)
struct Division {
    int64_t q, r;
};
__device__ __forceinline__ Division divide(int64_t i, int64_t n)
{
    if ((static_cast<uint64_t>(i) | static_cast<uint64_t>(n)) >> 32 == 0) {
        const uint32_t q = static_cast<uint32_t>(i) / static_cast<uint32_t>(n);
        return {q, static_cast<uint32_t>(i) - q * static_cast<uint32_t>(n)};
    }
    return {i / n, i % n};
}

// tokens of row n, clamped to the array
__device__ __forceinline__ int64_t row_length(const int32_t *lengths, int64_t n, int64_t T)
{
    if (lengths == nullptr) return T;
    const int64_t len = lengths[n];
    return len < 0 ? 0 : (len < T ? len : T);
}

// Blocks of rows of unlike lengths.  Blocks that walk whole rows take the time
// of their row, and half as long again where they share an SM, so the order
// matters in which the GPU takes them: the longest rows first.  A grid between
// one and two blocks an SM fills every SM once before any twice; there the
// second blocks come with the shortest rows first, beside the longest.
// Measured (ragged, rows as they are / longest first / with the second blocks
// turned round): scan 8 x 4096 x 4096 640, 588, 578 us, 16 x 1024 x 2048 158,
// 148, 138; 24 x 1024 x 4096 398, 332; gradients 24 x 512 x 2048 with the
// forward pass 753, 675.  With 200 rows finding the order cost more than it
// gave (96 tokens: 142, 160), with 64 it did not (512 tokens: 228, 214).
constexpr int kOrderedRows = 64;
__device__ __forceinline__ int64_t by_length(const int32_t *lengths, int N, int64_t blocks, int64_t sms, int *smem)
{
    const int64_t grid = N * blocks, place = blockIdx.x;
    int64_t rank = place;
    if (grid <= 2 * sms && place >= sms) rank = grid - 1 - (place - sms);
    const Division at = divide(rank, blocks);
    for (int i = threadIdx.x; i < N; i += blockDim.x) smem[i] = lengths[i];
    __syncthreads();
    for (int i = threadIdx.x; i < N; i += blockDim.x) {
        const int own = smem[i];
        int longer = 0;
#pragma unroll 8
        for (int j = 0; j < N; ++j) longer += smem[j] > own || (smem[j] == own && j < i);
        if (longer == at.q) smem[N] = i;
    }
    __syncthreads();
    const int row = static_cast<int>(__reduce_max_sync(0xffffffffu, smem[N]));  // the same value: into a uniform register
    __syncthreads();
    return row * blocks + at.r;
}

// ---- pairs of float32 in one register pair (PTX f32x2) -----------------------
// The pipe runs 128 float32 lanes a clock and SM either way; a pair halves the
// instructions, which these kernels run out of first (measured: an
// exponential with four multiply-adds a value, 31.5 values/clk/SM in pairs,
// 24.7 one by one).
using f2 = unsigned long long;

__device__ __forceinline__ f2 pair(float lo, float hi)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 halves(f2 v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 both(float v) { return pair(v, v); }
__device__ __forceinline__ f2 exp2_fast(f2 v)
{
    const float2 h = halves(v);
    return pair(exp2_fast(h.x), exp2_fast(h.y));
}
__device__ __forceinline__ float decay(float dt, float A2) { return exp2_fast(fmaf(dt, A2, kDecayShift)); }
__device__ __forceinline__ f2 decay(f2 dt, f2 A2) { return exp2_fast(fma2(dt, A2, both(kDecayShift))); }
__device__ __forceinline__ f2 rcp_fast(f2 v)
{
    const float2 h = halves(v);
    return pair(rcp_fast(h.x), rcp_fast(h.y));
}
__device__ __forceinline__ f2 sigmoid(f2 v) { return rcp_fast(add2(both(1.f), exp2_fast(mul2(v, both(-kLog2e))))); }

// softplus of both halves, as softplus(float)
__device__ __forceinline__ f2 softplus(f2 v)
{
    const float2 h = halves(v);
    const f2 e = exp2_fast(mul2(pair(fabsf(h.x), fabsf(h.y)), both(-kLog2e)));
    const f2 s = mul2(e, rcp_fast(add2(both(2.f), e)));
    const f2 q = mul2(s, s);
    f2 p = both(1.f / 13.f);
    p = fma2(p, q, both(1.f / 11.f));
    p = fma2(p, q, both(1.f / 9.f));
    p = fma2(p, q, both(1.f / 7.f));
    p = fma2(p, q, both(1.f / 5.f));
    p = fma2(p, q, both(1.f / 3.f));
    p = fma2(p, q, both(1.f));
    return fma2(add2(s, s), p, pair(fmaxf(h.x, 0.f), fmaxf(h.y, 0.f)));
}

// ---- loads from shared memory that stores do not hold up --------------------
// To the compiler these depend on their address alone, so it may move them
// over stores, which plain loads of possibly the same memory have to wait
// for.  `anchor` gives an address that it takes for new: loads through it
// stay behind the anchor, and it stays behind the barrier in front of it.
__device__ __forceinline__ uint32_t anchor(const void *p)
{
    uint32_t r;
    asm volatile("mov.u32 %0, %1;" : "=r"(r) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))) : "memory");
    return r;
}
__device__ __forceinline__ void load_pairs(f2 &a, f2 &b, uint32_t at)
{
    asm("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(at));
}
__device__ __forceinline__ float load_value(uint32_t at, float)
{
    float v;
    asm("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ float load_value(uint32_t at, bf16)
{
    uint32_t v;
    asm("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(at));
    return __uint_as_float(v << 16);
}

// ---- asynchronous copies into shared memory ---------------------------------
// `bytes` (0..16, rest zero-filled) of a 16-byte chunk, or 4 bytes
__device__ __forceinline__ void copy16(void *dst, const void *src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy4(void *dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy8(void *dst, const void *src, int bytes)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// A tile of ROWS tokens x WIDTH values in shared memory (rows PITCH bytes
// apart) from rows `row_bytes` apart at `src`: `rows` of them hold tokens and
// `width` values of each are inside the array; the rest of the tile becomes
// 0.  CHUNK is the unit of the copies: 16 or 4 bytes, asynchronous, where
// addresses and strides are multiples of it, or 0 for single values.
template <class T, int ROWS, int WIDTH, int PITCH, int CHUNK, int THREADS>
__device__ __forceinline__ void load_tile(char *dst, const T *src, int64_t stride, int rows, int width)
{
    if constexpr (CHUNK == 0) {
        constexpr int N = ROWS * WIDTH;
#pragma unroll 8
        for (int i = threadIdx.x; i < N; i += THREADS) {
            const int r = i / WIDTH, c = i % WIDTH;
            T v = from_f<T>(0.f);
            if (r < rows && c < width) v = src[r * stride + c];
            *reinterpret_cast<T *>(dst + r * PITCH + c * sizeof(T)) = v;
        }
    } else {
        constexpr int PER = CHUNK / static_cast<int>(sizeof(T)), CPR = WIDTH / PER, N = ROWS * CPR;
        static_assert(WIDTH % PER == 0 && PITCH % CHUNK == 0 && (THREADS % CPR == 0 || CPR % THREADS == 0));
        // a thread keeps its column and steps over rows (or, of wide rows, over columns)
        constexpr int STEP = THREADS >= CPR ? THREADS / CPR : 1, ACROSS = THREADS >= CPR ? 1 : CPR / THREADS;
        const int r0 = threadIdx.x / CPR, c0 = threadIdx.x % CPR * PER;
        if (N < THREADS && threadIdx.x >= N) return;
        const T *from = src + r0 * stride + c0;
        char *to = dst + r0 * PITCH + c0 * static_cast<int>(sizeof(T));
#pragma unroll
        for (int r = 0; r < ROWS; r += STEP) {
#pragma unroll
            for (int x = 0; x < ACROSS; ++x) {
                const int have = (width - c0 - x * THREADS * PER) * static_cast<int>(sizeof(T));
                const int bytes = r0 + r < rows && have > 0 ? (have < CHUNK ? have : CHUNK) : 0;
                const T *at = bytes > 0 ? from + x * THREADS * PER : src;
                char *into = to + r * PITCH + x * THREADS * PER * static_cast<int>(sizeof(T));
                if constexpr (CHUNK == 16)
                    copy16(into, at, bytes);
                else
                    copy4(into, at, bytes);
            }
            from += STEP * stride;
        }
    }
}

// The chunk that fits a set of arrays: `add` each one's address and strides.
struct Chunk {
    uint64_t bits = 0;
    void add(const void *p, int64_t row_stride, int64_t token_stride, int size)
    {
        bits |= reinterpret_cast<uintptr_t>(p) | static_cast<uint64_t>(row_stride) * size |
                static_cast<uint64_t>(token_stride) * size;
    }
    int size() const { return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 0; }
};

// Launch that lets the kernel's start overlap the end of the kernel before
// it; every such kernel begins with ptx::pdl_wait_prerequisites().
template <class K, class... Args>
inline rlscan_status launch(bool overlapped, K kernel, int64_t grid, int threads, size_t smem, cudaStream_t stream,
                            Args... args)
{
    if (grid > 0x7fffffff) return RLSCAN_ERR_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = overlapped && pdl_enabled() ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return RLSCAN_ERR_CUDA;
    }
    return RLSCAN_OK;
}

template <class K, class... Args>
inline rlscan_status launch_overlapped(K kernel, int64_t grid, int threads, size_t smem, cudaStream_t stream,
                                       Args... args)
{
    return launch(true, kernel, grid, threads, smem, stream, args...);
}

inline bool ok(cudaError_t e)
{
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess;
}

// The current device (-1 on an error).
inline int current_device()
{
    int dev = 0;
    return ok(cudaGetDevice(&dev)) ? dev : -1;
}

// The device's SM count (0 on an error).
inline int sm_count()
{
    static PerDevice counts;
    const int dev = current_device();
    if (dev < 0) return 0;
    return counts.get(dev, [&] {
        int n = 0;
        return ok(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) ? n : 0;
    });
}

// Lets `kernel` have `bytes` of dynamic shared memory on the current device;
// `raised` is the kernel's own.
template <class K>
inline bool raise_smem(PerDevice &raised, K kernel, size_t bytes)
{
    if (bytes <= 48 * 1024) return true;
    return raised.get(current_device(), [&] {
        return ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes))) ? 1 : 0;
    }) > 0;
}

// SMs for by_length, or 0 where the order of the rows is left alone
inline int64_t order_sms(const int32_t *lengths, int64_t N, int64_t blocks, int64_t chunks)
{
    const int64_t sms = sm_count() > 0 ? sm_count() : 152;
    return lengths != nullptr && N > 1 && N <= kOrderedRows && chunks == 1 && N * blocks > sms ? sms : 0;
}

// Whether the second blocks are to come after every SM has its first.  Started
// while the kernel before it still runs, such a grid goes in pairs to the SMs
// that are done first (gradients of ragged 8 x 2048 x 4096 with the forward
// pass: 1885 us, started behind it 1754).
inline bool spread_out(int64_t grid, int64_t sms) { return sms > 0 && grid <= 2 * sms; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Lanes of a channel's states, four states each: 1, 2, 4, ... 32.
inline int state_lanes(int64_t S)
{
    int lanes = 1;
    while (4 * lanes < S) lanes *= 2;
    return lanes;
}

rlscan_status launch_selective_scan(const rlscan_selective_scan_args &a, void *y, float *final_state,
                                    float *checkpoints, void *ws, cudaStream_t s);
size_t selective_scan_workspace(const rlscan_selective_scan_args &a);
// The gradient's message behind each chunk of tokens (states [N][chunks][D][S]);
// spans [N][chunks][D] and cuts [N][chunks] are scratch.
rlscan_status launch_back_states(const rlscan_selective_scan_args &a, const rlscan_array3 &grad_y, const float *grad_final,
                                 int64_t chunk, int64_t chunks, float *states, float *spans, uint8_t *cuts,
                                 cudaStream_t s);
rlscan_status launch_selective_scan_step(const rlscan_selective_scan_args &a, float *state, int64_t P,
                                         const int32_t *slots, void *y, cudaStream_t s);
rlscan_status launch_selective_scan_backward(const rlscan_selective_scan_args &a, const rlscan_array3 &grad_y,
                                             const float *grad_final_state, const float *checkpoints,
                                             const rlscan_selective_scan_grads &g, void *ws, cudaStream_t s);
size_t selective_scan_backward_workspace(const rlscan_selective_scan_args &a);
rlscan_status launch_causal_conv(const rlscan_causal_conv_args &a, void *y, void *final_state, cudaStream_t s);
rlscan_status launch_causal_conv_step(const rlscan_causal_conv_args &a, void *state, int64_t P, const int32_t *slots,
                                      void *y, cudaStream_t s);
rlscan_status launch_causal_conv_backward(const rlscan_causal_conv_args &a, const rlscan_array3 &grad_y,
                                          const void *grad_final_state, void *grad_x, float *grad_weight,
                                          float *grad_bias, void *grad_initial_state, void *ws, cudaStream_t s);
size_t causal_conv_backward_workspace(const rlscan_causal_conv_args &a);

struct NormArgs {
    const void *x, *residual;
    int64_t x_stride, residual_stride;
    const float *weight;
    int64_t M, D;
    float eps;
    void *y;
    float *scales;
    void *residual_out;
    bool vec = false;  // set by the launcher
};
rlscan_status launch_add_rms_norm(const NormArgs &a, bool bf16_io, bool bf16_residual, cudaStream_t s);

struct NormGradArgs {
    const void *grad_y, *h, *grad_residual;
    int64_t grad_y_stride, h_stride, grad_residual_stride;
    const float *weight;
    int64_t M, D;
    float eps;
    void *grad_x, *grad_h;
    float *grad_weight;
    bool vec = false;  // set by the launcher
};
rlscan_status launch_add_rms_norm_backward(const NormGradArgs &a, bool bf16_io, bool bf16_h, void *ws, cudaStream_t s);
size_t add_rms_norm_backward_workspace(int64_t M, int64_t D);

// (`on_device`: whether all [N,T,D] arrays are device memory, which bulk copies are for)
rlscan_status launch_gated_scan(const rlscan_gated_scan_args &a, void *y, float *final_state, float *checkpoints,
                                bool on_device, cudaStream_t s);
rlscan_status launch_gated_scan_step(const rlscan_gated_scan_args &a, float *state, int64_t P, const int32_t *slots,
                                     void *y, cudaStream_t s);
rlscan_status launch_gated_scan_backward(const rlscan_gated_scan_args &a, const rlscan_array3 &grad_y,
                                         const float *grad_final_state, const float *checkpoints,
                                         const rlscan_gated_scan_grads &g, void *ws, bool on_device, cudaStream_t s);
size_t gated_scan_backward_workspace(const rlscan_gated_scan_args &a);
rlscan_status gated_scan_status(cudaStream_t s);           // whether a wait ran out
rlscan_status gated_scan_backward_status(cudaStream_t s);

// Sums over parts, several in one launch:
// out[i] = sum over w < parts of part[w * pitch + i], i < m, in a fixed order.
struct SumJobs {
    static constexpr int kMost = 5, kColumns = 32;  // columns of a block
    struct Job {
        const float *part;
        int64_t parts, pitch, m;
        void *out;
        bool bf16_out, vec;  // vec: columns in whole, aligned units of four
        int64_t first;       // its first block
    } job[kMost];
    int count = 0;
    int64_t blocks = 0;
    void add(const float *part, int64_t parts, int64_t pitch, int64_t m, void *out, bool bf16_out)
    {
        if (m == 0) return;
        const bool vec = m % 4 == 0 && pitch % 4 == 0 && (reinterpret_cast<uintptr_t>(part) & 15u) == 0;
        job[count++] = Job{part, parts, pitch, m, out, bf16_out, vec, blocks};
        blocks += (m + kColumns - 1) / kColumns;
    }
};
rlscan_status launch_sums(const SumJobs &jobs, cudaStream_t s);

inline rlscan_status launched()
{
    return cudaGetLastError() == cudaSuccess ? RLSCAN_OK : RLSCAN_ERR_CUDA;
}

}  // namespace seq
}  // namespace rlscan
