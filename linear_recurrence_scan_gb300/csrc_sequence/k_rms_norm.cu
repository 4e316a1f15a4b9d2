// k_rms_norm.cu -- root-mean-square norm with the residual's addition, its
// 8-bit output with a scale for each 128 columns, and its gradients.
//
// One pass: a warp or a block takes a row and keeps it in registers (two
// chunks of 16 bytes of x a thread) between the sum of squares and the
// outputs.  Bytes bound it: 32768 x 4096 bf16 with 8-bit output 143 us,
// 6.6 TB/s; 16384 x 2560 bf16 with gradients 113 us, 5.9 TB/s.
#include <cuda_fp8.h>

#include "sequence.cuh"

namespace rlscan {
namespace seq {
namespace {

// Registers of a thread.  Measured (bf16): forward 32768 x 4096 to 8 bits
// with 64: 154 us, 80: 152, 104: 175; gradients 16384 x 2560 with the
// forward pass with 80: 176 us, 104: 136, 128: 133.
constexpr int kNormRegisters = 80, kGradRegisters = 128;
constexpr int kChunks = 2;  // chunks of a thread
constexpr int kMostThreads = 512;
constexpr int kRowWarps = 4;  // rows of a block whose rows take a warp each

template <class T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

// Threads of a row: whole warps, two chunks a thread; 0 if the row is too long.
template <class T>
int row_threads(int64_t D)
{
    const int64_t t = (D + kChunks * kVec<T> * 32 - 1) / (kChunks * kVec<T> * 32) * 32;
    return t <= kMostThreads ? static_cast<int>(t) : 0;
}

// Where a thread's values lie in its row.  VEC: V neighbours, chunk j at
// column (j threads + tid) V.  Otherwise single values, neighbouring lanes
// side by side: value i of chunk j at column (j V + i) threads + tid.
template <bool VEC, int V>
struct Columns {
    int tid, threads, D;
    __device__ __forceinline__ int first(int j) const { return VEC ? (j * threads + tid) * V : j * V * threads + tid; }
    __device__ __forceinline__ int at(int j, int i) const { return VEC ? first(j) + i : first(j) + i * threads; }
};

// The values of a chunk as loaded: V side by side, or a register each (put
// together at once they would wait for their loads at once).
template <bool VEC, class E, int V>
struct Held {
    Words<E, VEC ? V : 1> v[VEC ? 1 : V];
    __device__ __forceinline__ float operator[](int i) const
    {
        if constexpr (VEC) return v[0][i];
        return v[VEC ? 0 : i][0];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (VEC ? 1 : V); ++i) v[i].zero();
    }
};

// chunk j of a row, 0 past its end
template <bool VEC, class E, int V>
__device__ __forceinline__ void load_chunk(Held<VEC, E, V> &r, const E *p, const Columns<VEC, V> &c, int j)
{
    r.zero();
#pragma unroll
    for (int i = 0; i < (VEC ? 1 : V); ++i)
        if (c.at(j, i) < c.D) r.v[i].load(p + c.at(j, i));
}

template <bool VEC, class E, int V>
__device__ __forceinline__ void store_chunk(E *p, const float *v, const Columns<VEC, V> &c, int j)
{
    if constexpr (VEC) {
        Words<E, V> r;
#pragma unroll
        for (int i = 0; i < V; i += 2) r.set(i / 2, v[i], v[i + 1]);
        if (c.first(j) < c.D) r.store(p + c.first(j));
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (c.at(j, i) < c.D) p[c.at(j, i)] = from_f<E>(v[i]);
    }
}

// Sums of v[0..N) over the threads of a row (WARP: a warp's, else the
// block's), the same bits in each.  `flip` alternates, so that one barrier
// suffices: a half is written again only after the next call's barrier.
template <bool WARP, int N>
__device__ __forceinline__ void row_sums(float *v, float (*scratch)[32][N], int flip)
{
#pragma unroll
    for (int m = 16; m > 0; m /= 2)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
    if constexpr (!WARP) {
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) scratch[flip][threadIdx.x / 32][i] = v[i];
        __syncthreads();
        const int warps = blockDim.x / 32;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.f;
        for (int w = 0; w < warps; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += scratch[flip][w][i];
    }
}

// A block walks rows in strides of the grid: the next row's loads are in
// flight while this row's sum and outputs are made.
template <class T, class R, bool WARP, bool VEC>
__global__ void __maxnreg__(VEC ? kNormRegisters : 128) norm_kernel(const __grid_constant__ NormArgs a)
{
    constexpr int V = kVec<T>;
    __shared__ float scratch[2][32][1];
    __shared__ uint32_t tops[WARP ? kRowWarps : 1][VEC ? 1 : kMostThreads * kChunks * V / kScaleBlock];
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int threads = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x, D = static_cast<int>(a.D);
    const int64_t rows = WARP ? kRowWarps : 1, step = gridDim.x * rows;
    int64_t row = blockIdx.x * rows + (WARP ? threadIdx.x / 32 : 0);
    const Columns<VEC, V> col{tid, threads, D};
    const bool summed = a.residual != nullptr;
    Held<VEC, T, V> x[kChunks];
    Held<VEC, R, V> r[kChunks];
    auto load = [&](int64_t at) {
        const T *xp = static_cast<const T *>(a.x) + at * a.x_stride;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) load_chunk<VEC>(x[j], xp, col, j);
        if (summed) {
            const R *rp = static_cast<const R *>(a.residual) + at * a.residual_stride;
#pragma unroll
            for (int j = 0; j < kChunks; ++j) load_chunk<VEC>(r[j], rp, col, j);
        }
    };
    Held<VEC, float, V> w[kChunks];
    if (row < a.M) load(row);
#pragma unroll
    for (int j = 0; j < kChunks; ++j) load_chunk<VEC>(w[j], a.weight, col, j);
    const float over = 1.f / static_cast<float>(D);
    const int blocks = (D + kScaleBlock - 1) / kScaleBlock;
    for (int flip = 0; row < a.M; row += step, flip ^= 1) {
        float h[kChunks][V], ss[1] = {0.f};
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                h[j][i] = x[j][i];
                if (summed) h[j][i] += r[j][i];
                ss[0] = fmaf(h[j][i], h[j][i], ss[0]);
            }
            if (summed) store_chunk<VEC>(static_cast<R *>(a.residual_out) + row * a.D, h[j], col, j);
        }
        if (row + step < a.M) load(row + step);
        row_sums<WARP, 1>(ss, scratch, flip);
        const float inv = rsqrtf(fmaf(ss[0], over, a.eps));
#pragma unroll
        for (int j = 0; j < kChunks; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) h[j][i] = h[j][i] * inv * w[j][i];
        if (a.scales == nullptr) {
#pragma unroll
            for (int j = 0; j < kChunks; ++j) store_chunk<VEC>(static_cast<T *>(a.y) + row * a.D, h[j], col, j);
            continue;
        }
        uint8_t *y = static_cast<uint8_t *>(a.y) + row * a.D;
        float *scales = a.scales + row * blocks;
        // the bits of |v| order like |v|, with infinities and NaN on top
        auto scale_of = [](uint32_t top) {
            return top < 0x7f800000u ? fmaxf(__uint_as_float(top), kScaleFloor) / kE4m3Max : __int_as_float(0x7fffffff);
        };
        if constexpr (VEC) {
            // kScaleBlock / V neighbouring lanes hold a block of columns
#pragma unroll
            for (int j = 0; j < kChunks; ++j) {
                const int c = col.first(j);
                uint32_t top = 0;
#pragma unroll
                for (int i = 0; i < V; ++i) top = max(top, __float_as_uint(h[j][i]) & 0x7fffffffu);
#pragma unroll
                for (int m = kScaleBlock / V / 2; m > 0; m /= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, m));
                const float scale = scale_of(top), back = 1.f / scale;
                uint32_t q[V / 4];
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(h[j][i] * back, h[j][i + 1] * back),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(h[j][i + 2] * back, h[j][i + 3] * back),
                                                                 __NV_SATFINITE, __NV_E4M3);
                    q[i / 4] = lo | hi << 16;
                }
                if (c < D) {
                    if constexpr (V == 8)
                        *reinterpret_cast<uint2 *>(y + c) = make_uint2(q[0], q[1]);
                    else
                        *reinterpret_cast<uint32_t *>(y + c) = q[0];
                    if (c % kScaleBlock == 0) scales[c / kScaleBlock] = scale;
                }
            }
        } else {
            // a warp's value lies in one block of columns (threads are whole
            // warps, 32 divides 128); the block's largest is kept in shared
            // memory (a maximum does not depend on the order)
            uint32_t *top = tops[WARP ? threadIdx.x / 32 : 0];
            auto rows_barrier = [] {
                if constexpr (WARP)
                    __syncwarp();
                else
                    __syncthreads();
            };
            rows_barrier();  // the row before has been read
            for (int b = tid; b < blocks; b += threads) top[b] = 0u;
            rows_barrier();
#pragma unroll
            for (int j = 0; j < kChunks; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = col.at(j, i), b = (c - (tid & 31)) / kScaleBlock;
                    const uint32_t v = __reduce_max_sync(0xffffffffu, c < D ? __float_as_uint(h[j][i]) & 0x7fffffffu : 0u);
                    if ((tid & 31) == 0 && b < blocks) atomicMax(&top[b], v);
                }
            rows_barrier();
            for (int b = tid; b < blocks; b += threads) {
                const float scale = scale_of(top[b]);
                scales[b] = scale;
                top[b] = __float_as_uint(1.f / scale);
            }
            rows_barrier();
#pragma unroll
            for (int j = 0; j < kChunks; ++j)
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const int c = col.at(j, i);
                    if (c < D)
                        y[c] = __nv_cvt_float_to_fp8(h[j][i] * __uint_as_float(top[c / kScaleBlock]), __NV_SATFINITE,
                                                     __NV_E4M3);
                }
        }
    }
}

// Rows of any length: a block of 1024 threads walks the row twice.
constexpr int kLongThreads = 1024;

template <class T, class R>
__global__ void __launch_bounds__(kLongThreads) long_norm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float scratch[2][32][1];
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + row * a.x_stride;
    const R *r = a.residual != nullptr ? static_cast<const R *>(a.residual) + row * a.residual_stride : nullptr;
    auto sum_at = [&](int64_t c) { return to_f(x[c]) + (r != nullptr ? to_f(r[c]) : 0.f); };
    float ss[1] = {0.f};
    for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) {
        const float h = sum_at(c);
        ss[0] = fmaf(h, h, ss[0]);
        if (r != nullptr) static_cast<R *>(a.residual_out)[row * a.D + c] = from_f<R>(h);
    }
    row_sums<false, 1>(ss, scratch, 0);
    const float inv = rsqrtf(ss[0] / static_cast<float>(a.D) + a.eps);
    if (a.scales == nullptr) {
        for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads)
            static_cast<T *>(a.y)[row * a.D + c] = from_f<T>(sum_at(c) * inv * a.weight[c]);
        return;
    }
    const int64_t blocks = (a.D + kScaleBlock - 1) / kScaleBlock;
    const int lane = threadIdx.x & 31;
    for (int64_t b = threadIdx.x / 32; b < blocks; b += kLongThreads / 32) {
        float v[kScaleBlock / 32], top = 0.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < kScaleBlock / 32; ++i) {
            const int64_t c = b * kScaleBlock + i * 32 + lane;
            v[i] = c < a.D ? sum_at(c) * inv * a.weight[c] : 0.f;
            top = fmaxf(top, fabsf(v[i]));
            bad = bad || !(fabsf(v[i]) <= 3.402823466e38f);
        }
#pragma unroll
        for (int m = 16; m > 0; m /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        bad = __any_sync(0xffffffffu, bad);
        const float scale = bad ? __int_as_float(0x7fffffff) : fmaxf(top, kScaleFloor) / kE4m3Max;
#pragma unroll
        for (int i = 0; i < kScaleBlock / 32; ++i) {
            const int64_t c = b * kScaleBlock + i * 32 + lane;
            if (c < a.D)
                static_cast<__nv_fp8_storage_t *>(a.y)[row * a.D + c] =
                    __nv_cvt_float_to_fp8(v[i] / scale, __NV_SATFINITE, __NV_E4M3);
        }
        if (lane == 0) a.scales[row * blocks + b] = scale;
    }
}

// Gradients: dh = r (gn - n mean(gn n)) + grad_residual.  Rows as above; a
// row's threads keep their sums of dy n in registers and write them as one
// row of `part` at the end.
template <class T, class R, bool WARP, bool VEC>
__global__ void __maxnreg__(kGradRegisters)
    norm_grad_kernel(const __grid_constant__ NormGradArgs a, float *part)
{
    constexpr int V = kVec<T>;
    __shared__ float scratch[2][32][2];
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int threads = WARP ? 32 : blockDim.x, tid = WARP ? threadIdx.x & 31 : threadIdx.x, D = static_cast<int>(a.D);
    const int64_t rows = WARP ? kRowWarps : 1, step = gridDim.x * rows;
    const int64_t slot = blockIdx.x * rows + (WARP ? threadIdx.x / 32 : 0);
    int64_t row = slot;
    const Columns<VEC, V> col{tid, threads, D};
    Held<VEC, T, V> gy[kChunks];
    Held<VEC, R, V> hr[kChunks], gr[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) gr[j].zero();
    auto load = [&](int64_t at) {
        const T *gp = static_cast<const T *>(a.grad_y) + at * a.grad_y_stride;
        const R *hp = static_cast<const R *>(a.h) + at * a.h_stride;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            load_chunk<VEC>(hr[j], hp, col, j);
            load_chunk<VEC>(gy[j], gp, col, j);
        }
        if (a.grad_residual != nullptr) {
            const R *rp = static_cast<const R *>(a.grad_residual) + at * a.grad_residual_stride;
#pragma unroll
            for (int j = 0; j < kChunks; ++j) load_chunk<VEC>(gr[j], rp, col, j);
        }
    };
    if (row < a.M) load(row);
    Held<VEC, float, V> w[kChunks];
#pragma unroll
    for (int j = 0; j < kChunks; ++j) load_chunk<VEC>(w[j], a.weight, col, j);
    float dw[kChunks][V];
#pragma unroll
    for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) dw[j][i] = 0.f;
    const float over = 1.f / static_cast<float>(D);
    for (int flip = 0; row < a.M; row += step, flip ^= 1) {
        Held<VEC, T, V> g0[kChunks];
        Held<VEC, R, V> h0[kChunks], r0[kChunks];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            g0[j] = gy[j];
            h0[j] = hr[j];
            r0[j] = gr[j];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s[0] = fmaf(h0[j][i], h0[j][i], s[0]);
                s[1] = fmaf(g0[j][i] * w[j][i], h0[j][i], s[1]);
            }
        }
        if (row + step < a.M) load(row + step);
        row_sums<WARP, 2>(s, scratch, flip);
        const float inv = rsqrtf(fmaf(s[0], over, a.eps)), mean = s[1] * inv * over;
#pragma unroll
        for (int j = 0; j < kChunks; ++j) {
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float nv = h0[j][i] * inv, gv = g0[j][i];
                dw[j][i] = fmaf(gv, nv, dw[j][i]);
                v[i] = fmaf(inv, fmaf(-nv, mean, gv * w[j][i]), r0[j][i]);
            }
            store_chunk<VEC>(static_cast<T *>(a.grad_x) + row * a.D, v, col, j);
            if (a.grad_h != nullptr) store_chunk<VEC>(static_cast<R *>(a.grad_h) + row * a.D, v, col, j);
        }
    }
    if (part != nullptr) {
#pragma unroll
        for (int j = 0; j < kChunks; ++j) store_chunk<VEC>(part + slot * a.D, dw[j], col, j);
    }
}

template <class T, class R>
__global__ void __launch_bounds__(kLongThreads) long_norm_grad_kernel(const __grid_constant__ NormGradArgs a, float *part)
{
    __shared__ float scratch[2][32][2];
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    for (int64_t row = blockIdx.x, flip = 0; row < a.M; row += gridDim.x, flip ^= 1) {
        const T *gy = static_cast<const T *>(a.grad_y) + row * a.grad_y_stride;
        const R *h = static_cast<const R *>(a.h) + row * a.h_stride;
        const R *gr = a.grad_residual != nullptr ? static_cast<const R *>(a.grad_residual) + row * a.grad_residual_stride
                                                 : nullptr;
        float s[2] = {0.f, 0.f};
        for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) {
            const float hv = to_f(h[c]);
            s[0] = fmaf(hv, hv, s[0]);
            s[1] = fmaf(to_f(gy[c]) * a.weight[c], hv, s[1]);
        }
        row_sums<false, 2>(s, scratch, static_cast<int>(flip));
        const float inv = rsqrtf(s[0] / static_cast<float>(a.D) + a.eps), mean = s[1] * inv / static_cast<float>(a.D);
        for (int64_t c = threadIdx.x; c < a.D; c += kLongThreads) {
            const float nv = to_f(h[c]) * inv, gv = to_f(gy[c]);
            const float gh = inv * fmaf(-nv, mean, gv * a.weight[c]) + (gr != nullptr ? to_f(gr[c]) : 0.f);
            static_cast<T *>(a.grad_x)[row * a.D + c] = from_f<T>(gh);
            if (a.grad_h != nullptr) static_cast<R *>(a.grad_h)[row * a.D + c] = from_f<R>(gh);
            if (part != nullptr) {
                float *p = part + blockIdx.x * a.D + c;
                *p = (row == blockIdx.x ? 0.f : *p) + gv * nv;
            }
        }
    }
}

// Blocks of a call: a wave of resident ones, at most what kWaveThreads allows
// (the workspace's bound, from sizes alone).
constexpr int kWaveThreads = 1536;

int64_t row_blocks(int64_t M, int threads) { return threads == 32 ? ceil_div(M, kRowWarps) : M; }
int block_threads(int threads) { return threads == 32 ? 32 * kRowWarps : threads; }

int64_t most_blocks(int threads)
{
    const int64_t sms = sm_count() > 0 ? sm_count() : 152;
    const int per_sm = kWaveThreads / block_threads(threads);
    return sms * (per_sm > 0 ? per_sm : 1);
}

// Resident blocks of a kernel on the device, asked once for each kernel (the
// kernel itself, not its type: the types' kernels share one and differ in
// registers), block size and device.
template <auto KERNEL>
int64_t resident(int threads)
{
    static PerDevice known[kMostThreads / 32 + 1];
    const int n = known[threads / 32].get(current_device(), [&] {
        int blocks = 0;
        return ok(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, KERNEL, threads, 0)) ? blocks : 0;
    });
    return static_cast<int64_t>(n > 0 ? n : 1) * (sm_count() > 0 ? sm_count() : 1);
}

template <auto KERNEL>
int64_t wave(int64_t M, int threads)
{
    int64_t grid = row_blocks(M, threads);
    for (int64_t most : {most_blocks(threads), resident<KERNEL>(block_threads(threads))})
        if (grid > most) grid = most;
    return grid;
}

template <auto KERNEL>
rlscan_status forward_rows(const NormArgs &a, int threads, cudaStream_t s)
{
    return launch_overlapped(KERNEL, wave<KERNEL>(a.M, threads), block_threads(threads), 0, s, a);
}

template <auto KERNEL>
rlscan_status backward_rows(const NormGradArgs &a, int threads, float *part, int64_t &parts, cudaStream_t s)
{
    const int64_t grid = wave<KERNEL>(a.M, threads);
    parts = grid * (threads == 32 ? kRowWarps : 1);
    return launch_overlapped(KERNEL, grid, block_threads(threads), 0, s, a, part);
}

template <class T, class R>
rlscan_status forward(const NormArgs &a, cudaStream_t s)
{
    const int t = row_threads<T>(a.D);
    if (t == 0) return launch_overlapped(long_norm_kernel<T, R>, a.M, kLongThreads, 0, s, a);
    if (t == 32)
        return a.vec ? forward_rows<norm_kernel<T, R, true, true>>(a, t, s)
                     : forward_rows<norm_kernel<T, R, true, false>>(a, t, s);
    return a.vec ? forward_rows<norm_kernel<T, R, false, true>>(a, t, s)
                 : forward_rows<norm_kernel<T, R, false, false>>(a, t, s);
}

// most rows of `part` that a call fills
template <class T>
int64_t most_parts(int64_t M, int64_t D)
{
    const int t = row_threads<T>(D);
    const int64_t need = row_blocks(M, t), most = most_blocks(t == 0 ? kLongThreads : t);
    return (need < most ? need : most) * (t == 32 ? kRowWarps : 1);
}

// launches, and says how many rows of `part` it fills
template <class T, class R>
rlscan_status backward(const NormGradArgs &a, float *part, int64_t &parts, cudaStream_t s)
{
    const int t = row_threads<T>(a.D);
    if (t == 0) {
        const int64_t most = most_blocks(kLongThreads);
        parts = a.M < most ? a.M : most;
        return launch_overlapped(long_norm_grad_kernel<T, R>, parts, kLongThreads, 0, s, a, part);
    }
    if (t == 32)
        return a.vec ? backward_rows<norm_grad_kernel<T, R, true, true>>(a, t, part, parts, s)
                     : backward_rows<norm_grad_kernel<T, R, true, false>>(a, t, part, parts, s);
    return a.vec ? backward_rows<norm_grad_kernel<T, R, false, true>>(a, t, part, parts, s)
                 : backward_rows<norm_grad_kernel<T, R, false, false>>(a, t, part, parts, s);
}

uint64_t low_bits(const void *p) { return reinterpret_cast<uintptr_t>(p); }

}  // namespace

rlscan_status launch_add_rms_norm(const NormArgs &args, bool bf16_io, bool bf16_residual, cudaStream_t s)
{
    NormArgs a = args;
    const int ts = bf16_io ? 2 : 4, rs = bf16_residual ? 2 : 4;
    // wide accesses: whole chunks in every row, 16-byte aligned rows
    uint64_t bits = low_bits(a.x) | a.x_stride * ts | a.D * ts | low_bits(a.y) | low_bits(a.weight);
    if (a.residual != nullptr) bits |= low_bits(a.residual) | a.residual_stride * rs | low_bits(a.residual_out);
    a.vec = bits % 16 == 0;
    if (!bf16_io) return forward<float, float>(a, s);
    return bf16_residual ? forward<bf16, bf16>(a, s) : forward<bf16, float>(a, s);
}

size_t add_rms_norm_backward_workspace(int64_t M, int64_t D)
{
    const int64_t f = most_parts<float>(M, D), b = most_parts<bf16>(M, D);
    return sizeof(float) * static_cast<size_t>(f > b ? f : b) * D;
}

rlscan_status launch_add_rms_norm_backward(const NormGradArgs &args, bool bf16_io, bool bf16_h, void *ws, cudaStream_t s)
{
    NormGradArgs a = args;
    const int ts = bf16_io ? 2 : 4, hs = bf16_h ? 2 : 4;
    uint64_t bits = low_bits(a.grad_y) | a.grad_y_stride * ts | a.D * ts | low_bits(a.h) | a.h_stride * hs |
                    low_bits(a.grad_x) | low_bits(a.grad_h) | low_bits(a.weight);
    if (a.grad_residual != nullptr) bits |= low_bits(a.grad_residual) | a.grad_residual_stride * hs;
    a.vec = bits % 16 == 0;
    float *part = a.grad_weight != nullptr ? static_cast<float *>(ws) : nullptr;
    int64_t parts = 0;
    if (a.M > 0) {
        const rlscan_status st = !bf16_io ? backward<float, float>(a, part, parts, s)
                                 : bf16_h ? backward<bf16, bf16>(a, part, parts, s)
                                          : backward<bf16, float>(a, part, parts, s);
        if (st != RLSCAN_OK) return st;
    }
    if (a.grad_weight == nullptr) return RLSCAN_OK;
    SumJobs jobs;
    jobs.add(part, parts, a.D, a.D, a.grad_weight, false);
    return launch_sums(jobs, s);
}

}  // namespace seq
}  // namespace rlscan
