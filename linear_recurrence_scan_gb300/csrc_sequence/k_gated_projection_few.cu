// k_gated_projection_few.cu -- the gated feed-forward block's projections for a
// few rows (a decoding step): the weights are read once for all of them.
#include "gated_projection.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kWarps = 8, kFeatures = 16;  // of a block

// D += A B over 16 values of K: A 16 features x 16, B 16 x 8 rows of x
__device__ __forceinline__ void multiply(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// eight values from k on of a row of D, 0 past its end
template <bool VEC>
__device__ __forceinline__ Words<bf16, 8> eight(const bf16 *row, int64_t k, int64_t D)
{
    Words<bf16, 8> w;
    w.zero();
    if constexpr (VEC) {
        if (k < D) w.load(row + k);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w.set(i, k + 2 * i < D ? to_f(row[k + 2 * i]) : 0.f, k + 2 * i + 1 < D ? to_f(row[k + 2 * i + 1]) : 0.f);
    }
    return w;
}

// A block makes 16 features of both projections for up to 8 NT rows.  Its warps
// share K out; a lane loads 16 bytes of a weight's row at a time and gives them
// to the products as they are: which of the 16 values of K a register holds is
// the same for weights and rows, and their sum does not mind the order.  The
// weights' bytes bound it, not the products, so the tensor cores' older warp
// form, which takes its operands from registers, is the one that fits.
// Measured: 1 x 2048 x 8192 16 us, by the tiles of 256 rows 24 (the call on the
// host 7); 8 x 4096 x 12288 34 us, 5.9 TB/s, 16 rows 43, 32 rows 62, by the
// tiles 54 for any of them; 32 x 2047 x 8192, read value by value, 46 us, by the
// tiles, which need copies of such weights, 100.
template <int NT, bool VEC>
__global__ void __launch_bounds__(32 * kWarps, NT == 4 ? 2 : 3)
    few_kernel(const __grid_constant__ rlscan_gated_projection_args a, bf16 *h)
{
    __shared__ float part[kWarps][2][NT][4][32];
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = lane >> 2, quad = lane & 3;
    const int64_t f0 = static_cast<int64_t>(blockIdx.x) * kFeatures;
    const int64_t fa = f0 + row < a.F ? f0 + row : a.F - 1, fb = f0 + row + 8 < a.F ? f0 + row + 8 : a.F - 1;
    const bf16 *gate = static_cast<const bf16 *>(a.gate_weight), *up = static_cast<const bf16 *>(a.up_weight);
    const bf16 *ga = gate + fa * a.gate_stride, *gb = gate + fb * a.gate_stride;
    const bf16 *ua = up + fa * a.up_stride, *ub = up + fb * a.up_stride;
    const bf16 *x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) x[n] = static_cast<const bf16 *>(a.x) + (8 * n + row < a.M ? (8 * n + row) * a.x_stride : 0);
    float z[NT][4] = {}, u[NT][4] = {};
    const int64_t rounds = (a.D + 31) / 32;
#pragma unroll(NT == 1 ? 4 : 2)  // more loads ahead spill
    for (int64_t r = warp; r < rounds; r += kWarps) {
        const int64_t k = r * 32 + quad * 8;
        const Words<bf16, 8> wga = eight<VEC>(ga, k, a.D), wgb = eight<VEC>(gb, k, a.D);
        const Words<bf16, 8> wua = eight<VEC>(ua, k, a.D), wub = eight<VEC>(ub, k, a.D);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const Words<bf16, 8> v = eight<VEC>(x[n], k, a.D);
            multiply(z[n], wga.w[0], wgb.w[0], wga.w[1], wgb.w[1], v.w[0], v.w[1]);
            multiply(z[n], wga.w[2], wgb.w[2], wga.w[3], wgb.w[3], v.w[2], v.w[3]);
            multiply(u[n], wua.w[0], wub.w[0], wua.w[1], wub.w[1], v.w[0], v.w[1]);
            multiply(u[n], wua.w[2], wub.w[2], wua.w[3], wub.w[3], v.w[2], v.w[3]);
        }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[warp][0][n][i][lane] = z[n][i], part[warp][1][n][i][lane] = u[n][i];
    __syncthreads();
    // a value is one lane's of one of its four: row 8 (i / 2) + lane / 4, column 2 (lane % 4) + i % 2
    for (int v = threadIdx.x; v < NT * 128; v += 32 * kWarps) {
        const int n = v / 128, i = v / 32 % 4, l = v % 32;
        float zz = 0.f, uu = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) zz += part[w][0][n][i][l], uu += part[w][1][n][i][l];
        const int64_t f = f0 + 8 * (i / 2) + l / 4, m = 8 * n + 2 * (l % 4) + i % 2;
        if (f < a.F && m < a.M) h[m * a.F + f] = from_f<bf16>(halves((a.activation == RLSCAN_SILU ? silu(both(zz)) : gelu(both(zz))).value).x * uu);
    }
}

// Rows in whole units of 16 bytes
bool in_units(const rlscan_gated_projection_args &a)
{
    const uint64_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.gate_weight) | reinterpret_cast<uintptr_t>(a.up_weight) |
                          static_cast<uint64_t>((a.M > 1 ? a.x_stride : 0) * 2) |
                          static_cast<uint64_t>(a.F > 1 ? (a.gate_stride | a.up_stride) * 2 : 0);
    return bits % 16 == 0 && a.D % 8 == 0;
}

}  // namespace

// Up to 16 rows; up to 32 of arrays that tensor maps do not take
bool projection_is_few(const rlscan_gated_projection_args &a) { return a.M <= 16 || (a.M <= 32 && !in_units(a)); }

rlscan_status launch_gated_projection_few(const rlscan_gated_projection_args &a, void *h, cudaStream_t s)
{
    const bool vec = in_units(a);
    const int64_t grid = ceil_div(a.F, kFeatures);
    bf16 *out = static_cast<bf16 *>(h);
    auto go = [&](auto kernel) { return launch_overlapped(kernel, grid, 32 * kWarps, 0, s, a, out); };
    if (a.M <= 8) return vec ? go(few_kernel<1, true>) : go(few_kernel<1, false>);
    if (a.M <= 16) return vec ? go(few_kernel<2, true>) : go(few_kernel<2, false>);
    return go(few_kernel<4, false>);
}

}  // namespace seq
}  // namespace rlscan
