// k_distill_short.cu -- distillation from a teacher's top logits where a row of
// the student's fits a warp's registers.
#include "distill_rows.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kRows = 8;  // of a block: a warp each
constexpr int kMostValues = kShortUnits * 8 + 7;              // of a row: its units, and less than one more
constexpr int kSeenWords = (kMostValues / 32 / 32 + 1) * 32;  // a bit for each of them, a word a lane at a time

// A warp holds a row, UNITS times 16 bytes a lane, and goes with it.  Its loads
// are all under way at once, and the other warps of an SM cover its chain of
// steps (the teacher's tokens, the logits there, the sums, the gradient), which
// bounds it together with the instructions that a row takes whatever its length.
// Measured, loss and gradient, 32768 rows of K = 8 bfloat16: V 100 26 us, 400 25,
// 1500 64 (their bytes' time 2, 7 and 30; by the blocks that stay for many rows,
// whose last warp brings one row after the other, 1500 took 106).  Rows in two
// warps' registers are no faster than by those (V 4096: 132 us, 121).  Whether a
// token comes twice is found with a bit for each: K = 100 90 us, with each place
// compared with all others 136.
template <class T, int UNITS, Part PART>
__global__ void __launch_bounds__(32 * kRows, UNITS == 8 ? 3 : UNITS == 4 ? 4 : 5)
    distill_short_kernel(const __grid_constant__ rlscan_distill_args a, const __grid_constant__ DistillOut o)
{
    constexpr int PER = Unit<T>::PER;
    extern __shared__ __align__(16) float teachers[];
    __shared__ uint32_t seen[kRows][kSeenWords];  // the teacher's tokens of a row
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, slot = threadIdx.x >> 5, K = static_cast<int>(a.K);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + slot;
    if (row >= a.N * a.T) return;
    const Division at = divide(row, a.T);
    const Row<T> in(static_cast<const T *>(a.logits.data) + at.q * a.logits.row_stride + at.r * a.logits.token_stride, a.V);
    T *out = static_cast<T *>(o.grad) + row * a.V;
    const bool aligned = (reinterpret_cast<uintptr_t>(out + in.head) & 15u) == 0;  // units of the gradient as of the logits
    const int edge = in.edge(lane);                                              // the lane's value outside the units
    auto clear = [&] {
        for (int e = lane; e < in.V; e += 32) out[e] = from_f<T>(0.f);
    };
    if (a.mask != nullptr && load_byte(a.mask + row) == 0u) {
        if (PART != Part::Grad && lane == 0) {
            o.loss[row] = 0.f;
            keep_normalizers(o.normalizers, row, 0.f, 1.f);
        }
        if constexpr (PART != Part::Loss) clear();
        return;
    }
    Unit<T> v[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;  // -infinity
        v[i].v = make_uint4(none, none, none, none);
        if (lane + 32 * i < in.units) v[i] = in.load(lane + 32 * i);
    }
    const float at_edge = edge >= 0 ? to_f(in.p[edge]) : -INFINITY;
    const float c = kLog2e / static_cast<float>(a.temperature), rtau = 1.f / static_cast<float>(a.temperature);
    const float weight = PART != Part::Loss ? o.grad_loss[row] * rtau : 0.f;
    const int padded = (K + 3) / 4 * 4;
    Teacher of(teachers + slot * 3 * padded, padded);
    if (lane < padded - K) of.token[K + lane] = -1;
    of.gather<2>(a, in, row, 0, K, lane);
    const bool taught = of.softmax(K, lane, c, rtau);
    bool twice = false;  // whether a token comes twice
    if constexpr (PART != Part::Loss) {
#pragma unroll
        for (int i = 0; i < kSeenWords; i += 32) seen[slot][i + lane] = 0u;
        __syncwarp();
        for (int k = lane; k < K; k += 32) {
            const int32_t token = of.token[k];
            if (token >= 0) twice = twice || (atomicOr(&seen[slot][token / 32], 1u << token % 32) >> token % 32 & 1u) != 0u;
        }
        twice = __any_sync(0xffffffffu, twice);
    }
    float m = fmaxf(-FLT_MAX, at_edge), s = 0.f;
    if constexpr (PART == Part::Grad) {
        m = o.normalizers[2 * row], s = o.normalizers[2 * row + 1];
    } else {
#pragma unroll
        for (int i = 0; i < UNITS; ++i) m = fmaxf(m, v[i].max());
        m = warp_max(m);
        const Shift shift(m, c);
        if (!shift.wide) {
            f2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
#pragma unroll
                for (int j = 0; j < Unit<T>::PAIRS; j += 2) {
                    s0 = add2(s0, shift.exp(v[i].get(j)));
                    s1 = add2(s1, shift.exp(v[i].get(j + 1)));
                }
            const float2 f = halves(add2(s0, s1));
            s = (f.x + f.y) * shift.exact();
        } else {
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
#pragma unroll
                for (int j = 0; j < PER; ++j) s += exp2_fast((v[i].value(j) - m) * c);
        }
        s = warp_sum(s + exp2_fast((at_edge - m) * c));
    }
    if constexpr (PART != Part::Loss) {
        const Shift shift(m, c);
        const float scale = weight / s;
        auto value = [&](float z) { return from_f<T>(exp2_fast((z - m) * c) * scale); };
        const f2 factor = both(scale * shift.exact());
#pragma unroll
        for (int i = 0; i < UNITS; ++i) {
            const int u = lane + 32 * i;
            if (u >= in.units) break;
            if (aligned && !shift.wide) {
                Words<T, PER> w;
#pragma unroll
                for (int j = 0; j < PER / 2; ++j) {
                    const float2 f = halves(mul2(shift.exp(v[i].get(j)), factor));
                    w.set(j, f.x, f.y);
                }
                *reinterpret_cast<uint4 *>(out + in.first(u)) = make_uint4(w.w[0], w.w[1], w.w[2], w.w[3]);
            } else {
#pragma unroll
                for (int j = 0; j < PER; ++j) out[in.first(u) + j] = value(v[i].value(j));
            }
        }
        if (edge >= 0) out[edge] = value(at_edge);
        __syncwarp();  // over what has been written: the teacher's tokens,
        if (taught) {
            for (int k = lane; k < K; k += 32) {
                const int32_t token = of.token[k];
                float q = of.q[k];
                if (token < 0 || (twice && !taught_at(of.q, of.token, k, padded, q))) continue;
                out[token] = from_f<T>(exp2_fast((of.z[k] - m) * c) * scale - q * weight);
            }
        } else {
            clear();  // or, where there is nothing to learn from, zeros
        }
    }
    if constexpr (PART != Part::Grad) {
        const float cross = taught ? cross_of(of.q, of.z, K, lane, m, rtau) : 0.f;
        if (lane == 0) {
            o.loss[row] = taught ? of.entropy - cross + logf(s) : 0.f;
            keep_normalizers(o.normalizers, row, m, s);
        }
    }
}

template <class T, int UNITS, Part PART>
rlscan_status launch_short(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s)
{
    const size_t smem = static_cast<size_t>(kRows) * 12 * ((a.K + 3) / 4 * 4);  // at most 24 KB
    return launch_overlapped(distill_short_kernel<T, UNITS, PART>, ceil_div(a.N * a.T, kRows), 32 * kRows, smem, s, a, o);
}

// A lane's units: the fewest that hold the row.
template <class T, Part PART>
rlscan_status run(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s)
{
    const int64_t units = a.V / Unit<T>::PER;
    if (units <= 32) return launch_short<T, 1, PART>(a, o, s);
    if (units <= 64) return launch_short<T, 2, PART>(a, o, s);
    if (units <= 128) return launch_short<T, 4, PART>(a, o, s);
    return launch_short<T, 8, PART>(a, o, s);
}
template <Part PART>
rlscan_status run_typed(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s)
{
    return a.dtype == RLSCAN_BF16 ? run<bf16, PART>(a, o, s) : run<float, PART>(a, o, s);
}

}  // namespace

rlscan_status launch_distill_short(const rlscan_distill_args &a, Part part, const DistillOut &o, cudaStream_t s)
{
    switch (part) {
    case Part::Loss: return run_typed<Part::Loss>(a, o, s);
    case Part::Grad: return run_typed<Part::Grad>(a, o, s);
    default: return run_typed<Part::Both>(a, o, s);
    }
}

}  // namespace seq
}  // namespace rlscan
