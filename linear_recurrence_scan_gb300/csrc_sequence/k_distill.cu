// k_distill.cu -- distillation from a teacher's top logits, for each token:
//   q = softmax(teacher / tau) over its K tokens,  p = softmax(logits / tau)
//   loss = sum_k q_k (log q_k - log p_k),  dlogits = grad_loss / tau (p - q).
#include <cfloat>

#include "distill.cuh"
#include "gated_scan.cuh"

namespace rlscan {
namespace seq {
namespace {

enum class Part { Loss, Grad, Both };

// 16 bytes of a row of logits
template <class T>
struct Unit {
    static constexpr int PER = 16 / static_cast<int>(sizeof(T)), PAIRS = PER / 2;
    uint4 v;
    __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
    __device__ __forceinline__ f2 get(int j) const
    {
        if constexpr (sizeof(T) == 2) return pair(__uint_as_float(word(j) << 16), __uint_as_float(word(j) & 0xffff0000u));
        return pair(__uint_as_float(word(2 * j)), __uint_as_float(word(2 * j + 1)));
    }
    __device__ __forceinline__ float value(int i) const
    {
        const float2 h = halves(get(i / 2));
        return i % 2 == 0 ? h.x : h.y;
    }
    __device__ __forceinline__ float max() const
    {
        if constexpr (sizeof(T) == 2) {
            auto as2 = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162 *>(&w); };
            const __nv_bfloat162 m = __hmax2(__hmax2(as2(v.x), as2(v.y)), __hmax2(as2(v.z), as2(v.w)));
            return fmaxf(__low2float(m), __high2float(m));
        } else {
            return fmaxf(fmaxf(value(0), value(1)), fmaxf(value(2), value(3)));
        }
    }
};

// A row of V values as units of 16 bytes of memory: the first and the last
// may hold others' values, and are then taken value by value.
template <class T>
struct Row {
    const T *aligned;  // start of the first unit
    int64_t off, V;    // values of the first unit in front of the row
    __device__ __forceinline__ Row(const T *p, int64_t n)
        : aligned(reinterpret_cast<const T *>(reinterpret_cast<uintptr_t>(p) & ~static_cast<uintptr_t>(15))),
          off(p - aligned), V(n)
    {
    }
    __device__ __forceinline__ int64_t units() const { return (off + V + Unit<T>::PER - 1) / Unit<T>::PER; }
    __device__ __forceinline__ int64_t first(int64_t u) const { return u * Unit<T>::PER - off; }
    __device__ __forceinline__ bool whole(int64_t u) const { return first(u) >= 0 && first(u) + Unit<T>::PER <= V; }
    // unit u; -infinity where it lies outside the row
    __device__ __forceinline__ Unit<T> load(int64_t u, int64_t end) const
    {
        Unit<T> r;
        const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
        r.v = make_uint4(none, none, none, none);
        if (u >= end) return r;
        if (whole(u)) {
            asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(r.v.x), "=r"(r.v.y), "=r"(r.v.z), "=r"(r.v.w)
                         : "l"(aligned + u * Unit<T>::PER));
            return r;
        }
        float f[Unit<T>::PER];
#pragma unroll
        for (int i = 0; i < Unit<T>::PER; ++i) {
            const int64_t e = first(u) + i;
            f[i] = e >= 0 && e < V ? to_f(aligned[u * Unit<T>::PER + i]) : -INFINITY;
        }
        Words<T, Unit<T>::PER> w;
#pragma unroll
        for (int i = 0; i < Unit<T>::PAIRS; ++i) w.set(i, f[2 * i], f[2 * i + 1]);
        r.v = make_uint4(w.w[0], w.w[1], w.w[2], w.w[3]);
        return r;
    }
};

struct Stats {
    float m, s;  // the largest logit and sum exp((z - m) / tau)
};

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int i = 16; i > 0; i /= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, i));
    return v;
}
__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int i = 16; i > 0; i /= 2) v += __shfl_xor_sync(0xffffffffu, v, i);
    return v;
}
__device__ __forceinline__ Stats join(Stats a, Stats b, float c)
{
    const float m = fmaxf(a.m, b.m);
    return {m, a.s * exp2_fast((a.m - m) * c) + b.s * exp2_fast((b.m - m) * c)};
}

// A row belongs to a warp (THREADS = 32: four rows a block), to a block, or,
// CLUSTER, to the blocks of a cluster, each with a slice.  A thread holds
// UNITS units of 16 bytes in registers, all in flight together.  Part::Both
// reads the logits once: largest value and sum from the registers, joined
// over lanes, warps and blocks, then the gradient from the same registers.
// Loss walks longer rows in several rounds with a running maximum and sum;
// Grad starts from the kept maximum and sum, its blocks share nothing.  The
// maximum starts at the lowest finite number, not at -infinity, so that rows
// and parts of rows without a finite value need no case of their own (their
// sum is 0), and values enter as (z - m) / tau, which is 0 for the largest
// whatever its size.
template <class T, int THREADS, int UNITS, Part PART, bool CLUSTER>
__global__ void __launch_bounds__(THREADS == 32 ? 128 : THREADS, THREADS == 512 ? 2 : 6)
    distill_kernel(const __grid_constant__ rlscan_distill_args a, const __grid_constant__ DistillOut o, int ranks)
{
    constexpr bool WARP = THREADS == 32;
    constexpr int GROUPS = WARP ? 4 : 1, WARPS = WARP ? 1 : THREADS / 32, PER = Unit<T>::PER;
    struct Teacher {
        float q[kMostTeacher], z[kMostTeacher];
        int32_t token[kMostTeacher];
    };
    __shared__ Teacher teachers[GROUPS];
    __shared__ Stats of_warp[WARPS];
    __shared__ float4 of_rank[CLUSTER ? kGatedCluster : 1];
    __shared__ float logs[GROUPS];  // sum of q log q
    __shared__ int taught[GROUPS];  // whether a teacher's token is left
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int g = WARP ? threadIdx.x / 32 : 0, t = WARP ? threadIdx.x % 32 : threadIdx.x, lane = threadIdx.x & 31;
    const int rank = WARP ? 0 : static_cast<int>(blockIdx.x % static_cast<unsigned>(ranks));
    const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * GROUPS + g : blockIdx.x / static_cast<unsigned>(ranks);
    if (row >= a.N * a.T) return;  // a whole warp
    auto sync = [] {
        if constexpr (WARP) __syncwarp();
        else __syncthreads();
    };
    const Division at = divide(row, a.T);
    const Row<T> in(static_cast<const T *>(a.logits.data) + at.q * a.logits.row_stride + at.r * a.logits.token_stride, a.V);
    // the slice of this rank, in whole rounds of the block
    const int64_t all = in.units(), share = (all + ranks - 1) / ranks, u0 = rank * share, end = u0 + share < all ? u0 + share : all;
    T *out = static_cast<T *>(o.grad) + row * a.V;
    const bool same = PART != Part::Loss && (reinterpret_cast<uintptr_t>(out) & 15u) == static_cast<uintptr_t>(in.off) * sizeof(T);
    // a unit of the gradient, from fp32 values that `value` gives
    auto put = [&](int64_t u, auto value) {
        if (same && in.whole(u)) {
            Words<T, PER> w;
#pragma unroll
            for (int i = 0; i < PER / 2; ++i) {
                const float2 h = halves(value(i));
                w.set(i, h.x, h.y);
            }
            *reinterpret_cast<uint4 *>(out + in.first(u)) = make_uint4(w.w[0], w.w[1], w.w[2], w.w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < PER / 2; ++i) {
                const float2 h = halves(value(i));
                const int64_t e = in.first(u) + 2 * i;
                if (e >= 0 && e < a.V) out[e] = from_f<T>(h.x);
                if (e + 1 >= 0 && e + 1 < a.V) out[e + 1] = from_f<T>(h.y);
            }
        }
    };
    if (a.mask != nullptr && a.mask[row] == 0) {  // neither its logits nor its teacher are read
        if (PART != Part::Grad && rank == 0 && t == 0) {
            o.loss[row] = 0.f;
            if (o.normalizers != nullptr) reinterpret_cast<float2 *>(o.normalizers)[row] = make_float2(0.f, 1.f);
        }
        if constexpr (PART != Part::Loss)
            for (int64_t u = u0 + t; u < end; u += THREADS) put(u, [](int) { return both(0.f); });
        return;
    }
    const float c = kLog2e / static_cast<float>(a.temperature), rtau = 1.f / static_cast<float>(a.temperature);
    Unit<T> v[UNITS];
    auto load = [&](int64_t first) {
#pragma unroll
        for (int i = 0; i < UNITS; ++i) v[i] = in.load(first + i * THREADS + t, end);
    };
    load(u0);
    if constexpr (CLUSTER && PART != Part::Grad) cluster_arrive();
    Teacher &teach = teachers[g];
    const int K = static_cast<int>(a.K);
    if (t < 32) {  // the teacher's probabilities, by one warp
        float largest = -INFINITY, sum = 0.f;
        for (int k = lane; k < K; k += 32) {
            const int64_t i = row * a.K + k;
            const int64_t token = a.token_bytes == 8 ? static_cast<const int64_t *>(a.teacher_tokens)[i]
                                                     : static_cast<const int32_t *>(a.teacher_tokens)[i];
            const bool valid = token >= 0 && token < a.V;
            teach.token[k] = valid ? static_cast<int32_t>(token) : -1;
            const float x = a.teacher_dtype == RLSCAN_BF16 ? to_f(static_cast<const bf16 *>(a.teacher_logits)[i])
                                                           : static_cast<const float *>(a.teacher_logits)[i];
            teach.q[k] = valid ? x : -INFINITY;
            teach.z[k] = valid ? to_f(in.aligned[in.off + token]) : 0.f;
            if (valid) largest = x > largest || x != x ? x : largest;  // a NaN stays
        }
        const bool nan = __any_sync(0xffffffffu, largest != largest);
        largest = nan ? NAN : warp_max(largest);
        if (lane == 0) taught[g] = largest != -INFINITY;
        if (largest != -INFINITY) {
            for (int k = lane; k < K; k += 32) sum += exp2_fast((teach.q[k] - largest) * c);
            sum = warp_sum(sum);
            const float log_sum = logf(sum);
            float entropy = 0.f;  // sum of q log q
            for (int k = lane; k < K; k += 32) {
                const float lq = (teach.q[k] - largest) * rtau - log_sum, q = exp2_fast((teach.q[k] - largest) * c) / sum;
                if (!(q == 0.f)) entropy += q * lq;
                teach.q[k] = q;
            }
            entropy = warp_sum(entropy);
            if (lane == 0) logs[g] = entropy;
        }
    }
    Stats st{-FLT_MAX, 0.f};
    if constexpr (PART == Part::Grad) {
        const float2 kept = reinterpret_cast<const float2 *>(o.normalizers)[row];
        st = {kept.x, kept.y};
        sync();
    } else {
        for (int64_t first = u0;;) {
            float m = st.m;
#pragma unroll
            for (int i = 0; i < UNITS; ++i) m = fmaxf(m, v[i].max());
            const f2 low = both(-m), scale = both(c);
            f2 s0 = both(0.f), s1 = both(0.f);
#pragma unroll
            for (int i = 0; i < UNITS; ++i)
#pragma unroll
                for (int j = 0; j < Unit<T>::PAIRS; ++j) {
                    f2 &s = j % 2 == 0 ? s0 : s1;
                    s = add2(s, exp2_fast(mul2(add2(v[i].get(j), low), scale)));
                }
            const float2 h = halves(add2(s0, s1));
            st = {m, st.s * exp2_fast((st.m - m) * c) + (h.x + h.y)};
            first += THREADS * UNITS;
            if (PART == Part::Both || first >= end) break;
            load(first);
        }
        const float m = warp_max(st.m);
        st = {m, warp_sum(st.s * exp2_fast((st.m - m) * c))};
        if constexpr (!WARP) {
            if (lane == 0) of_warp[threadIdx.x / 32] = st;
            __syncthreads();
            st = of_warp[0];
#pragma unroll
            for (int i = 1; i < WARPS; ++i) st = join(st, of_warp[i], c);
        } else {
            __syncwarp();
        }
        if constexpr (CLUSTER) {
            cluster_wait();
            if (t < ranks) store_to_rank(&of_rank[rank], t, make_float4(st.m, st.s, 0.f, 0.f));
            cluster_arrive();
            cluster_wait();
            st = {of_rank[0].x, of_rank[0].y};
            for (int i = 1; i < ranks; ++i) st = join(st, Stats{of_rank[i].x, of_rank[i].y}, c);
        }
        if (rank == 0 && t < 32) {
            float cross = 0.f;
            for (int k = lane; k < K; k += 32) {
                const float q = teach.q[k];
                if (!(q == 0.f)) cross += q * ((teach.z[k] - st.m) * rtau);
            }
            cross = warp_sum(cross);
            if (lane == 0) {
                o.loss[row] = taught[g] ? logs[g] - cross + logf(st.s) : 0.f;
                if (o.normalizers != nullptr) reinterpret_cast<float2 *>(o.normalizers)[row] = make_float2(st.m, st.s);
            }
        }
    }
    if constexpr (PART != Part::Loss) {
        const bool some = taught[g] != 0;
        const float weight = some ? o.grad_loss[row] * rtau : 0.f, scale = weight / st.s;
        const f2 low = both(-st.m), c2 = both(c), scale2 = both(scale);
        // The registers keep the logits as they were read: without this the
        // compiler keeps the widened values from the first pass to this one.
        if constexpr (PART == Part::Both) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i) asm volatile("" : "+r"(v[i].v.x), "+r"(v[i].v.y), "+r"(v[i].v.z), "+r"(v[i].v.w));
        }
        for (int64_t first = u0;;) {
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                const int64_t u = first + i * THREADS + t;
                if (u < end)
                    put(u, [&](int j) {
                        const f2 e = mul2(exp2_fast(mul2(add2(v[i].get(j), low), c2)), scale2);
                        return some ? e : both(0.f);
                    });
            }
            first += THREADS * UNITS;
            if (PART == Part::Both || first >= end) break;
            load(first);
        }
        sync();  // the teacher's tokens over what has been written
        if (some)
            for (int k = t; k < K; k += THREADS) {
                const int32_t token = teach.token[k];
                const int64_t u = (in.off + token) / PER;
                if (token < 0 || u < u0 || u >= end) continue;
                float q = 0.f;
                bool first = true;  // a token that comes twice counts twice, and is written once
                for (int j = 0; j < K; ++j)
                    if (teach.token[j] == token) {
                        first = first && j >= k;
                        q += teach.q[j];
                    }
                if (first) out[token] = from_f<T>(exp2_fast((teach.z[k] - st.m) * c) * scale - q * weight);
            }
    }
}

// Loss, or loss and gradient: threads and blocks of a row.
struct Plan {
    int threads, ranks;
};

constexpr int kUnits = 8;  // of a thread

// Units that a row may touch: one more than its own where it starts inside one
int64_t most_units(const rlscan_distill_args &a)
{
    const int64_t per = a.dtype == RLSCAN_BF16 ? 8 : 4;
    return ceil_div(a.V + per - 1, per);
}

// Rows of up to a warp's or a small block's registers stay there; longer ones
// are split while they do not fit a block of 512 threads (`hold`), or while
// there are too few rows to give every SM two blocks.
Plan plan(const rlscan_distill_args &a, bool hold)
{
    const int64_t units = most_units(a), rows = a.N * a.T, sms = sm_count() > 0 ? sm_count() : 152;
    if (units <= 32 * kUnits) return {32, 1};
    if (units <= 128 * kUnits) return {128, 1};
    int ranks = 1;
    while (ranks < kGatedCluster &&
           ((hold && ceil_div(units, ranks) > 512 * kUnits) || (rows * ranks < 2 * sms && ceil_div(units, ranks) > 512)))
        ranks *= 2;
    return {512, ranks};
}

template <class T, Part PART>
rlscan_status run(const rlscan_distill_args &a, const DistillOut &o, Plan p, cudaStream_t s)
{
    const int64_t rows = a.N * a.T;
    if (p.threads == 32)
        return launch_overlapped(distill_kernel<T, 32, kUnits, PART, false>, ceil_div(rows, 4), 128, 0, s, a, o, 1);
    if (p.threads == 128)
        return launch_overlapped(distill_kernel<T, 128, kUnits, PART, false>, rows * p.ranks, 128, 0, s, a, o, p.ranks);
    if constexpr (PART == Part::Grad) {
        return launch_overlapped(distill_kernel<T, 512, kUnits, PART, false>, rows * p.ranks, 512, 0, s, a, o, p.ranks);
    } else {
        if (p.ranks > 1)
            return launch_cluster(distill_kernel<T, 512, kUnits, PART, true>, rows * p.ranks, 512, 0, p.ranks, s, a, o, p.ranks);
        return launch_overlapped(distill_kernel<T, 512, kUnits, PART, false>, rows, 512, 0, s, a, o, 1);
    }
}

template <Part PART>
rlscan_status run_typed(const rlscan_distill_args &a, const DistillOut &o, Plan p, cudaStream_t s)
{
    return a.dtype == RLSCAN_BF16 ? run<bf16, PART>(a, o, p, s) : run<float, PART>(a, o, p, s);
}

}  // namespace

rlscan_status launch_distill(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s)
{
    return run_typed<Part::Loss>(a, o, plan(a, false), s);
}

rlscan_status launch_distill_backward(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s)
{
    Plan p = plan(a, false);
    if (p.threads == 512) p.ranks = static_cast<int>(ceil_div(most_units(a), 512 * kUnits));
    return run_typed<Part::Grad>(a, o, p, s);
}

bool distill_fits(const rlscan_distill_args &a) { return most_units(a) <= static_cast<int64_t>(kGatedCluster) * 512 * kUnits; }

rlscan_status launch_distill_both(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s)
{
    return run_typed<Part::Both>(a, o, plan(a, true), s);
}

}  // namespace seq
}  // namespace rlscan
