// distill_rows.cuh -- what the distillation's kernels share: a row of logits,
// its maximum and sum, and the teacher's tokens of a row.
#pragma once

#include <cfloat>

#include "distill.cuh"
#include "sequence.cuh"

namespace rlscan {
namespace seq {

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

// A row of V values: `units` whole units of 16 bytes of memory from `p + head`
// on, and the values in front of and behind them (`head` and `tail`, at most
// PER - 1 each), which are taken one by one.
template <class T>
struct Row {
    const T *p;
    int V, head, units, tail;
    __device__ __forceinline__ Row(const T *row, int64_t n) : p(row), V(static_cast<int>(n))
    {
        constexpr int PER = Unit<T>::PER;
        head = (PER - static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T))) % PER;
        head = head < V ? head : V;
        units = (V - head) / PER;
        tail = V - head - units * PER;
    }
    __device__ __forceinline__ int64_t first(int u) const { return head + static_cast<int64_t>(u) * Unit<T>::PER; }
    __device__ __forceinline__ Unit<T> load(int u) const
    {
        Unit<T> r;
        asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r.v.x), "=r"(r.v.y), "=r"(r.v.z), "=r"(r.v.w)
                     : "l"(p + first(u)));
        return r;
    }
    // the t-th value outside the units: its place, or -1
    __device__ __forceinline__ int edge(int t) const { return t < head ? t : t < head + tail ? V - tail + (t - head) : -1; }
};

struct Stats {
    float m, s;  // the largest logit and sum exp((z - m) / tau)
};

// A row's two normalizers, each by itself: the array is aligned as floats are.
__device__ __forceinline__ void keep_normalizers(float *normalizers, int64_t row, float m, float s)
{
    if (normalizers != nullptr) normalizers[2 * row] = m, normalizers[2 * row + 1] = s;
}

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
// exp((z - m) / tau) of a pair, for a logit z and its row's largest m: one
// multiply-add in front of the exponential, z c - m c with c = log2 e / tau.
// m c is rounded, by the same `rest` for every logit, which `exact` takes back
// from a sum or a factor.  Below 2^24 `rest` is at most 1/2; it grows with m c,
// and from 2^32 on 2^rest and 2^-rest leave the type's range.  So from 2^24 on
// (logits far from 0 or low temperatures, rows masked throughout with -1e10,
// say) values are taken one by one, the difference z - m first.
struct Shift {
    f2 c, mc;
    float rest;
    bool wide;
    __device__ __forceinline__ Shift(float m, float c1)
    {
        const float product = m * c1;
        c = both(c1);
        mc = both(-product);
        wide = !(fabsf(product) < 0x1p24f);  // (NaN too)
        rest = wide ? 0.f : fmaf(m, c1, -product);
    }
    __device__ __forceinline__ f2 exp(f2 z) const { return exp2_fast(fma2(z, c, mc)); }
    __device__ __forceinline__ float exact() const { return exp2_fast(-rest); }
};

// ---- the teacher's tokens of a row, a warp's work -----------------------------------
__device__ __forceinline__ int32_t token_at(const rlscan_distill_args &a, int64_t row, int k)  // -1: none
{
    const int64_t i = row * a.K + k;
    const int64_t id = a.token_bytes == 8 ? static_cast<const int64_t *>(a.teacher_tokens)[i]
                                          : static_cast<const int32_t *>(a.teacher_tokens)[i];
    return id >= 0 && id < a.V ? static_cast<int32_t>(id) : -1;
}
__device__ __forceinline__ float logit_at(const rlscan_distill_args &a, int64_t row, int k)
{
    const int64_t i = row * a.K + k;
    return a.teacher_dtype == RLSCAN_BF16 ? to_f(static_cast<const bf16 *>(a.teacher_logits)[i])
                                          : static_cast<const float *>(a.teacher_logits)[i];
}

// In shared memory: the teacher's probabilities, the row's logits at its tokens,
// the tokens, `padded` places each.
struct Teacher {
    float *q, *z;
    int32_t *token;
    float largest = -INFINITY, entropy = 0.f;  // entropy: sum of q log q
    __device__ __forceinline__ Teacher(float *at, int padded)
        : q(at), z(at + padded), token(reinterpret_cast<int32_t *>(at + 2 * padded))
    {
    }
    __device__ __forceinline__ void place(int k, int32_t id, float x, float logit)
    {
        token[k] = id;
        q[k] = id >= 0 ? x : -INFINITY;
        z[k] = logit;
        if (id >= 0) largest = x > largest || x != x ? x : largest;  // a NaN stays
    }
    // Places from `k0` on, k = k0 + lane, k0 + lane + 32, ...: EACH a lane are on
    // their way at once, tokens and logits first, then the row's logits there.
    template <int EACH, class R>
    __device__ __forceinline__ void gather(const rlscan_distill_args &a, const R &in, int64_t row, int k0, int K, int lane)
    {
        for (; k0 < K; k0 += 32 * EACH) {
            int32_t id[EACH];
            float x[EACH], logit[EACH];
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                const int k = k0 + 32 * i + lane;
                id[i] = k < K ? token_at(a, row, k) : -1;
                x[i] = k < K ? logit_at(a, row, k) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < EACH; ++i) logit[i] = id[i] >= 0 ? to_f(in.p[id[i]]) : 0.f;
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                if (k0 + 32 * i + lane < K) place(k0 + 32 * i + lane, id[i], x[i], logit[i]);
        }
    }
    // q = softmax of what every lane has placed (k = lane, lane + 32, ...); whether there is anything
    __device__ __forceinline__ bool softmax(int K, int lane, float c, float rtau)
    {
        largest = __any_sync(0xffffffffu, largest != largest) ? NAN : warp_max(largest);
        if (largest == -INFINITY) return false;
        float sum = 0.f;
        for (int k = lane; k < K; k += 32) sum += exp2_fast((q[k] - largest) * c);
        sum = warp_sum(sum);
        const float log_sum = logf(sum);
        for (int k = lane; k < K; k += 32) {
            const float lq = (q[k] - largest) * rtau - log_sum, p = exp2_fast((q[k] - largest) * c) / sum;
            if (!(p == 0.f)) entropy += p * lq;
            q[k] = p;
        }
        entropy = warp_sum(entropy);
        return true;
    }
};

// sum of q (z - m) / tau, by a warp.  The temperature comes last: a type's lowest
// value over a low one is past float32 where its part of the sum is not, and q
// over a high one may be 0, which would hide a z of -infinity.  Halves are summed,
// which stay finite where z - m, or q that sum to a little over 1, would not.
__device__ __forceinline__ float cross_of(const float *q, const float *z, int K, int lane, float m, float rtau)
{
    const float half = 0.5f * m;
    float cross = 0.f;
    for (int k = lane; k < K; k += 32)
        if (!(q[k] == 0.f)) cross += q[k] * fmaf(0.5f, z[k], -half);
    return warp_sum(cross) * (2.f * rtau);
}

// The probability of the k-th place's token: one that comes twice counts twice,
// and its first place (true) is the one that writes it.
__device__ __forceinline__ bool taught_at(const float *q_of, const int32_t *token_of, int k, int padded, float &q)
{
    const int32_t token = token_of[k];
    bool first = true;
    q = 0.f;
    for (int j = 0; j < padded; j += 4) {
        const int4 four = *reinterpret_cast<const int4 *>(token_of + j);
        const int same = (four.x == token ? 1 : 0) | (four.y == token ? 2 : 0) | (four.z == token ? 4 : 0) | (four.w == token ? 8 : 0);
        if (same != 0)
            for (int i = 0; i < 4; ++i)
                if ((same >> i & 1) != 0) {
                    first = first && j + i >= k;
                    q += q_of[j + i];
                }
    }
    return first;
}

}  // namespace seq
}  // namespace rlscan
