// k_distill.cu -- distillation from a teacher's top logits, for each token:
//   q = softmax(teacher / tau) over its K tokens,  p = softmax(logits / tau)
//   loss = sum_k q_k (log q_k - log p_k),  dlogits = grad_loss / tau (p - q).
#include <cfloat>

#include "distill.cuh"
#include "distill_rows.cuh"
#include "gated_scan.cuh"

namespace rlscan {
namespace seq {
namespace {

__device__ unsigned int g_timed_out;  // a wait ran out on this device

// The maxima and sums of a row's warps, of all the blocks that share it.  Two
// buffers take turns: who has all of a row's knows that all have read those of
// the row before.
template <int WARPS, bool CLUSTER>
struct Meeting {
    float2 of_warp[2][CLUSTER ? kGatedCluster * WARPS : WARPS];
    uint64_t bar[2];
};

// What comes with a row's last part in shared memory: the teacher's
// probabilities, the logits at its tokens, the tokens (K each, behind the
// stages), and the row's values outside units.
struct Head {
    float edge[16];
    float entropy;     // sum of q log q
    float m, s;        // Part::Grad: the kept maximum and sum
    float weight;      // grad_loss / tau
    int taught;
};

constexpr int kStages = 2;
constexpr int kStageUnits[] = {768, 1600, 3000};  // of 64, 128 and 256 consumers: 12, 25 and 47 KB
constexpr int kWideUnits = 6400;                       // one block an SM: 100 KB
constexpr int kMostConsumers = 256;

__device__ __forceinline__ void copy_bulk(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes),
                 "r"(bar)
                 : "memory");
}

// Blocks that stay for many rows.  The last warp runs ahead: it brings the
// next part of the row's logits into shared memory (one copy a stage) and works
// out the teacher's probabilities there; CONSUMERS threads take a part's sums
// and write its gradient.  So copies are in flight while sums, the meeting of
// blocks and the stores of the row before take their time.  Part::Both reads
// the logits once: a block's slice of a row is one part; CLUSTER: a row is
// several blocks' slices, whose maxima and sums meet.  Loss and Grad walk
// longer rows in several parts.  The maximum starts at the lowest finite
// number, not at -infinity, so that rows and parts of rows without a finite
// value need no case of their own (their sum is 0).
// The loss of long rows is bound by its bytes (8 x 1024 x 131072 bfloat16 302
// us, 7.1 TB/s); loss and gradient by a row's chain of steps (sums, meeting,
// gradient), of which an SM has two to eight side by side, and by
// instructions: 4 x 1023 x 50257 134 us, its bytes' time 106 (blocks that held
// one row in registers and went with it 197 us; a row's gradient behind the
// next row's sums, which takes a third stage, 187 us against 169 then), 16 x
// 2048 x 6000 176 us, its bytes' time 118.
template <class T, int CONSUMERS, Part PART, bool CLUSTER>
__global__ void __launch_bounds__(CONSUMERS + 32, CONSUMERS == 64 ? 8 : CONSUMERS == 128 ? 4 : 2)
    distill_kernel(const __grid_constant__ rlscan_distill_args a, const __grid_constant__ DistillOut o, int ranks, int stage_units)
{
    constexpr int WARPS = CONSUMERS / 32, PER = Unit<T>::PER, ROUND = 4;
    extern __shared__ __align__(16) char buffers[];
    __shared__ Head heads[kStages];
    __shared__ Meeting<WARPS, CLUSTER> meeting;
    __shared__ uint64_t full[kStages], empty[kStages];
    __shared__ int gave_up;
    ptx::pdl_trigger_dependents();
    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(&full[i], 2);  // the copy has been asked for; the head is there
            ptx::mbar_init(&empty[i], WARPS);
        }
        for (int i = 0; i < 2; ++i) ptx::mbar_init(&meeting.bar[i], 1);
        ptx::fence_mbar_init();
    }
    __syncthreads();
    if constexpr (CLUSTER) {
        cluster_arrive();
        cluster_wait();  // all can be written to
    }
    ptx::pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, rank = static_cast<int>(blockIdx.x % static_cast<unsigned>(ranks)), K = static_cast<int>(a.K);
    const int padded = (K + 3) / 4 * 4;  // of the teacher's arrays: the tokens are looked through by fours
    auto teacher = [&](int st) { return reinterpret_cast<float *>(buffers + static_cast<size_t>(kStages) * stage_units * 16) + st * 3 * padded; };
    const int64_t rows = a.N * a.T, stride = gridDim.x / static_cast<unsigned>(ranks), row0 = blockIdx.x / static_cast<unsigned>(ranks);
    const float c = kLog2e / static_cast<float>(a.temperature), rtau = 1.f / static_cast<float>(a.temperature);
    auto row_of = [&](int64_t row) {
        const Division at = divide(row, a.T);
        return Row<T>(static_cast<const T *>(a.logits.data) + at.q * a.logits.row_stride + at.r * a.logits.token_stride, a.V);
    };
    // the rank's units of a row: from `u0` to `end`
    auto slice = [&](const Row<T> &in, int &u0, int &end) {
        const int share = (in.units + ranks - 1) / ranks;
        u0 = rank * share < in.units ? rank * share : in.units;
        end = u0 + share < in.units ? u0 + share : in.units;
    };
    int stage = 0;
    uint32_t parity = 0;
    auto next = [&] {
        if (++stage == kStages) stage = 0, parity ^= 1u;
    };
    // Brings rows, by the last warp.
    auto bring = [&] {
        // Of the loss of a row of many parts the warp has the next row's first 64
        // teacher's tokens, their logits and the row's there before the row's
        // last part: loaded behind that part's copy, one after the other, they
        // held up the next row's first (8 x 1024 x 131072: 350 us, so 325).
        // Shorter rows lose by it: theirs are held up in front of the copy.
        constexpr int AHEAD = PART == Part::Loss && CONSUMERS == 128 ? 2 : 0;
        int32_t next_token[AHEAD + 1];
        float next_x[AHEAD + 1], next_z[AHEAD + 1];
        auto look = [&](const Row<T> &in, int64_t row) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int k = 32 * i + lane;
                next_token[i] = k < K ? token_at(a, row, k) : -1;
                next_x[i] = k < K ? logit_at(a, row, k) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) next_z[i] = next_token[i] >= 0 ? to_f(in.p[next_token[i]]) : 0.f;
        };
        // The head of a row: the teacher's tokens (-1: none), q = softmax of its
        // logits over them, the row's logits there.
        auto teach = [&](Head &h, float *q_of, const Row<T> &in, int64_t row, bool looked) {
            if (lane < padded - K) reinterpret_cast<int32_t *>(q_of + 2 * padded)[K + lane] = -1;
            if (rank == 0 && in.edge(lane) >= 0) h.edge[lane] = to_f(in.p[in.edge(lane)]);
            Teacher of(q_of, padded);
            if (looked) {
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    if (32 * i + lane < K) of.place(32 * i + lane, next_token[i], next_x[i], next_z[i]);
            }
            of.template gather<2>(a, in, row, looked ? 32 * AHEAD : 0, K, lane);
            const bool taught = of.softmax(K, lane, c, rtau);
            if (lane == 0) h.taught = taught, h.entropy = of.entropy;
        };
        uint32_t mask = a.mask != nullptr && row0 < rows ? load_byte(a.mask + row0) : 1u;
        for (int64_t row = row0; row < rows; row += stride) {
            const Row<T> in = row_of(row);
            int u0, end;
            slice(in, u0, end);
            const bool masked = mask == 0u, ahead = AHEAD > 0 && !masked && end - u0 > 3 * stage_units;
            if (a.mask != nullptr && row + stride < rows) mask = load_byte(a.mask + row + stride);
            for (int u = u0;;) {  // a masked row is one part without logits
                const int n = masked ? 0 : end - u < stage_units ? end - u : stage_units;
                const bool last = masked || u + n >= end;
                if (!wait_warp(ptx::smem_u32(&empty[stage]), parity ^ 1u, &gave_up)) return;
                if (lane == 0) {
                    if (n > 0) {
                        ptx::mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(n) * 16);
                        copy_bulk(ptx::smem_u32(buffers) + stage * stage_units * 16, in.p + in.first(u), static_cast<uint32_t>(n) * 16,
                                  ptx::smem_u32(&full[stage]));
                    } else {
                        ptx::mbar_arrive(&full[stage]);
                    }
                }
                Head &h = heads[stage];
                if (lane == 0) {
                    if (PART != Part::Loss && !masked) h.weight = o.grad_loss[row] * rtau;
                    if (PART == Part::Grad && !masked) {
                        h.m = o.normalizers[2 * row], h.s = o.normalizers[2 * row + 1];
                    }
                }
                if (last && !masked) teach(h, teacher(stage), in, row, ahead);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&full[stage]);
                if (ahead && u == u0) look(in, row);
                next();
                if (last) break;
                u += n;
            }
        }
    };
    if (threadIdx.x >= CONSUMERS) {
        bring();
    } else {  // ---- sums and gradients
        const int t = threadIdx.x;
        auto sync = [] { ptx::named_barrier(1, CONSUMERS); };
        auto release = [&] {
            __syncwarp();
            if (lane == 0 && !has_given_up(&gave_up)) ptx::mbar_arrive(&empty[stage]);
            next();
        };
        int turn = 0;
        // What decides which barriers a row takes is read from memory by all.
        uint32_t mask = a.mask != nullptr && row0 < rows ? load_byte(a.mask + row0) : 1u;
        for (int64_t row = row0; row < rows; row += stride) {
            const Row<T> in = row_of(row);
            int u0, end;
            slice(in, u0, end);
            const bool masked = mask == 0u;
            if (a.mask != nullptr && row + stride < rows) mask = load_byte(a.mask + row + stride);
            T *out = static_cast<T *>(o.grad) + row * a.V;
            const bool aligned = (reinterpret_cast<uintptr_t>(out + in.head) & 15u) == 0;  // units of the gradient as of the logits
            const int edge = rank == 0 ? in.edge(t) : -1;                                // the thread's value outside the units
            auto clear = [&] {
                if (edge >= 0) out[edge] = from_f<T>(0.f);
                if (aligned) {
                    for (int u = u0 + t; u < end; u += CONSUMERS) *reinterpret_cast<uint4 *>(out + in.first(u)) = make_uint4(0u, 0u, 0u, 0u);
                } else {
                    for (int64_t e = in.first(u0) + t; e < in.first(end); e += CONSUMERS) out[e] = from_f<T>(0.f);
                }
            };
            Stats st{-FLT_MAX, 0.f};
            for (int u = u0;;) {
                wait(ptx::smem_u32(&full[stage]), parity, &gave_up);
                const Head &h = heads[stage];
                const float *q_of = teacher(stage), *z_of = q_of + padded;
                const int32_t *token_of = reinterpret_cast<const int32_t *>(q_of + 2 * padded);
                const uint4 *part = reinterpret_cast<const uint4 *>(buffers + static_cast<size_t>(stage) * stage_units * 16);
                if (masked) {
                    if (PART != Part::Grad && rank == 0 && t == 0) {
                        o.loss[row] = 0.f;
                        keep_normalizers(o.normalizers, row, 0.f, 1.f);
                    }
                    if constexpr (PART != Part::Loss) clear();
                    release();
                    break;
                }
                const int n = end - u < stage_units ? end - u : stage_units;
                const bool last = u + n >= end;
                if constexpr (PART == Part::Grad) {
                    st = {h.m, h.s};
                } else {
                    const float at_edge = last && edge >= 0 ? h.edge[t] : -INFINITY;
                    if (last && edge >= 0) {
                        const float m = fmaxf(st.m, at_edge);
                        st = {m, st.s * exp2_fast((st.m - m) * c) + exp2_fast((at_edge - m) * c)};
                    }
                    auto round = [&](int i0, auto units) {  // as many units, from i0 on
                        constexpr int UNITS = decltype(units)::value;
                        Unit<T> v[UNITS];
                        float m = st.m;
#pragma unroll
                        for (int i = 0; i < UNITS; ++i) {
                            v[i].v = part[i0 + i * CONSUMERS];
                            m = fmaxf(m, v[i].max());
                        }
                        const Shift shift(m, c);
                        float more = 0.f;
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
                            more = (f.x + f.y) * shift.exact();
                        } else {  // value by value
                            for (int i = 0; i < UNITS; ++i) {
                                const T *at = reinterpret_cast<const T *>(part + i0 + i * CONSUMERS);
                                for (int j = 0; j < PER; ++j) more += exp2_fast((to_f(at[j]) - m) * c);
                            }
                        }
                        st = {m, fmaf(st.s, exp2_fast((st.m - m) * c), more)};
                    };
                    int i0 = t;
                    for (; i0 + (ROUND - 1) * CONSUMERS < n; i0 += ROUND * CONSUMERS) round(i0, std::integral_constant<int, ROUND>());
                    for (; i0 < n; i0 += CONSUMERS) round(i0, std::integral_constant<int, 1>());
                }
                if (PART != Part::Grad && last) {
                    // lanes, then the warps' results in every warp: the same sums in all
                    const int p = turn & 1;
                    const float m = warp_max(st.m);
                    st = {m, warp_sum(st.s * exp2_fast((st.m - m) * c))};
                    if constexpr (CLUSTER) {
                        const int mine = rank * WARPS + t / 32;
                        const bool fine = !has_given_up(&gave_up);
                        if (fine && t == 0) ptx::mbar_arrive_expect_tx(&meeting.bar[p], static_cast<uint32_t>(ranks * WARPS) * sizeof(float2));
                        if (fine && lane < ranks) {
                            uint32_t to, signal;
                            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(ptx::smem_u32(&meeting.of_warp[p][mine])), "r"(lane));
                            asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(signal) : "r"(ptx::smem_u32(&meeting.bar[p])), "r"(lane));
                            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to),
                                         "f"(st.m), "f"(st.s), "r"(signal)
                                         : "memory");
                        }
                        wait(ptx::smem_u32(&meeting.bar[p]), static_cast<uint32_t>(turn >> 1) & 1u, &gave_up);
                    } else {
                        if (lane == 0) meeting.of_warp[p][t / 32] = make_float2(st.m, st.s);
                        sync();
                    }
                    const int all = CLUSTER ? ranks * WARPS : WARPS;
                    Stats some{-FLT_MAX, 0.f};
                    for (int i = lane; i < all; i += 32) {
                        const float2 one = meeting.of_warp[p][i];
                        const float top = fmaxf(some.m, one.x);
                        some = {top, some.s * exp2_fast((some.m - top) * c) + one.y * exp2_fast((one.x - top) * c)};
                    }
                    const float top = warp_max(some.m);
                    st = {top, warp_sum(some.s * exp2_fast((some.m - top) * c))};
                    ++turn;
                }
                if constexpr (PART != Part::Loss) {
                    const Shift shift(st.m, c);
                    const float scale = h.weight / st.s;
                    auto value = [&](float z) { return from_f<T>(exp2_fast((z - st.m) * c) * scale); };
                    if (aligned && !shift.wide) {
                        const f2 factor = both(scale * shift.exact());
#pragma unroll 4
                        for (int i = t; i < n; i += CONSUMERS) {
                            Unit<T> v;
                            v.v = part[i];
                            Words<T, PER> w;
#pragma unroll
                            for (int j = 0; j < PER / 2; ++j) {
                                const float2 f = halves(mul2(shift.exp(v.get(j)), factor));
                                w.set(j, f.x, f.y);
                            }
                            *reinterpret_cast<uint4 *>(out + in.first(u + i)) = make_uint4(w.w[0], w.w[1], w.w[2], w.w[3]);
                        }
                    } else {
                        const T *from = reinterpret_cast<const T *>(part);
                        const int64_t first = in.first(u);
                        for (int i = t; i < n * PER; i += CONSUMERS) out[first + i] = value(to_f(from[i]));
                    }
                    if (last) {
                        if (edge >= 0) out[edge] = value(h.edge[t]);
                        sync();  // over what has been written: the teacher's tokens,
                        if (h.taught) {
                            for (int k = CONSUMERS - 1 - t; k < K; k += CONSUMERS) {  // (the first warp has the loss to do)
                                const int32_t token = token_of[k];
                                // the rank that has written the token's place
                                const bool outside = token < in.head || token >= in.V - in.tail;
                                const int at = (token - in.head) / PER;
                                if (token < 0 || token >= in.V || (outside ? rank != 0 : at < u0 || at >= end)) continue;
                                float q;
                                if (taught_at(q_of, token_of, k, padded, q))
                                    out[token] = from_f<T>(exp2_fast((z_of[k] - st.m) * c) * scale - q * h.weight);
                            }
                        } else {
                            clear();  // or, where there is nothing to learn from, zeros
                        }
                    }
                }
                if (PART != Part::Grad && last && rank == 0 && t < 32) {
                    const float cross = h.taught ? cross_of(q_of, z_of, K, lane, st.m, rtau) : 0.f;
                    if (lane == 0) {
                        o.loss[row] = h.taught ? h.entropy - cross + logf(st.s) : 0.f;
                        keep_normalizers(o.normalizers, row, st.m, st.s);
                    }
                }
                release();
                if (last) break;
                u += n;
            }
        }
    }
    __syncwarp();
    leave(&gave_up, &g_timed_out);
}

// Threads that take a row's sums and the bytes of a stage: larger ones for
// longer rows, so that what a row costs beside its bytes (the reduction, the
// hand-over) stays in proportion, as many blocks an SM as fit beside each
// other.
struct Plan {
    int consumers, stage_units, ranks;
    bool cluster;
};
// Units of 16 bytes that a row may have
int64_t most_units(const rlscan_distill_args &a) { return a.V / (a.dtype == RLSCAN_BF16 ? 8 : 4); }

// Part::Both keeps a block's slice of a row in one stage: of 25 KB where up to
// eight blocks hold a row so (4 x 1023 x 50257 bfloat16 134 us; of 47 KB, two
// blocks an SM instead of four, 169), of 47 KB and then of 100 KB for longer
// ones.  The others take longer rows in several parts, the loss in the smaller
// ones (8 x 1024 x 131072 302 us, in the larger 318), the gradient, which has no
// sums to wait for, in the larger (4 x 1023 x 50257 121 us, in ones of 34 KB
// 128).  Rows are split further while there are too few of them to give every
// SM two blocks (four, where as many fit: 1 x 64 x 50257 both 19 us, so 14).
Plan plan(const rlscan_distill_args &a, Part part)
{
    const int64_t units = most_units(a), rows = a.N * a.T, sms = sm_count() > 0 ? sm_count() : 152;
    if (units <= kStageUnits[0]) return {64, kStageUnits[0], 1, false};
    if (units <= kStageUnits[1]) return {128, kStageUnits[1], 1, false};
    Plan p{kMostConsumers, kStageUnits[2], 1, false};
    if (part == Part::Loss || (part == Part::Both && units <= kGatedCluster * kStageUnits[1])) p = {128, kStageUnits[1], 1, false};
    if (part == Part::Both) {
        if (units > int64_t{kGatedCluster} * p.stage_units) p.stage_units = kWideUnits;
        p.ranks = static_cast<int>(ceil_div(units, p.stage_units));
    }
    while (2 * p.ranks <= kGatedCluster && rows * p.ranks < 2 * sms && ceil_div(units, p.ranks) > 512) p.ranks *= 2;
    p.cluster = p.ranks > 1 && part != Part::Grad;
    return p;
}

template <class T, int CONSUMERS, Part PART, bool CLUSTER>
rlscan_status launch_stream(const rlscan_distill_args &a, const DistillOut &o, Plan p, cudaStream_t s)
{
    auto kernel = distill_kernel<T, CONSUMERS, PART, CLUSTER>;
    // as much shared memory as any call of this kernel takes, for the limit and for the blocks that fit
    const bool wide = p.stage_units == kWideUnits;
    const size_t stages = static_cast<size_t>(kStages) * p.stage_units * 16, smem = stages + kStages * 12 * ((a.K + 3) / 4 * 4);
    const size_t limit = static_cast<size_t>(kStages) * (CONSUMERS == kMostConsumers ? kWideUnits : p.stage_units) * 16 + kStages * 12 * kMostTeacher;
    static PerDevice raised, resident[2][kGatedCluster + 1];
    const int device = current_device();
    if (raised.get(device, [&] {
            return ok(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(limit))) ? 1 : 0;
        }) <= 0)
        return RLSCAN_ERR_CUDA;
    const int cluster = CLUSTER ? p.ranks : 1;
    const int groups_fit = resident[wide ? 1 : 0][cluster].get(device, [&] {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(cluster));
        cfg.blockDim = dim3(CONSUMERS + 32);
        cfg.dynamicSmemBytes = stages + kStages * 12 * 64;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        return ok(cudaOccupancyMaxActiveClusters(&n, kernel, &cfg)) ? n : 0;
    });
    const int64_t rows = a.N * a.T, fit = groups_fit > 0 ? groups_fit : 1;
    int64_t groups = CLUSTER ? fit : fit / p.ranks;  // that share a row
    groups = groups < 1 ? 1 : groups < rows ? groups : rows;
    return launch_cluster(groups * p.ranks <= sm_count(), kernel, groups * p.ranks, CONSUMERS + 32, smem, cluster, s, a, o, p.ranks, p.stage_units);
}

template <class T, Part PART>
rlscan_status run(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s)
{
    if (most_units(a) <= kShortUnits) return launch_distill_short(a, PART, o, s);
    const Plan p = plan(a, PART);
    switch (p.consumers) {
    case 64: return launch_stream<T, 64, PART, false>(a, o, p, s);
    case 128:
        if constexpr (PART != Part::Grad)
            if (p.cluster) return launch_stream<T, 128, PART, true>(a, o, p, s);
        return launch_stream<T, 128, PART, false>(a, o, p, s);
    default:  // (the loss takes long rows with 128)
        if constexpr (PART == Part::Both)
            if (p.cluster) return launch_stream<T, kMostConsumers, PART, true>(a, o, p, s);
        if constexpr (PART != Part::Loss) return launch_stream<T, kMostConsumers, PART, false>(a, o, p, s);
        return RLSCAN_ERR_SHAPE;
    }
}

template <Part PART>
rlscan_status run_typed(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s)
{
    return a.dtype == RLSCAN_BF16 ? run<bf16, PART>(a, o, s) : run<float, PART>(a, o, s);
}

}  // namespace

rlscan_status launch_distill(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s) { return run_typed<Part::Loss>(a, o, s); }

rlscan_status launch_distill_backward(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s)
{
    return run_typed<Part::Grad>(a, o, s);
}

bool distill_fits(const rlscan_distill_args &a) { return most_units(a) <= int64_t{kGatedCluster} * kWideUnits; }

rlscan_status launch_distill_both(const rlscan_distill_args &a, const DistillOut &o, cudaStream_t s) { return run_typed<Part::Both>(a, o, s); }

rlscan_status distill_status(cudaStream_t s) { return take_flag(g_timed_out, s); }

}  // namespace seq
}  // namespace rlscan
