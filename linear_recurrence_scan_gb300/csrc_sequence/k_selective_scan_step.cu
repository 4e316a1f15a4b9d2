// k_selective_scan_step.cu -- the selective scan for one token of each of many
// sequences, their states in slots that are updated in place.
#include "sequence.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kThreads = 128;

// One token: a lane has four states of one channel, of ROWS sequences, whose
// states are in flight together and share its row of A.  What a sequence and
// channel need once (softplus, the gate, the output) is shared out over the
// channel's lanes, one sequence a lane.  VEC: states and A, B and C in whole
// units of four.  Bound by the states' bytes, then by instructions: 256 x
// 4096 x 16 bf16 takes 27 us with four sequences a lane (142 MB, 5.3 TB/s),
// 34 us with two, 36 us with one.
struct StepArgs {
    float *state;
    int64_t P;
    const int32_t *slots;
    void *y;
};

template <class T, int LANES, int ROWS, bool VEC>
__global__ void __launch_bounds__(kThreads)
    step_kernel(const __grid_constant__ rlscan_selective_scan_args a, const __grid_constant__ StepArgs q)
{
    constexpr int CH = kThreads / LANES, SHARE = LANES / ROWS;  // lanes that prepare the same sequence
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, sl = lane % LANES, s0 = 4 * sl, S = static_cast<int>(a.S);
    const Division at_block = divide(blockIdx.x, (a.D + CH - 1) / CH);
    const int64_t d = at_block.r * CH + threadIdx.x / LANES, n0 = at_block.q * ROWS;
    const bool live = d < a.D, mine = live && s0 < S;
    const int64_t dd = live ? d : a.D - 1;
    float *state[ROWS];  // the lane's, null: idle
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t n = n0 + r;
        const int64_t slot = n < a.N ? (q.slots != nullptr ? q.slots[n] : n) : -1;
        state[r] = slot >= 0 && slot < q.P ? q.state + (slot * a.D + dd) * S + s0 : nullptr;
    }
    auto four = [&](auto &v, const auto *p, bool on) {  // states s0 .. s0+3, 0 past the last
        v.zero();
        if constexpr (VEC) {
            if (on) v.load(p);
        } else {
            const float e0 = on ? to_f(p[0]) : 0.f, e1 = on && s0 + 1 < S ? to_f(p[1]) : 0.f;
            const float e2 = on && s0 + 2 < S ? to_f(p[2]) : 0.f, e3 = on && s0 + 3 < S ? to_f(p[3]) : 0.f;
            v.set(0, e0, e1);
            v.set(1, e2, e3);
        }
    };
    Words<float, 4> h[ROWS], A;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) four(h[r], state[r], mine && state[r] != nullptr);
    // the sequence that the lane prepares
    const int64_t n = n0 + sl / SHARE, nn = n < a.N ? n : a.N - 1;
    Words<T, 1> xw, dw, zw;
    xw.load(static_cast<const T *>(a.x.data) + nn * a.x.row_stride + dd);
    dw.load(static_cast<const T *>(a.delta.data) + nn * a.delta.row_stride + dd);
    zw.zero();
    if (a.z.data != nullptr) zw.load(static_cast<const T *>(a.z.data) + nn * a.z.row_stride + dd);
    Words<T, 4> B[ROWS], C[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t m = n0 + r < a.N ? n0 + r : a.N - 1;
        four(B[r], static_cast<const T *>(a.B.data) + m * a.B.row_stride + s0, s0 < S);
        four(C[r], static_cast<const T *>(a.C.data) + m * a.C.row_stride + s0, s0 < S);
    }
    four(A, a.A + dd * S + s0, s0 < S);
    const float bias = a.delta_bias != nullptr ? a.delta_bias[dd] : 0.f, skip = a.skip != nullptr ? a.skip[dd] : 0.f;
    const float xv = xw[0], zv = zw[0];
    float dt = dw[0] + bias;
    if (a.delta_softplus) dt = softplus(dt);
    const float dtx = dt * xv;
    float A2[4], sum[ROWS];
#pragma unroll
    for (int i = 0; i < 4; ++i) A2[i] = A[i] * kLog2e;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const float t = __shfl_sync(0xffffffffu, dt, r * SHARE, LANES), tx = __shfl_sync(0xffffffffu, dtx, r * SHARE, LANES);
        float v[4];
        sum[r] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = fmaf(decay(t, A2[i]), h[r][i], tx * B[r][i]);
            sum[r] = fmaf(C[r][i], v[i], sum[r]);
        }
        if (mine && state[r] != nullptr) {
            if constexpr (VEC) {
                *reinterpret_cast<float4 *>(state[r]) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (s0 + i < S) state[r][i] = v[i];
            }
        }
    }
    bool idle = false;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) idle = r == sl / SHARE ? state[r] == nullptr : idle;
    scatter_sums<ROWS, LANES / 2, 1>(sum, lane);  // leaves the lane its sequence's
    float v = fmaf(skip, xv, sum[0]);
    if (a.z.data != nullptr) v *= zv * sigmoid(zv);
    if (live && sl % SHARE == 0 && n < a.N) static_cast<T *>(q.y)[n * a.D + d] = from_f<T>(idle ? 0.f : v);
}

template <class T>
rlscan_status step_typed(const rlscan_selective_scan_args &a, float *state, int64_t P, const int32_t *slots, void *y,
                         cudaStream_t s)
{
    const StepArgs q{state, P, slots, y};
    Chunk bc;
    for (const rlscan_array3 *v : {&a.B, &a.C}) bc.add(v->data, v->row_stride, 0, sizeof(T));
    const bool vec = a.S % 4 == 0 && bc.bits % (4 * sizeof(T)) == 0 &&
                     ((reinterpret_cast<uintptr_t>(state) | reinterpret_cast<uintptr_t>(a.A)) & 15u) == 0;
    auto go = [&](auto lanes) {
        constexpr int LANES = decltype(lanes)::value, MANY = LANES < 4 ? LANES : 4;
        const int64_t across = ceil_div(a.D, kThreads / LANES), sms = sm_count() > 0 ? sm_count() : 152;
        // several sequences a lane while that leaves two blocks an SM
        if (ceil_div(a.N, MANY) * across >= 2 * sms)
            return vec ? launch_overlapped(step_kernel<T, LANES, MANY, true>, ceil_div(a.N, MANY) * across, kThreads, 0, s, a, q)
                       : launch_overlapped(step_kernel<T, LANES, MANY, false>, ceil_div(a.N, MANY) * across, kThreads, 0, s, a, q);
        return vec ? launch_overlapped(step_kernel<T, LANES, 1, true>, a.N * across, kThreads, 0, s, a, q)
                   : launch_overlapped(step_kernel<T, LANES, 1, false>, a.N * across, kThreads, 0, s, a, q);
    };
    switch (state_lanes(a.S)) {
    case 1: return go(std::integral_constant<int, 1>());
    case 2: return go(std::integral_constant<int, 2>());
    case 4: return go(std::integral_constant<int, 4>());
    case 8: return go(std::integral_constant<int, 8>());
    case 16: return go(std::integral_constant<int, 16>());
    default: return go(std::integral_constant<int, 32>());
    }
}

}  // namespace

rlscan_status launch_selective_scan_step(const rlscan_selective_scan_args &a, float *state, int64_t P,
                                         const int32_t *slots, void *y, cudaStream_t s)
{
    return a.dtype == RLSCAN_BF16 ? step_typed<bf16>(a, state, P, slots, y, s)
                                  : step_typed<float>(a, state, P, slots, y, s);
}

}  // namespace seq
}  // namespace rlscan
