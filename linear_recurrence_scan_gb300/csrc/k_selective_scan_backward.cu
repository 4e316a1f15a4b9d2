// k_selective_scan_backward.cu -- gradients of the selective scan.
//
// With g the gradient of sum_s C h and G_t = C_t g_t + exp(dt_{t+1} A) G_{t+1}
// the gradient of h_t, segments of kCheckpoint tokens are taken from the last
// to the first: the states are made again from the segment's checkpoint and
// kept in registers, then G runs back over them.  exp(dt A) h_{t-1} is
// h_t - dt x B, so that the previous state is not needed.
#include "sequence.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kThreads = 128;
constexpr int L = kCheckpoint;

struct GradArgs {
    rlscan_array3 grad_y;
    const float *grad_final, *checkpoints;
    void *x, *delta, *z;
    float *initial_state;
    float *part_B, *part_C;  // [channel blocks][N T S]
    float *part_A;           // [N][D S]
    float *part_d;           // [N][2][D]: skip, delta_bias
};

template <class T, int LANES>
__global__ void __launch_bounds__(kThreads)
    grad_kernel(const __grid_constant__ rlscan_selective_scan_args a, const __grid_constant__ GradArgs g)
{
    constexpr int CH = 32 / LANES;
    const int lane = threadIdx.x & 31, sl = lane % LANES;
    const int64_t blocks = (a.D + CH - 1) / CH;
    const int64_t warp = blockIdx.x * static_cast<int64_t>(kThreads / 32) + threadIdx.x / 32;
    if (warp >= a.N * blocks) return;
    const int64_t n = warp / blocks, block = warp % blocks, d = block * CH + lane / LANES;
    const bool live = d < a.D;
    const int64_t dd = live ? d : a.D - 1;
    const int s0 = 4 * sl, S = static_cast<int>(a.S);
    const int64_t marks = (a.T + L - 1) / L;
    float A1[4], G[4], dA[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        A1[i] = s0 + i < S ? a.A[dd * S + s0 + i] : 0.f;
        G[i] = live && s0 + i < S && g.grad_final != nullptr ? g.grad_final[(n * a.D + dd) * S + s0 + i] : 0.f;
    }
    const float bias = a.delta_bias != nullptr ? a.delta_bias[dd] : 0.f;
    const float skip = a.skip != nullptr ? a.skip[dd] : 0.f;
    const T *x = static_cast<const T *>(a.x.data) + n * a.x.row_stride + dd;
    const T *delta = static_cast<const T *>(a.delta.data) + n * a.delta.row_stride + dd;
    const T *z = a.z.data != nullptr ? static_cast<const T *>(a.z.data) + n * a.z.row_stride + dd : nullptr;
    const T *gy = static_cast<const T *>(g.grad_y.data) + n * g.grad_y.row_stride + dd;
    const T *B = static_cast<const T *>(a.B.data) + n * a.B.row_stride;
    const T *C = static_cast<const T *>(a.C.data) + n * a.C.row_stride;
    T *gx = static_cast<T *>(g.x), *gdelta = static_cast<T *>(g.delta), *gz = static_cast<T *>(g.z);
    const int64_t len = row_length(a.lengths, n, a.T);
    float dskip = 0.f, dbias = 0.f;

    for (int64_t t = a.T - 1; t >= len; --t) {
        const int64_t e = (n * a.T + t) * a.D + dd;
        if (live && sl == 0) {
            gx[e] = from_f<T>(0.f);
            if (gdelta != nullptr) gdelta[e] = from_f<T>(0.f);
            if (gz != nullptr) gz[e] = from_f<T>(0.f);
        }
        if (lane < LANES)
            for (int i = 0; i < 4; ++i)
                if (s0 + i < S) {
                    const int64_t p = (block * a.N * a.T + n * a.T + t) * S + s0 + i;
                    if (g.part_B != nullptr) g.part_B[p] = 0.f;
                    if (g.part_C != nullptr) g.part_C[p] = 0.f;
                }
    }
    for (int64_t m = (len + L - 1) / L - 1; m >= 0; --m) {
        const int64_t t0 = m * L;
        const int count = static_cast<int>(len - t0 < L ? len - t0 : L);
        float h[L][4];
        float start[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            start[i] = s0 + i < S ? g.checkpoints[((n * marks + m) * a.D + dd) * S + s0 + i] : 0.f;
#pragma unroll
        for (int k = 0; k < L; ++k) {
            const int64_t t = t0 + k;
            if (k < count) {
                const bool reset = a.resets != nullptr && a.resets[n * a.T + t] != 0;
                const float xv = to_f(x[t * a.x.token_stride]);
                float dt = to_f(delta[t * a.delta.token_stride]) + bias;
                if (a.delta_softplus) dt = softplus(dt);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float b = s0 + i < S ? to_f(B[t * a.B.token_stride + s0 + i]) : 0.f;
                    const float before = reset ? 0.f : (k > 0 ? h[k > 0 ? k - 1 : 0][i] : start[i]);
                    h[k][i] = fmaf(exp2_fast(dt * (A1[i] * kLog2e)), before, dt * xv * b);
                }
            }
        }
#pragma unroll
        for (int k = L - 1; k >= 0; --k) {
            const int64_t t = t0 + k;
            if (k >= count) continue;
            const bool reset = a.resets != nullptr && a.resets[n * a.T + t] != 0;
            const float xv = to_f(x[t * a.x.token_stride]);
            const float pre = to_f(delta[t * a.delta.token_stride]) + bias;
            const float dt = a.delta_softplus ? softplus(pre) : pre;
            const float dtx = dt * xv;
            float gv = live ? to_f(gy[t * g.grad_y.token_stride]) : 0.f;
            float zv = 0.f, sg = 0.f, out = gv;
            if (z != nullptr) {
                zv = to_f(z[t * a.z.token_stride]);
                sg = sigmoid(zv);
                gv = out * (zv * sg);
            }
            float u = 0.f, w = 0.f, yv = 0.f, gB[4], gC[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float b = s0 + i < S ? to_f(B[t * a.B.token_stride + s0 + i]) : 0.f;
                const float c = s0 + i < S ? to_f(C[t * a.C.token_stride + s0 + i]) : 0.f;
                G[i] = fmaf(c, gv, G[i]);
                yv = fmaf(c, h[k][i], yv);
                gC[i] = gv * h[k][i];
                gB[i] = G[i] * dtx;
                u = fmaf(G[i], b, u);
                const float q = reset ? 0.f : G[i] * fmaf(-dtx, b, h[k][i]);
                w = fmaf(q, A1[i], w);
                dA[i] = fmaf(q, dt, dA[i]);
                G[i] = reset ? 0.f : G[i] * exp2_fast(dt * (A1[i] * kLog2e));
            }
#pragma unroll
            for (int s = LANES / 2; s > 0; s /= 2) {
                u += __shfl_xor_sync(0xffffffffu, u, s);
                w += __shfl_xor_sync(0xffffffffu, w, s);
                yv += __shfl_xor_sync(0xffffffffu, yv, s);
            }
            // over the warp's channels
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                gB[i] = live ? gB[i] : 0.f;
                gC[i] = live ? gC[i] : 0.f;
            }
#pragma unroll
            for (int s = 16; s >= LANES; s /= 2)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    gB[i] += __shfl_xor_sync(0xffffffffu, gB[i], s);
                    gC[i] += __shfl_xor_sync(0xffffffffu, gC[i], s);
                }
            if (lane < LANES)
                for (int i = 0; i < 4; ++i)
                    if (s0 + i < S) {
                        const int64_t p = (block * a.N * a.T + n * a.T + t) * S + s0 + i;
                        if (g.part_B != nullptr) g.part_B[p] = gB[i];
                        if (g.part_C != nullptr) g.part_C[p] = gC[i];
                    }
            float gd = fmaf(u, xv, w);
            if (a.delta_softplus) gd *= sigmoid(pre);
            dskip = fmaf(gv, xv, dskip);
            dbias += gd;
            if (live && sl == 0) {
                const int64_t e = (n * a.T + t) * a.D + d;
                gx[e] = from_f<T>(fmaf(u, dt, gv * skip));
                if (gdelta != nullptr) gdelta[e] = from_f<T>(gd);
                if (gz != nullptr)
                    gz[e] = from_f<T>(out * fmaf(skip, xv, yv) * sg * fmaf(zv, 1.f - sg, 1.f));
            }
        }
    }
    if (!live) return;
    for (int i = 0; i < 4; ++i) {
        if (s0 + i >= S) break;
        if (g.initial_state != nullptr) g.initial_state[(n * a.D + d) * S + s0 + i] = G[i];
        if (g.part_A != nullptr) g.part_A[(n * a.D + d) * S + s0 + i] = dA[i];
    }
    if (g.part_d != nullptr && sl == 0) {
        g.part_d[(n * 2 + 0) * a.D + d] = dskip;
        g.part_d[(n * 2 + 1) * a.D + d] = dbias;
    }
}

__global__ void sum_parts_kernel(const float *part, int64_t parts, int64_t pitch, int64_t m, void *out, int bf16_out)
{
    const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
    if (i >= m) return;
    float acc = 0.f;
    for (int64_t w = 0; w < parts; ++w) acc += part[w * pitch + i];
    if (bf16_out)
        static_cast<bf16 *>(out)[i] = from_f<bf16>(acc);
    else
        static_cast<float *>(out)[i] = acc;
}

struct Layout {
    int64_t blocks;
    size_t B, C, A, d, bytes;
};

Layout layout(const rlscan_selective_scan_args &a)
{
    Layout l;
    l.blocks = ceil_div(a.D, 32 / state_lanes(a.S));
    const size_t bc = sizeof(float) * static_cast<size_t>(l.blocks) * a.N * a.T * a.S;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    l.B = 0;
    l.C = up(bc);
    l.A = l.C + up(bc);
    l.d = l.A + up(sizeof(float) * static_cast<size_t>(a.N) * a.D * a.S);
    l.bytes = l.d + up(sizeof(float) * 2 * static_cast<size_t>(a.N) * a.D);
    return l;
}

template <class T>
rlscan_status launch_typed(const rlscan_selective_scan_args &a, const GradArgs &g, cudaStream_t s)
{
    const int lanes = state_lanes(a.S);
    const unsigned grid = static_cast<unsigned>(ceil_div(a.N * ceil_div(a.D, 32 / lanes), kThreads / 32));
    switch (lanes) {
    case 1: grad_kernel<T, 1><<<grid, kThreads, 0, s>>>(a, g); break;
    case 2: grad_kernel<T, 2><<<grid, kThreads, 0, s>>>(a, g); break;
    case 4: grad_kernel<T, 4><<<grid, kThreads, 0, s>>>(a, g); break;
    case 8: grad_kernel<T, 8><<<grid, kThreads, 0, s>>>(a, g); break;
    case 16: grad_kernel<T, 16><<<grid, kThreads, 0, s>>>(a, g); break;
    default: grad_kernel<T, 32><<<grid, kThreads, 0, s>>>(a, g); break;
    }
    return launched();
}

}  // namespace

rlscan_status launch_sum_parts(const float *part, int64_t parts, int64_t pitch, int64_t m, void *out, bool bf16_out,
                               cudaStream_t s)
{
    if (m == 0) return RLSCAN_OK;
    sum_parts_kernel<<<static_cast<unsigned>(ceil_div(m, 256)), 256, 0, s>>>(part, parts, pitch, m, out, bf16_out);
    return launched();
}

size_t selective_scan_backward_workspace(const rlscan_selective_scan_args &a) { return layout(a).bytes; }

rlscan_status launch_selective_scan_backward(const rlscan_selective_scan_args &a, const rlscan_array3 &grad_y,
                                             const float *grad_final_state, const float *checkpoints,
                                             const rlscan_selective_scan_grads &g, void *ws, cudaStream_t s)
{
    const Layout l = layout(a);
    char *w = static_cast<char *>(ws);
    GradArgs k;
    k.grad_y = grad_y;
    k.grad_final = grad_final_state;
    k.checkpoints = checkpoints;
    k.x = g.x;
    k.delta = g.delta;
    k.z = g.z;
    k.initial_state = g.initial_state;
    k.part_B = g.B != nullptr ? reinterpret_cast<float *>(w + l.B) : nullptr;
    k.part_C = g.C != nullptr ? reinterpret_cast<float *>(w + l.C) : nullptr;
    k.part_A = g.A != nullptr ? reinterpret_cast<float *>(w + l.A) : nullptr;
    k.part_d = g.skip != nullptr || g.delta_bias != nullptr ? reinterpret_cast<float *>(w + l.d) : nullptr;
    const bool b16 = a.dtype == RLSCAN_BF16;
    if (a.N > 0) {
        const rlscan_status st = b16 ? launch_typed<bf16>(a, k, s) : launch_typed<float>(a, k, s);
        if (st != RLSCAN_OK) return st;
    }
    const int64_t bc = a.N * a.T * a.S;
    rlscan_status st = RLSCAN_OK;
    if (g.B != nullptr) st = launch_sum_parts(k.part_B, l.blocks, bc, bc, g.B, b16, s);
    if (st == RLSCAN_OK && g.C != nullptr) st = launch_sum_parts(k.part_C, l.blocks, bc, bc, g.C, b16, s);
    if (st == RLSCAN_OK && g.A != nullptr) st = launch_sum_parts(k.part_A, a.N, a.D * a.S, a.D * a.S, g.A, false, s);
    if (st == RLSCAN_OK && g.skip != nullptr) st = launch_sum_parts(k.part_d, a.N, 2 * a.D, a.D, g.skip, false, s);
    if (st == RLSCAN_OK && g.delta_bias != nullptr)
        st = launch_sum_parts(k.part_d + a.D, a.N, 2 * a.D, a.D, g.delta_bias, false, s);
    return st;
}

}  // namespace seq
}  // namespace rlscan
