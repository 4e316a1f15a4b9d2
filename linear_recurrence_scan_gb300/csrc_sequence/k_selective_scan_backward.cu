// k_selective_scan_backward.cu -- gradients of the selective scan.
//
// With g the gradient of sum_s C h and G_t = C_t g_t + exp(dt_{t+1} A) G_{t+1}
// the gradient of h_t, tiles of 16 tokens are taken from the last to the
// first.  The states are made again from the tile's checkpoint, 4 tokens at a
// time, and stay in registers while G runs back over them.  G exp(dt A) h_{t-1}
// is the message to the token before, which is needed anyway, times its state;
// h_t - dt x B in its place would leave the rounding of h_t, far above the
// gradient of a rate that decays within a token (rate 16, time steps of about
// 0.7, 1.3, 2.1: that gradient 3e-7, 2e-7, 6e-7 off, by the difference 6e-5,
// 2e-3, 1.8).
//
// A lane holds four channels x four states, in pairs of channels: the sums
// over channels (dB, dC) start in its registers, which leaves an eighth of
// the shuffles that one channel a lane would need.  What each channel and
// token needs once (softplus, the gate, the outputs) is shared out over the
// lanes through shared memory.
//
// Instructions bound it, 408 for a warp (32 channels x 16 states) and token,
// at the two warps a scheduler that 255 registers leave.  Measured, 8 x 512 x
// 4096 x 16 bf16: 379 us, 59 % of the issue slots where an SM has two blocks;
// 8 x 2048 x 4096 with the forward pass 1989 us.  (Tried when that was 1994:
// three blocks an SM at 168 registers, with spills, 3088; two channels a lane
// and four blocks 2234.)
#include "scan_plan.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kTile = kCheckpoint;
// Tokens whose states are in registers.  Eight need fewer steps made again,
// but their code no longer fits the instruction cache (measured, 8 x 2048 x
// 4096 bf16 with the forward pass: 8: 2992 us, 4: 2294 us).
constexpr int kSub = 4;
constexpr float kLn2 = 0.6931471805599453f;

struct GradArgs {
    rlscan_array3 grad_y;
    const float *grad_final;  // of the final state; with chunks the messages behind them [N][chunks][D][S]
    const float *checkpoints;
    int64_t chunk, chunks;    // rows in chunks of tokens
    void *x, *delta, *z;
    float *initial_state;
    float *part_B, *part_C;  // [channel blocks][N T S]
    float *part_A;           // [N chunks][D S]
    float *part_d;           // [N chunks][2][D]: skip, delta_bias
    int unit;                // bytes of the copies into shared memory: 16, 4 or 0 (single values)
    bool vec;                // checkpoints in whole 16-byte units
    int64_t sms;             // as ScanOut's
};

template <class T, int LANES>
struct Shape {
    static constexpr int WARPS = LANES == 2 ? 2 : 4, THREADS = 32 * WARPS;
    static constexpr int GROUPS = 32 / LANES;
    static constexpr int CW = 4 * GROUPS, CH = WARPS * CW;  // channels of a warp, of a block
    static constexpr int SP = 4 * LANES;                    // states, padded
    static constexpr int SHARE = LANES >= 4 ? LANES / 4 : 1;  // lanes that end up with the same sums
    static constexpr int CPL = CW > 32 ? CW / 32 : 1;       // channels a lane prepares
    static constexpr int ITEMS = CW * kTile / 32;           // (channel, token) pairs a lane prepares
    static constexpr int PITCH = CH * static_cast<int>(sizeof(T));
    static constexpr int BPITCH = SP * static_cast<int>(sizeof(T));
    static constexpr int ACT = kTile * PITCH, BC = kTile * BPITCH, MARK = THREADS * 64;
    // two stages, or one where two would leave a single block an SM (float32)
    static constexpr int STAGE = 4 * ACT + 2 * BC + MARK, STAGES = sizeof(T) == 4 ? 1 : 2;
    static constexpr int F = kTile * CW;                    // floats of one array of a warp
    static constexpr int MINE = LANES >= 4 ? 1 : 4 / LANES;  // channels whose sums a lane ends up with
    static constexpr int WIDE = 2 * kTile * SP * 8;         // B and C, each value twice
    static constexpr int RED = WARPS * kTile * 2 * SP * 4;
    static constexpr int KEEP = (kTile / kSub - 2) * MARK;   // states between the sub-tiles
    static constexpr size_t SMEM = STAGES * STAGE + WARPS * 3 * F * 4 + WIDE + RED + KEEP + MARK;
    static_assert(ACT % 16 == 0 && BC % 16 == 0 && BPITCH % 16 == 0 && PITCH % 16 == 0);
};

template <class T, int LANES>
__global__ void __launch_bounds__(Shape<T, LANES>::THREADS)
    grad_kernel(const __grid_constant__ rlscan_selective_scan_args a, const __grid_constant__ GradArgs g)
{
    using P = Shape<T, LANES>;
    extern __shared__ __align__(16) char smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, sl = lane % LANES, group = lane / LANES;
    float *F0 = reinterpret_cast<float *>(smem + P::STAGES * P::STAGE) + warp * 3 * P::F;  // dt
    float *F1 = F0 + P::F, *F2 = F1 + P::F;                                               // dt x, g
    char *wide = smem + P::STAGES * P::STAGE + P::WARPS * 3 * P::F * 4;
    float *red = reinterpret_cast<float *>(wide + P::WIDE);
    char *keep = wide + P::WIDE + P::RED + threadIdx.x * 16;  // the lane's own, as the checkpoint's
    char *sumA = keep + P::KEEP;  // dA: a tile's sum is in registers, the sum over tiles here (two short sums, not one long)
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int64_t blocks = (a.D + P::CH - 1) / P::CH;
    const int64_t place =
        g.sms > 0 ? by_length(a.lengths, static_cast<int>(a.N), blocks, g.sms, reinterpret_cast<int *>(smem)) : blockIdx.x;
    const Division at_block = divide(place, blocks), at_row = divide(at_block.q, g.chunks);
    const int64_t block = at_block.r;
    const int64_t chunk = at_row.r, n = at_row.q;
    const int64_t first = chunk * g.chunk, last = first + g.chunk < a.T ? first + g.chunk : a.T;
    const int64_t c0 = block * P::CH;
    const int S = static_cast<int>(a.S), s0 = 4 * sl;
    const int width = static_cast<int>(a.D - c0 < P::CH ? a.D - c0 : P::CH);
    const int cw = warp * P::CW, c4 = cw + 4 * group;  // the warp's and the lane's first channel in the block
    const int64_t marks = (a.T + kTile - 1) / kTile;
    const int64_t all = row_length(a.lengths, n, a.T), len = all < last ? all : last;  // tokens first <= t < len
    const int64_t low = first / kTile, tiles = len > first ? (len + kTile - 1) / kTile : low;  // tiles low .. tiles-1
    const bool gated = a.z.data != nullptr;
    const uint32_t gate = gated ? ~0u : 0u, soft = a.delta_softplus ? ~0u : 0u;

    const T *x = static_cast<const T *>(a.x.data) + n * a.x.row_stride + c0;
    const T *delta = static_cast<const T *>(a.delta.data) + n * a.delta.row_stride + c0;
    const T *z = static_cast<const T *>(a.z.data) + n * a.z.row_stride + c0;
    const T *gy = static_cast<const T *>(g.grad_y.data) + n * g.grad_y.row_stride + c0;
    const T *B = static_cast<const T *>(a.B.data) + n * a.B.row_stride;
    const T *C = static_cast<const T *>(a.C.data) + n * a.C.row_stride;
    const uint8_t *resets = a.resets != nullptr ? a.resets + n * a.T : nullptr;
    const float *mark = g.checkpoints + (n * marks * a.D + c0 + c4) * S + s0;

    auto copy_tile = [&](auto unit, char *st, int64_t t, int rows) {
        constexpr int CHUNK = decltype(unit)::value;
        load_tile<T, kTile, P::CH, P::PITCH, CHUNK, P::THREADS>(st, x + t * a.x.token_stride, a.x.token_stride, rows, width);
        load_tile<T, kTile, P::CH, P::PITCH, CHUNK, P::THREADS>(st + P::ACT, delta + t * a.delta.token_stride,
                                                                a.delta.token_stride, rows, width);
        if (gated)
            load_tile<T, kTile, P::CH, P::PITCH, CHUNK, P::THREADS>(st + 2 * P::ACT, z + t * a.z.token_stride,
                                                                    a.z.token_stride, rows, width);
        load_tile<T, kTile, P::CH, P::PITCH, CHUNK, P::THREADS>(st + 3 * P::ACT, gy + t * g.grad_y.token_stride,
                                                                g.grad_y.token_stride, rows, width);
        load_tile<T, kTile, P::SP, P::BPITCH, CHUNK, P::THREADS>(st + 4 * P::ACT, B + t * a.B.token_stride,
                                                                 a.B.token_stride, rows, S);
        load_tile<T, kTile, P::SP, P::BPITCH, CHUNK, P::THREADS>(st + 4 * P::ACT + P::BC, C + t * a.C.token_stride,
                                                                 a.C.token_stride, rows, S);
    };
    auto issue = [&](int64_t tile) {  // tiles go down
        if (tile >= low) {
            char *st = smem + tile % P::STAGES * P::STAGE;
            const int64_t t = tile * kTile, left = len - t;
            const int rows = left < kTile ? static_cast<int>(left) : kTile;
            if (g.unit == 16)
                copy_tile(std::integral_constant<int, 16>(), st, t, rows);
            else if (g.unit == 4)
                copy_tile(std::integral_constant<int, 4>(), st, t, rows);
            else
                copy_tile(std::integral_constant<int, 0>(), st, t, rows);
            // the lane's own states, four of each of its channels
            char *own = st + 4 * P::ACT + 2 * P::BC + threadIdx.x * 16;
            const float *m = mark + tile * a.D * S;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const bool on = c4 + c < width;
                if (g.vec) {
                    const bool have = on && s0 < S;
                    copy16(own + c * P::THREADS * 16, have ? m + c * S : g.checkpoints, have ? 16 : 0);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const bool have = on && s0 + i < S;
                        copy4(own + c * P::THREADS * 16 + 4 * i, have ? m + c * S + i : g.checkpoints, have ? 4 : 0);
                    }
                }
            }
        }
        copies_commit();
    };

    // padding: zeros
    for (int64_t t = tiles * kTile; t < last; ++t) {
        const int64_t row = n * a.T + t;
        for (int c = threadIdx.x; c < width; c += P::THREADS) {
            static_cast<T *>(g.x)[row * a.D + c0 + c] = from_f<T>(0.f);
            if (g.delta != nullptr) static_cast<T *>(g.delta)[row * a.D + c0 + c] = from_f<T>(0.f);
            if (g.z != nullptr) static_cast<T *>(g.z)[row * a.D + c0 + c] = from_f<T>(0.f);
        }
        for (int s = threadIdx.x; s < S; s += P::THREADS) {
            if (g.part_B != nullptr) g.part_B[(block * a.N * a.T + row) * S + s] = 0.f;
            if (g.part_C != nullptr) g.part_C[(block * a.N * a.T + row) * S + s] = 0.f;
        }
    }
    issue(tiles - 1);

    // [pair of channels][state]
    f2 A2[2][4], G[2][4], dA[2][4];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[2], f[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int c = c4 + 2 * p + q;
                const bool on = c < width && s0 + i < S;
                v[q] = on ? a.A[(c0 + c) * S + s0 + i] * kLog2e : 0.f;
                f[q] = on && g.grad_final != nullptr ? g.grad_final[((n * g.chunks + chunk) * a.D + c0 + c) * S + s0 + i] : 0.f;
            }
            A2[p][i] = pair(v[0], v[1]);
            G[p][i] = pair(f[0], f[1]);
            dA[p][i] = 0ull;
        }
    auto add_dA = [&](bool first_tile) {
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ulonglong2 *at = reinterpret_cast<ulonglong2 *>(sumA + (2 * p + h) * P::THREADS * 16);
                ulonglong2 v = make_ulonglong2(dA[p][2 * h], dA[p][2 * h + 1]);
                if (!first_tile) v = make_ulonglong2(add2(v.x, at->x), add2(v.y, at->y));
                *at = v;
                dA[p][2 * h] = dA[p][2 * h + 1] = 0ull;
            }
    };
    add_dA(true);
    float bias[P::CPL];  // of the channels the lane prepares
#pragma unroll
    for (int j = 0; j < P::CPL; ++j) {
        const int c = cw + (lane + 32 * j) % P::CW;
        bias[j] = a.delta_bias != nullptr && c < width ? a.delta_bias[c0 + c] : 0.f;
    }
    // the channels whose outputs the lane writes: those that scatter_sums leaves it
    const int mine = 4 * group + (LANES >= 4 ? sl / P::SHARE : sl * P::MINE);
    const bool writes = sl % P::SHARE == 0;
    float obias[P::MINE], skip[P::MINE], dskip[P::MINE], dbias[P::MINE];
#pragma unroll
    for (int i = 0; i < P::MINE; ++i) {
        const int c = cw + mine + i;
        obias[i] = a.delta_bias != nullptr && c < width ? a.delta_bias[c0 + c] : 0.f;
        skip[i] = a.skip != nullptr && c < width ? a.skip[c0 + c] : 0.f;
        dskip[i] = dbias[i] = 0.f;
    }

    for (int64_t tile = tiles - 1; tile >= low; --tile) {
        const int64_t t0 = tile * kTile;
        const int left = len - t0 < kTile ? static_cast<int>(len - t0) : kTile;
        copies_wait<0>();
        __syncthreads();  // the tile is here, and the buffer of the one before is free
        if (P::STAGES > 1) issue(tile - 1);
        const char *st = smem + tile % P::STAGES * P::STAGE;
        const uint32_t starts =
            resets != nullptr ? __ballot_sync(0xffffffffu, lane < left && resets[t0 + lane] != 0) : 0u;
        for (int i = threadIdx.x; i < 2 * kTile * P::SP; i += P::THREADS) {
            const float v = to_f(reinterpret_cast<const T *>(st + 4 * P::ACT)[i]);  // C lies behind B
            reinterpret_cast<float2 *>(wide)[i] = make_float2(v, v);
        }
        const T *xs = reinterpret_cast<const T *>(st) + cw, *ds = reinterpret_cast<const T *>(st + P::ACT) + cw,
                *zs = reinterpret_cast<const T *>(st + 2 * P::ACT) + cw, *ys = reinterpret_cast<const T *>(st + 3 * P::ACT) + cw;
#pragma unroll
        for (int j = 0; j < P::ITEMS; j += 2) {  // two (channel, token) pairs at once
            float xv[2], pre[2], zv[2], gv[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int item = lane + 32 * (j + q), at = item / P::CW * P::CH + item % P::CW;
                xv[q] = to_f(xs[at]);
                zv[q] = to_f(zs[at]);
                gv[q] = to_f(ys[at]);
                pre[q] = to_f(ds[at]) + bias[(j + q) % P::CPL];
            }
            const float2 sp = halves(softplus(pair(pre[0], pre[1]))), sg = halves(sigmoid(pair(zv[0], zv[1])));
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int item = lane + 32 * (j + q);
                const float dt = item / P::CW < left ? choose(soft, q == 0 ? sp.x : sp.y, pre[q]) : 0.f;
                F0[item] = dt;
                F1[item] = dt * xv[q];
                F2[item] = gv[q] * choose(gate, zv[q] * (q == 0 ? sg.x : sg.y), 1.f);
            }
        }
        __syncthreads();
        float sk[P::MINE], sb[P::MINE];  // the tile's share of dskip, dbias: short sums
#pragma unroll
        for (int i = 0; i < P::MINE; ++i) sk[i] = sb[i] = 0.f;

        auto off = [&](const void *p) { return static_cast<uint32_t>(static_cast<const char *>(p) - smem); };
        const uint32_t oB = off(wide) + 32 * sl, oC = oB + kTile * P::SP * 8;
        const uint32_t o0 = off(F0) + 16 * group, o1 = o0 + P::F * 4, o2 = o1 + P::F * 4;
        const char *own = st + 4 * P::ACT + 2 * P::BC + threadIdx.x * 16;
        auto row = [&](uint32_t f, int k, f2 *v) { load_pairs(v[0], v[1], f + k * (P::CW * 4)); };  // a token's four channels
        auto states = [&](uint32_t w, int k, f2 *v) {  // a token's four states, each twice
            load_pairs(v[0], v[1], w + k * (P::SP * 8));
            load_pairs(v[2], v[3], w + k * (P::SP * 8) + 16);
        };
        auto begin = [&](f2 (*h)[4], const char *from) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const float4 u = *reinterpret_cast<const float4 *>(from + 2 * p * P::THREADS * 16);
                const float4 v = *reinterpret_cast<const float4 *>(from + (2 * p + 1) * P::THREADS * 16);
                h[p][0] = pair(u.x, v.x);
                h[p][1] = pair(u.y, v.y);
                h[p][2] = pair(u.z, v.z);
                h[p][3] = pair(u.w, v.w);
            }
        };
        auto save = [&](const f2 (*h)[4], char *to) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const float2 a0 = halves(h[p][0]), a1 = halves(h[p][1]), a2 = halves(h[p][2]), a3 = halves(h[p][3]);
                *reinterpret_cast<float4 *>(to + 2 * p * P::THREADS * 16) = make_float4(a0.x, a1.x, a2.x, a3.x);
                *reinterpret_cast<float4 *>(to + (2 * p + 1) * P::THREADS * 16) = make_float4(a0.y, a1.y, a2.y, a3.y);
            }
        };
        const uint32_t oX = off(xs) + mine * static_cast<uint32_t>(sizeof(T));  // the lane's channel in the raw rows
        const int64_t out = (n * a.T + t0) * a.D + c0 + cw + mine;
        auto walk = [&](auto fast) {
            constexpr bool FAST = decltype(fast)::value;
            auto step = [&](uint32_t base, int k, const f2 (*from)[4], f2 (*to)[4]) {
                f2 d[2], dx[2], b[4];
                row(base + o0, k, d);
                row(base + o1, k, dx);
                states(base + oB, k, b);
                const bool cut = !FAST && (starts >> k & 1u) != 0;
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f2 before = cut ? 0ull : from[p][i];
                        to[p][i] = fma2(dx[p], b[i], mul2(decay(d[p], A2[p][i]), before));
                    }
            };
            // the states at each sub-tile's start: the first is the checkpoint,
            // the last stays in registers, those between go to the lane's own place
            f2 h0[2][4];
            begin(h0, own);
#pragma unroll 1
            for (int k = 0; k < kTile - kSub; k += kSub) {
                if (k > 0) save(h0, keep + (k / kSub - 1) * P::MARK);
                const uint32_t base = anchor(smem);
#pragma unroll
                for (int u = 0; u < kSub; ++u) step(base, k + u, h0, h0);
            }
#pragma unroll 1
            for (int k0 = kTile - kSub; k0 >= 0; k0 -= kSub) {
                f2 h[kSub - 1][2][4];  // the sub-tile's last states are made where they are used
                if (k0 < kTile - kSub) begin(h0, k0 > 0 ? keep + (k0 / kSub - 1) * P::MARK : own);
                uint32_t base = anchor(smem);
#pragma unroll
                for (int k = 0; k < kSub - 1; ++k) step(base, k0 + k, k > 0 ? h[k > 0 ? k - 1 : 0] : h0, h[k]);
                // a new anchor for each part: its loads are its own, not registers held since the part before
                base = anchor(smem);
                constexpr int KEPT = P::GROUPS >= 8 ? 1 : 8 / P::GROUPS;
#pragma unroll
                for (int j = kSub - 1; j >= 0; --j) {
                    const int k = k0 + j;
                    f2 d[2], dx[2], gv[2], b[4], c[4], u[2], w[2], y[2], gB[4], gC[4];
                    row(base + o0, k, d);
                    row(base + o1, k, dx);
                    row(base + o2, k, gv);
                    states(base + oB, k, b);
                    states(base + oC, k, c);
                    const bool cut = !FAST && (starts >> k & 1u) != 0;
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const f2 prior = j > 0 ? h[j > 0 ? j - 1 : 0][p][i] : h0[p][i];
                            const f2 e = decay(d[p], A2[p][i]);
                            const f2 Gt = fma2(c[i], gv[p], G[p][i]);
                            f2 hv, q;  // h_t, G exp(dt A) h_{t-1}
                            if (j == kSub - 1) {
                                const f2 eh = mul2(e, cut ? 0ull : prior);
                                hv = fma2(dx[p], b[i], eh);
                                q = mul2(Gt, eh);
                                G[p][i] = mul2(Gt, e);
                            } else {
                                hv = h[j < kSub - 1 ? j : 0][p][i];
                                G[p][i] = mul2(Gt, e);
                                q = mul2(G[p][i], prior);
                            }
                            if (!FAST) {
                                q = cut ? 0ull : q;
                                G[p][i] = cut ? 0ull : G[p][i];
                            }
                            y[p] = i == 0 ? mul2(hv, c[i]) : fma2(hv, c[i], y[p]);
                            gC[i] = p == 0 ? mul2(hv, gv[p]) : fma2(hv, gv[p], gC[i]);
                            gB[i] = p == 0 ? mul2(Gt, dx[p]) : fma2(Gt, dx[p], gB[i]);
                            u[p] = i == 0 ? mul2(Gt, b[i]) : fma2(Gt, b[i], u[p]);
                            w[p] = i == 0 ? mul2(q, A2[p][i]) : fma2(q, A2[p][i], w[p]);
                            dA[p][i] = fma2(q, d[p], dA[p][i]);
                        }
                    }
                    float bc[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 vb = halves(gB[i]), vc = halves(gC[i]);
                        bc[i] = vb.x + vb.y;
                        bc[4 + i] = vc.x + vc.y;
                    }
                    base = anchor(smem);  // the next token's loads may start here, no sooner
                    const int kept = scatter_sums<8, 16, LANES>(bc, lane);
#pragma unroll
                    for (int i = 0; i < KEPT; ++i) {
                        const int v = kept + i;
                        red[((warp * kTile + k) * 2 + v / 4) * P::SP + s0 + v % 4] = bc[i];
                    }
                    float uv[4], wv[4], yv[4];
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const float2 a0 = halves(u[p]), a1 = halves(w[p]), a2 = halves(y[p]);
                        uv[2 * p] = a0.x;
                        uv[2 * p + 1] = a0.y;
                        wv[2 * p] = a1.x;
                        wv[2 * p + 1] = a1.y;
                        yv[2 * p] = a2.x;
                        yv[2 * p + 1] = a2.y;
                    }
                    scatter_sums<4, LANES / 2, 1>(uv, lane);
                    scatter_sums<4, LANES / 2, 1>(wv, lane);
                    scatter_sums<4, LANES / 2, 1>(yv, lane);
                    const bool on = FAST || k < left;
#pragma unroll
                    for (int m = 0; m < P::MINE; ++m) {
                        const uint32_t raw = base + oX + (k * P::CH + m) * static_cast<uint32_t>(sizeof(T));
                        const float xv = load_value(raw, T()), pre = load_value(raw + P::ACT, T()) + obias[m];
                        const float zv = load_value(raw + 2 * P::ACT, T()), go = load_value(raw + 3 * P::ACT, T());
                        const float dt = load_value(base + off(F0) + (k * P::CW + mine + m) * 4, 0.f), sg = sigmoid(zv);
                        const float gm = go * choose(gate, zv * sg, 1.f);
                        float gd = fmaf(uv[m], xv, wv[m] * kLn2);
                        gd = on ? gd * choose(soft, sigmoid(pre), 1.f) : 0.f;
                        const float gx = on ? fmaf(uv[m], dt, gm * skip[m]) : 0.f;
                        const float gz = on ? go * fmaf(skip[m], xv, yv[m]) * sg * fmaf(zv, 1.f - sg, 1.f) : 0.f;
                        sk[m] = fmaf(gm, xv, sk[m]);
                        sb[m] += gd;
                        const bool st = writes && cw + mine + m < width && (FAST || t0 + k < last);
                        const int64_t e = out + k * a.D + m;
                        if (st) static_cast<T *>(g.x)[e] = from_f<T>(gx);
                        if (st && g.delta != nullptr) static_cast<T *>(g.delta)[e] = from_f<T>(gd);
                        if (st && g.z != nullptr) static_cast<T *>(g.z)[e] = from_f<T>(gz);
                    }
                }
            }
        };
        if (starts == 0 && left == kTile)
            walk(std::true_type());
        else
            walk(std::false_type());
        __syncthreads();
        if (P::STAGES == 1) issue(tile - 1);
        add_dA(false);
#pragma unroll
        for (int m = 0; m < P::MINE; ++m) {
            dskip[m] += sk[m];
            dbias[m] += sb[m];
        }
        // the block's sums over its channels
        for (int i = threadIdx.x; i < 2 * kTile * P::SP; i += P::THREADS) {
            const int k = i / (2 * P::SP), which = i / P::SP % 2, s = i % P::SP;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < P::WARPS; ++w) v += red[w * kTile * 2 * P::SP + i];
            float *part = which == 0 ? g.part_B : g.part_C;
            if (part != nullptr && s < S && t0 + k < a.T)
                part[((block * a.N + n) * a.T + t0 + k) * S + s] = k < left ? v : 0.f;
        }
    }

#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 gi = halves(G[p][i]);
            const float2 ga = halves(reinterpret_cast<const f2 *>(sumA + (2 * p + i / 2) * P::THREADS * 16)[i % 2]);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int c = c4 + 2 * p + q;
                if (c >= width || s0 + i >= S) continue;
                const int64_t e = (c0 + c) * S + s0 + i;
                if (g.initial_state != nullptr && chunk == 0) g.initial_state[n * a.D * S + e] = q == 0 ? gi.x : gi.y;
                if (g.part_A != nullptr) g.part_A[(n * g.chunks + chunk) * a.D * S + e] = q == 0 ? ga.x : ga.y;
            }
        }
    if (g.part_d != nullptr && writes) {
#pragma unroll
        for (int m = 0; m < P::MINE; ++m) {
            const int c = cw + mine + m;
            if (c >= width) break;
            float *part = g.part_d + (n * g.chunks + chunk) * 2 * a.D + c0 + c;
            part[0] = dskip[m];
            part[a.D] = dbias[m];
        }
    }
}

// A block takes 32 columns: 8 threads of four columns x 32 slices of the
// parts.  A slice adds its parts in order, then the slices are added in order.
constexpr int kSlices = 32, kColumns = SumJobs::kColumns;

__global__ void __launch_bounds__(8 * kSlices) sums_kernel(const __grid_constant__ SumJobs jobs)
{
    __shared__ float scratch[kSlices][kColumns + 4];
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    int which = 0;
#pragma unroll
    for (int j = 1; j < SumJobs::kMost; ++j)
        if (j < jobs.count && blockIdx.x >= jobs.job[j].first) which = j;
    const SumJobs::Job &job = jobs.job[which];
    const int slice = threadIdx.x / 8, quad = threadIdx.x % 8;
    const int64_t c0 = (blockIdx.x - job.first) * kColumns, c = c0 + 4 * quad;
    const float *p = job.part + c;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    if (job.vec) {
        if (c < job.m) {
#pragma unroll 4
            for (int64_t w = slice; w < job.parts; w += kSlices) {
                const float4 v = *reinterpret_cast<const float4 *>(p + w * job.pitch);
                acc[0] += v.x;
                acc[1] += v.y;
                acc[2] += v.z;
                acc[3] += v.w;
            }
        }
    } else {
        for (int64_t w = slice; w < job.parts; w += kSlices)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + i < job.m) acc[i] += p[w * job.pitch + i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) scratch[slice][4 * quad + i] = acc[i];
    __syncthreads();
    const int64_t out = c0 + threadIdx.x;
    if (threadIdx.x >= kColumns || out >= job.m) return;
    float sum = scratch[0][threadIdx.x];
#pragma unroll
    for (int s = 1; s < kSlices; ++s) sum += scratch[s][threadIdx.x];
    if (job.bf16_out)
        static_cast<bf16 *>(job.out)[out] = from_f<bf16>(sum);
    else
        static_cast<float *>(job.out)[out] = sum;
}

int grad_lanes(int64_t S)
{
    const int lanes = state_lanes(S);
    return lanes < 2 ? 2 : lanes;
}

// How a call is laid out, and its workspace.  Rows are split into chunks of
// tokens, whose messages take a pass of their own (about a quarter of the
// work), while there are less than 1.5 blocks an SM without; the chunks fill
// whole waves of two blocks an SM.  Measured with the forward pass, against
// chunks for two waves, whole or not, of 64 tokens or more (us): 1 x 509 x
// 1536 126, 96 (chunks of 32);  2 x 300 x 768 113, 88 (32);  2 x 8192 x 1024
// 601, 581;  8 x 500 x 3000 480, 461.  Of rows with lengths nobody knows here
// how many blocks have tokens: chunks for three waves, short enough that the
// last one costs little (ragged 3 x 1500 x 3000: 128: 454, as if all rows were
// full, 384: 488;  4 x 1024 x 2048: 80: 332, 256: 363;  3 x 1001 x 1111 float32:
// 48: 188, 64: 200, 96: 194).
struct Layout {
    int64_t blocks, chunk, chunks;
    size_t B, C, A, d, states, spans, cuts, realigned, bytes;
};

Layout layout(const rlscan_selective_scan_args &a)
{
    Layout l;
    const int lanes = grad_lanes(a.S);
    const int64_t sms = sm_count() > 0 ? sm_count() : 152;
    l.blocks = ceil_div(a.D, (lanes == 2 ? 2 : 4) * 4 * (32 / lanes));
    l.chunk = ceil_div(a.T > 0 ? a.T : 1, kTile) * kTile;
    if (a.N * l.blocks > 0 && a.T > 128 && 2 * a.N * l.blocks < 3 * sms) {
        const int64_t want = ceil_div(6 * sms, a.N * l.blocks), even = ceil_div(ceil_div(a.T, want), kTile) * kTile;
        if (a.lengths != nullptr)
            l.chunk = even < 48 ? 48 : even;
        else
            l.chunk = wave_chunk(a.T, a.N * l.blocks, 2 * sms, 4, a.T + kTile);
    }
    l.chunks = ceil_div(a.T > 0 ? a.T : 1, l.chunk);
    const size_t each = static_cast<size_t>(a.N) * l.chunks, F = sizeof(float);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    l.B = take(F * l.blocks * a.N * a.T * a.S);
    l.C = take(F * l.blocks * a.N * a.T * a.S);
    l.A = take(F * each * a.D * a.S);
    l.d = take(F * each * 2 * a.D);
    const bool split = l.chunks > 1;
    l.states = take(split ? F * each * a.D * a.S : 0);
    l.spans = take(split ? F * each * a.D : 0);
    l.cuts = take(split ? each : 0);
    l.realigned = take(realign_workspace(a, true));
    l.bytes = at;
    return l;
}

template <class T, int LANES>
rlscan_status launch_shape(const rlscan_selective_scan_args &a, const GradArgs &g, cudaStream_t s)
{
    using P = Shape<T, LANES>;
    auto kernel = grad_kernel<T, LANES>;
    static PerDevice raised;
    if (!raise_smem(raised, kernel, P::SMEM)) return RLSCAN_ERR_CUDA;
    const int64_t grid = a.N * ceil_div(a.D, P::CH) * g.chunks;
    return launch(!spread_out(grid, g.sms), kernel, grid, P::THREADS, P::SMEM, s, a, g);
}

template <class T>
rlscan_status launch_typed(const rlscan_selective_scan_args &a, GradArgs g, cudaStream_t s)
{
    Chunk c;
    for (const rlscan_array3 *v : {&a.x, &a.delta, &a.B, &a.C, static_cast<const rlscan_array3 *>(&g.grad_y)})
        c.add(v->data, v->row_stride, v->token_stride, sizeof(T));
    if (a.z.data != nullptr) c.add(a.z.data, a.z.row_stride, a.z.token_stride, sizeof(T));
    g.unit = c.size();
    g.vec = a.S % 4 == 0 && (reinterpret_cast<uintptr_t>(g.checkpoints) & 15u) == 0;
    switch (grad_lanes(a.S)) {
    case 2: return launch_shape<T, 2>(a, g, s);
    case 4: return launch_shape<T, 4>(a, g, s);
    case 8: return launch_shape<T, 8>(a, g, s);
    case 16: return launch_shape<T, 16>(a, g, s);
    default: return launch_shape<T, 32>(a, g, s);
    }
}

}  // namespace

rlscan_status launch_sums(const SumJobs &jobs, cudaStream_t s)
{
    if (jobs.blocks == 0) return RLSCAN_OK;
    return launch_overlapped(sums_kernel, jobs.blocks, 8 * kSlices, 0, s, jobs);
}

size_t selective_scan_backward_workspace(const rlscan_selective_scan_args &a) { return layout(a).bytes; }

rlscan_status launch_selective_scan_backward(const rlscan_selective_scan_args &args, const rlscan_array3 &grad,
                                             const float *grad_final_state, const float *checkpoints,
                                             const rlscan_selective_scan_grads &g, void *ws, cudaStream_t s)
{
    rlscan_selective_scan_args a = args;
    rlscan_array3 grad_y = grad;
    const Layout l = layout(a);
    char *w = static_cast<char *>(ws);
    if (realign_workspace(a, true) > 0) {
        const rlscan_status st = realign(a, &grad_y, w + l.realigned, s);
        if (st != RLSCAN_OK) return st;
    }
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
    k.chunk = l.chunk;
    k.chunks = l.chunks;
    k.sms = order_sms(a.lengths, a.N, l.blocks, l.chunks);
    if (a.N > 0 && a.D > 0) {
        if (l.chunks > 1) {
            float *states = reinterpret_cast<float *>(w + l.states);
            const rlscan_status st =
                launch_back_states(a, grad_y, grad_final_state, l.chunk, l.chunks, states,
                                   reinterpret_cast<float *>(w + l.spans), reinterpret_cast<uint8_t *>(w + l.cuts), s);
            if (st != RLSCAN_OK) return st;
            k.grad_final = states;
        }
        const rlscan_status st = b16 ? launch_typed<bf16>(a, k, s) : launch_typed<float>(a, k, s);
        if (st != RLSCAN_OK) return st;
    }
    const int64_t bc = a.N * a.T * a.S;
    SumJobs jobs;
    if (g.B != nullptr) jobs.add(k.part_B, l.blocks, bc, bc, g.B, b16);
    if (g.C != nullptr) jobs.add(k.part_C, l.blocks, bc, bc, g.C, b16);
    if (g.A != nullptr) jobs.add(k.part_A, a.N * l.chunks, a.D * a.S, a.D * a.S, g.A, false);
    if (g.skip != nullptr) jobs.add(k.part_d, a.N * l.chunks, 2 * a.D, a.D, g.skip, false);
    if (g.delta_bias != nullptr) jobs.add(k.part_d + a.D, a.N * l.chunks, 2 * a.D, a.D, g.delta_bias, false);
    return launch_sums(jobs, s);
}

}  // namespace seq
}  // namespace rlscan
