// selective_scan.cuh -- the selective scan over prompts, for one activation
// type: the kernels, and the launches that k_selective_scan_*.cu instantiate
// (a translation unit for each type, which halves the build).
//
//   h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,   y_t = (C_t h_t + skip x_t) silu(z_t)
//
// A lane holds SPT states of one channel in registers and walks the
// tokens in order; LANES lanes share a channel.  Tiles of 16 tokens come into
// shared memory by asynchronous copies, two tiles ahead.  A tile's tokens are
// shared out over a channel's lanes: each prepares its own (softplus, dt x,
// the gate), hands dt and dt x to the others with shuffles, and gets its
// tokens' sums over the states back.
//
// An exponential and four multiply-adds a state value bound it: in pairs they
// run at 31.5 values a clock and SM.
// Measured, S 16 bf16: 8 x 4096 x 4096 675 us, 3.2e12 values/s, 63 % of the
// issue slots where an SM has two blocks; with ragged rows (62 % of the
// tokens) 500 to 530 us back to back.  1 x 4096 x 2048 in chunks of 128: 35 us for the chunks' states (69 % of
// the exponential units), 8 for joining them, 54 for the outputs.
#pragma once

#include "scan_plan.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kTile = kCheckpoint;

template <class T, int SPT, int LANES, bool SPLIT>
struct Shape {
    static constexpr int CH = kScanThreads / LANES;     // channels of a block
    static constexpr int SP = SPT * LANES;          // states, padded
    // Tokens taken at once, and registers: calls whose rows are whole have few
    // warps and live on the overlap of 16 tokens; those in chunks have many
    // (measured, unsplit 8 x 4096 x 4096 ragged: 16 tokens 652 us, 8: 695;
    // in chunks, 2 x 16384 x 2048: 16 tokens 570 us, 8 with four blocks 525).
    static constexpr int MOST = SPLIT ? 8 : 16, WALK = LANES > MOST ? LANES : MOST;
    static constexpr int PER = WALK / LANES;              // of them a lane prepares sl, sl + LANES, ...
    // rows of the lanes that share a channel lie in different banks
    static constexpr int ROWB = 32 / LANES * static_cast<int>(sizeof(T));
    static constexpr int PITCH = CH * static_cast<int>(sizeof(T)) + (ROWB > 16 ? ROWB : 16);
    static constexpr int BW = SP * sizeof(T) < 16 ? 16 / static_cast<int>(sizeof(T)) : SP;  // whole 16-byte units
    static constexpr int BPITCH = BW * static_cast<int>(sizeof(T));
    static constexpr int ACT = kTile * PITCH, BC = kTile * BPITCH;
    static constexpr int STAGE = 3 * ACT + 2 * BC;
    static constexpr int STAGES = 3;
    static constexpr bool CONVERT = sizeof(T) == 2;
    static constexpr int WIDE = CONVERT ? 2 * kTile * SP * 4 : 0;  // B and C in float32
    static constexpr size_t SMEM = STAGES * STAGE + 2 * WIDE;
    static constexpr int BLOCKS = SPLIT ? 4 : (SPT == 16 ? 2 : 3);
    static_assert(ACT % 16 == 0 && BC % 16 == 0);
};

template <class T, int SPT>
__device__ __forceinline__ void load_states(f2 *h, const float *p, int s0, int S, bool on)
{
#pragma unroll
    for (int i = 0; i < SPT / 2; ++i) {
        const int s = s0 + 2 * i;
        h[i] = pair(on && s < S ? p[s] : 0.f, on && s + 1 < S ? p[s + 1] : 0.f);
    }
}

template <int SPT>
__device__ __forceinline__ void store_states(float *p, const f2 *h, int s0, int S, bool vec)
{
    if (vec) {
#pragma unroll
        for (int i = 0; i < SPT / 4; ++i) {
            const float2 a = halves(h[2 * i]), b = halves(h[2 * i + 1]);
            if (s0 + 4 * i < S) *reinterpret_cast<float4 *>(p + s0 + 4 * i) = make_float4(a.x, a.y, b.x, b.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < SPT / 2; ++i) {
            const float2 a = halves(h[i]);
            if (s0 + 2 * i < S) p[s0 + 2 * i] = a.x;
            if (s0 + 2 * i + 1 < S) p[s0 + 2 * i + 1] = a.y;
        }
    }
}

// FULL: outputs.  PART: a chunk's end state from 0 and its sum of dt.  BACK:
// the same for the gradient of the states, from the chunk's last token to
// its first: E_t = exp(dt_t A) (E_{t+1} + C_t g_t), with grad_y in x's place
// and C in B's.
enum Mode { FULL_SCAN, PART, BACK };

template <class T, int SPT, int LANES, int MODE, bool SPLIT>
__global__ void __launch_bounds__(kScanThreads, Shape<T, SPT, LANES, SPLIT>::BLOCKS)
    scan_kernel(const __grid_constant__ rlscan_selective_scan_args a, const __grid_constant__ ScanOut o)
{
    using P = Shape<T, SPT, LANES, SPLIT>;
    constexpr bool FULL = MODE == FULL_SCAN;
    extern __shared__ __align__(16) char smem[];
    float *wide = reinterpret_cast<float *>(smem + P::STAGES * P::STAGE);
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, sl = lane % LANES, ch = threadIdx.x / LANES;
    const int64_t blocks = (a.D + P::CH - 1) / P::CH;
    const int64_t place = FULL && !SPLIT && o.sms > 0
                              ? by_length(a.lengths, static_cast<int>(a.N), blocks, o.sms, reinterpret_cast<int *>(smem))
                              : blockIdx.x;
    const Division at_block = divide(place, blocks), at_row = divide(at_block.q, o.chunks);
    const int64_t c0 = at_block.r * P::CH, chunk = at_row.r, n = at_row.q;
    const int64_t d = c0 + ch;
    const bool live = d < a.D;
    const int64_t dd = live ? d : a.D - 1;
    const int s0 = SPT * sl, S = static_cast<int>(a.S);
    const int width = static_cast<int>(a.D - c0 < P::CH ? a.D - c0 : P::CH);
    const bool gated = MODE != PART && a.z.data != nullptr;
    const uint32_t gate = gated ? ~0u : 0u, soft = a.delta_softplus ? ~0u : 0u;
    const int64_t first = chunk * o.chunk, last = first + o.chunk < a.T ? first + o.chunk : a.T;
    const int64_t len = row_length(a.lengths, n, a.T);
    const int64_t stop = len < last ? len : last;  // tokens first <= t < stop are scanned

    const rlscan_array3 &in = MODE == BACK ? o.grad_y : a.x, &drive = MODE == BACK ? a.C : a.B;
    const T *x = static_cast<const T *>(in.data) + n * in.row_stride + first * in.token_stride + c0;
    const T *delta = static_cast<const T *>(a.delta.data) + n * a.delta.row_stride + first * a.delta.token_stride + c0;
    const T *z = static_cast<const T *>(a.z.data) + n * a.z.row_stride + first * a.z.token_stride + c0;
    const T *B = static_cast<const T *>(drive.data) + n * drive.row_stride + first * drive.token_stride;
    const T *C = static_cast<const T *>(a.C.data) + n * a.C.row_stride + first * a.C.token_stride;
    const uint8_t *resets = a.resets != nullptr ? a.resets + n * a.T + first : nullptr;

    const int64_t count = stop - first, tiles = count > 0 ? (count + kTile - 1) / kTile : 0;
    auto copy_tile = [&](auto unit, int64_t tile) {
        constexpr int CHUNK = decltype(unit)::value;
        const int64_t t = (MODE == BACK ? tiles - 1 - tile : tile) * kTile, left = count - t;
        char *st = smem + tile % P::STAGES * P::STAGE;
        const int rows = left < kTile ? static_cast<int>(left) : kTile;
        load_tile<T, kTile, P::CH, P::PITCH, CHUNK, kScanThreads>(st, x + t * in.token_stride, in.token_stride, rows, width);
        load_tile<T, kTile, P::CH, P::PITCH, CHUNK, kScanThreads>(st + P::ACT, delta + t * a.delta.token_stride,
                                                              a.delta.token_stride, rows, width);
        load_tile<T, kTile, P::BW, P::BPITCH, CHUNK, kScanThreads>(st + 3 * P::ACT, B + t * drive.token_stride,
                                                               drive.token_stride, rows, S);
        if (gated)
            load_tile<T, kTile, P::CH, P::PITCH, CHUNK, kScanThreads>(st + 2 * P::ACT, z + t * a.z.token_stride,
                                                                  a.z.token_stride, rows, width);
        if (FULL) {
            load_tile<T, kTile, P::BW, P::BPITCH, CHUNK, kScanThreads>(st + 3 * P::ACT + P::BC, C + t * a.C.token_stride,
                                                                   a.C.token_stride, rows, S);
        }
    };
    auto issue = [&](int64_t tile) {
        if (tile < tiles) {
            if (o.unit == 16)
                copy_tile(std::integral_constant<int, 16>(), tile);
            else if (o.unit == 4)
                copy_tile(std::integral_constant<int, 4>(), tile);
            else
                copy_tile(std::integral_constant<int, 0>(), tile);
        }
        copies_commit();
    };
    issue(0);
    issue(1);

    f2 A2[SPT / 2], h[SPT / 2];
    load_states<T, SPT>(A2, a.A + dd * S, s0, S, true);
#pragma unroll
    for (int i = 0; i < SPT / 2; ++i) A2[i] = mul2(A2[i], both(kLog2e));
    if (FULL && o.chunks > 1)
        load_states<T, SPT>(h, o.states + ((n * o.chunks + chunk) * a.D + dd) * S, s0, S, true);
    else
        load_states<T, SPT>(h, a.initial_state + (n * a.D + dd) * S, s0, S, FULL && a.initial_state != nullptr);
    const float bias = a.delta_bias != nullptr ? a.delta_bias[dd] : 0.f;
    const float skip = FULL && a.skip != nullptr ? a.skip[dd] : 0.f;
    const int64_t marks = (a.T + kTile - 1) / kTile;
    T *y = static_cast<T *>(o.y) + (n * a.T + first) * a.D + dd;
    float *mark = o.checkpoints != nullptr ? o.checkpoints + ((n * marks + first / kTile) * a.D + dd) * S : nullptr;
    float span = 0.f;
    uint32_t cut = 0;

    auto flag_at = [&](int64_t tile) {
        const int64_t t = (MODE == BACK ? tiles - 1 - tile : tile) * kTile + lane;
        return resets != nullptr && lane < kTile && t >= 0 && t < count ? static_cast<uint32_t>(resets[t]) : 0u;
    };
    uint32_t flag = flag_at(0);  // one tile ahead
    for (int64_t tile = 0; tile < tiles; ++tile) {
        const int64_t t0 = (MODE == BACK ? tiles - 1 - tile : tile) * kTile;
        copies_wait<1>();
        __syncthreads();  // the tile is here, and its predecessor's buffer is free
        issue(tile + 2);
        const char *st = smem + tile % P::STAGES * P::STAGE;
        const float *Bw, *Cw;
        if constexpr (P::CONVERT) {
            float *w = wide + (tile & 1) * (2 * kTile * P::SP);
            constexpr int QUADS = kTile * P::SP / 4;
#pragma unroll
            for (int i = threadIdx.x; i < (FULL ? 2 : 1) * QUADS; i += kScanThreads) {
                const int k = i / QUADS, r = i / (P::SP / 4) % kTile, c = i % (P::SP / 4);
                const uint2 v = *reinterpret_cast<const uint2 *>(st + 3 * P::ACT + k * P::BC + r * P::BPITCH + c * 8);
                *reinterpret_cast<float4 *>(w + 4 * i) =
                    make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                                __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
            }
            __syncthreads();
            Bw = w + s0;
            Cw = w + kTile * P::SP + s0;
        } else {
            Bw = reinterpret_cast<const float *>(st + 3 * P::ACT) + s0;
            Cw = Bw + P::BC / 4;
        }
        const uint32_t starts = resets != nullptr ? __ballot_sync(0xffffffffu, flag != 0) : 0u;
        if (resets != nullptr) flag = tile + 1 < tiles ? flag_at(tile + 1) : 0u;
        cut |= starts;
        if (FULL && mark != nullptr && live) store_states<SPT>(mark + tile * a.D * S, h, s0, S, o.vec);
        const int left = count - t0 < kTile ? static_cast<int>(count - t0) : kTile;
        const T *xs = reinterpret_cast<const T *>(st) + ch, *ds = reinterpret_cast<const T *>(st + P::ACT) + ch,
                *zs = reinterpret_cast<const T *>(st + 2 * P::ACT) + ch;
        constexpr int ROW = P::PITCH / static_cast<int>(sizeof(T));
        constexpr int BROW = P::CONVERT ? P::SP : P::BPITCH / 4;
        T *yt = y + t0 * a.D;
        // FAST: 16 tokens of one episode, without a branch, so that the tokens' work overlaps
        auto walk = [&](auto fast, int w0) {
            constexpr bool FAST = decltype(fast)::value;
            float xv[P::PER], dt[P::PER], dtx[P::PER], part[P::WALK];
            // f(first, how many) for the lane's tokens, two at once where it has two
            auto by_pairs = [](auto f) {
                if constexpr (P::PER == 1) {
                    f(0, std::integral_constant<int, 1>());
                } else {
#pragma unroll
                    for (int p = 0; p < P::PER; p += 2) f(p, std::integral_constant<int, 2>());
                }
            };
            auto gate_of = [&](int p) {  // of tokens p and p + 1
                const float z0 = to_f(zs[(w0 + p * LANES + sl) * ROW]);
                const float z1 = P::PER > 1 ? to_f(zs[(w0 + (p + 1) * LANES + sl) * ROW]) : 0.f;
                const f2 z = pair(z0, z1);
                const float2 v = halves(mul2(z, sigmoid(z)));
                return pair(choose(gate, v.x, 1.f), choose(gate, v.y, 1.f));
            };
            by_pairs([&](int p, auto two) {
                constexpr int Q = decltype(two)::value - 1;
                xv[p] = to_f(xs[(w0 + p * LANES + sl) * ROW]);
                xv[p + Q] = to_f(xs[(w0 + (p + Q) * LANES + sl) * ROW]);
                const f2 pre = add2(pair(to_f(ds[(w0 + p * LANES + sl) * ROW]), to_f(ds[(w0 + (p + Q) * LANES + sl) * ROW])),
                                    both(bias));
                const float2 s = halves(softplus(pre)), r = halves(pre);
                dt[p] = choose(soft, s.x, r.x);
                dt[p + Q] = choose(soft, Q == 0 ? s.x : s.y, Q == 0 ? r.x : r.y);
                if (!FAST) {  // past the last token the state stays
                    dt[p] = w0 + p * LANES + sl < left ? dt[p] : 0.f;
                    dt[p + Q] = w0 + (p + Q) * LANES + sl < left ? dt[p + Q] : 0.f;
                }
                const float2 v = halves(mul2(pair(xv[p], xv[p + Q]), MODE == BACK ? gate_of(p) : pair(dt[p], dt[p + Q])));
                dtx[p] = v.x;
                dtx[p + Q] = Q == 0 ? v.x : v.y;
                if (!FULL) span += Q == 0 ? dt[p] : dt[p] + dt[p + Q];
            });
#pragma unroll
            for (int kk = 0; kk < P::WALK; ++kk) {
                const int j = MODE == BACK ? P::WALK - 1 - kk : kk, k = w0 + j;
                float dj = dt[j / LANES], xj = dtx[j / LANES];
                if constexpr (LANES > 1) {
                    dj = __shfl_sync(0xffffffffu, dj, j % LANES, LANES);
                    xj = __shfl_sync(0xffffffffu, xj, j % LANES, LANES);
                }
                if (!FAST && MODE != BACK && (starts >> k & 1u) != 0) {
#pragma unroll
                    for (int i = 0; i < SPT / 2; ++i) h[i] = 0ull;
                }
                const f2 dp = both(dj), xp = both(xj);
                f2 acc[2] = {0ull, 0ull};
#pragma unroll
                for (int i = 0; i < SPT / 4; ++i) {
                    const ulonglong2 b = *reinterpret_cast<const ulonglong2 *>(Bw + k * BROW + 4 * i);
                    const f2 e0 = decay(dp, A2[2 * i]), e1 = decay(dp, A2[2 * i + 1]);
                    if constexpr (MODE == BACK) {
                        h[2 * i] = mul2(e0, fma2(xp, b.x, h[2 * i]));
                        h[2 * i + 1] = mul2(e1, fma2(xp, b.y, h[2 * i + 1]));
                    } else {
                        // xp is the same register for all states: one new operand less than e h + (x B)
                        h[2 * i] = fma2(xp, b.x, mul2(e0, h[2 * i]));
                        h[2 * i + 1] = fma2(xp, b.y, mul2(e1, h[2 * i + 1]));
                    }
                    if (FULL) {
                        const ulonglong2 c = *reinterpret_cast<const ulonglong2 *>(Cw + k * BROW + 4 * i);
                        acc[0] = i == 0 ? mul2(c.x, h[0]) : fma2(c.x, h[2 * i], acc[0]);
                        acc[1] = i == 0 ? mul2(c.y, h[1]) : fma2(c.y, h[2 * i + 1], acc[1]);
                    }
                }
                if (!FAST && MODE == BACK && (starts >> k & 1u) != 0) {
#pragma unroll
                    for (int i = 0; i < SPT / 2; ++i) h[i] = 0ull;
                }
                if (FULL) {
                    const float2 v = halves(add2(acc[0], acc[1]));
                    part[j] = v.x + v.y;
                }
            }
            if constexpr (FULL) {
                by_pairs([&](int p, auto two) {
                    constexpr int Q = decltype(two)::value - 1;
                    // leaves lane sl the sums of its tokens
                    scatter_sums<LANES, LANES / 2, 1>(part + p * LANES, lane);
                    if (Q > 0) scatter_sums<LANES, LANES / 2, 1>(part + (p + Q) * LANES, lane);
                    const float2 v = halves(mul2(
                        fma2(both(skip), pair(xv[p], xv[p + Q]), pair(part[p * LANES], part[(p + Q) * LANES])), gate_of(p)));
#pragma unroll
                    for (int q = 0; q <= Q; ++q) {
                        const int k = w0 + (p + q) * LANES + sl;
                        const float out = q == 0 ? v.x : v.y;
                        if (FAST) {
                            if (live) yt[k * a.D] = from_f<T>(out);
                        } else if (live && t0 + k < last - first) {
                            yt[k * a.D] = from_f<T>(k < left ? out : 0.f);
                        }
                    }
                });
            }
        };
#pragma unroll 1
        for (int w = 0; w < kTile; w += P::WALK) {
            const int w0 = MODE == BACK ? kTile - P::WALK - w : w;
            if (starts == 0 && left == kTile)
                walk(std::true_type(), w0);
            else
                walk(std::false_type(), w0);
        }
    }
    if (!FULL) {
        if constexpr (LANES > 1) {
#pragma unroll
            for (int m = LANES / 2; m > 0; m /= 2) span += __shfl_xor_sync(0xffffffffu, span, m);
        }
        if (live) {
            const int64_t at = (n * o.chunks + chunk) * a.D + d;
            store_states<SPT>(o.states + at * S, h, s0, S, o.vec);
            if (sl == 0) o.spans[at] = span;
        }
        if (c0 == 0 && threadIdx.x == 0) o.cuts[n * o.chunks + chunk] = cut != 0;
        return;
    }
    if (!live) return;
    // padding behind the last tile; checkpoints there hold the final state
    for (int64_t t = tiles * kTile + sl; t < last - first; t += LANES) y[t * a.D] = from_f<T>(0.f);
    if (mark != nullptr)
        for (int64_t m = tiles; m * kTile < last - first; ++m) store_states<SPT>(mark + m * a.D * S, h, s0, S, o.vec);
    // the chunk with the row's last token (the first chunk of an empty row)
    if (o.final_state != nullptr && (len > first ? len <= last : len == 0 && chunk == 0))
        store_states<SPT>(o.final_state + (n * a.D + d) * S, h, s0, S, o.vec);
}

// The state in front of each chunk: carry = exp(A span) carry + the chunk's
// own end state, or that alone where an episode starts in the chunk.  BACK:
// the gradient's message behind each chunk, from the last to the first.
// Eight chunks' loads are in flight before their states are replaced.
template <bool REVERSE>
__global__ void __launch_bounds__(256) chunk_kernel(const __grid_constant__ rlscan_selective_scan_args a,
                                                    const __grid_constant__ ScanOut o, const float *start)
{
    constexpr int AHEAD = 8;
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int64_t i = blockIdx.x * 256ll + threadIdx.x, DS = a.D * a.S;
    if (i >= a.N * DS) return;
    const Division at = divide(i, DS);
    const int64_t n = at.q, e = at.r, d = divide(e, a.S).q;
    const float A2 = a.A[e] * kLog2e;
    float carry = start != nullptr ? start[i] : 0.f;
    float *st = o.states + n * o.chunks * DS + e;
    const float *sp = o.spans + n * o.chunks * a.D + d;
    const uint8_t *cut = o.cuts + n * o.chunks;
    for (int64_t base = 0; base < o.chunks; base += AHEAD) {
        float own[AHEAD], span[AHEAD];
        uint8_t cuts[AHEAD];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (base + u >= o.chunks) break;
            const int64_t c = REVERSE ? o.chunks - 1 - base - u : base + u;
            own[u] = st[c * DS];
            span[u] = sp[c * a.D];
            cuts[u] = cut[c];
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (base + u >= o.chunks) break;
            const int64_t c = REVERSE ? o.chunks - 1 - base - u : base + u;
            st[c * DS] = carry;
            carry = cuts[u] != 0 ? own[u] : fmaf(exp2_fast(A2 * span[u]), carry, own[u]);
        }
    }
}

template <class T, int SPT, int LANES, int MODE, bool SPLIT>
rlscan_status launch_mode(const rlscan_selective_scan_args &a, ScanOut o, cudaStream_t s)
{
    using P = Shape<T, SPT, LANES, SPLIT>;
    o.sms = order_sms(a.lengths, a.N, ceil_div(a.D, P::CH), o.chunks);
    auto kernel = scan_kernel<T, SPT, LANES, MODE, SPLIT>;
    static PerDevice raised;
    if (!raise_smem(raised, kernel, P::SMEM)) return RLSCAN_ERR_CUDA;
    const int64_t grid = a.N * ceil_div(a.D, P::CH) * o.chunks;
    return launch(!spread_out(grid, o.sms), kernel, grid, kScanThreads, P::SMEM, s, a, o);
}

template <class T, int SPT, int LANES>
rlscan_status launch_shape(const rlscan_selective_scan_args &a, const ScanOut &o, cudaStream_t s)
{
    if (o.chunks == 1) return launch_mode<T, SPT, LANES, FULL_SCAN, false>(a, o, s);
    rlscan_status st = launch_mode<T, SPT, LANES, PART, true>(a, o, s);
    if (st == RLSCAN_OK)
        st = launch_overlapped(chunk_kernel<false>, ceil_div(a.N * a.D * a.S, 256), 256, 0, s, a, o, a.initial_state);
    if (st != RLSCAN_OK) return st;
    return launch_mode<T, SPT, LANES, FULL_SCAN, true>(a, o, s);
}

template <class T, int SPT>
rlscan_status by_lanes(int lanes, const rlscan_selective_scan_args &a, const ScanOut &o, cudaStream_t s)
{
    switch (lanes) {
    case 1: return launch_shape<T, SPT, 1>(a, o, s);
    case 2: return launch_shape<T, SPT, 2>(a, o, s);
    case 4: return launch_shape<T, SPT, 4>(a, o, s);
    case 8: return launch_shape<T, SPT, 8>(a, o, s);
    default: return launch_shape<T, SPT, 16>(a, o, s);
    }
}

// The gradient's messages, for the backward pass: its own shape of lanes.
template <class T, int SPT, int LANES>
rlscan_status launch_back(const rlscan_selective_scan_args &a, const ScanOut &o, const float *grad_final, cudaStream_t s)
{
    const rlscan_status st = launch_mode<T, SPT, LANES, BACK, true>(a, o, s);
    if (st != RLSCAN_OK) return st;
    return launch_overlapped(chunk_kernel<true>, ceil_div(a.N * a.D * a.S, 256), 256, 0, s, a, o, grad_final);
}

}  // namespace

template <class T>
rlscan_status scan_typed(const Plan &p, const rlscan_selective_scan_args &a, ScanOut o, cudaStream_t s)
{
    Chunk c;
    for (const rlscan_array3 *v : {&a.x, &a.delta, &a.B, &a.C}) c.add(v->data, v->row_stride, v->token_stride, sizeof(T));
    if (a.z.data != nullptr) c.add(a.z.data, a.z.row_stride, a.z.token_stride, sizeof(T));
    o.unit = c.size();
    o.vec = a.S % 4 == 0 &&
            ((reinterpret_cast<uintptr_t>(o.final_state) | reinterpret_cast<uintptr_t>(o.checkpoints)) & 15u) == 0;
    if (p.spt == 16) return by_lanes<T, 16>(p.lanes, a, o, s);
    return by_lanes<T, 8>(p.lanes, a, o, s);
}

template <class T>
rlscan_status back_states_typed(const rlscan_selective_scan_args &a, ScanOut o, const float *grad_final, cudaStream_t s)
{
    Chunk c;
    for (const rlscan_array3 *v : {static_cast<const rlscan_array3 *>(&o.grad_y), &a.delta, &a.C})
        c.add(v->data, v->row_stride, v->token_stride, sizeof(T));
    if (a.z.data != nullptr) c.add(a.z.data, a.z.row_stride, a.z.token_stride, sizeof(T));
    o.unit = c.size();
    o.vec = a.S % 4 == 0;
    if (a.S <= 8) return launch_back<T, 8, 1>(a, o, grad_final, s);
    if (a.S <= 16) return launch_back<T, 8, 2>(a, o, grad_final, s);
    if (a.S <= 32) return launch_back<T, 8, 4>(a, o, grad_final, s);
    if (a.S <= 64) return launch_back<T, 8, 8>(a, o, grad_final, s);
    return launch_back<T, 8, 16>(a, o, grad_final, s);
}

}  // namespace seq
}  // namespace rlscan
