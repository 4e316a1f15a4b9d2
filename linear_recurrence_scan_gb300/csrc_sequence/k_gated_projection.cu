// k_gated_projection.cu -- the gated feed-forward block's two projections with
// the activation and the product, and its gradients:
//   z = x Wg^T,  u = x Wu^T,  h = act(z) u
//   gz = grad_h u act'(z),  gu = grad_h act(z)
//   dx = gz Wg + gu Wu,  dWg = gz^T x,  dWu = gu^T x
// Four products on the tensor cores; the first two share their main loop.
#include "gated_projection.cuh"
#include "gated_scan.cuh"
#include "umma.cuh"

namespace rlscan {
namespace seq {
namespace {

__device__ unsigned int g_timed_out;  // a wait ran out on this device

// Forward: z and u, then h.  Gates: z and u, then gz and gu.  Input: dx, the
// sum over both gates' columns.  Weights: dWg and dWu.
enum class Job { Forward, Gates, Input, Weights };

struct Maps {
    CUtensorMap a[2], b[2], out[2];
};

struct Work {
    int64_t M, D, F;
    int64_t tiles_m, tiles_n, steps;  // steps: blocks of 64 values of K
    int act;
    const bf16 *grad_h;
    int64_t grad_h_stride;
    bool grad_h_vec;
    bf16 *out[2];
    int64_t out_stride;
    bool out_mapped;  // outputs leave through maps.out
    int64_t parts, part_steps;  // K in `parts` of `part_steps` steps (1: whole)
    float *sums;                // of parts > 1: [parts][rows of all outputs][columns]
};

constexpr int kBlockK = 64;  // values of K in a stage: a row of 128 bytes
constexpr int kStages = 5, kThreads = 384, kSumWarps = 8;
constexpr uint32_t kTileBytes = 128 * kBlockK * 2, kStageBytes = 2 * kTileBytes;
constexpr uint32_t kOutBytes = 32 * 128;  // 32 rows of 64 values, two of a warp that takes sums out
constexpr size_t kSmem = kStages * kStageBytes + kSumWarps * 2 * kOutBytes + 1024;

// 32 neighbouring values into half `h` of the lane's row of an output box, with
// its swizzle: the 16-byte units of a row change places by the row's number
__device__ __forceinline__ void box_row(char *box, int lane, int h, const float (&v)[32])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        Words<bf16, 8> w;
#pragma unroll
        for (int j = 0; j < 4; ++j) w.set(j, v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
        w.store(reinterpret_cast<bf16 *>(box + lane * 128 + (((4 * h + i) ^ (lane & 7)) * 16)));
    }
}
// A box to rows of any alignment, row by row: neighbouring lanes write
// neighbouring values (each lane its own row's: 32 sectors a store, which
// made all gradients of 1 x 2047 x 8192 three times as long)
__device__ __forceinline__ void copy_box(bf16 *to, int64_t stride, const char *box, int lane, int64_t rows, int64_t columns)
{
    for (int r = 0; r < 32 && r < rows; ++r, to += stride) {
#pragma unroll
        for (int c = lane; c < 64; c += 32)
            if (c < columns) to[c] = *reinterpret_cast<const bf16 *>(box + r * 128 + (((c / 8) ^ (r & 7)) * 16) + c % 8 * 2);
    }
}
__device__ __forceinline__ void store_box2(const CUtensorMap *map, int64_t x, int64_t y, const char *box)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(static_cast<int>(x)),
                 "r"(static_cast<int>(y)), "r"(ptx::smem_u32(box))
                 : "memory");
}
__device__ __forceinline__ void load_row(Words<bf16, 8> (&w)[4], const bf16 *p, int64_t n, bool vec)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        w[i].zero();
        if (vec && 8 * i + 8 <= n) {
            w[i].load(p + 8 * i);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = 8 * i + 2 * j;
                w[i].set(j, at < n ? to_f(p[at]) : 0.f, at + 1 < n ? to_f(p[at + 1]) : 0.f);
            }
        }
    }
}

// A pair of blocks, one on each of two SMs, makes tiles of 256 x 256: each
// block has 128 rows of A and half the columns of B in its shared memory, and
// one thread of the pair's first block multiplies for both.  For z and u the
// halves are 128 columns of z and the same 128 of u, so that the epilogue
// finds both of a value in its own tensor memory.  Warps: 0 copies, 1
// multiplies (the first block's), 2 holds the tensor memory, 4 to 11 take the
// sums out while the next tile's are made in the other half of the 512 columns.
// Bound by the products where K is long (forward 16384 x 4096 x 12288 1838 us,
// 1.79 PFLOP/s of the 1.89 that the library's plain product reaches), by the
// epilogue and the outputs' bytes where it is short (3636 x 64 x 4016 26 us).
// Four warps for the sums held the products up: gradients of 16384 x 512 x 512
// 130 us, with eight 107.
template <Job JOB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    projection_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Work k)
{
    constexpr bool kGates = JOB == Job::Forward || JOB == Job::Gates;
    constexpr bool kAMn = JOB == Job::Weights, kBMn = !kGates;
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t full[kStages], empty[kStages], sums_full[2], sums_empty[2];
    __shared__ uint32_t tmem_at;
    __shared__ int gave_up;
    ptx::pdl_trigger_dependents();
    char *raw_aligned = reinterpret_cast<char *>(raw) + ((1024u - (ptx::smem_u32(raw) & 1023u)) & 1023u);
    const uint32_t smem = ptx::smem_u32(raw_aligned), rank = umma::cluster_rank();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        gave_up = 0;
        for (int i = 0; i < kStages; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&sums_full[i], 1);
            ptx::mbar_init(&sums_empty[i], 2 * kSumWarps);  // a warp's arrival each, of both blocks
        }
        ptx::fence_mbar_init();
    }
    if (warp == 2) umma::tmem_alloc(ptx::smem_u32(&tmem_at), 512);
    umma::fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    umma::fence_after();
    const uint32_t tmem = tmem_at;
    ptx::pdl_wait_prerequisites();
    const int64_t items = k.tiles_m * k.tiles_n * k.parts, first_item = blockIdx.x / 2, pairs = gridDim.x / 2;
    // Tiles in bands of eight rows of tiles, column after column: the pairs at
    // work share rows of A and columns of B in L2.
    auto place = [&](int64_t tile, int64_t &m, int64_t &n) {
        constexpr int64_t kBand = 8;
        const int64_t band = tile / (kBand * k.tiles_n), in = tile - band * kBand * k.tiles_n;
        const int64_t high = k.tiles_m - band * kBand < kBand ? k.tiles_m - band * kBand : kBand;
        m = band * kBand + in % high;
        n = in / high;
    };
    // An item is a tile, or a part of its K
    auto first_step = [&](int64_t item) { return item % k.parts * k.part_steps; };
    auto last_step = [&](int64_t item) {
        const int64_t e = (item % k.parts + 1) * k.part_steps;
        return e < k.steps ? e : k.steps;
    };
    if (warp == 0 && lane == 0) {  // copies
        uint32_t stage = 0, phase = 1;  // the first wait on an empty stage passes
        int64_t issued = 0;
        const int64_t half = kGates ? 0 : JOB == Job::Input ? k.steps / 2 : k.tiles_m / 2;
        for (int64_t item = first_item; item < items && !has_given_up(&gave_up); item += pairs) {
            int64_t tm, tn;
            place(item / k.parts, tm, tn);
            for (int64_t s = first_step(item), e = last_step(item); s < e; ++s) {
                if (!wait(ptx::smem_u32(&empty[stage]), phase, &gave_up)) break;
                const uint32_t bar = umma::of_rank(ptx::smem_u32(&full[stage]), 0);
                const uint32_t a = smem + stage * kStageBytes, b = a + kTileBytes;
                if (rank == 0) ptx::mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
                if constexpr (kGates) {
                    const int k0 = static_cast<int>(s) * kBlockK;
                    umma::load_box(a, &maps.a[0], k0, static_cast<int>(tm * 256 + rank * 128), bar);
                    umma::load_box(b, &maps.b[rank], k0, static_cast<int>(tn * 128), bar);
                } else if constexpr (JOB == Job::Input) {
                    const int part = s >= half ? 1 : 0, k0 = static_cast<int>(s - part * half) * kBlockK;
                    umma::load_box(a, &maps.a[part], k0, static_cast<int>(tm * 256 + rank * 128), bar);
                    for (int i = 0; i < 2; ++i)
                        umma::load_box(b + i * (kTileBytes / 2), &maps.b[part], static_cast<int>(tn * 256 + rank * 128 + 64 * i), k0, bar);
                } else {
                    const int part = tm >= half ? 1 : 0, k0 = static_cast<int>(s) * kBlockK;
                    const int f0 = static_cast<int>((tm - part * half) * 256 + rank * 128);
                    for (int i = 0; i < 2; ++i) {
                        umma::load_box(a + i * (kTileBytes / 2), &maps.a[part], f0 + 64 * i, k0, bar);
                        umma::load_box(b + i * (kTileBytes / 2), &maps.b[0], static_cast<int>(tn * 256 + rank * 128 + 64 * i), k0, bar);
                    }
                }
                ++issued;
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
        }
        // The block stays until the products have taken its last copies.
        for (int64_t i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
            if (!wait(ptx::smem_u32(&empty[i % kStages]), static_cast<uint32_t>(i / kStages) & 1u, &gave_up)) break;
    } else if (warp == 1 && lane == 0 && rank == 0) {  // products
        constexpr uint32_t kInstruction = umma::instruction(kAMn, kBMn, 256, 256);
        uint32_t stage = 0, phase = 0, buffer = 0, buffer_phase = 1;
        for (int64_t item = first_item; item < items; item += pairs) {
            if (!wait(ptx::smem_u32(&sums_empty[buffer]), buffer_phase, &gave_up)) break;
            umma::fence_after();
            bool fine = true;
            const int64_t begin = first_step(item), stop = last_step(item);
            for (int64_t s = begin; s < stop && fine; ++s) {
                fine = wait(ptx::smem_u32(&full[stage]), phase, &gave_up);
                if (!fine) break;
                umma::fence_after();
                const uint32_t a = smem + stage * kStageBytes, b = a + kTileBytes;
#pragma unroll
                for (int j = 0; j < kBlockK / 16; ++j)
                    umma::multiply(tmem + buffer * 256, umma::descriptor(a + j * (kAMn ? 2048 : 32), kTileBytes / 2),
                                   umma::descriptor(b + j * (kBMn ? 2048 : 32), kTileBytes / 2), kInstruction, s > begin || j > 0);
                umma::commit(ptx::smem_u32(&empty[stage]));
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
            if (!fine) break;
            umma::commit(ptx::smem_u32(&sums_full[buffer]));
            buffer ^= 1;
            if (buffer == 0) buffer_phase ^= 1;
        }
    } else if (warp >= 4) {  // sums
        uint32_t buffer = 0, phase = 0;
        // a warp reaches a quarter of the tensor memory's rows; two warps share it, half of the columns each
        const int part = warp % 4, side = (warp - 4) / 4;
        char *boxes = raw_aligned + kStages * kStageBytes + (warp - 4) * 2 * kOutBytes;
        // the box that comes next has been read: all of the warp's, or (two take turns) all but the last
        auto free_box = [&](bool turns) {
            if (lane == 0) {
                if (turns) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                else asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            }
            __syncwarp();
        };
        int turn = 0;  // of Forward's two boxes
        auto put_box = [&](int i, int64_t x, int64_t y, int64_t rows, int64_t columns, const char *box) {
            const bool some = y < rows && x < columns;
            if (k.out_mapped) {
                fence_async();
                __syncwarp();
                if (lane == 0 && some) store_box2(&maps.out[i], x, y, box);
                if (lane == 0) stores_commit();
            } else {
                __syncwarp();
                if (some) copy_box(k.out[i] + y * k.out_stride + x, k.out_stride, box, lane, rows - y, columns - x);
            }
        };
        for (int64_t item = first_item; item < items; item += pairs) {
            int64_t tm, tn;
            place(item / k.parts, tm, tn);
            const int64_t half = k.tiles_m / 2;
            const int which = JOB == Job::Weights && tm >= half ? 1 : 0;
            const int64_t row = (tm - which * half) * 256 + rank * 128 + part * 32 + lane;
            const int64_t rows = JOB == Job::Weights ? k.F : k.M;
            if (!wait(ptx::smem_u32(&sums_full[buffer]), phase, &gave_up)) break;
            umma::fence_after();
            const uint32_t at = tmem + buffer * 256 + (static_cast<uint32_t>(part * 32) << 16);
            const int64_t row0 = row - lane;  // of the warp
            if constexpr (kGates) {
                const int64_t f0 = tn * 128;
#pragma unroll 1
                for (int c = side * 64; c < side * 64 + 64; c += 32) {
                    const int64_t n = row < rows ? k.F - f0 - c : 0;
                    uint32_t z[32], u[32];
                    Words<bf16, 8> gh[4];
                    if constexpr (JOB == Job::Gates) load_row(gh, k.grad_h + row * k.grad_h_stride + f0 + c, n, k.grad_h_vec);
                    umma::tmem_load(z, at + c);
                    umma::tmem_load(u, at + 128 + c);
                    umma::tmem_loaded();
                    float v[32], w[32];
                    auto outputs = [&](auto act) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            const f2 uu = pair(__uint_as_float(u[i]), __uint_as_float(u[i + 1]));
                            const Activated of = act(pair(__uint_as_float(z[i]), __uint_as_float(z[i + 1])));
                            if constexpr (JOB == Job::Forward) {
                                const float2 h = halves(mul2(of.value, uu));
                                v[i] = h.x, v[i + 1] = h.y;
                            } else {
                                const f2 g = pair(gh[i / 8][i % 8], gh[i / 8][i % 8 + 1]);
                                const float2 gz = halves(mul2(mul2(g, uu), of.slope)), gu = halves(mul2(g, of.value));
                                v[i] = gz.x, v[i + 1] = gz.y, w[i] = gu.x, w[i + 1] = gu.y;
                            }
                        }
                    };
                    if (k.act == RLSCAN_SILU) outputs([](f2 x) { return silu(x); });
                    else outputs([](f2 x) { return gelu(x); });
                    const int h = c / 32 % 2;
                    char *box = boxes + (JOB == Job::Forward ? turn * kOutBytes : 0);
                    if (h == 0) free_box(JOB == Job::Forward);
                    box_row(box, lane, h, v);
                    if constexpr (JOB == Job::Gates) box_row(boxes + kOutBytes, lane, h, w);
                    if (h == 1) {
                        const int64_t x = f0 + c - 32;
                        put_box(0, x, row0, rows, k.F, box);
                        turn ^= 1;
                        if constexpr (JOB == Job::Gates) put_box(1, x, row0, rows, k.F, boxes + kOutBytes);
                    }
                }
            } else {
                const int64_t d0 = tn * 256;
#pragma unroll 1
                for (int c = side * 128; c < side * 128 + 128; c += 32) {
                    uint32_t v[32];
                    umma::tmem_load(v, at + c);
                    umma::tmem_loaded();
                    float f[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
                    if (k.parts > 1) {
                        const int64_t all = JOB == Job::Weights ? 2 * rows : rows, n = row < rows ? k.D - d0 - c : 0;
                        float *to = k.sums + ((item % k.parts) * all + which * rows + row) * k.D + d0 + c;
                        if (k.D % 4 == 0) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                if (i < n) *reinterpret_cast<float4 *>(to + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (i < n) to[i] = f[i];
                        }
                    } else {
                        char *box = boxes + c / 64 % 2 * kOutBytes;
                        const int h = c / 32 % 2;
                        if (h == 0) free_box(true);
                        box_row(box, lane, h, f);
                        if (h == 1) put_box(which, d0 + c - 32, row0, rows, k.D, box);
                    }
                }
            }
            umma::fence_before();
            __syncwarp();
            if (lane == 0) umma::arrive_cluster(umma::of_rank(ptx::smem_u32(&sums_empty[buffer]), 0));
            buffer ^= 1;
            if (buffer == 0) phase ^= 1;
        }
        if (lane == 0) stores_read();
    }
    __syncwarp();
    umma::fence_before();
    __syncthreads();
    leave(&gave_up, &g_timed_out);
    __syncwarp();
    cluster_arrive();
    cluster_wait();  // neither block leaves while the other may still reach it
    umma::fence_after();
    if (warp == 2) umma::tmem_free(tmem, 512);
}

// Outputs from the sums of parts of K, `half` values of out[0], then out[1]'s
__global__ void __launch_bounds__(256) join_kernel(const float *sums, int64_t parts, int64_t all, int64_t half, bf16 *out0, bf16 *out1)
{
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < all; i += static_cast<int64_t>(gridDim.x) * 256) {
        float v = 0.f;
#pragma unroll 4
        for (int64_t p = 0; p < parts; ++p) v += sums[p * all + i];
        (i < half ? out0[i] : out1[i - half]) = from_f<bf16>(v);
    }
}

// Rows of `columns` values into rows `pitch` values apart, a warp a row
__global__ void __launch_bounds__(256) pack_kernel(const bf16 *from, int64_t stride, bf16 *to, int64_t pitch, int64_t rows, int64_t columns)
{
    constexpr int AHEAD = 8;
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; r < rows; r += static_cast<int64_t>(gridDim.x) * 8) {
        const uint16_t *in = reinterpret_cast<const uint16_t *>(from + r * stride);
        uint16_t *out = reinterpret_cast<uint16_t *>(to + r * pitch);
        for (int64_t c = lane; c < columns; c += 32 * AHEAD) {
            uint32_t v[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (c + 32 * i < columns) asm volatile("ld.global.u16 %0, [%1];" : "=r"(v[i]) : "l"(in + c + 32 * i));
#pragma unroll
            for (int i = 0; i < AHEAD; ++i)
                if (c + 32 * i < columns) out[c + 32 * i] = static_cast<uint16_t>(v[i]);
        }
    }
}

int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

// Tensor maps take arrays whose address and row stride are multiples of 16
// bytes; others are copied first.
bool fits_map(const void *p, int64_t rows, int64_t columns, int64_t stride)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows <= 1 || (stride % 8 == 0 && stride >= columns && stride < (int64_t{1} << 38)));
}

struct Operand {
    const void *p;
    int64_t rows, columns, pitch;
    bool packed;
};

Operand operand(const void *p, int64_t rows, int64_t columns, int64_t stride)
{
    const bool fits = fits_map(p, rows, columns, stride);
    return {p, rows, columns, fits && rows > 1 ? stride : up8(columns), !fits};
}

size_t bytes_of(const Operand &o) { return o.packed ? static_cast<size_t>(o.rows) * o.pitch * 2 : 0; }
size_t up256(size_t n) { return (n + 255) / 256 * 256; }

struct Layout {
    Operand x, gate, up;
    size_t at_x, at_gate, at_up, bytes;
};

Layout layout(const rlscan_gated_projection_args &a)
{
    Layout l;
    l.x = operand(a.x, a.M, a.D, a.x_stride);
    l.gate = operand(a.gate_weight, a.F, a.D, a.gate_stride);
    l.up = operand(a.up_weight, a.F, a.D, a.up_stride);
    l.at_x = 0;
    l.at_gate = l.at_x + up256(bytes_of(l.x));
    l.at_up = l.at_gate + up256(bytes_of(l.gate));
    l.bytes = l.at_up + up256(bytes_of(l.up));
    return l;
}

rlscan_status pack(Operand &o, int64_t stride, void *to, cudaStream_t s)
{
    if (!o.packed) return RLSCAN_OK;
    const int64_t blocks = ceil_div(o.rows, 8), most = 8 * (sm_count() > 0 ? sm_count() : 152);
    const rlscan_status st = launch_overlapped(pack_kernel, blocks < most ? blocks : most, 256, 0, s, static_cast<const bf16 *>(o.p),
                                               stride, static_cast<bf16 *>(to), o.pitch, o.rows, o.columns);
    o.p = to;
    return st;
}

rlscan_status pack_all(const rlscan_gated_projection_args &a, Layout &l, char *ws, cudaStream_t s)
{
    rlscan_status st = pack(l.x, a.x_stride, ws + l.at_x, s);
    if (st == RLSCAN_OK) st = pack(l.gate, a.gate_stride, ws + l.at_gate, s);
    if (st == RLSCAN_OK) st = pack(l.up, a.up_stride, ws + l.at_up, s);
    return st;
}

bool map_of(CUtensorMap *m, const Operand &o, uint32_t box) { return umma::encode(m, o.p, o.rows, o.columns, o.pitch, box); }

// Few tiles of a long K leave pairs without work: K is then taken in parts, at
// least four steps each, whose sums are joined in order by another kernel.
// Measured, gradients of 8 x 4096 x 12288 (dx: 16 tiles of 384 steps) 250 us
// whole, 166 in four parts of 96 steps (and dW of 16384 x 512 x 512 in parts: all
// gradients 132 and 70).
struct Split {
    int64_t parts, steps;
};
Split split_of(int64_t tiles, int64_t steps)
{
    const int64_t pairs = (sm_count() > 0 ? sm_count() : 152) / 2;
    int64_t parts = tiles > 0 ? pairs / tiles : 1;
    if (parts > steps / 4) parts = steps / 4;
    if (parts < 2) return {1, steps};
    const int64_t each = ceil_div(steps, parts);
    return {ceil_div(steps, each), each};
}
struct GradSplits {
    Split input, weights;
    size_t bytes;  // of the sums of either, which take turns
};
GradSplits splits_of(const rlscan_gated_projection_args &a)
{
    GradSplits g;
    g.input = split_of(ceil_div(a.M, 256) * ceil_div(a.D, 256), 2 * ceil_div(a.F, kBlockK));
    g.weights = split_of(2 * ceil_div(a.F, 256) * ceil_div(a.D, 256), ceil_div(a.M, kBlockK));
    const int64_t x = g.input.parts > 1 ? g.input.parts * a.M * a.D : 0, w = g.weights.parts > 1 ? g.weights.parts * 2 * a.F * a.D : 0;
    g.bytes = static_cast<size_t>(x > w ? x : w) * sizeof(float);
    return g;
}

rlscan_status join(const Work &w, int64_t rows, cudaStream_t s)
{
    const int64_t half = rows * w.D, all = w.out[1] != nullptr ? 2 * half : half, most = 16 * (sm_count() > 0 ? sm_count() : 152);
    const int64_t blocks = ceil_div(all, 256);
    return launch_overlapped(join_kernel, blocks < most ? blocks : most, 256, 0, s, w.sums, w.parts, all, half, w.out[0], w.out[1]);
}

template <Job JOB>
rlscan_status launch_job(const Maps &maps, Work &w, cudaStream_t s)
{
    static PerDevice raised, pairs_of;
    if (!raise_smem(raised, projection_kernel<JOB>, kSmem)) return RLSCAN_ERR_CUDA;
    const int most = pairs_of.get(current_device(), [] {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        return ok(cudaOccupancyMaxActiveClusters(&n, projection_kernel<JOB>, &cfg)) ? n : 0;
    });
    const int64_t tiles = w.tiles_m * w.tiles_n * w.parts, pairs = most > 0 ? most : 1;
    if (w.M > 0x7fffffff - 256 || w.F > 0x7fffffff - 256 || w.D > 0x7fffffff - 256) return RLSCAN_ERR_SHAPE;
    return launch(true, projection_kernel<JOB>, 2 * (tiles < pairs ? tiles : pairs), kThreads, kSmem, s, maps, w);
}

// An output [rows, columns] that leaves in boxes of 64 columns x 32 rows, where its alignment allows
void map_out(Maps &m, int i, Work &w, void *p, int64_t rows, int64_t columns, int64_t pitch)
{
    w.out[i] = static_cast<bf16 *>(p);
    w.out_stride = pitch;
    w.out_mapped = (i == 0 || w.out_mapped) && fits_map(p, rows, columns, pitch) && umma::encode(&m.out[i], p, rows, columns, up8(pitch), 32);
}

bool vec_rows(const void *p, int64_t stride) { return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(stride * 2)) & 15u) == 0; }

}  // namespace

size_t gated_projection_workspace(const rlscan_gated_projection_args &a)
{
    return a.M == 0 || a.F == 0 || a.D == 0 || projection_is_few(a) ? 0 : layout(a).bytes;
}

rlscan_status launch_gated_projection(const rlscan_gated_projection_args &a, void *h, void *ws, cudaStream_t s)
{
    if (a.D == 0) return ok(cudaMemsetAsync(h, 0, static_cast<size_t>(a.M) * a.F * 2, s)) ? RLSCAN_OK : RLSCAN_ERR_CUDA;
    if (projection_is_few(a)) return launch_gated_projection_few(a, h, s);
    Layout l = layout(a);
    rlscan_status st = pack_all(a, l, static_cast<char *>(ws), s);
    if (st != RLSCAN_OK) return st;
    Maps m = {};
    if (!map_of(&m.a[0], l.x, 128) || !map_of(&m.b[0], l.gate, 128) || !map_of(&m.b[1], l.up, 128)) return RLSCAN_ERR_CUDA;
    Work w = {};
    w.M = a.M, w.D = a.D, w.F = a.F, w.act = static_cast<int>(a.activation);
    w.tiles_m = ceil_div(a.M, 256), w.tiles_n = ceil_div(a.F, 128), w.steps = ceil_div(a.D, kBlockK);
    w.parts = 1, w.part_steps = w.steps;
    map_out(m, 0, w, h, a.M, a.F, a.F);
    return launch_job<Job::Forward>(m, w, s);
}

size_t gated_projection_backward_workspace(const rlscan_gated_projection_args &a)
{
    if (a.M == 0 || a.F == 0 || a.D == 0) return 0;
    return layout(a).bytes + up256(static_cast<size_t>(a.M) * 2 * up8(a.F) * 2) + splits_of(a).bytes;
}

rlscan_status launch_gated_projection_backward(const rlscan_gated_projection_args &a, const void *grad_h,
                                               int64_t grad_h_stride, void *grad_x, void *grad_gate, void *grad_up,
                                               void *ws, cudaStream_t s)
{
    if (a.M == 0 || a.F == 0 || a.D == 0) {  // sums of nothing
        const size_t w = static_cast<size_t>(a.F) * a.D * 2, x = static_cast<size_t>(a.M) * a.D * 2;
        for (void *p : {grad_gate, grad_up})
            if (p != nullptr && w > 0 && !ok(cudaMemsetAsync(p, 0, w, s))) return RLSCAN_ERR_CUDA;
        if (grad_x != nullptr && x > 0 && !ok(cudaMemsetAsync(grad_x, 0, x, s))) return RLSCAN_ERR_CUDA;
        return RLSCAN_OK;
    }
    Layout l = layout(a);
    rlscan_status st = pack_all(a, l, static_cast<char *>(ws), s);
    if (st != RLSCAN_OK) return st;
    const int64_t pitch = up8(a.F);
    bf16 *g = reinterpret_cast<bf16 *>(static_cast<char *>(ws) + l.bytes);  // [M, 2 pitch]: gz, gu
    Maps m = {};
    if (!map_of(&m.a[0], l.x, 128) || !map_of(&m.b[0], l.gate, 128) || !map_of(&m.b[1], l.up, 128)) return RLSCAN_ERR_CUDA;
    Work w = {};
    w.M = a.M, w.D = a.D, w.F = a.F, w.act = static_cast<int>(a.activation);
    w.tiles_m = ceil_div(a.M, 256), w.tiles_n = ceil_div(a.F, 128), w.steps = ceil_div(a.D, kBlockK);
    w.grad_h = static_cast<const bf16 *>(grad_h), w.grad_h_stride = grad_h_stride, w.grad_h_vec = vec_rows(grad_h, grad_h_stride);
    w.parts = 1, w.part_steps = w.steps;
    map_out(m, 0, w, g, a.M, a.F, 2 * pitch);
    map_out(m, 1, w, g + pitch, a.M, a.F, 2 * pitch);
    st = launch_job<Job::Gates>(m, w, s);
    if (st != RLSCAN_OK) return st;
    const GradSplits splits = splits_of(a);
    w.sums = reinterpret_cast<float *>(reinterpret_cast<char *>(g) + up256(static_cast<size_t>(a.M) * 2 * pitch * 2));
    const Operand gz{g, a.M, a.F, 2 * pitch, false}, gu{g + pitch, a.M, a.F, 2 * pitch, false};
    if (grad_x != nullptr) {
        Maps mx = {};
        if (!map_of(&mx.a[0], gz, 128) || !map_of(&mx.a[1], gu, 128) || !map_of(&mx.b[0], l.gate, 64) || !map_of(&mx.b[1], l.up, 64))
            return RLSCAN_ERR_CUDA;
        w.tiles_n = ceil_div(a.D, 256), w.steps = 2 * ceil_div(a.F, kBlockK);
        w.parts = splits.input.parts, w.part_steps = splits.input.steps;
        map_out(mx, 0, w, grad_x, a.M, a.D, a.D);
        w.out[1] = nullptr;
        st = launch_job<Job::Input>(mx, w, s);
        if (st == RLSCAN_OK && w.parts > 1) st = join(w, a.M, s);
        if (st != RLSCAN_OK) return st;
    }
    if (grad_gate != nullptr) {
        Maps mw = {};
        if (!map_of(&mw.a[0], gz, 64) || !map_of(&mw.a[1], gu, 64) || !map_of(&mw.b[0], l.x, 64)) return RLSCAN_ERR_CUDA;
        w.tiles_m = 2 * ceil_div(a.F, 256), w.tiles_n = ceil_div(a.D, 256), w.steps = ceil_div(a.M, kBlockK);
        map_out(mw, 0, w, grad_gate, a.F, a.D, a.D);
        map_out(mw, 1, w, grad_up, a.F, a.D, a.D);
        w.parts = splits.weights.parts, w.part_steps = splits.weights.steps;
        st = launch_job<Job::Weights>(mw, w, s);
        if (st == RLSCAN_OK && w.parts > 1) st = join(w, a.F, s);
    }
    return st;
}

rlscan_status gated_projection_status(cudaStream_t s) { return take_flag(g_timed_out, s); }

}  // namespace seq
}  // namespace rlscan
