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

// Forward: z and u, then h.  Gates: z and u, then gz and gu.  Grads: dx, the sum
// over both gates' columns, and dWg and dWu.  gz and gu are rounded to bfloat16,
// the type of the last products' operands: the gradients are 0.0023 of their size
// off, which with 32 bits there would be 0.0017, the outputs' own rounding.  A
// second bfloat16 part of each would keep those bits, and make the last products,
// two thirds of all operations, twice as many.
enum class Job { Forward, Gates, Grads };

struct Maps {
    CUtensorMap a[4], b[3], out[3];  // Grads: dx's, then the weights'
};

// A product: its tiles, each in `parts` of `part_steps` steps (blocks of 64
// values of K; 1: whole), which are the items of work.
struct Product {
    bool weights;
    int64_t tiles_m, tiles_n, steps, parts, part_steps;
    float *sums;  // of parts > 1: [parts][rows of all outputs][columns]
    __host__ __device__ int64_t items() const { return tiles_m * tiles_n * parts; }
};

struct Work {
    int64_t M, D, F;
    int act;
    const bf16 *grad_h;
    int64_t grad_h_stride;
    bool grad_h_vec;
    Product product[2];  // the one of longer items first; the second may have none
    int64_t items[2], whole, high, extra;  // see item_of: items of both, whole rounds of the first's, pairs with one more
    bf16 *out[3];
    int64_t out_stride;
    bool out_mapped[3];  // the output leaves through maps.out
};

// The i-th item of a pair of blocks, -1 behind its last: the first product's in
// turn; then the pairs that had one less of them take `extra` of the second's,
// which last as long, and all take the rest in turn.
__device__ __forceinline__ int64_t item_of(const Work &k, int64_t at, int64_t pairs, int64_t i)
{
    const int64_t a = k.items[0], b = k.items[1], high = k.high, mine = k.whole + (at < high ? 1 : 0);
    if (i < mine) return at + i * pairs;
    int64_t j = i - mine;
    const int64_t low = high > 0 ? pairs - high : 0;
    if (low > 0 && at >= high) {
        if (j < k.extra) {
            const int64_t first = at - high + j * low;
            return first < b ? a + first : -1;
        }
        j -= k.extra;
    }
    const int64_t rest = k.extra * low + (at >= high ? at - high : at - high + pairs) + j * pairs;
    return rest < b ? a + rest : -1;
}

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
// Bound by the products where K is long (forward 16384 x 4096 x 12288 back to
// back 1810 to 1900 us, 1.74 to 1.82 PFLOP/s of the 1.89 that the library's plain
// product reaches in a burst; a pass, inputs cold, 1940 to 2060), by the epilogue and
// the outputs' bytes where it is short (3636 x 64 x 4016, gelu, 26 us).
// Four warps for the sums held the products up: gradients of 16384 x 512 x 512
// 130 us, with eight 107.
template <Job JOB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    projection_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Work k)
{
    constexpr bool kGates = JOB == Job::Forward || JOB == Job::Gates;
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
    const int64_t at_pair = blockIdx.x / 2, pairs = gridDim.x / 2;
    // Tiles in bands of eight rows of tiles, column after column: the pairs at
    // work share rows of A and columns of B in L2.
    auto place = [&](const Product &of, int64_t tile, int64_t &m, int64_t &n) {
        constexpr int64_t kBand = 8;
        const int64_t band = tile / (kBand * of.tiles_n), in = tile - band * kBand * of.tiles_n;
        const int64_t high = of.tiles_m - band * kBand < kBand ? of.tiles_m - band * kBand : kBand;
        m = band * kBand + in % high;
        n = in / high;
    };
    // The item's product, and the item's number among the product's
    auto product_of = [&](int64_t &item) -> const Product & {
        if (item < k.items[0]) return k.product[0];
        item -= k.items[0];
        return k.product[1];
    };
    // An item is a tile, or a part of its K
    auto first_step = [](const Product &of, int64_t item) { return item % of.parts * of.part_steps; };
    auto last_step = [](const Product &of, int64_t item) {
        const int64_t e = (item % of.parts + 1) * of.part_steps;
        return e < of.steps ? e : of.steps;
    };
    if (warp == 0 && lane == 0) {  // copies
        uint32_t stage = 0, phase = 1;  // the first wait on an empty stage passes
        int64_t issued = 0;
        for (int64_t i = 0, item; !has_given_up(&gave_up) && (item = item_of(k, at_pair, pairs, i)) >= 0; ++i) {
            const Product &of = product_of(item);
            int64_t tm, tn;
            place(of, item / of.parts, tm, tn);
            for (int64_t s = first_step(of, item), e = last_step(of, item); s < e; ++s) {
                // (a look at the flag here, behind a wait that has passed, made the
                // gradients of 5000 x 2560 x 6912 701 us long, so 660)
                if (!wait(ptx::smem_u32(&empty[stage]), phase, &gave_up)) break;
                const uint32_t bar = umma::of_rank(ptx::smem_u32(&full[stage]), 0);
                const uint32_t a = smem + stage * kStageBytes, b = a + kTileBytes;
                if (rank == 0) ptx::mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
                if constexpr (kGates) {
                    const int k0 = static_cast<int>(s) * kBlockK;
                    umma::load_box(a, &maps.a[0], k0, static_cast<int>(tm * 256 + rank * 128), bar);
                    umma::load_box(b, &maps.b[rank], k0, static_cast<int>(tn * 128), bar);
                } else if (!of.weights) {
                    const int64_t half = of.steps / 2;
                    const int part = s >= half ? 1 : 0, k0 = static_cast<int>(s - part * half) * kBlockK;
                    umma::load_box(a, &maps.a[part], k0, static_cast<int>(tm * 256 + rank * 128), bar);
                    for (int i = 0; i < 2; ++i)
                        umma::load_box(b + i * (kTileBytes / 2), &maps.b[part], static_cast<int>(tn * 256 + rank * 128 + 64 * i), k0, bar);
                } else {
                    const int64_t half = of.tiles_m / 2;
                    const int part = tm >= half ? 1 : 0, k0 = static_cast<int>(s) * kBlockK;
                    const int f0 = static_cast<int>((tm - part * half) * 256 + rank * 128);
                    for (int i = 0; i < 2; ++i) {
                        umma::load_box(a + i * (kTileBytes / 2), &maps.a[2 + part], f0 + 64 * i, k0, bar);
                        umma::load_box(b + i * (kTileBytes / 2), &maps.b[2], static_cast<int>(tn * 256 + rank * 128 + 64 * i), k0, bar);
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
        uint32_t stage = 0, phase = 0, buffer = 0, buffer_phase = 1;
        for (int64_t i = 0, item; (item = item_of(k, at_pair, pairs, i)) >= 0; ++i) {
            const Product &of = product_of(item);
            // rows of A and columns of B lie along K (Forward, Gates; dx's A) or across it
            const bool a_across = !kGates && of.weights;
            const uint32_t instruction = kGates ? umma::instruction(false, false, 256, 256)
                                         : a_across ? umma::instruction(true, true, 256, 256) : umma::instruction(false, true, 256, 256);
            if (!wait(ptx::smem_u32(&sums_empty[buffer]), buffer_phase, &gave_up)) break;
            umma::fence_after();
            bool fine = true;
            const int64_t begin = first_step(of, item), stop = last_step(of, item);
            for (int64_t s = begin; s < stop && fine; ++s) {
                fine = wait(ptx::smem_u32(&full[stage]), phase, &gave_up);
                if (!fine) break;
                umma::fence_after();
                const uint32_t a = smem + stage * kStageBytes, b = a + kTileBytes;
#pragma unroll
                for (int j = 0; j < kBlockK / 16; ++j)
                    umma::multiply(tmem + buffer * 256, umma::descriptor(a + j * (a_across ? 2048 : 32), kTileBytes / 2),
                                   umma::descriptor(b + j * (kGates ? 32 : 2048), kTileBytes / 2), instruction, s > begin || j > 0);
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
            if (k.out_mapped[i]) {
                fence_async();
                __syncwarp();
                if (lane == 0 && some) store_box2(&maps.out[i], x, y, box);
            } else {
                __syncwarp();
                if (some) copy_box(k.out[i] + y * k.out_stride + x, k.out_stride, box, lane, rows - y, columns - x);
            }
            // (one group a box, an empty one too: free_box counts them, and Grads' outputs may leave either way)
            if (lane == 0) stores_commit();
        };
        for (int64_t i = 0, item; (item = item_of(k, at_pair, pairs, i)) >= 0; ++i) {
            const Product &of = product_of(item);
            int64_t tm, tn;
            place(of, item / of.parts, tm, tn);
            const int64_t half = of.tiles_m / 2;
            const int which = of.weights && tm >= half ? 1 : 0;
            const int64_t row = (tm - which * half) * 256 + rank * 128 + part * 32 + lane;
            const int64_t rows = of.weights ? k.F : k.M;
            if (!wait_warp(ptx::smem_u32(&sums_full[buffer]), phase, &gave_up)) break;
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
                    if (of.parts > 1) {
                        const int64_t all = of.weights ? 2 * rows : rows, n = row < rows ? k.D - d0 - c : 0;
                        float *to = of.sums + ((item % of.parts) * all + which * rows + row) * k.D + d0 + c;
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
                        if (h == 1) put_box(of.weights ? 1 + which : 0, d0 + c - 32, row0, rows, k.D, box);
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

// The gradients' two products share a launch, the longer items first.  Few
// tiles of a long K leave pairs without work: a tile of more steps than a pair's
// average load is taken in parts, of at least four steps each, whose sums are
// joined in order by another kernel.  Taking a tile's sums out counts as eight
// steps.  Measured, gradients of 8 x 4096 x 12288 (dx: 16 tiles of 384 steps) 209
// us whole, 168 in parts (and dW of 16384 x 512 x 512 in parts: all gradients 125
// and 66).
struct GradPlan {
    Product input, weights;
    int64_t load;              // steps of a pair, on average
    size_t at_weights, bytes;  // of the sums of parts
};
GradPlan plan_of(const rlscan_gated_projection_args &a, bool want_x, bool want_weights)
{
    constexpr int64_t kEnd = 8;
    GradPlan g = {};
    g.input = {false, want_x ? ceil_div(a.M, 256) : 0, ceil_div(a.D, 256), 2 * ceil_div(a.F, kBlockK), 1, 0, nullptr};
    g.weights = {true, want_weights ? 2 * ceil_div(a.F, 256) : 0, ceil_div(a.D, 256), ceil_div(a.M, kBlockK), 1, 0, nullptr};
    const int64_t pairs = (sm_count() > 0 ? sm_count() : 152) / 2;
    g.load = (g.input.items() * (g.input.steps + kEnd) + g.weights.items() * (g.weights.steps + kEnd)) / pairs;
    size_t at = 0;
    for (Product *p : {&g.input, &g.weights}) {
        const int64_t each = g.load > 4 ? g.load : 4;
        p->parts = p->items() > 0 && p->steps > each ? ceil_div(p->steps, each) : 1;
        if (p->parts > p->steps / 4) p->parts = p->steps / 4 > 1 ? p->steps / 4 : 1;
        p->part_steps = ceil_div(p->steps, p->parts);
        p->parts = ceil_div(p->steps, p->part_steps);
        if (p == &g.weights) g.at_weights = at;
        if (p->parts > 1) at += up256(static_cast<size_t>(p->parts) * (p->weights ? 2 * a.F : a.M) * a.D * sizeof(float));
    }
    g.bytes = at;
    return g;
}

rlscan_status join(const Product &p, int64_t rows, int64_t columns, bf16 *out0, bf16 *out1, cudaStream_t s)
{
    const int64_t half = rows * columns, all = out1 != nullptr ? 2 * half : half, most = 16 * (sm_count() > 0 ? sm_count() : 152);
    const int64_t blocks = ceil_div(all, 256);
    return launch_overlapped(join_kernel, blocks < most ? blocks : most, 256, 0, s, p.sums, p.parts, all, half, out0, out1);
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
    for (int i = 0; i < 2; ++i) w.items[i] = w.product[i].items();
    const int64_t items = w.items[0] + w.items[1], pairs = most > 0 && most < items ? most : most > 0 ? items : 1;
    w.whole = w.items[0] / pairs, w.high = w.items[0] % pairs;
    const int64_t each = w.product[1].part_steps + 1;  // (an item takes a little time beside its steps)
    w.extra = (w.product[0].part_steps + each / 2) / each;
    if (w.M > 0x7fffffff - 256 || w.F > 0x7fffffff - 256 || w.D > 0x7fffffff - 256) return RLSCAN_ERR_SHAPE;
    return launch(true, projection_kernel<JOB>, 2 * pairs, kThreads, kSmem, s, maps, w);
}

// An output [rows, columns] that leaves in boxes of 64 columns x 32 rows, where its alignment allows
void map_out(Maps &m, int i, Work &w, void *p, int64_t rows, int64_t columns, int64_t pitch)
{
    w.out[i] = static_cast<bf16 *>(p);
    w.out_stride = pitch;
    w.out_mapped[i] = fits_map(p, rows, columns, pitch) && umma::encode(&m.out[i], p, rows, columns, up8(pitch), 32);
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
    w.product[0] = {false, ceil_div(a.M, 256), ceil_div(a.F, 128), ceil_div(a.D, kBlockK), 1, ceil_div(a.D, kBlockK), nullptr};
    map_out(m, 0, w, h, a.M, a.F, a.F);
    return launch_job<Job::Forward>(m, w, s);
}

size_t gated_projection_backward_workspace(const rlscan_gated_projection_args &a)
{
    if (a.M == 0 || a.F == 0 || a.D == 0) return 0;
    size_t sums = 0;  // of whichever gradients are asked for: one alone may be in more parts
    for (const bool x : {true, false})
        for (const bool weights : {true, false}) {
            const size_t n = plan_of(a, x, weights).bytes;
            sums = n > sums ? n : sums;
        }
    return layout(a).bytes + up256(static_cast<size_t>(a.M) * 2 * up8(a.F) * 2) + sums;
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
    w.product[0] = {false, ceil_div(a.M, 256), ceil_div(a.F, 128), ceil_div(a.D, kBlockK), 1, ceil_div(a.D, kBlockK), nullptr};
    w.grad_h = static_cast<const bf16 *>(grad_h), w.grad_h_stride = grad_h_stride, w.grad_h_vec = vec_rows(grad_h, grad_h_stride);
    map_out(m, 0, w, g, a.M, a.F, 2 * pitch);
    map_out(m, 1, w, g + pitch, a.M, a.F, 2 * pitch);
    st = launch_job<Job::Gates>(m, w, s);
    if (st != RLSCAN_OK || (grad_x == nullptr && grad_gate == nullptr)) return st;
    GradPlan p = plan_of(a, grad_x != nullptr, grad_gate != nullptr);
    char *sums = reinterpret_cast<char *>(g) + up256(static_cast<size_t>(a.M) * 2 * pitch * 2);
    p.input.sums = reinterpret_cast<float *>(sums);
    p.weights.sums = reinterpret_cast<float *>(sums + p.at_weights);
    const Operand gz{g, a.M, a.F, 2 * pitch, false}, gu{g + pitch, a.M, a.F, 2 * pitch, false};
    Maps mg = {};
    if (grad_x != nullptr) {
        if (!map_of(&mg.a[0], gz, 128) || !map_of(&mg.a[1], gu, 128) || !map_of(&mg.b[0], l.gate, 64) || !map_of(&mg.b[1], l.up, 64))
            return RLSCAN_ERR_CUDA;
        map_out(mg, 0, w, grad_x, a.M, a.D, a.D);
    }
    if (grad_gate != nullptr) {
        if (!map_of(&mg.a[2], gz, 64) || !map_of(&mg.a[3], gu, 64) || !map_of(&mg.b[2], l.x, 64)) return RLSCAN_ERR_CUDA;
        map_out(mg, 1, w, grad_gate, a.F, a.D, a.D);
        map_out(mg, 2, w, grad_up, a.F, a.D, a.D);
    }
    const bool input_first = p.weights.items() == 0 || (p.input.items() > 0 && p.input.part_steps >= p.weights.part_steps);
    w.product[0] = input_first ? p.input : p.weights;
    w.product[1] = input_first ? p.weights : p.input;
    // Much work gains nothing by sharing a launch, and the most loses by it: the
    // pairs, no longer at the same steps of K, find less of their operands in L2.
    // Measured, all gradients, one launch and two: 375 x 2912 x 368 (15 steps a
    // pair) 36 and 45 us, 5000 x 2560 x 6912 (1207) 665 and 708, 8192 x 4096 x 8192
    // (3610) 2059 and 2065, 16384 x 4096 x 6144 (5362) 3121 and 3130, 16384 x 4096
    // x 12288 (10617) 6420 and 6370, 30000 x 4096 x 12288 (19378) 11829 and 11627.
    if (p.load > 4096) {
        const Product second = w.product[1];
        w.product[1] = {};
        st = launch_job<Job::Grads>(mg, w, s);
        w.product[0] = second;
    }
    if (st == RLSCAN_OK && w.product[0].items() > 0) st = launch_job<Job::Grads>(mg, w, s);
    if (st == RLSCAN_OK && p.input.parts > 1) st = join(p.input, a.M, a.D, static_cast<bf16 *>(grad_x), nullptr, s);
    if (st == RLSCAN_OK && p.weights.parts > 1)
        st = join(p.weights, a.F, a.D, static_cast<bf16 *>(grad_gate), static_cast<bf16 *>(grad_up), s);
    return st;
}

rlscan_status gated_projection_status(cudaStream_t s) { return take_flag(g_timed_out, s); }

}  // namespace seq
}  // namespace rlscan
