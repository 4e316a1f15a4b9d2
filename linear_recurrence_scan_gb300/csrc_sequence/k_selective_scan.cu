// k_selective_scan.cu -- the layout of a call of the selective scan and its
// workspace; the kernels are in selective_scan.cuh.
#include "scan_plan.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kTile = kCheckpoint;


// Sixteen states a lane need the fewest instructions a state, eight give
// twice the warps; chunks give as many warps as a row has tokens for, but
// compute every state twice.  Measured (D 2048, S 16, bf16, microseconds; the
// states a lane and the chunk in parentheses):
//   one row    T 256: 27 unsplit;  T 512: 48 unsplit, 28 (8, 64);  T 1024: 91, 40 (8, 64);
//              T 2048: 173, 61 (16, 128);  T 8192: 668, 151 (16, 128)
//   four rows  T 512: 50, 56 (8, 64);  T 1024: 91, 93 (16, 128);  T 2048: 174, 148 (16, 128);
//              T 8192: 666, 500 (16, 128)
//   eight rows T 512: 62 unsplit with 16, 66 with 8;  T 2048: 222 and 236, 268 (16, 256);
//              T 8192: 861 and 914, 944 (16, 256)
// so rows are split while the unsplit call with eight states a lane has less
// than 1.5 blocks an SM (up to 1024 tokens: less than 0.75).  The chunks fill
// the four blocks an SM: against those of 64 or 128 tokens,
//   1 x 509 x 1536 31 us, 26 (chunks of 32);  2 x 700 x 2048 49, 45 (80);  1 x 2048 x 4096 93, 87 (112);
//   3 x 2048 x 2048 129, 120 (176);  2 x 16384 x 2048 509, 508 (224), ragged 421, 400
// Rows too long for that in eight half waves take chunks of 128 (2 x 16384 x
// 2048: 64: 556 us, 128: 509, 288: 488, 864: 498; ragged 461, 421, 415, 494).
Plan plan(const rlscan_selective_scan_args &a)
{
    const int64_t sms = sm_count() > 0 ? sm_count() : 152;
    auto lanes_of = [&](int spt) {
        int lanes = 1;
        while (spt * lanes < a.S) lanes *= 2;
        return lanes;
    };
    auto blocks_of = [&](int spt) { return a.N * ceil_div(a.D * lanes_of(spt), kScanThreads); };
    Plan p;
    const int64_t narrow = blocks_of(8);  // 0 without rows or channels
    const bool split = narrow > 0 && a.T > 256 && 2 * narrow < 3 * sms && !(4 * narrow >= 3 * sms && a.T <= 1024);
    p.spt = a.S > 8 && (split ? a.T >= 2048 : 2 * narrow >= 3 * sms) ? 16 : 8;
    p.chunk = ceil_div(a.T > 0 ? a.T : 1, kTile) * kTile;
    p.lanes = lanes_of(p.spt);
    if (split) {
        const int64_t chunk = wave_chunk(a.T, blocks_of(p.spt), 4 * sms, 8, 256);
        p.chunk = chunk > 0 ? chunk : 128;
    }
    p.chunks = ceil_div(a.T > 0 ? a.T : 1, p.chunk);
    return p;
}

size_t up(size_t v) { return (v + 255) / 256 * 256; }

size_t chunk_workspace(const rlscan_selective_scan_args &a, const Plan &p)
{
    if (p.chunks <= 1) return 0;
    const size_t each = static_cast<size_t>(a.N) * p.chunks;
    return up(each * a.D * a.S * 4) + up(each * a.D * 4) + up(each);
}

// ---- rows of 2-byte alignment -----------------------------------------------

constexpr int kRealigned = 6;  // x, delta, z, grad_y, B, C

struct RealignJobs {
    struct Job {
        rlscan_array3 from;
        uint32_t *to;        // rows of `words` pairs of values
        int64_t T, width, words, rows;
    } job[kRealigned];
    int jobs;
};

int64_t padded(int64_t width) { return (width + 7) / 8 * 8; }

// A warp copies a row, neighbouring lanes neighbouring pairs of values.
__global__ void __launch_bounds__(256) realign_kernel(const __grid_constant__ RealignJobs r)
{
    ptx::pdl_trigger_dependents();
    ptx::pdl_wait_prerequisites();
    const RealignJobs::Job &job = r.job[blockIdx.y];
    const int lane = threadIdx.x & 31, width = static_cast<int>(job.width), words = static_cast<int>(job.words);
    for (int64_t row = blockIdx.x * 8ll + threadIdx.x / 32; row < job.rows; row += gridDim.x * 8ll) {
        const Division at = divide(row, job.T);
        const uint16_t *p =
            static_cast<const uint16_t *>(job.from.data) + at.q * job.from.row_stride + at.r * job.from.token_stride;
        uint32_t *to = job.to + row * words;
#pragma unroll 8
        for (int i = lane; i < words; i += 32) {
            const uint32_t lo = 2 * i < width ? p[2 * i] : 0u, hi = 2 * i + 1 < width ? p[2 * i + 1] : 0u;
            to[i] = lo | hi << 16;
        }
    }
}

bool odd_rows(const rlscan_selective_scan_args &a)
{
    Chunk c;
    for (const rlscan_array3 *v : {&a.x, &a.delta, &a.B, &a.C}) c.add(v->data, v->row_stride, v->token_stride, 2);
    if (a.z.data != nullptr) c.add(a.z.data, a.z.row_stride, a.z.token_stride, 2);
    return c.size() == 0;
}

}  // namespace

size_t realign_workspace(const rlscan_selective_scan_args &a, bool backward)
{
    if (a.dtype != RLSCAN_BF16 || a.N * a.T * a.D < (1 << 18) || !odd_rows(a)) return 0;
    const size_t rows = 2 * static_cast<size_t>(a.N) * a.T;
    return up(rows * padded(a.D)) * (backward ? 4 : 3) + up(rows * padded(a.S)) * 2;
}

rlscan_status realign(rlscan_selective_scan_args &a, rlscan_array3 *grad_y, char *ws, cudaStream_t s)
{
    RealignJobs r;
    r.jobs = 0;
    auto take = [&](rlscan_array3 &v, int64_t width) {
        if (v.data == nullptr) return;
        RealignJobs::Job &j = r.job[r.jobs++];
        j.from = v;
        j.to = reinterpret_cast<uint32_t *>(ws);
        j.T = a.T;
        j.width = width;
        j.words = padded(width) / 2;
        j.rows = a.N * a.T;
        v.data = ws;
        v.token_stride = padded(width);
        v.row_stride = a.T * v.token_stride;
        ws += up(2 * static_cast<size_t>(a.N) * a.T * padded(width));
    };
    take(a.x, a.D);
    take(a.delta, a.D);
    take(a.z, a.D);
    take(a.B, a.S);
    take(a.C, a.S);
    if (grad_y != nullptr) take(*grad_y, a.D);
    const int64_t sms = sm_count() > 0 ? sm_count() : 152, need = ceil_div(a.N * a.T, 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(need < 8 * sms ? need : 8 * sms), static_cast<unsigned>(r.jobs));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, realign_kernel, r) != cudaSuccess) {
        cudaGetLastError();
        return RLSCAN_ERR_CUDA;
    }
    return RLSCAN_OK;
}

size_t selective_scan_workspace(const rlscan_selective_scan_args &a)
{
    return chunk_workspace(a, plan(a)) + realign_workspace(a, false);
}

rlscan_status launch_selective_scan(const rlscan_selective_scan_args &args, void *y, float *final_state,
                                    float *checkpoints, void *ws, cudaStream_t s)
{
    rlscan_selective_scan_args a = args;
    const Plan p = plan(a);
    if (realign_workspace(a, false) > 0) {
        const rlscan_status st = realign(a, nullptr, static_cast<char *>(ws) + chunk_workspace(a, p), s);
        if (st != RLSCAN_OK) return st;
    }
    ScanOut o{y, final_state, checkpoints, p.chunk, p.chunks, 0, false, nullptr, nullptr, nullptr, {}};
    if (p.chunks > 1) {
        const size_t each = static_cast<size_t>(a.N) * p.chunks;
        char *w = static_cast<char *>(ws);
        o.states = reinterpret_cast<float *>(w);
        o.spans = reinterpret_cast<float *>(w + up(each * a.D * a.S * 4));
        o.cuts = reinterpret_cast<uint8_t *>(w + up(each * a.D * a.S * 4) + up(each * a.D * 4));
    }
    return a.dtype == RLSCAN_BF16 ? scan_typed<bf16>(p, a, o, s) : scan_typed<float>(p, a, o, s);
}

rlscan_status launch_back_states(const rlscan_selective_scan_args &a, const rlscan_array3 &grad_y, const float *grad_final,
                                 int64_t chunk, int64_t chunks, float *states, float *spans, uint8_t *cuts,
                                 cudaStream_t s)
{
    const ScanOut o{nullptr, nullptr, nullptr, chunk, chunks, 0, false, states, spans, cuts, grad_y};
    return a.dtype == RLSCAN_BF16 ? back_states_typed<bf16>(a, o, grad_final, s) : back_states_typed<float>(a, o, grad_final, s);
}

}  // namespace seq
}  // namespace rlscan
