// k_selective_scan.cu -- the layout of a call of the selective scan and its
// workspace; the kernels are in selective_scan.cuh.
#include "scan_plan.cuh"

namespace rlscan {
namespace seq {
namespace {

constexpr int kTile = kCheckpoint;


// Sixteen states a lane need the fewest instructions a state, eight give
// twice the warps; chunks give as many warps as a row has tokens for, but
// compute every state twice.  Measured (D 2048, S 16, bf16, microseconds):
//   one row    T 512: 60 unsplit (8 states), 34 in chunks of 64;
//              T 2048: 213, 68 (128);  T 8192: 829, 185 (16 states, 512)
//   four rows  T 512: 60, 65;  T 2048: 214, 175 (16, 128);  T 8192: 830, 563 (16, 512)
//   eight rows T 2048: 267 (8) and 279 (16), 301 (16, 256);  T 8192: 1037 (8), 1081 (16, 512)
// so rows are split while the unsplit call has less than 1.5 blocks an SM.
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
    const int64_t narrow = blocks_of(8);
    const bool split = a.T > 256 && 2 * narrow < 3 * sms && !(4 * narrow >= 3 * sms && a.T <= 1024);
    p.spt = a.S > 8 && (split ? a.T >= 1024 : narrow >= 3 * sms) ? 16 : 8;
    p.chunk = ceil_div(a.T > 0 ? a.T : 1, kTile) * kTile;
    if (split) {
        p.chunk = a.T < 1024 ? 64 : 256;
        while (p.chunk > 64 && blocks_of(p.spt) * ceil_div(a.T, p.chunk) < sms) p.chunk /= 2;
    }
    p.lanes = lanes_of(p.spt);
    p.chunks = ceil_div(a.T > 0 ? a.T : 1, p.chunk);
    return p;
}

size_t up(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

size_t selective_scan_workspace(const rlscan_selective_scan_args &a)
{
    const Plan p = plan(a);
    if (p.chunks <= 1) return 0;
    const size_t each = static_cast<size_t>(a.N) * p.chunks;
    return up(each * a.D * a.S * 4) + up(each * a.D * 4) + up(each);
}

rlscan_status launch_selective_scan(const rlscan_selective_scan_args &a, void *y, float *final_state,
                                    float *checkpoints, void *ws, cudaStream_t s)
{
    const Plan p = plan(a);
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
