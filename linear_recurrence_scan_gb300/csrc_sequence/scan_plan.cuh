// scan_plan.cuh -- how a call of the selective scan is laid out, and what its
// kernels write.
#pragma once

#include "sequence.cuh"

namespace rlscan {
namespace seq {

constexpr int kScanThreads = 128;

struct ScanOut {
    void *y;
    float *final_state, *checkpoints;
    // rows in `chunks` chunks of `chunk` tokens
    int64_t chunk, chunks;
    int unit;        // bytes of the copies into shared memory: 16, 4 or 0 (single values)
    bool vec;        // states in whole 16-byte units
    float *states;   // [N][chunks][D][S]: a chunk's own end state, then the state in front of it
    float *spans;    // [N][chunks][D]: the chunk's sum of dt
    uint8_t *cuts;   // [N][chunks]: an episode starts in the chunk
    rlscan_array3 grad_y;  // BACK
    int64_t sms;           // rows in the order of their lengths, for so many SMs; 0: as they are
};

// How a call is laid out: states per lane, and chunks of each row.
struct Plan {
    int spt, lanes;
    int64_t chunk, chunks;
};

// Tokens of a chunk where a chunk of every row takes `each` blocks and `slots`
// blocks run at once: chunks that fill whole waves, or half of the last one
// (whose blocks have an SM to fewer and take about 0.8 of the time).  A
// block's time is that of its tokens and of about eight more.  Of up to
// `halves` half waves the least time; 0 if all have more than `most` tokens.
inline int64_t wave_chunk(int64_t T, int64_t each, int64_t slots, int halves, int64_t most)
{
    int64_t best = 0, least = 0;
    for (int k = 1; k <= halves; ++k) {
        const int64_t count = k * slots / 2 / each;
        if (count < 1) continue;
        int64_t chunk = ceil_div(ceil_div(T, count), kCheckpoint) * kCheckpoint;
        chunk = chunk < 32 ? 32 : chunk;
        if (chunk > most) continue;
        const int64_t blocks = ceil_div(T, chunk) * each, rest = blocks % slots;
        const int64_t cost = (blocks / slots * 10 + (rest == 0 ? 0 : 2 * rest <= slots ? 8 : 10)) * (chunk + 8);
        if (best == 0 || cost < least) {
            best = chunk;
            least = cost;
        }
    }
    return best;
}

// Arrays whose rows are aligned to 2 bytes alone would come into shared memory
// value by value (measured, 8 x 2048 x 2049 x 16 bf16: 765 us, with aligned
// rows 236); a call that is large enough for another launch copies them into
// aligned rows first.  Whether it does, and the copies' bytes; then the
// copies, which replace the arrays in `a` (and *grad_y, where given).
size_t realign_workspace(const rlscan_selective_scan_args &a, bool backward);
rlscan_status realign(rlscan_selective_scan_args &a, rlscan_array3 *grad_y, char *ws, cudaStream_t s);

template <class T>
rlscan_status scan_typed(const Plan &p, const rlscan_selective_scan_args &a, ScanOut o, cudaStream_t s);
template <class T>
rlscan_status back_states_typed(const rlscan_selective_scan_args &a, ScanOut o, const float *grad_final, cudaStream_t s);

}  // namespace seq
}  // namespace rlscan
