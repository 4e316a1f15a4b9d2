// k_selective_scan_bf16.cu -- the selective scan's kernels for bfloat16 activations.
#include "selective_scan.cuh"

namespace rlscan {
namespace seq {

template rlscan_status scan_typed<bf16>(const Plan &, const rlscan_selective_scan_args &, ScanOut, cudaStream_t);
template rlscan_status back_states_typed<bf16>(const rlscan_selective_scan_args &, ScanOut, const float *, cudaStream_t);

}  // namespace seq
}  // namespace rlscan
