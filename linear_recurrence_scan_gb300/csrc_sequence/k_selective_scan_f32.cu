// k_selective_scan_f32.cu -- the selective scan's kernels for float32 activations.
#include "selective_scan.cuh"

namespace rlscan {
namespace seq {

template rlscan_status scan_typed<float>(const Plan &, const rlscan_selective_scan_args &, ScanOut, cudaStream_t);
template rlscan_status back_states_typed<float>(const rlscan_selective_scan_args &, ScanOut, const float *, cudaStream_t);

}  // namespace seq
}  // namespace rlscan
