// The root-mean-square norm's kernels over bf16 activations (see dyt_rms_select.cuh).
#include "dyt_rms_select_impl.cuh"

namespace dyt {
namespace norm {
DYT_INSTANTIATE_RMS(__nv_bfloat16)
}  // namespace norm
}  // namespace dyt
