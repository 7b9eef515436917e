// The root-mean-square norm's kernels over f16 activations (see dyt_rms_select.cuh).
#include "dyt_rms_select_impl.cuh"

namespace dyt {
namespace norm {
DYT_INSTANTIATE_RMS(__half)
}  // namespace norm
}  // namespace dyt
