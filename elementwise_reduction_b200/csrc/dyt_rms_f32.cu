// The root-mean-square norm's kernels over f32 activations (see dyt_rms_select.cuh).
#include "dyt_rms_select_impl.cuh"

namespace dyt {
namespace norm {
DYT_INSTANTIATE_RMS(float)
}  // namespace norm
}  // namespace dyt
