// Which root-mean-square norm kernel a plan runs. The selectors are instantiated
// once per activation dtype (dyt_rms_f32.cu, dyt_rms_bf16.cu, dyt_rms_f16.cu), so
// that the kernels compile in parallel.
#pragma once

#include "dyt_rms.cuh"
#include "dyt_rows.h"

namespace dyt {
namespace norm {

using RmsFwdKernel = void (*)(RmsArgs);
using RmsBwdKernel = void (*)(RmsGradArgs);
using RmsBwdLongKernel = void (*)(RmsGradArgs, float *);
using RmsBwdColumnsKernel = void (*)(RmsGradArgs, const float *);

// res: with a residual (in the backward: the stored sum has a gradient). q8: an 8-bit output.
template <typename T>
RmsFwdKernel rms_fwd_kernel_of(const host::RowPlan &p, bool res, bool q8);
// Rows in registers.
template <typename T>
RmsBwdKernel rms_bwd_kernel_of(const host::RowPlan &p, bool res);
// Long rows: each row's sum, then dx and the column sums.
template <typename T>
RmsBwdLongKernel rms_bwd_rows_kernel_of(const host::RowPlan &p);
template <typename T>
RmsBwdColumnsKernel rms_bwd_columns_kernel_of(const host::RowPlan &p, bool res);

}  // namespace norm
}  // namespace dyt
