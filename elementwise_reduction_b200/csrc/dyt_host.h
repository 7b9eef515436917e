// Host helpers shared by the entry points' translation units: argument
// checks, per-device facts, error and launch records, and the programmatic
// launch configuration. The stateful ones are defined in dyt_api.cu.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "dyt.h"

namespace dyt {
namespace host {

// Keeps a failed CUDA call's code for dyt_last_cuda_error, clears the
// runtime's last-error state and returns DYT_ERR_CUDA.
dyt_status cuda_fail(cudaError_t e);

// The calling thread's record for dyt_last_launch_info.
void record_info(const dyt_launch_info &i);

// The current device and its SM count (cached).
dyt_status current_sms(int *dev_out, int *sms_out);
// CTAs of `block` threads of a kernel without dynamic shared memory that fit on an SM (cached).
dyt_status occupancy(int dev, const void *kernel, int block, int *ctas);
// Opt a kernel in to at least `bytes` of dynamic shared memory, once per device and size; safe from any thread.
dyt_status prepare_smem(int dev, const void *kernel, int bytes);

dyt_status check_shape(int64_t M, int64_t N, int xd);
dyt_status check_pitch(int64_t M, int64_t N, int64_t ld);

inline size_t dsize(int d) { return d == DYT_F32 ? 4 : 2; }
inline bool valid_dtype(int d) { return d == DYT_F32 || d == DYT_BF16 || d == DYT_F16; }
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
// A pointer to whole elements of `bytes` bytes (the kernels' loads need it).
inline bool elem_aligned(const void *p, size_t bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }
// Elements between the 16-byte boundary below p and p.
inline int shift_of(const void *p, size_t elem) { return (int)(((uintptr_t)p & 15u) / elem); }
// Two pointers at the same offset past a 16-byte boundary.
inline bool same_offset(const void *a, const void *b) { return (((uintptr_t)a ^ (uintptr_t)b) & 15u) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
// A row pitch of whole 16-byte vectors.
inline bool vec_pitch(int64_t ld, size_t elem) { return ((uint64_t)ld * elem) % 16 == 0; }

// Programmatic dependent launch: the kernel may be scheduled while its
// predecessor in the stream drains; its first instruction waits
// (griddepcontrol.wait) for that predecessor, so stream order holds.
struct PdlConfig {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg;
  PdlConfig(unsigned grid, unsigned block, size_t smem, cudaStream_t s) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

}  // namespace host
}  // namespace dyt
