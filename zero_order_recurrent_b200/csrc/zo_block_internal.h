// Host-side internals of the state-space block's calls: launchers and the
// rules that size their grids and workspaces.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/zo_block.h"

namespace zo {

// The grid rules count on a B200's SMs, so that workspace sizes need no device.
constexpr int kBlockSMs = 148;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Widest vector (in elements, at most `most`) with which a tensor's rows and
// steps can be accessed: its base, strides and `channels` must all keep to it.
inline int vec_width(const zo_tensor& t, int elem_bytes, int64_t channels, int most) {
  if (!t.ptr) return most;
  int v = most;
  while (v > 1 && (channels % v || t.row % v || t.step % v ||
                   reinterpret_cast<uintptr_t>(t.ptr) % (uintptr_t)(v * elem_bytes)))
    v /= 2;
  return v;
}


// Lets a kernel have `bytes` of dynamic shared memory.
template <class K>
cudaError_t allow_shared(K kernel, int bytes) {
  return bytes <= 48 * 1024
             ? cudaSuccess
             : cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

cudaError_t launch_conv(const zo_conv_args& a, cudaStream_t st);
int64_t conv_backward_workspace(const zo_conv_args& a);
cudaError_t launch_conv_backward(const zo_conv_args& a, const zo_conv_grads& g, float* ws,
                                 cudaStream_t st);
int64_t scan_workspace(const zo_scan_args& a);
int64_t scan_backward_workspace(const zo_scan_args& a);
cudaError_t launch_scan(const zo_scan_args& a, float* ws, cudaStream_t st);
cudaError_t launch_scan_step(const zo_scan_args& a, cudaStream_t st);
cudaError_t launch_scan_backward(const zo_scan_args& a, const zo_scan_grads& g, float* ws,
                                 cudaStream_t st);
cudaError_t launch_norm(const zo_norm_args& a, cudaStream_t st);
int64_t norm_backward_workspace(const zo_norm_args& a);
cudaError_t launch_norm_backward(const zo_norm_args& a, const zo_norm_grads& g, float* ws,
                                 cudaStream_t st);

// Partial sums are laid out [set][part][n values]; the values are those of up to three outputs
// one after the other, each n long; outputs without a pointer are left out.  Every value
// is the sum over the parts in a fixed order.
struct SumOut {
  zo_f32 out;
  int64_t n;
};
cudaError_t launch_sum_parts(const float* part, int sets, int64_t parts, int64_t n,
                             const SumOut* outs, int count, cudaStream_t st);

}  // namespace zo
