// Host-side helpers that the two handles' entry points share (kvring_api.cu
// defines the functions that are not inline).
#pragma once
#include <cmath>
#include <cstddef>
#include <cstdint>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "common.cuh"

namespace kvring_dev {

// Remember the CUDA error for kvring_last_cuda_error; returns KVRING_ERR_CUDA.
int cuda_fail(cudaError_t e);

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// omega_{a,j} = base^(-2j/d_a), fp64
inline double omega(double base, int d_axis, int j) { return std::pow(base, -2.0 * j / d_axis); }

inline bool rope_axes_ok(int n_axes, const int32_t* axis_dims, const int32_t* pos_count, int head_dim, double base) {
  if (n_axes < 1 || n_axes > kMaxAxes) return false;
  int sum = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (axis_dims[a] < 2 || axis_dims[a] % 2 || axis_dims[a] > head_dim) return false;
    if (pos_count[a] < 1 || pos_count[a] > (1 << 24)) return false;
    sum += axis_dims[a];
  }
  return sum == head_dim && base > 1.0 && std::isfinite(base);
}

}  // namespace kvring_dev
