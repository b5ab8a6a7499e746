// da_norm_f32.cu -- norm kernels for f32 rows.
#include "da_norm.cuh"

namespace da {

const void* norm_kernel_f32(int layout, int items, bool block, bool residual) {
  return norm_kernel_for<float>(layout, items, block, residual);
}

}  // namespace da
