// da_norm_f16.cu -- norm kernels for f16 rows.
#include "da_norm.cuh"

namespace da {

const void* norm_kernel_f16(int layout, int items, bool block, bool residual) {
  return norm_kernel_for<__half>(layout, items, block, residual);
}

}  // namespace da
