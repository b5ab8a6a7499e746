// da_norm_f32.cu -- norm kernels for f32 rows.
#include "da_norm.cuh"

namespace da {

const void* norm_kernel_f32(int layout, int items, bool block, bool residual) {
  return norm_kernel_for<float>(layout, items, block, residual);
}
const void* careful_norm_kernel_f32() { return reinterpret_cast<const void*>(&careful_norm_kernel<float>); }

}  // namespace da
