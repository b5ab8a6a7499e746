// da_norm_bf16.cu -- norm kernels for bf16 rows.
#include "da_norm.cuh"

namespace da {

const void* norm_kernel_bf16(int layout, int items, bool block, bool residual) {
  return norm_kernel_for<__nv_bfloat16>(layout, items, block, residual);
}
const void* careful_norm_kernel_bf16() { return reinterpret_cast<const void*>(&careful_norm_kernel<__nv_bfloat16>); }

}  // namespace da
