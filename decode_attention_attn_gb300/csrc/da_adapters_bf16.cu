// da_adapters_bf16.cu -- adapter kernels for bf16 rows.
#include "da_adapters.cuh"

namespace da {

const void* adapter_kernel_bf16(int rank, int tiles, bool vec) {
  return adapter_kernel_for<__nv_bfloat16>(rank, tiles, vec);
}

}  // namespace da
