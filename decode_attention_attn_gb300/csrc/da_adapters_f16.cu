// da_adapters_f16.cu -- adapter kernels for f16 rows.
#include "da_adapters.cuh"

namespace da {

const void* adapter_kernel_f16(int rank, int tiles, bool vec) {
  return adapter_kernel_for<__half>(rank, tiles, vec);
}

}  // namespace da
