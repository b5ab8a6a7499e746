// da_adapters_f32.cu -- adapter kernels for f32 rows.
#include "da_adapters.cuh"

namespace da {

const void* adapter_kernel_f32(int rank, int tiles, bool vec) {
  return adapter_kernel_for<float>(rank, tiles, vec);
}

}  // namespace da
