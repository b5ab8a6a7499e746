// da_rowvec.cuh -- what the row operators' kernels and launches share: wide accesses, conversions of
// pairs, strided row tensors' places in memory.
#pragma once

#include <algorithm>
#include <climits>
#include <cstdint>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "da_rows.h"

namespace da {

// 32 bytes a lane (aligned to 32): neighbouring lanes then fill whole sectors in one instruction,
// where two 16-byte accesses 32 bytes apart touch each sector twice (1.7 GB read back from FP8, 8 items a lane:
// 266 us, 340 with 16-byte stores; a rotary gradient 26.7, 27.4; a plain write of 134 MB 23.1, 24.0).
__device__ __forceinline__ void load32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                 "=r"(b.w)
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
// Two E4M3 codes, nearest even, |x| > 448 to +-448; `a` in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float a, float b) {
  uint32_t u;
  asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %2, %1;\n\tcvt.u32.u16 %0, c;\n\t}"
      : "=r"(u)
      : "f"(a), "f"(b));
  return u;
}

// A row tensor's places in memory, from its strides in elements (of which a byte's are a few bits more: larger
// ones than memory has are as good as the largest).
inline RowRuns runs(const void* p, long long rows, long long rs, long long heads, long long hs, int d, int es) {
  auto bytes = [es](long long s) {
    const long long most = INT64_MAX / 8;
    return std::min(std::max(s, -most), most) * es;
  };
  return {(uint64_t)(uintptr_t)p, rows, bytes(rs), heads, bytes(hs), (int64_t)d * es};
}

}  // namespace da
