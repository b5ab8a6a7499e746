// da_tcgen05.cuh -- the 5th-generation tensor cores' instructions as the kernels use them: tensor memory,
// matrix instructions and their descriptors, and the bounded waits of a warp.
#pragma once

#include <cstring>
#include <type_traits>

#include "da_device.cuh"

namespace da {

__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(slot)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// After the wait, `x` may be used: nothing that reads it can move above.
template <int N>
__device__ __forceinline__ void tmem_ready(float (&x)[N]) {
  tmem_wait_ld();
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+f"(x[k]));
}
template <int N>
__device__ __forceinline__ void tmem_ready(uint32_t (&x)[N]) {
  tmem_wait_ld();
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+r"(x[k]));
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// The thread of a converged warp that issues for it (the whole warp walks the issue loops, so that
// descriptors stay in uniform registers).
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}
// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}

// 32 columns of this warp's 32 TMEM lanes, one row a thread.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle: `block` is the distance between 64-element
// blocks along the contiguous dimension (read where that is M or N), `group` that between 8-row
// groups.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t block, uint32_t group) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(block >> 4) << 16 |
         (uint64_t)(group >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// fp32 accumulator, M = 128, N, 16-bit operands (bf16 or f16); trans_b: B's N is contiguous.
__host__ __device__ constexpr uint32_t mma_desc(bool bf16, int n, bool trans_b) {
  return 1u << 4 | (bf16 ? 1u : 0u) << 7 | (bf16 ? 1u : 0u) << 10 | (trans_b ? 1u : 0u) << 16 |
         (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}

__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// A pipeline wait that gives up, for every warp of the CTA, when one of them ran out of time: from
// then on nothing waits, no copy or MMA is issued, and every warp walks to its end (through all the
// CTA's barriers).
struct Waiter {
  int* abort_flag;
  int32_t* status;
  unsigned long long limit;
  bool dead;
  // warp-uniform
  __device__ __forceinline__ void operator()(uint64_t* bar, uint32_t parity) {
    bool ok = dead || mbar_try_wait(bar, parity);   // (the vote converges the warp either way)
    if (!__all_sync(0xffffffffu, ok)) {
      const unsigned long long t0 = global_timer_ns();
      while (!ok) {
#pragma unroll 1
        for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
        if (ok || *reinterpret_cast<volatile int*>(abort_flag)) break;
        if (global_timer_ns() - t0 > limit) {
          atomicOr(status, kStatusTimeout);
          atomicExch(abort_flag, 1);
          break;
        }
      }
      dead = __any_sync(0xffffffffu, !ok);
    }
  }
};

template <typename M>
__device__ __forceinline__ uint32_t pack_pair(float a, float b) {
  uint32_t u;
  if constexpr (std::is_same<M, __half>::value) {
    const __half2 h = __floats2half2_rn(a, b);
    memcpy(&u, &h, 4);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    memcpy(&u, &h, 4);
  }
  return u;
}
template <typename M>
__device__ __forceinline__ float2 unpack_pair(uint32_t u) {
  if constexpr (std::is_same<M, __half>::value) {
    __half2 h;
    memcpy(&h, &u, 4);
    return __half22float2(h);
  } else {
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
}

}  // namespace da
