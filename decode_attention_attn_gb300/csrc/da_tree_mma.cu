// da_tree_mma.cu -- tree attention on the 5th-generation tensor cores, for bf16, f16 and FP8
// caches.
//
// One CTA an SM walks its share of 128-token KV tiles for one tile of 128 query rows (rows =
// drafted tokens x heads of the group):
//   S = Q K^T     tcgen05.mma 128 x 128 x D, both operands in shared memory, into TMEM (two buffers)
//   P = 2^(S c - m)  8 warps: a thread holds one row's 64 columns of a tile, exchanges the row maximum
//                 with the thread of the other 64, and writes P back over S in TMEM
//   O += P V      tcgen05.mma 128 x D x 128 with P from TMEM and V from shared memory, O in TMEM
// While the softmax of tile i runs, the tensor core does S of tile i + 1 and O of tile i - 1.
// The maximum m is a reference that only moves when a tile exceeds it by more than 2^8, so O is
// rescaled (a TMEM round trip) once or twice a sequence, not per tile.
//
// P enters O += P V as hi + lo, two 16-bit parts (2^-17 of a weight is lost, as in the decode step):
// a bf16 P alone would cost as much accuracy as the bf16 output. The second product costs tensor
// time only where the step is not bound by memory. FP8 caches run on f16 operands (E4M3 codes are f16
// numbers) and take P as one f16 (2^-12) where the output is 16-bit: an eighth of a bf16 output's half
// step. q enters f16 scaled by a power of two per row, exact for every element above 2^-29 of the
// row's largest.
//
// What bounds it: up to 128 rows the KV stream (a 16-bit tile pair of 64 KB takes an SM 2800 cycles at
// the HBM rate, its MMAs 1536 and its softmax about as much); above, with R row tiles the SMs read
// every tile R times (once from HBM, then L2) and the tensor core is the bound.
#include <type_traits>

#include "da_tree_mma.cuh"

namespace da {
namespace {

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0;      // two S / P buffers of 128 columns
constexpr uint32_t kColO = 256;    // O: D columns
constexpr float kRescale = 8.f;    // log2: P <= 2^8 before the reference moves

// ---- tcgen05 -----------------------------------------------------------------------------
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
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
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

// Shared-memory operand descriptor, 128-byte swizzle: `lead` is the distance between 64-element
// blocks along the contiguous dimension (used where that is M or N), 1024 bytes that between
// 8-row groups.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | (uint64_t)(lead >> 4) << 16 |
         (uint64_t)(1024u >> 4) << 32 | 1ull << 46 | 2ull << 61;
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
    if (dead) return;
    bool ok = mbar_try_wait(bar, parity);
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

// The KV tiles of a CTA's share that have rows in its row tile, one after another.
struct Cursor {
  TreeWalk w;
  int kt = 0, piece = -1;
  __device__ __forceinline__ Cursor(const TreeParams& p, const TreeShare& sh) : w(p, sh) {
    w.t1 = 0;
  }
  __device__ __forceinline__ bool advance(const TreeParams& p, const TreeShare& sh) {
    if (piece >= 0 && kt + 1 < w.t1) {
      ++kt;
      return true;
    }
    while (w.next(p, sh)) {
      if (sh.row_tile * kTreeRows >= w.s.T * p.group) continue;
      kt = w.t0;
      ++piece;
      return true;
    }
    return false;
  }
  __device__ __forceinline__ bool first() const { return kt == w.t0; }
  __device__ __forceinline__ bool last() const { return kt + 1 == w.t1; }
};

template <typename T>
struct MmaOf {   // the operands' 16-bit type
  using type = T;
};
template <>
struct MmaOf<fp8e4m3> {
  using type = __half;
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

// Columns c < 64 of a half tile that a row attends to: its context (t < ctx) and its drafted tokens'
// bits; `off` = ctx minus the half tile's first token.
__device__ __forceinline__ unsigned long long visible(int off, unsigned long long word) {
  if (off >= 64) return ~0ull;
  if (off > 0) return ((1ull << off) - 1ull) | word << off;
  return off > -64 ? word >> -off : 0ull;
}

template <typename T, int D, bool kSplit>
__global__ void __launch_bounds__(tree_threads(std::is_same<T, fp8e4m3>::value), 1)
    tree_mma_kernel_t(const __grid_constant__ TreeParams p, const __grid_constant__ CUtensorMap tmq,
                      const __grid_constant__ CUtensorMap tmk,
                      const __grid_constant__ CUtensorMap tmv, const void* __restrict__ v_cache) {
  constexpr bool kFp8 = std::is_same<T, fp8e4m3>::value;
  using M = typename MmaOf<T>::type;
  constexpr TreeLayout L = tree_layout(D, kFp8);
  constexpr int kThreadsT = tree_threads(kFp8);
  constexpr uint32_t kTile = tree_tile_bytes(D);
  constexpr uint32_t kCode = 128u * D;
  constexpr int CH = D / 64;                 // 64-element blocks of a row
  constexpr int kBoxes = kFp8 ? 1 : CH;      // TMA boxes per run of tokens
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L.bar_off);
  uint64_t* k_full = bar;                 // the 16-bit tiles that the MMAs read
  uint64_t* k_empty = k_full + L.nk;
  uint64_t* v_full = k_empty + L.nk;
  uint64_t* v_empty = v_full + L.nv;
  uint64_t* q_full = v_empty + L.nv;
  uint64_t* q_empty = q_full + L.nq;
  uint64_t* s_full = q_empty + L.nq;      // S of a buffer done
  uint64_t* p_full = s_full + 2;          // P of a buffer written, O rescaled
  uint64_t* o_full = p_full + 2;          // O += P V done, tiles in turn
  uint64_t* rk_full = o_full + 2;         // FP8: tiles of codes
  uint64_t* rk_empty = rk_full + L.raw;
  uint64_t* rv_full = rk_empty + L.raw;
  uint64_t* rv_empty = rv_full + L.raw;
  uint64_t* drained = rv_empty + L.raw;
  static_assert(2 * L.nk + 2 * L.nv + 2 * L.nq + 7 + 4 * L.raw <= 48, "");
  float* exch = reinterpret_cast<float*>(smem + L.exch_off);
  signed char* qexp = reinterpret_cast<signed char*>(smem + L.qexp_off);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L.misc_off);
  int* abort_flag = reinterpret_cast<int*>(smem + L.misc_off + 4);
  unsigned long long* odd = reinterpret_cast<unsigned long long*>(smem + L.misc_off + 8);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const TreeShare sh = tree_schedule<kThreadsT>(p, *reinterpret_cast<TreeScratch*>(exch));
  if (sh.u1 <= sh.u0) return;   // the whole CTA
  if (tid == 0) {
    for (int i = 0; i < L.nk; ++i) {
      mbar_init(&k_full[i], kFp8 ? kTreeConvertWarps : 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < L.nv; ++i) {
      mbar_init(&v_full[i], kFp8 ? kTreeConvertWarps : 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < L.nq; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], kFp8 ? 1 + kTreeSoftmaxWarps : 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kTreeSoftmaxWarps);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(drained, 1);
    for (int i = 0; i < L.raw; ++i) {
      mbar_init(&rk_full[i], 1);
      mbar_init(&rk_empty[i], kTreeConvertWarps);
      mbar_init(&rv_full[i], 1);
      mbar_init(&rv_empty[i], kTreeConvertWarps);
    }
    // the swizzled tiles need a 1 KB boundary; elsewhere nothing may run
    *abort_flag = (smem_u32(smem) & 1023u) ? 1 : 0;
    if (*abort_flag) atomicOr(p.c.status, kStatusTimeout);
    *odd = 0;
    fence_mbar_init();
  }
  if (warp == kTreeSoftmaxWarps + 2) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Waiter wait{abort_flag, p.c.status, kWaitLimitNs, *abort_flag != 0};
  Cursor c(p, sh);

  if (warp < kTreeSoftmaxWarps) {
    // ---- softmax -----------------------------------------------------------------------
    const int half = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)quarter << 21);   // TMEM lane quarter * 32
    uint32_t it = 0;
    float m = -INFINITY, l = 0.f, factor = p.qscale;
    bool active = false;
    int r = 0;
    unsigned long long word = 0;
    while (c.advance(p, sh)) {
      const int R = c.w.s.T * p.group;
      if (c.first()) {
        r = sh.row_tile * kTreeRows + row;
        active = sh.row_tile * kTreeRows + quarter * 32 < R;   // this warp has rows
        const int i = r / p.group;
        word = r < R ? tree_word(p, c.w.s.row0 + i, i, c.w.s.T) : 0ull;
        m = -INFINITY;
        l = 0.f;
        if constexpr (kFp8) {
          const int qb = c.piece & 1;
          wait(&q_full[qb], (c.piece >> 1) & 1);
          factor = p.qscale * exp2f((float)qexp[qb * 128 + row]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_empty[qb]);
        }
      }
      const int buf = it & 1;
      const uint32_t s_addr = lane_addr + kColS + (uint32_t)buf * 128u;
      const int tok0 = c.kt * kTreeTokens;
      const bool tail = tok0 + kTreeTokens > c.w.s.ctx;   // drafted tokens or the end in this tile
      // O of tile it - 2 (complete: S of this tile was issued after it), so that every phase of the
      // two barriers is waited for in turn and a parity names one phase
      if (it >= 2) wait(&o_full[buf], ((it - 2) >> 1) & 1);
      wait(&s_full[buf], (it >> 1) & 1);
      tc_fence_after();
      if (active) {
        float x[64];
        tmem_ld32(s_addr + half * 64, reinterpret_cast<uint32_t*>(x));
        tmem_ld32(s_addr + half * 64 + 32, reinterpret_cast<uint32_t*>(x) + 32);
        tmem_wait_ld();
        const f32x2 f2 = f2_pack(factor, factor);
#pragma unroll
        for (int k = 0; k < 64; k += 2) f2_unpack(f2_mul(f2_pack(x[k], x[k + 1]), f2), x[k], x[k + 1]);
        if (tail) {
          const unsigned long long vis = visible(c.w.s.ctx - tok0 - half * 64, word);
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (!((k < 32 ? (uint32_t)vis : (uint32_t)(vis >> 32)) >> (k & 31) & 1u)) x[k] = -INFINITY;
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int k = 4; k < 64; ++k) mx[k & 3] = fmaxf(mx[k & 3], x[k]);
        float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        // the other half's maximum; P may be written over S once both have read it
        float* ex = exch + buf * 256;
        ex[half * 128 + row] = top;
        named_bar_sync(1 + quarter, 64);
        top = fmaxf(top, ex[(half ^ 1) * 128 + row]);
        bool move = false;
        float f = 1.f;
        if (c.first()) {
          m = top;
        } else if (top > m + kRescale) {
          f = fast_exp2(m - top);
          m = top;
          l *= f;
          move = true;
        }
        if (__any_sync(0xffffffffu, move)) {
          // O so far, relative to the new reference: this half's columns
          wait(&o_full[buf ^ 1], ((it - 1) >> 1) & 1);
          tc_fence_after();
#pragma unroll
          for (int cc = 0; cc < D / 64; ++cc) {
            uint32_t o[32];
            const uint32_t a = lane_addr + kColO + half * (D / 2) + cc * 32;
            tmem_ld32(a, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st32(a, o);
          }
          tmem_wait_st();
        }
        const float ref = m == -INFINITY ? 0.f : m;
        const f32x2 neg = f2_pack(-ref, -ref);
        uint32_t hi[32];
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          float a, b;
          f32x2 d = f2_pack(x[k], x[k + 1]);
          asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(neg));
          f2_unpack(d, a, b);
          a = fast_exp2(a);
          b = fast_exp2(b);
          sum[k & 2] += a;
          sum[(k & 2) + 1] += b;
          const uint32_t h = pack_pair<M>(a, b);
          hi[k / 2] = h;
          if constexpr (kSplit) {
            const float2 hf = unpack_pair<M>(h);
            x[k / 2] = __uint_as_float(pack_pair<M>(a - hf.x, b - hf.y));
          }
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_st32(s_addr + half * 32, hi);
        if constexpr (kSplit) tmem_st32(s_addr + 64 + half * 32, reinterpret_cast<uint32_t*>(x));
        tmem_wait_st();
      }
      if (tail) {
        // V rows that the MMA reads past the sequence's end are cleared, and values that are not
        // finite are taken out of drafted tokens' rows (0 * inf would reach rows that the token is
        // hidden from) and added to the rows that see them below.
        const uint32_t vs = it % L.nv;
        wait(&v_full[vs], (it / L.nv) & 1);
        const int valid = min(kTreeTokens, c.w.s.n - tok0);
        const int t = tid & 127, end = (valid + 15) / 16 * 16;
        uint4* vrow = reinterpret_cast<uint4*>(smem + L.v_off + vs * kTile + t * 128);
        for (int blk = tid >> 7; blk < CH; blk += 2) {
          uint4* v4 = vrow + blk * (128 * 128 / 16);
          if (t >= valid && t < end) {
#pragma unroll
            for (int k = 0; k < 8; ++k) v4[(k + t) & 7] = make_uint4(0u, 0u, 0u, 0u);
          } else if (t < valid && tok0 + t >= c.w.s.ctx) {
            constexpr uint32_t kInf = std::is_same<M, __half>::value ? 0x7c00u : 0x7f80u;
            bool found = false;
#pragma unroll 1
            for (int k = 0; k < 8; ++k) {
              uint4 v = v4[(k + t) & 7];
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
              bool here = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if ((w[e] & kInf) == kInf) {
                  w[e] &= 0xffff0000u;
                  here = true;
                }
                if ((w[e] >> 16 & kInf) == kInf) {
                  w[e] &= 0xffffu;
                  here = true;
                }
              }
              if (here) v4[(k + t) & 7] = make_uint4(w[0], w[1], w[2], w[3]);
              found |= here;
            }
            if (found) atomicOr(odd, 1ull << (tok0 + t - c.w.s.ctx));
          }
        }
        fence_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[buf]);

      if (c.last()) {
        // ---- a piece's end: normalise and store ----------------------------------------
        if (it >= 1) wait(&o_full[buf ^ 1], ((it - 1) >> 1) & 1);
        wait(&o_full[buf], (it >> 1) & 1);
        tc_fence_after();
        if (active) {
          float* ex = exch + (buf ^ 1) * 256;
          named_bar_sync(1 + quarter, 64);   // the other half has read its maximum of the tile before
          ex[half * 128 + row] = l;
          named_bar_sync(1 + quarter, 64);
          const float total = l + ex[(half ^ 1) * 128 + row];
          const float inv = total == 0.f ? 0.f : 1.f / total;
          const float lg = total == 0.f ? -INFINITY : m + log2f(total);
          const unsigned long long strange = *odd & word;
          const int i = r / p.group, h = c.w.kvh * p.group + r % p.group;
          const long long orow = (long long)(c.w.s.row0 + i) * p.c.hq + h;
          const long long prow =
              tree_slot(sh.owner, c.w.head, sh.row_tile, sh.row_tiles) * kTreeRows + row;
          if (half == 0 && r < R) {
            if (!c.w.whole) p.part_l[prow] = lg;
            else if (p.out_lse) p.out_lse[orow] = lg * 0.69314718055994531f;
          }
#pragma unroll
          for (int cc = 0; cc < D / 64; ++cc) {
            const int col = half * (D / 2) + cc * 32;
            float o[32];
            tmem_ld32(lane_addr + kColO + col, reinterpret_cast<uint32_t*>(o));
            tmem_wait_ld();
            if (r >= R) continue;
            for (unsigned long long rest = strange; rest; rest &= rest - 1) {   // rare
              const int t = c.w.s.ctx + __ffsll((long long)rest) - 1;
              const int entry = p.c.paged ? __ldg(p.c.block_table +
                                                  (long long)c.w.b * p.c.max_blocks + t / p.c.page_size)
                                          : 0;
              const long long at =
                  ((long long)token_row(p.c, c.w.b, t, entry) * p.c.hkv + c.w.kvh) * D + col;
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                float v;
                if constexpr (kFp8) {
                  const uint32_t hv = e4m3x2_to_f16x2(static_cast<const uint8_t*>(v_cache)[at + k]);
                  v = unpack_pair<__half>(hv).x;
                } else {
                  v = unpack_pair<M>(static_cast<const uint16_t*>(v_cache)[at + k]).x;
                }
                if (!isfinite(v)) o[k] += v;
              }
            }
            if (!c.w.whole) {
              float4* dst = reinterpret_cast<float4*>(p.part_o + prow * D + col);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                dst[k] = make_float4(o[4 * k] * inv, o[4 * k + 1] * inv, o[4 * k + 2] * inv,
                                     o[4 * k + 3] * inv);
            } else {
              const float g = inv * p.v_scale;
              if (p.c.out_dtype == kOutF32) {
                float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + orow * D + col);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  dst[k] = make_float4(o[4 * k] * g, o[4 * k + 1] * g, o[4 * k + 2] * g,
                                       o[4 * k + 3] * g);
              } else {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + orow * D + col);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  uint32_t w[4];
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const float a = o[8 * k + 2 * e] * g, b = o[8 * k + 2 * e + 1] * g;
                    w[e] = p.c.out_dtype == kOutF16 ? pack_pair<__half>(a, b)
                                                    : pack_pair<__nv_bfloat16>(a, b);
                  }
                  dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
            }
          }
        }
        // every warp has read `odd`; clear it for the next piece
        named_bar_sync(5, kTreeSoftmaxWarps * 32);
        if (tid == 0) *odd = 0;
        named_bar_sync(5, kTreeSoftmaxWarps * 32);
      }
      ++it;
    }
  } else if (warp == kTreeSoftmaxWarps || warp == kTreeSoftmaxWarps + 1) {
    // ---- K (V) producer ------------------------------------------------------------------
    const bool is_v = warp != kTreeSoftmaxWarps;
    const CUtensorMap* tm = is_v ? &tmv : &tmk;
    uint64_t* full = kFp8 ? (is_v ? rv_full : rk_full) : (is_v ? v_full : k_full);
    uint64_t* empty = kFp8 ? (is_v ? rv_empty : rk_empty) : (is_v ? v_empty : k_empty);
    const uint32_t slots = kFp8 ? L.raw : (is_v ? L.nv : L.nk);
    const uint32_t base = kFp8 ? (is_v ? L.rawv_off : L.rawk_off) : (is_v ? L.v_off : L.k_off);
    constexpr uint32_t kSlot = kFp8 ? kCode : kTile;
    constexpr uint32_t kRow = kFp8 ? (uint32_t)D : 128u;   // bytes of a token in a box
    const int box = p.c.box_tokens;
    if (lane == 0) prefetch_tensormap(tm);
    uint64_t pol;
    if (sh.row_tiles > 1)   // other CTAs read the same tiles: leave them in L2
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
    else
      pol = make_evict_first_policy();
    // the cache row that lane's box starts at: -2 past the end, -1 on a bad page
    auto lookup = [&](int kt) {
      const int t = kt * kTreeTokens + (lane / kBoxes) * box;
      if ((lane / kBoxes) * box >= kTreeTokens || t >= c.w.s.n) return -2;
      const int entry =
          p.c.paged ? __ldg(p.c.block_table + (long long)c.w.b * p.c.max_blocks + t / p.c.page_size)
                    : 0;
      return token_row(p.c, c.w.b, t, entry);
    };
    const int past = p.c.paged ? p.c.num_blocks * p.c.page_size : p.c.batch * p.c.max_seq_len;
    uint32_t it = 0, issued = 0;
    int z = -2;
    while (c.advance(p, sh)) {
      if (c.first()) z = lookup(c.kt);
      const int z_next = c.last() ? -2 : lookup(c.kt + 1);   // in flight during the wait
      const uint32_t slot = it % slots;
      wait(&empty[slot], ((it / slots) & 1) ^ 1);
      if (!wait.dead) {
        const int boxes = __popc(__ballot_sync(0xffffffffu, z != -2));
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], (uint32_t)(boxes * box) * kRow);
        __syncwarp();
        if (z != -2) {
          if (z < 0) atomicOr(p.c.status, kStatusBadBlockTable);
          const int row0 = z < 0 ? past : z;   // past the pool: zeros
          uint8_t* dst = smem + base + slot * kSlot + (uint32_t)((lane / kBoxes) * box) * kRow;
          if constexpr (kFp8) {
            tma_load_3d(dst, tm, &full[slot], 0, row0, c.w.kvh, pol);
          } else {
            const int blk = lane % kBoxes;
            tma_load_4d(dst + blk * (128 * 128), tm, &full[slot], 0, row0, blk, c.w.kvh, pol);
          }
        }
        issued = it + 1;
      }
      __syncwarp();
      z = z_next;
      ++it;
    }
    // never leave with copies in flight
    for (uint32_t k = issued > slots ? issued - slots : 0; k < issued; ++k)
      mbar_wait(&full[k % slots], (k / slots) & 1, kWaitLimitNs);
  } else if (warp == kTreeSoftmaxWarps + 2) {
    // ---- MMA issuer ------------------------------------------------------------------------
    constexpr bool kBf16 = std::is_same<M, __nv_bfloat16>::value;
    constexpr uint32_t kDescS = mma_desc(kBf16, kTreeTokens, false);
    constexpr uint32_t kDescO = mma_desc(kBf16, D, true);
    const uint32_t q_base = smem_u32(smem + L.q_off), k_base = smem_u32(smem + L.k_off);
    const uint32_t v_base = smem_u32(smem + L.v_off);
    Cursor d(p, sh);      // S runs a tile ahead of O
    uint32_t is = 0, io = 0;
    auto issue_s = [&]() {
      const uint32_t slot = is % L.nk, qb = d.piece & 1;
      if (d.first()) wait(&q_full[qb], (d.piece >> 1) & 1);
      wait(&k_full[slot], (is / L.nk) & 1);
      tc_fence_after();
      if (!wait.dead && lane == 0) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (uint32_t)(k / 4) * 16384u + (uint32_t)(k % 4) * 32u;
          mma_ss(tmem + kColS + (is & 1) * 128u, tile_desc(q_base + qb * kTile + off, 16),
                 tile_desc(k_base + slot * kTile + off, 16), kDescS, k != 0);
        }
        tc_commit(&k_empty[slot]);
        if (d.last()) tc_commit(&q_empty[qb]);
        tc_commit(&s_full[is & 1]);
      }
      __syncwarp();
      ++is;
    };
    bool more = d.advance(p, sh);
    if (more) issue_s();
    while (c.advance(p, sh)) {
      more = d.advance(p, sh);
      if (more) issue_s();
      const uint32_t slot = io % L.nv, buf = io & 1;
      wait(&v_full[slot], (io / L.nv) & 1);
      wait(&p_full[buf], (io >> 1) & 1);
      tc_fence_after();
      if (!wait.dead && lane == 0) {
        const int steps = (min(kTreeTokens, c.w.s.n - c.kt * kTreeTokens) + 15) / 16;
        const uint32_t pa = tmem + kColS + buf * 128u;
#pragma unroll 1
        for (int part = 0; part < (kSplit ? 2 : 1); ++part)
#pragma unroll 1
          for (int k = 0; k < steps; ++k)
            mma_ts(tmem + kColO, pa + part * 64u + k * 8u,
                   tile_desc(v_base + slot * kTile + k * 2048u, 16384), kDescO,
                   !c.first() || k != 0 || part != 0);
        tc_commit(&v_empty[slot]);
        tc_commit(&o_full[buf]);
      }
      __syncwarp();
      ++io;
    }
    // nothing leaves before the last MMA has completed (after a timeout too)
    if (lane == 0) tc_commit(drained);
    __syncwarp();
    mbar_wait(drained, 0, kWaitLimitNs);
  } else if (warp == kTreeSoftmaxWarps + 3) {
    // ---- q producer --------------------------------------------------------------------------
    int loaded = 0;
    // the merge reads the first piece of every owner, whether this row tile has rows in it or not
    {
      TreeWalk w(p, sh);
      if (w.next(p, sh) && sh.row_tile == 0 && lane == 0)
        p.info[sh.owner] = make_int4(w.b, w.kvh, w.t0, w.s.tiles);
    }
    while (c.advance(p, sh)) {
      if (!c.first()) {
        c.kt = c.w.t1 - 1;   // the rest of the piece
        continue;
      }
      const int qb = c.piece & 1;
      const int i0 = sh.row_tile * (kTreeRows / p.group);   // the tile's first drafted token
      wait(&q_empty[qb], ((c.piece >> 1) & 1) ^ 1);
      if (!wait.dead) {
        if constexpr (!kFp8) {
          if (lane == 0) {
            mbar_arrive_expect_tx(&q_full[qb], kTile);
            for (int blk = 0; blk < CH; ++blk)
              tma_load_4d(smem + L.q_off + qb * kTile + blk * (128 * 128), &tmq, &q_full[qb], 0,
                          c.w.kvh * p.group, c.w.s.row0 + i0, blk, make_evict_first_policy());
          }
          ++loaded;
        } else {
          // D / 8 lanes a row, 8 elements each: q as f16 times a power of two per row, so that its
          // largest element lies in [2^14, 2^15)
          constexpr int LR = D / 8, RW = 32 / LR;
          const int sub = lane / LR, e = lane % LR, R = c.w.s.T * p.group;
#pragma unroll 4
          for (int r8 = 0; r8 < kTreeRows; r8 += RW) {
            const int rr = r8 + sub, r = sh.row_tile * kTreeRows + rr;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (r < R)
              v = __ldg(reinterpret_cast<const uint4*>(
                            static_cast<const __nv_bfloat16*>(p.q) +
                            ((long long)(c.w.s.row0 + r / p.group) * p.c.hq + c.w.kvh * p.group +
                             r % p.group) * D) + e);
            float f[8];
            Elem<__nv_bfloat16>::to_f32(v, f);
            float big = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) big = fmaxf(big, fabsf(f[k]));
#pragma unroll
            for (int o = LR / 2; o > 0; o >>= 1)
              big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            // 2^(14 - exponent of the largest), within what an int8 holds; 1 for a row of zeros
            int s = big > 0.f && big < INFINITY ? 14 - ((int)(__float_as_uint(big) >> 23) - 127) : 0;
            s = min(max(s, -112), 126);
            const float mul = __uint_as_float((uint32_t)(s + 127) << 23);
            uint4 w;
            w.x = pack_pair<__half>(f[0] * mul, f[1] * mul);
            w.y = pack_pair<__half>(f[2] * mul, f[3] * mul);
            w.z = pack_pair<__half>(f[4] * mul, f[5] * mul);
            w.w = pack_pair<__half>(f[6] * mul, f[7] * mul);
            *reinterpret_cast<uint4*>(smem + L.q_off + qb * kTile + (e / 8) * (128 * 128) + rr * 128 +
                                      (((e & 7) ^ (rr & 7)) << 4)) = w;
            if (e == 0) qexp[qb * 128 + rr] = (signed char)-s;
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&q_full[qb]);
        }
      }
      __syncwarp();
    }
    if constexpr (!kFp8)
      for (int k = loaded > L.nq ? loaded - L.nq : 0; k < loaded; ++k)
        mbar_wait(&q_full[k & 1], (k >> 1) & 1, kWaitLimitNs);
  } else if constexpr (kFp8) {
    // ---- FP8: codes to f16 tiles ------------------------------------------------------------
    const int cw = warp - (kTreeSoftmaxWarps + 4);
    auto convert = [&](uint32_t n, uint64_t* rfull, uint64_t* rempty, uint32_t raw_off,
                       uint64_t* full, uint64_t* empty, uint32_t off, uint32_t slots) {
      const uint32_t rs = n % L.raw, ds = n % slots;
      wait(&rfull[rs], (n / L.raw) & 1);
      wait(&empty[ds], ((n / slots) & 1) ^ 1);
      if (!wait.dead) {
        constexpr int LR = D / 16, RW = 32 / LR;   // lanes a row (16 codes each), rows a pass
        const int seg = lane % LR, sub = lane / LR;
        const uint8_t* src = smem + raw_off + rs * kCode + cw * 32 * D + lane * 16;
        uint8_t* dst = smem + off + ds * kTile + (seg / 4) * (128 * 128);
        const int k0 = (seg & 3) * 2, flip = seg >> 2;   // the upper block's lanes store in the other
                                                         // order: 8 lanes then hit 8 different chunks
#pragma unroll
        for (int g = 0; g < 32; g += RW) {
          const int t = cw * 32 + g + sub;
          const uint4 v = *reinterpret_cast<const uint4*>(src + g * D);
          uint4 a, b;
          e4m3x4_to_f16x2(v.x, a.x, a.y);
          e4m3x4_to_f16x2(v.y, a.z, a.w);
          e4m3x4_to_f16x2(v.z, b.x, b.y);
          e4m3x4_to_f16x2(v.w, b.z, b.w);
          uint8_t* d = dst + t * 128;
          *reinterpret_cast<uint4*>(d + (((k0 + flip) ^ (t & 7)) << 4)) = flip ? b : a;
          *reinterpret_cast<uint4*>(d + (((k0 + 1 - flip) ^ (t & 7)) << 4)) = flip ? a : b;
        }
        fence_async_smem();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&rempty[rs]);
        mbar_arrive(&full[ds]);
      }
    };
    // in the order the MMAs take them: K 0, K 1, V 0, K 2, V 1, ...
    uint32_t nk = 0, nv = 0;
    while (c.advance(p, sh)) {
      convert(nk, rk_full, rk_empty, L.rawk_off, k_full, k_empty, L.k_off, L.nk);
      ++nk;
      if (nk >= 2) {
        convert(nv, rv_full, rv_empty, L.rawv_off, v_full, v_empty, L.v_off, L.nv);
        ++nv;
      }
    }
    for (; nv < nk; ++nv)
      convert(nv, rv_full, rv_empty, L.rawv_off, v_full, v_empty, L.v_off, L.nv);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kTreeSoftmaxWarps + 2) tmem_free(tmem, kTmemCols);
  pdl_launch_dependents();
}

template <typename T, bool kSplit>
const void* for_d(int D) {
  return D == 64    ? reinterpret_cast<const void*>(&tree_mma_kernel_t<T, 64, kSplit>)
         : D == 128 ? reinterpret_cast<const void*>(&tree_mma_kernel_t<T, 128, kSplit>)
                    : nullptr;
}

}  // namespace

const void* tree_mma_kernel(int dtype, bool fp8, int head_dim, bool split) {
  if (fp8) return split ? for_d<fp8e4m3, true>(head_dim) : for_d<fp8e4m3, false>(head_dim);
  if (!split) return nullptr;
  if (dtype == kOutF16) return for_d<__half, true>(head_dim);
  if (dtype == kOutBF16) return for_d<__nv_bfloat16, true>(head_dim);
  return nullptr;
}

}  // namespace da
