// da_tree_mma.cu -- tree attention on the 5th-generation tensor cores, for bf16, f16 and FP8
// caches.
//
// One CTA an SM walks its share of 128-token KV tiles for one tile of 128 query rows (rows =
// drafted tokens x heads of the group):
//   S = Q K^T     tcgen05.mma 128 x 128 x D into TMEM; K in shared memory, q there too (16-bit) or in TMEM
//   P = 2^(S c - m)  two teams of 4 warps, a thread a row, take the tiles in turn and write P over S
//   O += P V      tcgen05.mma 128 x D x 128 with P from TMEM and V from shared memory, O in TMEM
// S has three buffers in TMEM (16-bit caches) or two (FP8, whose q takes the columns of the third), so that
// the tensor core does S of later tiles and O of earlier ones while two tiles are in the softmax.
// The maximum m is a reference that only moves when a tile exceeds it by a few powers of two (Reference), so O
// is rescaled (a TMEM round trip) once or twice a sequence, not per tile. A thread holds a whole row, so a tile
// needs no exchange within a row, only the hand-over of m from team to team.
//
// P enters O += P V as hi + lo, two 16-bit parts. bf16 loses 2^-17 of a weight, as in the decode step; f16
// 2^-23 of it or 2^-36 of the row's largest, whichever is more:
// a bf16 P alone would cost as much accuracy as the bf16 output. The second product costs tensor
// time only where the step is not bound by memory. FP8 caches run on f16 operands (E4M3 codes are f16
// numbers); one f16 a weight took 339 instead of 386 us (64 drafted, 64 x 4350 tokens; 8 drafted 181
// instead of 195), but answered a drafted token less exactly than the decode step over the same cache, and cost
// an f16 result as much as its own rounding. q enters f16 scaled by a power of two per row, exact for every element above 2^-29 of the
// row's largest.
//
// What bounds it. 16-bit, up to 128 rows: the KV stream (64 KB of K and V a tile take an SM 2800 cycles at
// the HBM rate, the MMAs 1536): 64 paged sequences of 512 to 8192 tokens with 3 to 12 drafted, 197 us, 5.8
// TB/s, 87 % of a copy. With R row tiles every tile is read R times (once from HBM, then L2) and no part is the
// full one: 64 drafted tokens over 64 x 4350 cost 348 us, 846 TFLOP/s; without the second product of P's parts 6 %
// less, without forming them 6 %, without both 11 %. FP8: the chain S, softmax, O over two buffers (6300 cycles
// for two tiles), the conversion (192 KB a tile through shared memory) and the fetching of instructions for the
// many roles (a vote for a branch in every wait: 205 to 195 us) are even, whatever the rows: 8 drafted tokens 195
// us (2.9 TB/s), 64 drafted tokens 386 us (762 TFLOP/s). A single long sequence (32768 tokens, 16 drafted) takes 35
// us: 20 of stream, about 6 until the first tile is there (the schedule 2), the rest O's way out and the merge.
#include <type_traits>

#include "da_tcgen05.cuh"
#include "da_tree_mma.cuh"

namespace da {
namespace {

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 0;      // O: D columns
constexpr uint32_t kColS = 128;    // S / P buffers of 128 columns: 3, or 2 and
constexpr uint32_t kColQ = 384;    // FP8: two q tiles of D / 2 columns
__host__ __device__ constexpr uint32_t s_buffers(bool fp8) { return fp8 ? 2 : 3; }
// The reference that a row's weights are formed against, 2^(x - m): m lies kHead below the largest logit when
// it is set, and moves when a tile exceeds that by more than kMove (both log2). bf16's exponents reach as far as
// fp32's; f16 ends at 2^16 above and, hi and lo alike, at half a step of 2^-25 below, so its weights start at
// 2^11 and may grow to 2^15: what a weight loses is then at most 2^-36 of the row's largest. (8 and no headroom,
// as for bf16, would lose 2^-25: a 2^-12 of all weights 9 below one sink's logit, and all of those 18 below.)
template <typename M>
struct Reference {
  static constexpr float kHead = std::is_same<M, __half>::value ? 11.f : 0.f;
  static constexpr float kMove = std::is_same<M, __half>::value ? 4.f : 8.f;
};

// ---- TMA and tcgen05 -----------------------------------------------------------------------------
// 5-D tiled TMA load (a cache's [heads, tokens / 8, d / 64, 8, 64] view).
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar, int x,
                                            int y, int z, int w, int v, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v),
      "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ f32x2 f2_add(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Tiles that other CTAs read too (more row tiles) are left in L2.
__device__ __forceinline__ uint64_t kv_policy(int row_tiles) {
  if (row_tiles == 1) return make_evict_first_policy();
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void named_bar_arrive(int id, int nthreads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}

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

// The S / P buffer of a tile, and the parity of its barriers' phase.
template <uint32_t N>
struct TileSlot {
  uint32_t buf = 0, par = 0;
  __device__ __forceinline__ void next() {
    if (++buf == N) buf = 0, par ^= 1;
  }
  // those of the tile before
  __device__ __forceinline__ uint32_t before() const { return buf ? buf - 1 : N - 1; }
  __device__ __forceinline__ uint32_t before_par() const { return buf ? par : par ^ 1; }
};

template <typename T>
struct MmaOf {   // the operands' 16-bit type
  using type = T;
};
template <>
struct MmaOf<fp8e4m3> {
  using type = __half;
};

// Columns c < 32 of a quarter tile that a row attends to: its context (t < ctx) and its drafted tokens'
// bits; `off` = ctx minus the quarter's first token.
__device__ __forceinline__ uint32_t visible(int off, unsigned long long word) {
  if (off >= 32) return ~0u;
  if (off > 0) return ((1u << off) - 1u) | (uint32_t)word << off;
  return off > -64 ? (uint32_t)(word >> -off) : 0u;
}

// Adds what drafted tokens' V rows hold that is not finite (`odd`, tokens a row attends to) to 32
// columns of the row's stored result: the infinities and NaN that were taken out before the product.
// Rare.
template <typename T, int D>
__device__ __noinline__ void add_odd(const TreeParams& p, int b, int ctx, int kvh,
                                     unsigned long long odd, const void* v_cache, int col0, void* dst,
                                     long long row, int out_type) {
  constexpr bool kFp8 = std::is_same<T, fp8e4m3>::value;
#pragma unroll 1
  for (int col = col0; col < col0 + 32; ++col) {
    float sum = 0.f;
#pragma unroll 1
    for (unsigned long long rest = odd; rest; rest &= rest - 1) {
      const int t = ctx + __ffsll((long long)rest) - 1;
      const int entry = p.c.paged ? __ldg(p.c.block_table + (long long)b * p.c.max_blocks +
                                          t / p.c.page_size)
                                  : 0;
      const int z = token_row(p.c, b, t, entry);
      if (z < 0) continue;   // (a bad page holds zeros, unless the loads were given up)
      const long long at = ((long long)z * p.c.hkv + kvh) * D + col;
      float v;
      if constexpr (kFp8)
        v = unpack_pair<__half>(e4m3x2_to_f16x2(static_cast<const uint8_t*>(v_cache)[at])).x;
      else
        v = unpack_pair<typename MmaOf<T>::type>(static_cast<const uint16_t*>(v_cache)[at]).x;
      if (!isfinite(v)) sum += v;
    }
    if (isfinite(sum)) continue;
    const long long i = row * D + col;
    float o;
    if (out_type == kOutF32) o = static_cast<const float*>(dst)[i];
    else if (out_type == kOutF16) o = __half2float(static_cast<const __half*>(dst)[i]);
    else o = __bfloat162float(static_cast<const __nv_bfloat16*>(dst)[i]);
    store_out(dst, i, out_type, o + sum);
  }
}

template <typename T, int D>
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
  constexpr uint32_t NS = s_buffers(kFp8);
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L.bar_off);
  uint64_t* k_full = bar;                 // the 16-bit tiles that the MMAs read
  uint64_t* k_empty = k_full + L.nk;
  uint64_t* v_full = k_empty + L.nk;
  uint64_t* v_empty = v_full + L.nv;
  uint64_t* q_full = v_empty + L.nv;
  uint64_t* q_empty = q_full + L.nq;
  uint64_t* s_full = q_empty + L.nq;      // S of a buffer done
  uint64_t* p_full = s_full + NS;         // P of a buffer written, O rescaled
  uint64_t* o_full = p_full + NS;         // O += P V of a buffer done
  uint64_t* drained = o_full + NS;
  uint64_t* rk_full = drained + 2;        // FP8: tiles of codes
  uint64_t* rk_empty = rk_full + L.raw;
  uint64_t* rv_full = rk_empty + L.raw;
  uint64_t* rv_empty = rv_full + L.raw;
  static_assert(2 * L.nk + 2 * L.nv + 2 * L.nq + 3 * NS + 2 + 4 * L.raw <= 40, "");
  float* exch = reinterpret_cast<float*>(smem + L.exch_off);
  signed char* qexp = reinterpret_cast<signed char*>(smem + L.qexp_off);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L.misc_off);
  int* abort_flag = reinterpret_cast<int*>(smem + L.misc_off + 4);
  unsigned long long* odd = reinterpret_cast<unsigned long long*>(smem + L.misc_off + 8);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  // Before the kernel ahead in the stream has finished (this may be its programmatic dependent): barriers
  // and the tensor maps, whose first use would wait for their fetch. No TMEM: a kernel ahead that takes its
  // own after letting its dependents go, on the same SM, would wait for this CTA's, and this CTA for its end.
  if (tid == 0) {
    if (!kFp8) prefetch_tensormap(&tmq);
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    for (int i = 0; i < L.nk; ++i) {
      mbar_init(&k_full[i], kFp8 ? kTreeConvertWarps : 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < L.nv; ++i) {
      mbar_init(&v_full[i], kFp8 ? kTreeConvertWarps : 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < L.nq; ++i) {
      mbar_init(&q_full[i], kFp8 ? kTreeConvertWarps : 1);
      mbar_init(&q_empty[i], kFp8 ? 1 + kTreeSoftmaxWarps : 1);
    }
    for (int i = 0; i < (int)NS; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kTreeSoftmaxWarps / 2);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(&drained[0], 1);
    mbar_init(&drained[1], 1);
    for (int i = 0; i < L.raw; ++i) {
      mbar_init(&rk_full[i], 1);
      mbar_init(&rk_empty[i], kTreeConvertWarps);
      mbar_init(&rv_full[i], 1);
      mbar_init(&rv_empty[i], kTreeConvertWarps);
    }
    *abort_flag = 0;
    *odd = 0;
    fence_mbar_init();
  }
  pdl_wait();
  if (warp == kTreeSoftmaxWarps + 2) tmem_alloc(tmem_slot, kTmemCols);   // (beside the schedule's loads)
  tc_fence_before();
  // the share lies in shared memory: it is looked at once a piece, and registers are short
  TreeShare& sh = *reinterpret_cast<TreeShare*>(smem + L.misc_off + 16);
  bool any;
  {
    const TreeShare mine = tree_schedule<kThreadsT>(p, *reinterpret_cast<TreeScratch*>(exch));
    any = mine.u1 > mine.u0;
    if (tid == 0) sh = mine;
    if (tid == 0 && !any) tree_record(p, mine, false, TreeWalk(p, mine));
  }
  // the swizzled tiles need a 1 KB boundary; elsewhere nothing may run
  if (tid == 0 && any && (smem_u32(smem) & 1023u)) {
    *abort_flag = 1;
    atomicOr(p.c.status, kStatusTimeout);
  }
  __syncthreads();
  tc_fence_after();
  // The merge's launch runs beside this kernel; it waits for its end. Only now that the CTA has its TMEM: with
  // no merge (one CTA) the dependent is the caller's next kernel, which may take TMEM of its own.
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  if (!any) {   // the whole CTA
    if (warp == kTreeSoftmaxWarps + 2) tmem_free(tmem, kTmemCols);
    return;
  }
  // K and V tiles: distance between 64-element blocks and between 8-row groups
  const bool paired = !kFp8 && p.c.paged;
  const uint32_t blk_bytes = paired ? 1024u : 16384u, grp_bytes = paired ? CH * 1024u : 1024u;
  Waiter wait{abort_flag, p.c.status, p.c.wait_limit_ns, *abort_flag != 0};
  if constexpr (!kFp8) {
    if (warp < kTreeSoftmaxWarps)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTreeSoftmaxRegs));
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTreeOtherRegs));
  }
  if (warp < kTreeSoftmaxWarps) {
    // ---- softmax -----------------------------------------------------------------------
    // Team `team` (4 warps, a thread a row) takes the tiles it = team, team + 2, ...; while it
    // exponentiates one the other team reads the next. Both weigh against one reference per row, m in
    // shared memory, which belongs to O: before a tile's weights are formed its team learns that the tile
    // before has settled m (a barrier between the two warps of 32 rows, `settled`), moves it where the
    // tile exceeds it by too much, and passes on. Row sums are kept per team, relative to the
    // reference its thread saw last.
    Cursor c(p, sh);
    const int team = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)quarter << 21);   // TMEM lane quarter * 32
    const int settled = 1 + quarter * 2;                           // + the settling team
    uint32_t it = 0;
    TileSlot<NS> sl;
    float m = -INFINITY, l = 0.f, factor = p.qscale;
    bool active = false, due = false, masked = false;
    int r = 0;
    unsigned long long word = 0;
    while (c.advance(p, sh)) {
      float* const m_row = exch + (c.piece & 1) * 128 + row;
      if (c.first()) {
        const int R = c.w.s.T * p.group;
        r = sh.row_tile * kTreeRows + row;
        active = sh.row_tile * kTreeRows + quarter * 32 < R;   // this warp has rows
        const int i = r / p.group;
        // (the mask's word is on its way until a drafted token's tile needs it)
        word = r < R && p.mask ? __ldg(p.mask + c.w.s.row0 + i) : 0ull;
        if (r >= R) r = -1;
        masked = false;
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
      if ((it & 1) == team) {
        const uint32_t s_addr = lane_addr + kColS + sl.buf * 128u;
        const int tok0 = c.kt * kTreeTokens;
        const bool tail = tok0 + kTreeTokens > c.w.s.ctx;   // drafted tokens or the end in this tile
        if (tail && !masked) {
          word = r < 0 ? 0ull : tree_clip(p, word, r / p.group, c.w.s.T);
          masked = true;
        }
        wait(&s_full[sl.buf], sl.par);
        tc_fence_after();
        if (active) {
          auto tile = [&](auto tail_c) {
            constexpr bool kTail = decltype(tail_c)::value;
            // largest logit of the row's 128 columns (-inf: none seen)
            const float none = p.qscale >= 0.f ? -INFINITY : INFINITY;
            float top = none;
#pragma unroll 1
            for (int q2 = 0; q2 < 2; ++q2) {
              float x[64];
              tmem_ld32(s_addr + q2 * 64, reinterpret_cast<uint32_t*>(x));
              tmem_ld32(s_addr + q2 * 64 + 32, reinterpret_cast<uint32_t*>(x) + 32);
              tmem_ready(x);
              if constexpr (kTail) {
                const uint32_t v0 = visible(c.w.s.ctx - tok0 - q2 * 64, word);
                const uint32_t v1 = visible(c.w.s.ctx - tok0 - q2 * 64 - 32, word);
#pragma unroll
                for (int k = 0; k < 64; ++k)
                  if (!((k < 32 ? v0 : v1) >> (k & 31) & 1u)) x[k] = none;
              }
              float mx[4] = {top, x[0], x[1], x[2]};
              if (p.qscale >= 0.f) {
#pragma unroll
                for (int k = 3; k < 63; k += 2)
                  mx[k >> 1 & 3] = max3(mx[k >> 1 & 3], x[k], x[k + 1]);
                top = max3(max3(mx[0], mx[1], mx[2]), mx[3], x[63]);
              } else {
#pragma unroll
                for (int k = 3; k < 63; k += 2)
                  mx[k >> 1 & 3] = min3(mx[k >> 1 & 3], x[k], x[k + 1]);
                top = min3(min3(mx[0], mx[1], mx[2]), mx[3], x[63]);
              }
            }
            top = top == none ? -INFINITY : top * factor;
            if (due) named_bar_sync(settled + (team ^ 1), 64);   // the tile before has settled m
            constexpr float kHead = Reference<M>::kHead, kMove = Reference<M>::kMove;
            float now = top - kHead;
            if (!c.first()) {
              now = *m_row;
              if (now != m) {   // the other team moved it, or this is the team's first tile of the piece
                l *= fast_exp2(m - now);   // (0 where m was -inf: a sum of 0 stays 0, and NaN stays NaN)
                m = now;
              }
              float f = 1.f;
              if (top > now + (kHead + kMove)) {
                f = fast_exp2(now - (top - kHead));
                now = top - kHead;
                l *= f;
                *m_row = now;
              }
              if (__any_sync(0xffffffffu, f != 1.f)) {
                // O so far, relative to the new reference
                // (S of this tile waited for O of the tile NS before it, so the parity names one phase)
                wait(&o_full[sl.before()], sl.before_par());
                tc_fence_after();
#pragma unroll 1
                for (int cc = 0; cc < D; cc += 32) {
                  uint32_t o[32];
                  tmem_ld32(lane_addr + kColO + cc, o);
                  tmem_ready(o);
#pragma unroll
                  for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                  tmem_st32(lane_addr + kColO + cc, o);
                }
                tmem_wait_st();
              }
            } else {
              *m_row = now;
            }
            m = now;
            named_bar_arrive(settled + team, 64);
            // P over the columns of S that it comes from (S is read once more): for every 32 tokens 16
            // columns of hi, 16 of lo
            const float ref = m == -INFINITY ? 0.f : m;
            const f32x2 f2 = f2_pack(factor, factor), neg = f2_pack(-ref, -ref);
            f32x2 sum[2] = {0ull, 0ull};
            auto weigh = [&](float* x, int h) {
              uint32_t pk[32];
              uint32_t vis = ~0u;
              if constexpr (kTail) vis = visible(c.w.s.ctx - tok0 - h * 32, word);
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                f32x2 d = neg;
                f2_fma(d, f2_pack(x[k], x[k + 1]), f2);
                float a, b;
                f2_unpack(d, a, b);
                if constexpr (kTail) {
                  if (!(vis >> k & 1u)) a = -INFINITY;
                  if (!(vis >> (k + 1) & 1u)) b = -INFINITY;
                }
                a = fast_exp2(a);
                b = fast_exp2(b);
                const f32x2 e = f2_pack(a, b);
                sum[k >> 1 & 1] = f2_add(sum[k >> 1 & 1], e);
                const uint32_t hi = pack_pair<M>(a, b);
                pk[k / 2] = hi;
                const float2 hf = unpack_pair<M>(hi);
                float da, db;
                f2_unpack(f2_add(e, f2_pack(-hf.x, -hf.y)), da, db);
                pk[16 + k / 2] = pack_pair<M>(da, db);
              }
              tmem_st32(s_addr + h * 32, pk);
            };
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {   // (columns loaded ahead, in two copies of this, were no faster)
              float x[32];
              tmem_ld32(s_addr + h * 32, reinterpret_cast<uint32_t*>(x));
              tmem_ready(x);
              weigh(x, h);
            }
            float a, b;
            f2_unpack(f2_add(sum[0], sum[1]), a, b);
            l += a + b;
            tmem_wait_st();
          };
          if (tail) tile(std::true_type{});
          else tile(std::false_type{});
        } else {
          if (due) named_bar_sync(settled + (team ^ 1), 64);
          named_bar_arrive(settled + team, 64);
        }
        due = false;
        if (tail) {
          // V rows that the MMA reads past the sequence's end are cleared, and values that are not
          // finite are taken out of drafted tokens' rows (0 * inf would reach rows that the token is
          // hidden from) and added to the rows that see them below.
          const uint32_t vs = it % L.nv;
          wait(&v_full[vs], (it / L.nv) & 1);
          const int valid = min(kTreeTokens, c.w.s.n - tok0);
          const int end = (valid + 15) / 16 * 16, from = max(c.w.s.ctx - tok0, 0);
          constexpr uint32_t kInf = std::is_same<M, __half>::value ? 0x7c00u : 0x7f80u;
          // 16-byte chunks of rows from .. end - 1, a chunk a thread
#pragma unroll 1
          for (int i = tid & 127; i < (end - from) * (8 * CH); i += 128) {
            const int t = from + i / (8 * CH), k = i % (8 * CH);
            uint4* at = reinterpret_cast<uint4*>(smem + L.v_off + vs * kTile + (t >> 3) * grp_bytes +
                                                 (t & 7) * 128 + (k >> 3) * blk_bytes + (k & 7) * 16);
            if (t >= valid) {
              *at = make_uint4(0u, 0u, 0u, 0u);
              continue;
            }
            const uint4 v = *at;
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            bool here = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool lo = (w[e] & kInf) == kInf, hi = (w[e] >> 16 & kInf) == kInf;
              here |= lo | hi;
              w[e] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u);
            }
            if (here) {
              *at = make_uint4(w[0], w[1], w[2], w[3]);
              atomicOr(odd, 1ull << (tok0 + t - c.w.s.ctx));
            }
          }
          fence_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sl.buf]);
      } else {
        due = true;   // the other team settles m with this tile: learnt at the next one, or below
      }

      if (c.last()) {
        // ---- a piece's end: normalise and store, half of the columns a team ----------------
        wait(&s_full[sl.buf], sl.par);   // (O of this buffer's tile before is done: the next phase is its)
        wait(&o_full[sl.buf], sl.par);
        tc_fence_after();
        if (due) named_bar_sync(settled + (team ^ 1), 64);
        due = false;
        if (active) {
          // the final reference, settled by the last tile
          const float last = *m_row;
          if (last != m) {
            l *= fast_exp2(m - last);
            m = last;
          }
          float* const l_row = exch + 256 + row;
          l_row[team * 128] = l;
          __syncwarp();
          named_bar_sync(9 + quarter, 64);
          const float total = l_row[0] + l_row[128];
          const float inv = total == 0.f ? 0.f : 1.f / total;
          unsigned long long strange = *odd;
          if (strange && r >= 0)
            strange &= masked ? word : tree_clip(p, word, r / p.group, c.w.s.T);
          const bool whole = c.w.whole;
          // the row of out (and lse), or of the partials
          const long long at =
              whole ? (long long)(c.w.s.row0 + r / p.group) * p.c.hq + c.w.kvh * p.group + r % p.group
                    : (long long)tree_slot(sh.owner, c.w.head, sh.row_tiles * sh.heads,
                                           sh.head * sh.row_tiles + sh.row_tile) * kTreeRows + row;
          if (team == 0 && r >= 0) {
            const float lg = total == 0.f ? -INFINITY : m + log2f(total);
            if (!whole) p.part_l[at] = lg;
            else if (p.out_lse) p.out_lse[at] = lg * 0.69314718055994531f;
          }
          const float g = whole ? inv * p.v_scale : inv;
#pragma unroll 1
          for (int col = team * (D / 2); col < (team + 1) * (D / 2); col += 32) {
            float o[32];
            __syncwarp();   // rows that end in this warp's 32 leave some lanes without a store
            tmem_ld32(lane_addr + kColO + col, reinterpret_cast<uint32_t*>(o));
            tmem_ready(o);
            if (r < 0) {
              // nothing to store
            } else if (!whole || p.c.out_dtype == kOutF32) {
              float4* dst = reinterpret_cast<float4*>(
                  (whole ? static_cast<float*>(p.out) : p.part_o) + at * D + col);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                dst[k] = make_float4(o[4 * k] * g, o[4 * k + 1] * g, o[4 * k + 2] * g, o[4 * k + 3] * g);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * D + col);
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
            if (strange && r >= 0)
              add_odd<T, D>(p, c.w.b, c.w.s.ctx, c.w.kvh, strange, v_cache, col,
                            whole ? p.out : p.part_o, at, whole ? p.c.out_dtype : (int)kOutF32);
          }
          __syncwarp();
          tc_fence_before();
        }
        // O and `odd` have been read by everyone: the next piece may write them
        named_bar_sync(13, kTreeSoftmaxWarps * 32);
        if (tid == 0) *odd = 0;
        __syncwarp();
        named_bar_sync(13, kTreeSoftmaxWarps * 32);
      }
      ++it;
      sl.next();
    }
  } else if (warp < kTreeSoftmaxWarps + 2) {
    // ---- loaders: K (with q, for 16-bit caches) and V ------------------------------------------
    Cursor c(p, sh);
    const bool is_v = warp != kTreeSoftmaxWarps;
    const CUtensorMap* tm = is_v ? &tmv : &tmk;
    uint64_t* full = kFp8 ? (is_v ? rv_full : rk_full) : (is_v ? v_full : k_full);
    uint64_t* empty = kFp8 ? (is_v ? rv_empty : rk_empty) : (is_v ? v_empty : k_empty);
    const uint32_t slots = kFp8 ? L.raw : is_v ? L.nv : L.nk;
    uint8_t* const ring = smem + (kFp8 ? (is_v ? L.rawv_off : L.rawk_off) : (is_v ? L.v_off : L.k_off));
    constexpr uint32_t kSlot = kFp8 ? kCode : kTile;
    const uint64_t pol = kv_policy(sh.row_tiles);
    // Paged (and FP8) caches: lane i loads the i-th run of `box` tokens, whole rows. Contiguous 16-bit
    // caches: lane i loads block i of all tokens.
    const bool rows = kFp8 || p.c.paged;
    const int box = p.c.box_tokens;
    // lane's cache row of the cursor's tile; -2: nothing to load, -1: a bad page
    auto lookup = [&]() {
      const int t = c.kt * kTreeTokens + (rows ? lane * box : 0);
      if (rows ? lane * box >= kTreeTokens || t >= c.w.s.n : lane >= CH) return -2;
      const int entry =
          p.c.paged ? __ldg(p.c.block_table + (long long)c.w.b * p.c.max_blocks + t / p.c.page_size)
                    : 0;
      return token_row(p.c, c.w.b, t, entry);
    };
    const uint32_t lane_off = kFp8   ? (uint32_t)(lane * box) * D
                              : rows ? (uint32_t)(lane * box / 8) * grp_bytes
                                     : lane * blk_bytes;
    const uint32_t lane_bytes = (uint32_t)box * (kFp8 ? D : rows ? CH * 128 : 128);
    uint32_t slot = 0, par = 1, it = 0, issued = 0;
    int loaded = 0;
    // the cursor is a tile ahead of the loads, so that its page lookups are on their way meanwhile
    bool more = c.advance(p, sh);
    int z = more ? lookup() : -2;
    while (more) {
      const int kvh = c.w.kvh, row0 = c.w.s.row0, piece = c.piece, z_now = z;
      const bool first = c.first();
      more = c.advance(p, sh);
      z = more ? lookup() : -2;
      if (!kFp8 && !is_v && first) {
        const int qb = piece & 1;
        const int i0 = sh.row_tile * (kTreeRows / p.group);   // the tile's first drafted token
        wait(&q_empty[qb], ((piece >> 1) & 1) ^ 1);
        if (!wait.dead) {
          if (lane == 0) mbar_arrive_expect_tx(&q_full[qb], kTile);
          __syncwarp();
          if (lane < CH)
            tma_load_4d(smem + L.q_off + qb * kTile + lane * (128 * 128), &tmq, &q_full[qb], 0,
                        kvh * p.group, row0 + i0, lane, pol);
          ++loaded;
        }
      }
      wait(&empty[slot], par);
      // A converter that has given up frees tiles that it did not wait for: no copy may be armed on a barrier
      // whose last one is still under way. (What it arrived after, the flag, is seen once the wait has ended.)
      if (kFp8) wait.dead |= __any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(abort_flag));
      const bool left_out = p.stall == 1 + (int)is_v && blockIdx.x == 0 && it == 1;
      if (!wait.dead && !left_out) {
        const int boxes = __popc(__ballot_sync(0xffffffffu, z_now != -2));
        if (lane == 0) mbar_arrive_expect_tx(&full[slot], boxes * lane_bytes);
        __syncwarp();
        if (z_now != -2) {
          uint8_t* dst = ring + slot * kSlot + lane_off;
          // a bad page: past the pool, zeros
          if (z_now < 0) atomicOr(p.c.status, kStatusBadBlockTable);
          const int at = z_now < 0 ? p.c.num_blocks * p.c.page_size : z_now;
          if constexpr (kFp8) tma_load_3d(dst, tm, &full[slot], 0, at, kvh, pol);
          else if (rows) tma_load_5d(dst, tm, &full[slot], 0, 0, 0, at / 8, kvh, pol);
          else tma_load_4d(dst, tm, &full[slot], 0, at, lane, kvh, pol);
        }
        issued = it + 1;
      }
      __syncwarp();
      if (++slot == slots) slot = 0, par ^= 1;
      ++it;
    }
    // never leave with copies in flight
    for (uint32_t k = issued > slots ? issued - slots : 0; k < issued; ++k)
      mbar_wait(&full[k % slots], (k / slots) & 1, p.c.wait_limit_ns);
    for (int k = loaded > L.nq ? loaded - L.nq : 0; k < loaded; ++k)
      mbar_wait(&q_full[k & 1], (k >> 1) & 1, p.c.wait_limit_ns);
  } else if (warp == kTreeSoftmaxWarps + 2) {
    // ---- S = Q K^T issuer ------------------------------------------------------------------
    Cursor c(p, sh);
    constexpr bool kBf16 = std::is_same<M, __nv_bfloat16>::value;
    constexpr uint32_t kDescS = mma_desc(kBf16, kTreeTokens, false);
    // descriptors of the first tiles; an address step of b bytes adds b / 16 to them
    const uint64_t q_desc = tile_desc(smem_u32(smem + L.q_off), 16, 1024);
    const uint64_t k_desc = tile_desc(smem_u32(smem + L.k_off), 16, grp_bytes);
    const bool issuer = elect_one();
    uint32_t it = 0, k_slot = 0, k_par = 0;
    TileSlot<NS> sl;
    {
      TreeWalk w(p, sh);   // (the cursor passes over pieces without rows in this row tile)
      const bool any = w.next(p, sh);
      if (issuer) tree_record(p, sh, any, w);
    }
    while (c.advance(p, sh)) {
      const uint32_t qb = c.piece & 1, buf = sl.buf;
      const bool last = c.last();
      if (c.first()) wait(&q_full[qb], (c.piece >> 1) & 1);
      // the buffer's P has been used (its O is done); the softmax read its S before that
      if (it >= NS) wait(&o_full[buf], sl.par ^ 1);
      wait(&k_full[k_slot], k_par);
      tc_fence_after();
      if (!wait.dead && issuer) {
        const uint64_t kd = k_desc + k_slot * (kTile >> 4);
        const uint32_t s_col = tmem + kColS + buf * 128u;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t kk = kd + (uint32_t)(k / 4) * (blk_bytes >> 4) + (uint32_t)(k % 4) * 2u;
          if constexpr (kFp8) {
            mma_ts(s_col, tmem + kColQ + qb * (D / 2) + k * 8u, kk, kDescS, k != 0);
          } else {
            const uint32_t off = (uint32_t)(k / 4) * (16384u >> 4) + (uint32_t)(k % 4) * 2u;
            mma_ss(s_col, q_desc + qb * (kTile >> 4) + off, kk, kDescS, k != 0);
          }
        }
        tc_commit(&s_full[buf]);
        tc_commit(&k_empty[k_slot]);
        if (last) tc_commit(&q_empty[qb]);
      }
      __syncwarp();
      if (++k_slot == L.nk) k_slot = 0, k_par ^= 1;
      ++it;
      sl.next();
    }
    if (issuer) tc_commit(&drained[0]);   // nothing leaves before the last MMA has completed
    mbar_wait(&drained[0], 0, kWaitLimitNs);   // (issued MMAs end; no test hook holds them up)
  } else if (warp == kTreeSoftmaxWarps + 3) {
    // ---- O += P V issuer -------------------------------------------------------------------
    Cursor c(p, sh);
    constexpr bool kBf16 = std::is_same<M, __nv_bfloat16>::value;
    constexpr uint32_t kDescO = mma_desc(kBf16, D, true);
    const uint64_t v_desc = tile_desc(smem_u32(smem + L.v_off), blk_bytes, grp_bytes);
    const uint32_t v_step = 2u * grp_bytes >> 4;   // 16 tokens
    // P's columns of 16 tokens (hi): every 32 tokens' P lies over their S, lo 16 columns behind hi
    auto p_col = [](int k) { return (uint32_t)(k >> 1) * 32u + (uint32_t)(k & 1) * 8u; };
    const bool issuer = elect_one();
    uint32_t v_slot = 0, v_par = 0;
    TileSlot<NS> sl;
    while (c.advance(p, sh)) {
      const uint32_t buf = sl.buf;
      const uint64_t vd = v_desc + v_slot * (kTile >> 4);
      const uint32_t pa = tmem + kColS + buf * 128u, oc = tmem + kColO;
      const int valid = c.w.s.n - c.kt * kTreeTokens;
      const bool fresh = c.first();
      wait(&v_full[v_slot], v_par);
      wait(&p_full[buf], sl.par);
      tc_fence_after();
      if (!wait.dead && issuer) {
        if (valid >= kTreeTokens) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ts(oc, pa + p_col(k), vd + k * v_step, kDescO, k != 0 || !fresh);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ts(oc, pa + 16u + p_col(k), vd + k * v_step, kDescO, true);
        } else {   // the sequence ends in this tile
          const int steps = (valid + 15) / 16;
#pragma unroll 1
          for (int k = 0; k < steps; ++k) {
            mma_ts(oc, pa + p_col(k), vd + k * v_step, kDescO, k != 0 || !fresh);
            mma_ts(oc, pa + 16u + p_col(k), vd + k * v_step, kDescO, true);
          }
        }
        tc_commit(&o_full[buf]);
        tc_commit(&v_empty[v_slot]);
      }
      __syncwarp();
      if (++v_slot == L.nv) v_slot = 0, v_par ^= 1;
      sl.next();
    }
    if (issuer) tc_commit(&drained[1]);
    mbar_wait(&drained[1], 0, kWaitLimitNs);
  } else if constexpr (kFp8) {
    // ---- FP8: codes to f16 tiles, q ----------------------------------------------------------
    Cursor c(p, sh);
    const int cw = warp - (kTreeSoftmaxWarps + 4);
    // A warp converts 32 rows of a tile. 8 lanes take the same 16 codes of 8 rows, so that with both
    // tiles swizzled (the codes' by the TMA: 16-byte chunk ^= row % 8, or ^= row / 2 % 4 where a row is
    // 64 bytes) neither its loads nor its stores meet a bank twice.
    const int r7 = lane & 7, sg = lane >> 3;
    const uint32_t src0 = (uint32_t)(cw * 32 + r7) * D + ((D == 128 ? sg ^ r7 : sg ^ (r7 >> 1)) << 4);
    const uint32_t dst0 = (uint32_t)(cw * 32 + r7) * 128 + (((sg * 2) ^ r7) << 4);
    auto convert = [&](uint32_t from, uint32_t to) {   // 32 rows of a tile of codes to those of an f16 tile
      const uint8_t* src = smem + from + src0;
      uint8_t* dst = smem + to + dst0;
#pragma unroll
      for (int h = 0; h < CH; ++h) {
        uint4 v[4];
#pragma unroll
        for (int g = 0; g < 4; ++g)   // segment sg + 4 h: 64 bytes on, within the swizzle
          v[g] = *reinterpret_cast<const uint4*>(
              reinterpret_cast<const uint8_t*>(reinterpret_cast<uintptr_t>(src) ^ (h * 64)) + g * 8 * D);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          uint4 a, b;
          e4m3x4_to_f16x2(v[g].x, a.x, a.y);
          e4m3x4_to_f16x2(v[g].y, a.z, a.w);
          e4m3x4_to_f16x2(v[g].z, b.x, b.y);
          e4m3x4_to_f16x2(v[g].w, b.z, b.w);
          uint8_t* d = dst + h * 16384 + g * 1024;
          *reinterpret_cast<uint4*>(d) = a;
          *reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(d) ^ 16) = b;
        }
      }
    };
    // K of tile n and V of tile n - 1, which the MMAs take at about the same time, in one pass: the
    // waits, the fence and the arrivals cost more than a tile's conversion. There is one copy of the pass and
    // of the conversion: the warps' roles together run from more code than the instruction cache holds.
    auto pass = [&](bool k, bool v, uint32_t n, uint32_t rk, uint32_t rk_par) {
      const uint32_t i = n - 1, rv = rk ? rk - 1 : L.raw - 1, rv_par = rk ? rk_par : rk_par ^ 1;
#pragma unroll 1
      for (int s = k ? 0 : 1; s < (v ? 2 : 1); ++s) {
        wait(s ? &rv_full[rv] : &rk_full[rk], s ? rv_par : rk_par);
        wait(s ? &v_empty[i & 1] : &k_empty[n & 1], (((s ? i : n) >> 1) & 1) ^ 1);
        convert(s ? L.rawv_off + rv * kCode : L.rawk_off + rk * kCode,
                s ? L.v_off + (i & 1) * kTile : L.k_off + (n & 1) * kTile);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (k) {
          mbar_arrive(&k_full[n & 1]);
          mbar_arrive(&rk_empty[rk]);
        }
        if (v) {
          mbar_arrive(&v_full[i & 1]);
          mbar_arrive(&rv_empty[rv]);
        }
      }
    };
    static_assert(!kFp8 || (L.nk == 2 && L.nv == 2), "");
    uint32_t n = 0, rk = 0, rk_par = 0;
    bool more = c.advance(p, sh), left = false;   // left: V of tile n - 1 is to come
    while (more || left) {
      // a piece's first tile: the V that is left goes ahead, alone, then q
      const bool take = more && !(left && c.first());
      if (take && c.first()) {
        // q: a thread's row as f16 times a power of two, so that its largest element lies in
        // [2^14, 2^15), into TMEM
        const int qb = c.piece & 1, rr = cw * 32 + lane, r = sh.row_tile * kTreeRows + rr;
        wait(&q_empty[qb], ((c.piece >> 1) & 1) ^ 1);
        tc_fence_after();
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(p.q) +
            ((long long)(c.w.s.row0 + r / p.group) * p.c.hq + c.w.kvh * p.group + r % p.group) * D);
        const bool have = r < c.w.s.T * p.group;
        if (have) {   // its lines, and those of the next KV head's heads, which mostly come next
          const bool next = c.w.kvh + 1 < p.c.hkv;
          for (int j = 0; j < D / 8; j += 8) {
            prefetch_l2(src + j);
            if (next) prefetch_l2(src + p.group * (D / 8) + j);
          }
        }
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        float big = 0.f;
#pragma unroll 1
        for (int j = 0; j < D / 64; ++j) {   // a 128-byte line at a time: registers are short
          uint4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = have ? __ldg(src + j * 8 + k) : none;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack_pair<__nv_bfloat16>(u[e]);
              big = max3(big, fabsf(f.x), fabsf(f.y));
            }
          }
        }
        // 2^(14 - exponent of the largest), within what an int8 holds; 1 for a row of zeros
        int s = big > 0.f && big < INFINITY ? 14 - ((int)(__float_as_uint(big) >> 23) - 127) : 0;
        s = min(max(s, -112), 126);
        const float mul = __uint_as_float((uint32_t)(s + 127) << 23);
        const uint32_t q_addr = tmem + ((uint32_t)cw << 21) + kColQ + qb * (D / 2);
#pragma unroll 1
        for (int j = 0; j < D / 64; ++j) {
          uint32_t w[32];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint4 v = have ? __ldg(src + j * 8 + k) : none;
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack_pair<__nv_bfloat16>(u[e]);
              w[4 * k + e] = pack_pair<__half>(f.x * mul, f.y * mul);
            }
          }
          __syncwarp();   // (rows without a query load nothing)
          tmem_st32(q_addr + j * 32, w);
        }
        qexp[qb * 128 + rr] = (signed char)-s;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[qb]);
      }
      pass(take, left, n, rk, rk_par);
      left = take;
      if (take) {
        if (++rk == (uint32_t)L.raw) rk = 0, rk_par ^= 1;
        ++n;
        more = c.advance(p, sh);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kTreeSoftmaxWarps + 2) tmem_free(tmem, kTmemCols);
}

template <typename T>
const void* for_d(int D) {
  return D == 64    ? reinterpret_cast<const void*>(&tree_mma_kernel_t<T, 64>)
         : D == 128 ? reinterpret_cast<const void*>(&tree_mma_kernel_t<T, 128>)
                    : nullptr;
}

}  // namespace

const void* tree_mma_kernel(int dtype, bool fp8, int head_dim) {
  if (fp8) return for_d<fp8e4m3>(head_dim);
  if (dtype == kOutF16) return for_d<__half>(head_dim);
  if (dtype == kOutBF16) return for_d<__nv_bfloat16>(head_dim);
  return nullptr;
}

}  // namespace da
