// da_tree.cu -- attention for trees of drafted tokens over a cache: the fp32 kernel, the merge of
// partials, and the host side of decode_attn_tree_*.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>
#include <set>
#include <string>
#include <type_traits>
#include <utility>

#include "da_plan.h"
#include "da_tree_mma.cuh"

using namespace da;

struct da_tree_plan {
  da_problem prob;
  da_plan cache;                // the problem's cache layout (decode_attn_plan's fields)
  int max_tree, num_sms;
  int tile_rows, tile_tokens, max_row_tiles;
  int grid, stages, narrow;
  int stall;                    // test hook, see TreeParams
  unsigned char heads[kTreeMaxRowTiles + 1];
  size_t smem_bytes;
  size_t off_status, off_info, off_part_l, off_part_o, ws_bytes;
};

namespace {

// ---- fp32 caches: CUDA cores ------------------------------------------------------------------
constexpr int kCoreRows = 32;      // query rows per tile
constexpr int kCoreTokens = 64;    // KV tokens per tile
constexpr int kCoreThreads = 256;

template <int D>
struct CoreSmem {
  static constexpr int kStride = D + 4;        // rows 16 bytes apart mod 128: no bank conflicts
  float q[kCoreRows * kStride];
  float k[kCoreTokens * kStride];
  float v[kCoreTokens * D];
  float p[kCoreRows * (kCoreTokens + 4)];
  unsigned long long odd;                      // drafted tokens whose V has a value not finite
  TreeScratch sched;
};

// 16 bytes from global to shared memory, in the background; zeros where `valid` is false (src is then not
// read).
__device__ __forceinline__ void copy16_async(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {   // all but the N youngest groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A 32 x 64 tile of logits by 8 warps of 4 rows each: a lane holds its warp's rows at tokens lane and lane +
// 32 (what is read of q is the same for all lanes, what is read of K serves 4 rows); then the same rows of O at
// D / 32 columns. fp32 throughout. K and V rows past the
// sequence's end or on bad pages are zero in shared memory.
// Bound by the shared-memory reads that feed the FMAs (7800 wavefronts in the 11500 cycles of a tile; the FMAs
// take 4100, packed half) and the barriers between the phases; an fp32 cache has no tensor-core form that keeps
// its 24 bits. 8 sequences of 4350 tokens, 32/8 heads, 8 drafted (32 rows): 184 us, 25 TFLOP/s, 1.6 TB/s; with 1
// drafted token (4 rows) 98 us, 2.9 TB/s.
// Lanes of 2 rows x 4 tokens, with twice the reads of K: 205 and 92.
template <int D>
__global__ void __launch_bounds__(kCoreThreads) tree_core_kernel(const __grid_constant__ TreeParams p,
                                                                 const void* __restrict__ kc,
                                                                 const void* __restrict__ vc) {
  extern __shared__ __align__(16) uint8_t raw[];
  using Smem = CoreSmem<D>;
  Smem& sm = *reinterpret_cast<Smem*>(raw);
  constexpr int QS = Smem::kStride, PS = kCoreTokens + 4;
  constexpr int NR = 4, NC = D / 32;           // rows a warp, columns of O a lane
  using Vec = std::conditional_t<NC == 4, ulonglong2, f32x2>;
  const int tid = threadIdx.x, lane = tid & 31, row0 = (tid >> 5) * NR;
  const int G = p.group;
  pdl_wait();
  pdl_launch_dependents();   // the merge's launch runs beside this kernel; it waits for its end
  const TreeShare sh = tree_schedule<kCoreThreads>(p, sm.sched);
  TreeWalk w(p, sh);
  bool first_piece = true;
  if (sh.u1 <= sh.u0 && tid == 0) tree_record(p, sh, false, w);
  while (w.next(p, sh)) {
    if (first_piece && tid == 0) tree_record(p, sh, true, w);
    first_piece = false;
    const int R = w.s.T * G, r0 = sh.row_tile * kCoreRows;
    if (r0 >= R) continue;
    __syncthreads();
    if (tid == 0) sm.odd = 0;
    for (int i = tid; i < kCoreRows * D; i += kCoreThreads) {
      const int r = i / D, d = i % D, rr = r0 + r;
      float x = 0.f;
      if (rr < R) {
        x = __ldg(static_cast<const float*>(p.q) +
                  ((long long)(w.s.row0 + rr / G) * p.c.hq + w.kvh * G + rr % G) * D + d);
      }
      sm.q[r * QS + d] = x;
    }
    unsigned long long word[NR];
#pragma unroll
    for (int a = 0; a < NR; ++a) {
      const int rr = r0 + row0 + a, i = rr / G;
      word[a] = rr < R ? tree_clip(p, p.mask ? __ldg(p.mask + w.s.row0 + i) : 0ull, i, w.s.T) : 0ull;
    }
    const bool busy = r0 + row0 < R;   // a warp without rows only copies
    float m[NR], l[NR];
    f32x2 o2[NR][NC / 2] = {};   // pairs of columns
#pragma unroll
    for (int a = 0; a < NR; ++a) m[a] = -INFINITY, l[a] = 0.f;
    // A warp copies kCoreTokens / 8 rows of a tile; a lane looks one of them up. K of the next tile is on
    // its way from the end of S on, V from the end of O on.
    constexpr int kRows = kCoreTokens / 8, CH = D / 4;
    const int j0 = (tid >> 5) * kRows;
    int z = -1;   // cache row of tile row j0 + lane
    auto lookup = [&](int kt) {
      const int t = kt * kCoreTokens + j0 + lane;
      z = -1;
      if (lane < kRows && t < w.s.n) {
        const int entry = p.c.paged ? __ldg(p.c.block_table + (long long)w.b * p.c.max_blocks +
                                            t / p.c.page_size)
                                    : 0;
        z = token_row(p.c, w.b, t, entry);
        if (z < 0) atomicOr(p.c.status, kStatusBadBlockTable);
      }
    };
    // calls f(tile row, 16-byte chunk, cache row) for what this thread copies
    auto mine_of_tile = [&](auto f) {
#pragma unroll
      for (int n = 0; n < kRows * CH / 32; ++n) {
        const int r = n * 32 / CH + lane / CH;
        f(j0 + r, lane % CH, __shfl_sync(0xffffffffu, z, r));
      }
    };
    auto load = [&](const void* src, float* dst, int stride) {
      mine_of_tile([&](int jr, int c, int zr) {
        copy16_async(dst + jr * stride + c * 4,
                     static_cast<const uint4*>(src) + (zr < 0 ? 0ll : ((long long)zr * p.c.hkv + w.kvh) * CH + c),
                     zr >= 0);
      });
    };
    lookup(w.t0);
    __syncthreads();   // the piece before has been read
    load(kc, sm.k, QS);
    copies_commit();
    load(vc, sm.v, D);
    copies_commit();
    for (int kt = w.t0; kt < w.t1; ++kt) {
      copies_wait<1>();   // K
      __syncthreads();
      f32x2 s2[NR][2] = {};   // sums over even and over odd d
#pragma unroll 4
      for (int c = 0; c < (busy ? D / 4 : 0); ++c) {
        const ulonglong2 k0 = reinterpret_cast<const ulonglong2*>(sm.k + lane * QS)[c];
        const ulonglong2 k1 = reinterpret_cast<const ulonglong2*>(sm.k + (lane + 32) * QS)[c];
#pragma unroll
        for (int a = 0; a < NR; ++a) {
          const ulonglong2 q = reinterpret_cast<const ulonglong2*>(sm.q + (row0 + a) * QS)[c];
          f2_fma(s2[a][0], q.x, k0.x);
          f2_fma(s2[a][1], q.x, k1.x);
          f2_fma(s2[a][0], q.y, k0.y);
          f2_fma(s2[a][1], q.y, k1.y);
        }
      }
      __syncthreads();
      const int z_now = z;
      if (kt + 1 < w.t1) {
        lookup(kt + 1);
        load(kc, sm.k, QS);
      }
      copies_commit();
      if (busy) {
#pragma unroll
        for (int a = 0; a < NR; ++a) {
          float mx = m[a], s[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float even, odd;
            f2_unpack(s2[a][j], even, odd);
            const int t = kt * kCoreTokens + lane + 32 * j;
            const bool seen = t < w.s.ctx || (t < w.s.n && (word[a] >> (t - w.s.ctx) & 1ull));
            s[j] = seen ? (even + odd) * p.qscale : -INFINITY;
            mx = fmaxf(mx, s[j]);
          }
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
          const float ref = mx == -INFINITY ? 0.f : mx;
          const float f = exp2f(m[a] - ref);
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float e = exp2f(s[j] - ref);
            sum += e;
            sm.p[(row0 + a) * PS + lane + 32 * j] = e;
          }
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
          l[a] = l[a] * f + sum;
          m[a] = mx;
#pragma unroll
          for (int c = 0; c < NC / 2; ++c) o2[a][c] = f2_mul(o2[a][c], f2_pack(f, f));
        }
      }
      copies_wait<1>();   // V
      if ((kt + 1) * kCoreTokens > w.s.ctx) {
        // a drafted token may be hidden from some rows: its infinities and NaN must not reach
        // them as 0 * inf; they are set aside and added to the rows that see the token
        const int z_next = z;
        z = z_now;
        mine_of_tile([&](int jr, int c, int zr) {
          const int t = kt * kCoreTokens + jr;
          if (zr < 0 || t < w.s.ctx) return;
          float* const at = sm.v + jr * D + c * 4;
          bool odd = false;
#pragma unroll 1
          for (int k = 0; k < 4; ++k)
            if (!isfinite(at[k])) {
              odd = true;
              at[k] = 0.f;
            }
          if (odd) atomicOr(&sm.odd, 1ull << ((t - w.s.ctx) & 63));
        });
        z = z_next;
      }
      __syncthreads();   // V is there, and the warp's P
#pragma unroll 2
      for (int t = 0; t < (busy ? kCoreTokens : 0); t += 4) {
        float pr[NR][4];
#pragma unroll
        for (int a = 0; a < NR; ++a)
          *reinterpret_cast<float4*>(pr[a]) =
              *reinterpret_cast<const float4*>(sm.p + (row0 + a) * PS + t);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f32x2 v[NC / 2];
          *reinterpret_cast<Vec*>(v) = *reinterpret_cast<const Vec*>(sm.v + (t + e) * D + lane * NC);
#pragma unroll
          for (int a = 0; a < NR; ++a)
#pragma unroll
            for (int c = 0; c < NC / 2; ++c) f2_fma(o2[a][c], f2_pack(pr[a][e], pr[a][e]), v[c]);
        }
      }
      __syncthreads();
      if (kt + 1 < w.t1) load(vc, sm.v, D);
      copies_commit();
    }
#pragma unroll
    for (int a = 0; a < NR; ++a) {
      const int rr = r0 + row0 + a;
      if (rr >= R) continue;
      float o[NC];
#pragma unroll
      for (int c = 0; c < NC / 2; ++c) f2_unpack(o2[a][c], o[2 * c], o[2 * c + 1]);
      for (unsigned long long rest = sm.odd & word[a]; rest; rest &= rest - 1) {   // rare
        const int t = w.s.ctx + __ffsll((long long)rest) - 1;
        const int entry = p.c.paged ? __ldg(p.c.block_table + (long long)w.b * p.c.max_blocks +
                                            t / p.c.page_size)
                                    : 0;
        const int z = token_row(p.c, w.b, t, entry);
        for (int c = 0; c < NC; ++c) {
          const long long at = ((long long)z * p.c.hkv + w.kvh) * D + lane * NC + c;
          const float v = static_cast<const float*>(vc)[at];
          if (!isfinite(v)) o[c] += v;
        }
      }
      const float inv = l[a] == 0.f ? 0.f : 1.f / l[a];
      const float L = l[a] == 0.f ? -INFINITY : m[a] + log2f(l[a]);
      if (w.whole) {
        const long long row = (long long)(w.s.row0 + rr / G) * p.c.hq + w.kvh * G + rr % G;
        for (int c = 0; c < NC; ++c)
          store_out(p.out, row * D + lane * NC + c, p.c.out_dtype, o[c] * inv * p.v_scale);
        if (p.out_lse && lane == 0) p.out_lse[row] = L * 0.69314718055994531f;
      } else {
        const long long at =
            (long long)tree_slot(sh.owner, w.head, sh.row_tiles * sh.heads,
                                 sh.head * sh.row_tiles + sh.row_tile) * kCoreRows + row0 + a;
        for (int c = 0; c < NC; ++c) p.part_o[at * D + lane * NC + c] = o[c] * inv;
        if (lane == 0) p.part_l[at] = L;
      }
    }
  }
}

// ---- merge ----------------------------------------------------------------------------------
// o = sum_s 2^(L_s - L) o_s, L = log2 sum_s 2^(L_s). Block (x, y): what CTA x recorded (tree_record), rows
// y * 8 .. + 7 of its row tile and head, a warp a row, D / 32 columns a lane. A programmatic dependent of
// the attention kernel. Bound by latency, so it is two round trips to L2: the record, then a row's L's
// and its first partials together.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) tree_merge_kernel(
    const __grid_constant__ TreeParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rr = blockIdx.y * kMergeWarps + warp;
  pdl_wait();
  pdl_launch_dependents();   // the next run's attention kernel may set itself up; it waits for this one's end
  const int4 a = p.info[2 * blockIdx.x], b = p.info[2 * blockIdx.x + 1];
  const int n = a.x;
  if (n == 0 || rr >= b.y) return;
  constexpr int C = D / 32, K = 16;
  using Vec = std::conditional_t<C == 4, float4, float2>;
  auto slot = [&](int j) { return (long long)(a.y + (j ? a.z + (j - 1) * a.w : 0)) * p.tile_rows + rr; };
  auto part = [&](int j) {
    return *reinterpret_cast<const Vec*>(p.part_o + slot(j) * D + lane * C);
  };
  Vec v[K];
#pragma unroll
  for (int j = 0; j < K; ++j) v[j] = j < n ? part(j) : Vec{};
  float top = -INFINITY;
  for (int j = lane; j < n; j += 32) top = fmaxf(top, p.part_l[slot(j)]);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  // a NaN among the L's passes the maximum over; it comes back through the weights
  const float ref = top == -INFINITY ? 0.f : top;
  float acc[C] = {};
  float sum = 0.f;
  auto add = [&](float wgt, const Vec& x) {
    sum += wgt;
    acc[0] += wgt * x.x;
    acc[1] += wgt * x.y;
    if constexpr (C == 4) {
      acc[2] += wgt * x.z;
      acc[3] += wgt * x.w;
    }
  };
  for (int j0 = 0; j0 < n; j0 += 32) {
    const float wl = j0 + lane < n ? exp2f(p.part_l[slot(j0 + lane)] - ref) : 0.f;
    if (j0 == 0) {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const float wgt = __shfl_sync(0xffffffffu, wl, j);
        if (j < n) add(wgt, v[j]);   // (a weight of 0 for none would make NaN of an infinite partial)
      }
    }
#pragma unroll 8
    for (int j = j0 == 0 ? K : 0; j < min(32, n - j0); ++j)
      add(__shfl_sync(0xffffffffu, wl, j), part(j0 + j));
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int r = b.z + rr, i = r / p.group, h = b.w * p.group + r % p.group;
  const long long row = (long long)(b.x + i) * p.c.hq + h;
#pragma unroll
  for (int c = 0; c < C; ++c)
    store_out(p.out, row * D + lane * C + c, p.c.out_dtype, acc[c] * inv * p.v_scale);
  if (p.out_lse && lane == 0)
    p.out_lse[row] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
}

const void* core_kernel(int D) {
  return D == 64 ? reinterpret_cast<const void*>(&tree_core_kernel<64>)
                 : reinterpret_cast<const void*>(&tree_core_kernel<128>);
}

bool uses_mma(const da_problem& p) { return p.kv_fp8 || p.qkv_dtype != DA_F32; }

// The kernel's shared-memory limit, raised once per device and kernel. regs: the registers that the
// kernel must have been compiled to (its register split draws on them), or 0.
int raise_smem(const void* fn, size_t smem, int regs) {
  static std::mutex mu;
  static std::set<std::pair<int, const void*>> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(mu);
  if (done.count({dev, fn})) return DA_OK;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(tree kernel)");
  if (regs) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, fn);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncGetAttributes");
    if (fa.numRegs != regs) return text_fail("tree kernel not built to the registers of its split");
  }
  try {
    done.insert({dev, fn});
  } catch (...) {   // out of host memory: asked again next time
  }
  return DA_OK;
}

int encode(CUtensorMap* map, int es, int rank, const void* base, const cuuint64_t* dims,
           const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle,
           CUtensorMapL2promotion promote) {
  auto fn = encode_fn();
  if (!fn) return text_fail("cuTensorMapEncodeTiled is not available from the driver");
  const cuuint32_t ones[5] = {1u, 1u, 1u, 1u, 1u};
  const CUresult r =
      fn(map, es == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8,
         (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
         CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promote, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DA_OK : text_fail("cuTensorMapEncodeTiled refused a tensor map");
}

// [tokens, Hkv, D] cache, one box = `box` tokens of one KV head. FP8 caches: rows of codes, swizzled
// as wide as they are. 16-bit
// caches in 128-byte-swizzled blocks of 64 elements: contiguous ones as [Hkv, D / 64, tokens, 64], a
// box one block of 128 tokens; paged ones as [Hkv, tokens / 8, D / 64, 8, 64], a box whole rows.
int kv_map(const da_tree_plan& pl, const void* base, int box, CUtensorMap* map) {
  const da_problem& p = pl.prob;
  const cuuint64_t tokens = p.paged ? (cuuint64_t)p.num_physical_blocks * p.page_size
                                    : (cuuint64_t)p.batch * p.max_seq_len;
  const cuuint64_t D = p.head_dim, H = p.num_kv_heads;
  if (p.kv_fp8) {
    const cuuint64_t dims[3] = {D, tokens, H}, strides[2] = {H * D, D};
    const cuuint32_t b[3] = {(cuuint32_t)D, (cuuint32_t)box, 1u};
    return encode(map, 1, 3, base, dims, strides, b,
                  D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  D == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B);
  }
  const auto promote =
      D == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  if (p.paged) {   // pages hold at least 8 tokens
    const cuuint64_t dims[5] = {64, 8, D / 64, tokens / 8, H};
    const cuuint64_t strides[4] = {H * D * 2, 128, H * D * 16, D * 2};
    const cuuint32_t b[5] = {64u, 8u, (cuuint32_t)D / 64, (cuuint32_t)box / 8, 1u};
    return encode(map, 2, 5, base, dims, strides, b, CU_TENSOR_MAP_SWIZZLE_128B, promote);
  }
  const cuuint64_t dims[4] = {64, tokens, D / 64, H}, strides[3] = {H * D * 2, 128, D * 2};
  const cuuint32_t b[4] = {64u, (cuuint32_t)box, 1u, 1u};
  return encode(map, 2, 4, base, dims, strides, b, CU_TENSOR_MAP_SWIZZLE_128B, promote);
}

// [rows, Hq, D] q, one box = the G heads of a KV head of 128 / G drafted tokens, one 64-element block.
int q_map(const da_tree_plan& pl, const void* base, int rows, CUtensorMap* map) {
  const cuuint64_t D = pl.prob.head_dim, H = pl.prob.num_q_heads;
  const cuuint32_t G = (cuuint32_t)pl.cache.group;
  const cuuint64_t dims[4] = {64, H, (cuuint64_t)rows, D / 64}, strides[3] = {D * 2, H * D * 2, 128};
  const cuuint32_t b[4] = {64u, G, (cuuint32_t)kTreeRows / G, 1u};
  return encode(map, 2, 4, base, dims, strides, b, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
}

}  // namespace

extern "C" {

int decode_attn_tree_plan(const da_problem* problem, int max_tree, da_tree_plan** plan_out,
                          size_t* workspace_bytes_out) {
  if (!problem || !plan_out) return DA_ERR_INVALID_ARG;
  *plan_out = nullptr;
  if (max_tree < 1 || max_tree > DECODE_ATTN_MAX_TREE) return DA_ERR_INVALID_ARG;
  if (problem->mode != DA_SOFTMAX_SYNC) {
    const int v = validate_problem(*problem);
    return v != DA_OK ? v : DA_ERR_UNSUPPORTED;
  }
  if (problem->debug_stall_stage != 0) return DA_ERR_INVALID_ARG;
  da_plan* cache = nullptr;
  const int rc = decode_attn_plan(problem, 0, &cache, nullptr);
  if (rc != DA_OK) return rc;
  da_tree_plan* pl = new (std::nothrow) da_tree_plan();
  if (!pl) {
    decode_attn_destroy(cache);
    return DA_ERR_INVALID_ARG;
  }
  pl->cache = *cache;
  decode_attn_destroy(cache);
  pl->prob = *problem;
  const da_problem& p = pl->prob;
  pl->max_tree = max_tree;
  pl->num_sms = pl->cache.num_sms;
  const bool mma = uses_mma(p);
  if (mma) {
    const TreeLayout L = tree_layout(p.head_dim, p.kv_fp8 != 0);
    pl->tile_rows = kTreeRows;
    pl->tile_tokens = kTreeTokens;
    pl->stages = p.kv_fp8 ? 2 * L.raw : L.nk + L.nv;
    pl->smem_bytes = L.total;
  } else {
    pl->tile_rows = kCoreRows;
    pl->tile_tokens = kCoreTokens;
    pl->stages = 0;
    pl->smem_bytes = p.head_dim == 64 ? sizeof(CoreSmem<64>) : sizeof(CoreSmem<128>);
  }
  pl->max_row_tiles = (max_tree * pl->cache.group + pl->tile_rows - 1) / pl->tile_rows;
  const long long units = (long long)p.batch * p.num_kv_heads *
                          ((pl->cache.capacity + pl->tile_tokens - 1) / pl->tile_tokens);
  if (units >= (1ll << 31)) {   // the device schedule's 32-bit units
    delete pl;
    return DA_ERR_UNSUPPORTED;
  }
  pl->grid = (int)std::min<long long>(
      std::max(mma ? pl->num_sms : 2 * pl->num_sms, pl->max_row_tiles),
      units * pl->max_row_tiles);
  pl->narrow = (units + 1) * pl->grid < (1ll << 31) ? 1 : 0;
  for (int r = 1; r <= pl->max_row_tiles; ++r)
    pl->heads[r] = (unsigned char)tree_heads(pl->grid, r, p.num_kv_heads);
  const size_t slots = 2ull * pl->grid;   // two an owner and row tile; owners x row tiles <= grid
  size_t off = 0;
  pl->off_status = off;
  off = align256(off + 16);
  pl->off_info = off;
  off = align256(off + (size_t)pl->grid * 32);
  pl->off_part_l = off;
  off = align256(off + slots * pl->tile_rows * 4);
  pl->off_part_o = off;
  off = align256(off + slots * pl->tile_rows * p.head_dim * 4);
  pl->ws_bytes = off;
  *plan_out = pl;
  if (workspace_bytes_out) *workspace_bytes_out = pl->ws_bytes;
  return DA_OK;
}

int decode_attn_tree_plan_info(const da_tree_plan* plan, da_tree_plan_info* info) {
  if (!plan || !info) return DA_ERR_INVALID_ARG;
  info->grid_ctas = plan->grid;
  info->row_tiles = plan->max_row_tiles;
  info->tile_rows = plan->tile_rows;
  info->tile_tokens = plan->tile_tokens;
  info->stages = plan->stages;
  info->max_tree = plan->max_tree;
  info->workspace_bytes = plan->ws_bytes;
  info->smem_bytes = plan->smem_bytes;
  return DA_OK;
}

int decode_attn_tree_debug_stall(da_tree_plan* plan, int tensor) {
  if (!plan || tensor < 0 || tensor > 2) return DA_ERR_INVALID_ARG;
  if (plan->stages == 0) return DA_ERR_UNSUPPORTED;   // the fp32 kernel waits for its own copies alone
  plan->stall = tensor;
  return DA_OK;
}

void decode_attn_tree_destroy(da_tree_plan* plan) { delete plan; }

int decode_attn_tree_workspace_init(const da_tree_plan* plan, void* workspace,
                                    size_t workspace_bytes, void* cuda_stream) {
  if (!plan || !workspace || !aligned(workspace, 256)) return DA_ERR_INVALID_ARG;
  if (workspace_bytes < plan->ws_bytes) return DA_ERR_WORKSPACE_TOO_SMALL;
  const cudaError_t e = cudaMemsetAsync(static_cast<char*>(workspace) + plan->off_status, 0, 4,
                                        static_cast<cudaStream_t>(cuda_stream));
  return e == cudaSuccess ? DA_OK : cuda_fail(e, "cudaMemsetAsync(tree workspace)");
}

int decode_attn_tree_check_status(const da_tree_plan* plan, void* workspace, void* cuda_stream) {
  if (!plan || !workspace) return DA_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  char* ws = static_cast<char*>(workspace);
  int32_t st = 0;
  cudaError_t e = cudaMemcpyAsync(&st, ws + plan->off_status, 4, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemsetAsync(ws + plan->off_status, 0, 4, stream);
  if (e != cudaSuccess) return cuda_fail(e, "reading the device status");
  return status_to_error(st);
}

int decode_attn_tree_run(const da_tree_plan* plan, const da_tree_args* args) {
  if (!plan || !args) return DA_ERR_INVALID_ARG;
  const da_tree_plan& pl = *plan;
  const da_tree_args& a = *args;
  const da_problem& pr = pl.prob;
  if (a.rows < 0 || !a.row_offsets || !a.ctx_lens || !a.workspace || !std::isfinite(a.scale))
    return DA_ERR_INVALID_ARG;
  if (pr.paged ? !a.block_table : a.block_table != nullptr) return DA_ERR_INVALID_ARG;
  if (!aligned(a.row_offsets, 4) || !aligned(a.ctx_lens, 4) || !aligned(a.block_table, 4) ||
      !aligned(a.workspace, 256) || !aligned(a.tree_mask, 8) || !aligned(a.out_lse, 4))
    return DA_ERR_INVALID_ARG;
  if (a.workspace_bytes < pl.ws_bytes) return DA_ERR_WORKSPACE_TOO_SMALL;
  if (a.rows == 0) return DA_OK;
  if (!a.q || !a.k_cache || !a.v_cache || !a.out || !aligned(a.q, 16) || !aligned(a.k_cache, 16) ||
      !aligned(a.v_cache, 16) || !aligned(a.out, 16))
    return DA_ERR_INVALID_ARG;
  const long long elems = (long long)a.rows * pr.num_q_heads * pr.head_dim;
  if (overlap(a.q, elems * elem_size(pr.qkv_dtype), a.out, elems * elem_size(pr.out_dtype)))
    return DA_ERR_INVALID_ARG;
  TreeParams p;
  std::memset(&p, 0, sizeof p);
  fill_common(pl.cache, p.c, a.block_table, nullptr, nullptr);
  char* ws = static_cast<char*>(a.workspace);
  p.c.status = reinterpret_cast<int32_t*>(ws + pl.off_status);
  p.info = reinterpret_cast<int4*>(ws + pl.off_info);
  p.part_l = reinterpret_cast<float*>(ws + pl.off_part_l);
  p.part_o = reinterpret_cast<float*>(ws + pl.off_part_o);
  p.q = a.q;
  p.row_offsets = a.row_offsets;
  p.ctx_lens = a.ctx_lens;
  p.mask = reinterpret_cast<const unsigned long long*>(a.tree_mask);
  p.out = a.out;
  p.out_lse = a.out_lse;
  p.rows = a.rows;
  p.max_tree = pl.max_tree;
  p.group = pl.cache.group;
  p.tile_rows = pl.tile_rows;
  p.tile_tokens = pl.tile_tokens;
  p.max_row_tiles = pl.max_row_tiles;
  p.narrow = pl.narrow;
  p.stall = pl.stall;
  if (pl.stall) p.c.wait_limit_ns = kTestWaitLimitNs;
  std::memcpy(p.heads, pl.heads, sizeof p.heads);
  p.qscale = (float)((double)a.scale * 1.4426950408889634 * (pr.kv_fp8 ? (double)pr.k_scale : 1.0));
  p.v_scale = pr.kv_fp8 ? pr.v_scale : 1.f;
  if (!std::isfinite(p.qscale)) return DA_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(a.cuda_stream);
  cudaError_t e;
  if (pr.validate) {
    e = cudaMemsetAsync(ws + pl.off_status, 0, 4, stream);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(status)");
  }
  // Programmatic dependents of what is ahead of them set themselves up while it ends, and wait for its end
  // before they read or write anything of it. The merge is one; so is the attention kernel where a
  // sequence's rows fit one row tile (short tree, 640 tokens, a run in a row of runs: 17 % less time, 11.5 us
  // now). With more row tiles the CTAs that share KV tiles have to start as neighbours, which an early launch, as
  // SMs fall free, undoes (64 drafted tokens over FP8 pages: 16 % more time).
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)pl.grid);
  cfg.dynamicSmemBytes = pl.smem_bytes;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = pl.max_row_tiles == 1 ? 1 : 0;
  if (uses_mma(pr)) {
    const void* fn = tree_mma_kernel(pr.qkv_dtype, pr.kv_fp8 != 0, pr.head_dim);
    if (!fn) return DA_ERR_UNSUPPORTED;
    p.c.box_tokens = pr.paged ? std::min(pr.page_size, kTreeTokens) : kTreeTokens;
    CUtensorMap tmq, tmk, tmv;
    int rc = q_map(pl, a.q, a.rows, &tmq);
    if (rc == DA_OK) rc = kv_map(pl, a.k_cache, p.c.box_tokens, &tmk);
    if (rc == DA_OK) rc = kv_map(pl, a.v_cache, p.c.box_tokens, &tmv);
    if (rc == DA_OK) rc = raise_smem(fn, pl.smem_bytes, pr.kv_fp8 ? 0 : kTreeLaunchRegs);
    if (rc != DA_OK) return rc;
    const void* vc = a.v_cache;
    void* kargs[5] = {&p, &tmq, &tmk, &tmv, &vc};
    cfg.blockDim = dim3((unsigned)tree_threads(pr.kv_fp8 != 0));
    e = cudaLaunchKernelExC(&cfg, fn, kargs);
  } else {
    const void* fn = core_kernel(pr.head_dim);
    const int rc = raise_smem(fn, pl.smem_bytes, 0);
    if (rc != DA_OK) return rc;
    const void* kc = a.k_cache;
    const void* vc = a.v_cache;
    void* kargs[3] = {&p, &kc, &vc};
    cfg.blockDim = dim3(kCoreThreads);
    e = cudaLaunchKernelExC(&cfg, fn, kargs);
  }
  if (e != cudaSuccess) return cuda_fail(e, "launching the tree kernel");
  if (pl.grid > 1) {
    const int rows = std::min(pl.tile_rows, pl.max_tree * pl.cache.group);
    cfg.gridDim = dim3((unsigned)pl.grid, (unsigned)((rows + kMergeWarps - 1) / kMergeWarps));
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    void* margs[1] = {&p};
    const void* mf = pr.head_dim == 64 ? reinterpret_cast<const void*>(&tree_merge_kernel<64>)
                                       : reinterpret_cast<const void*>(&tree_merge_kernel<128>);
    e = cudaLaunchKernelExC(&cfg, mf, margs);
    if (e != cudaSuccess) return cuda_fail(e, "launching the merge kernel");
  }
  return pr.validate ? decode_attn_tree_check_status(plan, a.workspace, a.cuda_stream) : DA_OK;
}

}  // extern "C"
