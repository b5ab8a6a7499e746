// da_adapters.cuh -- low-rank adapters of many requests beside a shared projection: the kernel.
//
//     out[r, part s] = y[r, part s] + c_a (x[r] A_{a,s}^T) B_{a,s}^T,   a the adapter of row r's request,
//
// A_{a,s} [rank, width], B_{a,s} [width of part s, rank], s over the projection's parts (q, k and v).
//
// A step reads the weights of the adapters in use once, x and y once, and writes out once; at 2 rank products a
// number read or written this is bound by memory (few rows: the weights; prompts: x, y and out), so the legacy
// tensor path is enough, and its operands can come straight from memory into registers: an order of the
// contraction's index is free, so a lane takes 16 neighbouring bytes of a row and a weight as what two
// instructions want of it, with no transpose and nothing staged.
//
// One launch. A tile is up to 16 rows of one adapter, wherever they lie, and a cluster of CTAs takes it: each
// CTA contracts a share of x's width, the cluster's CTAs exchange their partial sums through distributed shared
// memory, and each then expands a share of the columns. Which rows are a tile's, every CTA finds for itself from
// the requests' offsets and adapters (a few KB), so that no schedule has to be launched ahead.
#pragma once

#include <cstring>
#include <type_traits>

#include "da_device.cuh"
#include "da_rowvec.cuh"

namespace da {

constexpr int kAdapterThreads = 256, kAdapterWarps = kAdapterThreads / 32;
constexpr int kMaxParts = 4;
// Rows of a tile. With more of them weights are read less often, but fewer CTAs are at work, one an SM from 64 rows on
// (at the best number of CTAs a tile: 2000 rows, rank 64, 4096 to 6144: 47 us with 16, 60 with 32, 89 with 64; 2300
// rows, rank 8: 14, 17 and 21).
constexpr int kAdapterTile = 16;

struct AdapterParams {
  const void *x, *y, *a, *b;
  void* out;
  const float* scales;          // of each adapter, or null
  const int32_t* row_offsets;
  const int32_t* ids;
  long long x_rs, y_rs, out_rs;
  int rows, batch, adapters, width, parts;
  int starts[kMaxParts + 1];    // columns of the parts
  int chunks[kMaxParts + 1];    // chunks of 32 columns ahead of each part
  int n_groups;                 // warps that share the low-rank columns
  int log_ranks;                // CTAs that share a tile
  int pitch;                    // floats of a row of partial sums
  int copy;                     // rows without an adapter are copied (out is not y)
  int x_unit, y_unit;           // bytes that x and A / y and out move by: 16, 8, 4 or an element's
  int tall;                     // requests of as many rows with an adapter are left to the tall kernels
};

// Requests of many rows: what their kernels take beside AdapterParams, in da_adapters_tall.cu.
constexpr int kTallRows = 64;           // rows from which a request is theirs, where they are launched
constexpr int kTallPieces = 8;          // sums of a tile, from as many CTAs at most
constexpr size_t kTallStatusBytes = 256;
struct TallParams {
  float4* sums;                 // [kTallPieces, low / 4, rows]: low-rank sums, four columns of a row
  int32_t* status;
  int rank, stages, most_tiles;
  int n;                        // low-rank columns, to a multiple of 16
  int blocks[kMaxParts + 1];    // blocks of 128 columns ahead of each part; all of them
};
long long most_tall_tiles(const AdapterParams& p);
bool tall_fits(const AdapterParams& p, int rank, int sms);
size_t tall_workspace(int rows, int low);
// The three launches, the short kernel's (`first` of `fn`) ahead.
int launch_tall(const AdapterParams& p, int rank, bool bf16, int sms, void* workspace, const cudaLaunchConfig_t& first,
                const void* fn);

// Bytes of dynamic shared memory: the partial sums of every group of warps (where the counts of rows lay before),
// the sums over the cluster, and them as operands.
inline size_t adapter_smem(int adapters, int parts, int rank, int es, int n_groups, int pitch) {
  const size_t rows = kAdapterTile;
  const size_t counts = 4 * ((size_t)adapters + 1), sums = rows * pitch * 4 * (kAdapterWarps / n_groups);
  const size_t steps = es == 4 ? rank / 8 : rank < 16 ? 1 : rank / 16;
  return std::max((counts + 15) / 16 * 16, sums) + rows * pitch * 4 + (size_t)parts * steps * 2 * 512;
}

// The contraction of 16 rows with 8 columns, 16 (8 for fp32, as tf32) deep.
template <typename T>
__device__ __forceinline__ void mma16x8(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, float>::value)
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An fp32 number as two tf32 ones: what is left is 2^-22 of it. An infinity, or what rounds to one, has no such parts
// unless CAREFUL: then an infinity or NaN is its first part alone, and tf32's largest number the first part of what is
// larger.
__device__ __forceinline__ uint32_t tf32(float x) {
  uint32_t u;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(u) : "f"(x));
  return u;
}
template <bool CAREFUL>
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  constexpr float kMost = 3.40116213421e38f;   // (2 - 2^-10) 2^127
  const bool finite = !CAREFUL || fabsf(x) <= 3.4028235e38f;
  hi = tf32(CAREFUL && finite ? fminf(fmaxf(x, -kMost), kMost) : x);
  lo = finite ? tf32(x - __uint_as_float(hi)) : 0u;
}
// c += a b of fp32 numbers in two tf32 parts: three of the four products (the last is 2^-22 of the first). They are
// added up from zero and then to c, as the instruction cuts off what it adds to a larger sum. An infinite part times
// the other number's rest is no share of the product (0 times it is NaN, a rest may have either sign): CAREFUL takes
// the large products alone where the small ones are not finite.
// The hot loops are not careful: a factor that is not finite leaves them a sum that is not either, and such sums are
// formed again, carefully (5 prompts of up to 300 rows, 1001 to 1076: 15.3 us; careful throughout 16.1; 700 rows of
// rank 128, 2048 wide to three parts, 90 and 129).
template <bool CAREFUL>
__device__ __forceinline__ void add_products(float* c, const uint32_t* hi, const uint32_t* lo, const uint32_t* bh,
                                             const uint32_t* bl) {
  float t[4] = {0.f, 0.f, 0.f, 0.f};
  mma16x8<float>(t, lo, bh[0], bh[1]);
  mma16x8<float>(t, hi, bl[0], bl[1]);
  if constexpr (CAREFUL) {
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = fabsf(t[e]) <= 3.4028235e38f ? t[e] : 0.f;
  }
  mma16x8<float>(t, hi, bh[0], bh[1]);
#pragma unroll
  for (int e = 0; e < 4; ++e) c[e] += t[e];
}
// Whether one of the warp's sums is not finite (0 times it is not 0).
template <int N>
__device__ __forceinline__ bool any_not_finite(const float (*c)[4]) {
  float z = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) z = fmaf(c[j][e], 0.f, z);
  return __any_sync(0xffffffffu, z != 0.f);
}
// Two fp32 numbers as two pairs of T: what is left is at most 2^-17 (bf16) or 2^-23 (f16) of them.
template <typename T>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack2(x, y, T());
  float hx, hy;
  if constexpr (std::is_same<T, __half>::value) {
    __half2 h;
    memcpy(&h, &hi, 4);
    const float2 f = __half22float2(h);
    hx = f.x;
    hy = f.y;
  } else {
    hx = __uint_as_float(hi << 16);
    hy = __uint_as_float(hi & 0xffff0000u);
  }
  lo = pack2(fabsf(hx) <= 3.4028235e38f ? x - hx : 0.f, fabsf(hy) <= 3.4028235e38f ? y - hy : 0.f, T());
}

// The larger of `most` and |v|, if v is finite.
__device__ __forceinline__ float most_finite(float most, float v) {
  return fabsf(v) <= 3.4028235e38f ? fmaxf(most, fabsf(v)) : most;
}
// The power of two that takes finite numbers of up to `most` below 2^8 (1: there are none but zeros).
__device__ __forceinline__ float low_rank_scale(float most) {
  const int e = most > 0.f ? (int)(__float_as_uint(most) >> 23) - 127 - 7 : 0;
  return __uint_as_float((uint32_t)(127 - min(max(e, -120), 120)) << 23);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// (aligned: by whole warps)
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 load_of_rank(const float* p, uint32_t rank) {
  uint32_t at;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// 16 bytes of T at row + k, of which the first `left` elements are there (none: zeros), `unit` bytes at a time:
// 16, an element's, or between them 8 or 4 (fp32: none between).
template <typename T>
__device__ __forceinline__ uint4 load16(const T* row, int k, int left, int unit) {
  constexpr int V = 16 / (int)sizeof(T);
  if (unit == 16) return left > 0 ? __ldg(reinterpret_cast<const uint4*>(row + k)) : make_uint4(0u, 0u, 0u, 0u);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (sizeof(T) == 2 && unit == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (i * (V / 2) < left) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + k) + i);
        w[2 * i] = v.x;
        w[2 * i + 1] = v.y;
      }
    }
  } else if (sizeof(T) == 4 || unit == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i * (V / 4) < left) w[i] = __ldg(reinterpret_cast<const uint32_t*>(row + k) + i);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < left) w[i / 2] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(row + k) + i) << (16 * (i & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The first `left` elements of 16 bytes of T to `to`, in the same way.
template <typename T>
__device__ __forceinline__ void store16(T* to, int left, int unit, const uint32_t* w) {
  constexpr int V = 16 / (int)sizeof(T);
  if (unit == 16) {
    if (left > 0) *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if (sizeof(T) == 2 && unit == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (i * (V / 2) < left) reinterpret_cast<uint2*>(to)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
  } else if (sizeof(T) == 4 || unit == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i * (V / 4) < left) reinterpret_cast<uint32_t*>(to)[i] = w[i];
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < left) reinterpret_cast<uint16_t*>(to)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
  }
}

struct AdapterShared {
  int sums[kAdapterWarps];
  int adapter, first, count, chunk_total;
};

// Sum over the threads before this one; the sum over all in sh.chunk_total. Two barriers.
__device__ __forceinline__ int block_prefix(int mine, AdapterShared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int below = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += below;
  }
  if (lane == 31) sh.sums[warp] = upto;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kAdapterWarps; ++w) {
    const int v = sh.sums[w];
    before += w < warp ? v : 0;
    all += v;
  }
  if (threadIdx.x == 0) sh.chunk_total = all;
  __syncthreads();
  return before + upto - mine;
}

// The same in a wider block, of whose threads only the first kAdapterThreads bring anything.
__device__ __forceinline__ int wide_prefix(int mine, AdapterShared& sh) {
  if (threadIdx.x < kAdapterThreads) return block_prefix(mine, sh);
  __syncthreads();
  __syncthreads();
  return 0;
}

// Rows of request b, and the adapter they take (`adapters`: none).
__device__ __forceinline__ int rows_of(const AdapterParams& p, int b, int& first) {
  first = min(max(__ldg(p.row_offsets + b), 0), p.rows);
  return max(min(max(__ldg(p.row_offsets + b + 1), 0), p.rows) - first, 0);
}
__device__ __forceinline__ int adapter_of(const AdapterParams& p, int b) {
  const int id = __ldg(p.ids + b);
  return id >= 0 && id < p.adapters ? id : p.adapters;
}

// A request ahead of the block's loops, of each thread: its first row, rows and adapter.
struct AdapterRequest {
  int row, n, adapter;
};

// Tile t in sh: its adapter, its first row's place among the adapter's rows and their count. Tiles go by adapter, an
// adapter's rows by request. Tiles behind the last: sh.adapter is p.adapters (rows without one), and sh.first which of
// them.
__device__ __forceinline__ void find_tile(const AdapterParams& p, int t, int* s_count, AdapterRequest& own,
                                          AdapterShared& sh) {
  constexpr int M = kAdapterTile;
  const int tid = threadIdx.x;
  for (int i = tid; i < p.adapters + 1; i += kAdapterThreads) s_count[i] = 0;
  if (tid == 0) sh.adapter = -1;
  __syncthreads();
  own.row = own.n = 0;
  own.adapter = -1;
  for (int b = tid; b < p.batch; b += kAdapterThreads) {
    int first_row;
    int n = rows_of(p, b, first_row);
    const int a = adapter_of(p, b);
    if (n >= p.tall && a < p.adapters) n = 0;
    if (n) atomicAdd(s_count + a, n);
    if (b == tid) own.row = first_row, own.n = n, own.adapter = a;
  }
  __syncthreads();
  int base = 0;
  for (int i0 = 0; i0 < p.adapters; i0 += kAdapterThreads) {
    const int i = i0 + tid, n = i < p.adapters ? s_count[i] : 0, tiles = (n + M - 1) / M;
    const int before = base + block_prefix(tiles, sh);
    if (before <= t && t < before + tiles) {
      sh.adapter = i;
      sh.first = (t - before) * M;
      sh.count = n;
    }
    base += sh.chunk_total;
    __syncthreads();
    if (base > t) return;
  }
  if (tid == 0) {
    sh.adapter = p.adapters;
    sh.first = t - base;
    sh.count = s_count[p.adapters];
  }
  __syncthreads();
}

// The rows of the tile of `adapter` that begins at `first` of its `count` rows, in s_row (which was all -1).
__device__ __forceinline__ void rows_of_tile(const AdapterParams& p, int adapter, int first, int count,
                                             const AdapterRequest& own, int* s_row, AdapterShared& sh) {
  constexpr int M = kAdapterTile;
  const int tid = threadIdx.x, end = first + min(M, count - first);
  for (int b0 = 0, base = 0; b0 < p.batch && base < end; b0 += kAdapterThreads) {
    const int b = b0 + tid;
    int row = 0, n = 0;
    if (b0 == 0) {
      row = own.row;
      n = own.adapter == adapter ? own.n : 0;
    } else if (b < p.batch && adapter_of(p, b) == adapter) {
      n = rows_of(p, b, row);
      if (n >= p.tall && adapter < p.adapters) n = 0;
    }
    const int before = base + block_prefix(n, sh);
    for (int i = max(first - before, 0); i < n && before + i < end; ++i) {
      const unsigned at = before + i - first;
      if (at >= M) break;   // (counts of offsets out of order may pass 32 bits)
      s_row[at] = row + i;
    }
    base += sh.chunk_total;
    __syncthreads();
  }
}

// VEC: rows and weights lie on 16-byte boundaries, parts and the width are multiples of 16 bytes.
// NT: 8-column tiles of low-rank columns that a warp holds (those behind the last repeat it).
template <typename T, int R, int NT, bool VEC>
__global__ void __launch_bounds__(kAdapterThreads, 2) adapter_kernel(const __grid_constant__ AdapterParams p) {
  constexpr int M = kAdapterTile;
  constexpr bool F32 = std::is_same<T, float>::value;
  constexpr int V = 16 / (int)sizeof(T);           // elements of 16 bytes
  constexpr int KB = 4 * V;                        // of the contraction a warp takes at once: 16 bytes a lane
  constexpr int STEPS = F32 ? R / 8 : R < 16 ? 1 : R / 16;   // instructions deep, of the expansion
  extern __shared__ __align__(16) char smem[];
  __shared__ AdapterShared sh;
  __shared__ int s_row[M];
  __shared__ int s_from[M];                        // rows to read: places without one read the tile's first
  __shared__ float s_scale[M * kMaxParts];         // f16: of a row's low-rank numbers, and back
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int rank = (int)cluster_rank(), log_ranks = p.log_ranks, ranks = 1 << log_ranks;
  const int tile = (int)(blockIdx.x >> log_ranks);
  const int low = p.parts * R, pitch = p.pitch;    // low-rank columns
  pdl_launch_dependents();                         // (the tall kernels' rows are others)

  const T* y = static_cast<const T*>(p.y);
  T* out = static_cast<T*>(p.out);
  AdapterRequest own;
  if (tid < M) s_row[tid] = -1;
  find_tile(p, tile, reinterpret_cast<int*>(smem), own, sh);
  const int adapter = min(max(sh.adapter, 0), p.adapters);
  if (adapter == p.adapters) {
    // no adapter: the clusters behind the last tile copy such rows, 16 at a time in turn
    const int copiers = (int)(gridDim.x >> log_ranks) - tile + sh.first;   // (tiles ahead: tile - sh.first)
    for (long long first = (long long)sh.first * M; p.copy && first < sh.count; first += (long long)copiers * M) {
      rows_of_tile(p, adapter, (int)first, sh.count, own, s_row, sh);
      for (int m = warp; m < M && s_row[m] >= 0; m += kAdapterWarps) {
        const T* from = y + s_row[m] * p.y_rs;
        T* to = out + s_row[m] * p.out_rs;
        const int c1 = p.starts[p.parts];
        for (int c = (rank * 32 + lane) * V; c < c1; c += 32 * V * ranks) {
          const uint4 v = load16<T>(from, c, c1 - c, VEC ? 16 : p.y_unit);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          store16<T>(to + c, c1 - c, VEC ? 16 : p.y_unit, w);
        }
      }
      __syncthreads();
      if (tid < M) s_row[tid] = -1;
      __syncthreads();
    }
    return;   // (the whole cluster)
  }
  rows_of_tile(p, adapter, sh.first, sh.count, own, s_row, sh);
  if (tid < M) s_from[tid] = min(max(s_row[tid] < 0 ? s_row[0] : s_row[tid], 0), p.rows - 1);
  __syncthreads();

  // the cluster's shares: of the width in blocks of KB, of the columns in chunks of 32
  const int blocks = (p.width + KB - 1) / KB, chunks = p.chunks[p.parts];
  const int k0 = blocks * rank >> log_ranks, k1 = blocks * (rank + 1) >> log_ranks;
  const int h0 = chunks * rank >> log_ranks, h1 = chunks * (rank + 1) >> log_ranks;
  auto part_of = [&](int h) {
    int s = 0;
    while (s + 1 < p.parts && h >= p.chunks[s + 1]) ++s;
    return s;
  };

  const T* a = static_cast<const T*>(p.a) + (long long)adapter * low * p.width;
  const T* b = static_cast<const T*>(p.b) + (long long)adapter * p.starts[p.parts] * R;

  float* s_part = reinterpret_cast<float*>(smem);
  const int k_groups = kAdapterWarps / p.n_groups;
  const size_t head = max(((size_t)(p.adapters + 1) * 4 + 15) / 16 * 16, (size_t)k_groups * M * pitch * 4);
  float* s_sum = reinterpret_cast<float*>(smem + head);
  uint4* s_frag = reinterpret_cast<uint4*>(s_sum + M * pitch);

  // ---- contraction: low[m][n] = sum over k of x[m][k] a[n][k]
  {
    const int kg = warp / p.n_groups, ng = warp % p.n_groups;
    float acc[NT][4];
    // (what places behind the tile's rows and low-rank columns hold is never looked at: they read others')
    const T* xr[2];
#pragma unroll
    for (int o = 0; o < 2; ++o) xr[o] = static_cast<const T*>(p.x) + s_from[8 * o + g] * p.x_rs;
    const int n0 = ng * NT * 8 + g;
    auto contract = [&](auto careful) {
      constexpr bool CAREFUL = decltype(careful)::value;
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll(CAREFUL ? 1 : 2)
      for (int kb = k0 + kg; kb < k1; kb += k_groups) {
        const int k = kb * KB + q * V, left = p.width - k;
        uint4 xv[2], av[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
          av[j] = load16<T>(a + (long long)min(n0 + j * 8, low - 1) * p.width, k, left, VEC ? 16 : p.x_unit);
#pragma unroll
        for (int o = 0; o < 2; ++o) xv[o] = load16<T>(xr[o], k, left, VEC ? 16 : p.x_unit);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if constexpr (!F32) {
            const uint32_t f[4] = {s ? xv[0].z : xv[0].x, s ? xv[1].z : xv[1].x, s ? xv[0].w : xv[0].y,
                                   s ? xv[1].w : xv[1].y};
#pragma unroll
            for (int j = 0; j < NT; ++j) mma16x8<T>(acc[j], f, s ? av[j].z : av[j].x, s ? av[j].w : av[j].y);
          } else {
            // each factor as two tf32 numbers
            uint32_t ah[NT][2], al[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              split_tf32<CAREFUL>(__uint_as_float(s ? av[j].z : av[j].x), ah[j][0], al[j][0]);
              split_tf32<CAREFUL>(__uint_as_float(s ? av[j].w : av[j].y), ah[j][1], al[j][1]);
            }
            uint32_t hi[4], lo[4];
            split_tf32<CAREFUL>(__uint_as_float(s ? xv[0].z : xv[0].x), hi[0], lo[0]);
            split_tf32<CAREFUL>(__uint_as_float(s ? xv[1].z : xv[1].x), hi[1], lo[1]);
            split_tf32<CAREFUL>(__uint_as_float(s ? xv[0].w : xv[0].y), hi[2], lo[2]);
            split_tf32<CAREFUL>(__uint_as_float(s ? xv[1].w : xv[1].y), hi[3], lo[3]);
#pragma unroll
            for (int j = 0; j < NT; ++j) add_products<CAREFUL>(acc[j], hi, lo, ah[j], al[j]);
          }
        }
      }
    };
    contract(std::false_type());
    if constexpr (F32) {
      if (any_not_finite<NT>(acc)) contract(std::true_type());
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = (ng * NT + j) * 8 + 2 * q;
      if (n >= low) continue;
      float* to = s_part + ((size_t)kg * M + g) * pitch + n;
      *reinterpret_cast<float2*>(to) = make_float2(acc[j][0], acc[j][1]);
      *reinterpret_cast<float2*>(to + 8 * pitch) = make_float2(acc[j][2], acc[j][3]);
    }
  }
  __syncthreads();
  if (k_groups > 1) {
    for (int i = tid; i < M * (low / 4); i += kAdapterThreads) {
      const int m = i / (low / 4), n = (i - m * (low / 4)) * 4;
      float4* at = reinterpret_cast<float4*>(s_part + (size_t)m * pitch + n);
      float4 v = *at;
      for (int k = 1; k < k_groups; ++k) {
        const float4 w = *reinterpret_cast<const float4*>(s_part + ((size_t)k * M + m) * pitch + n);
        v.x += w.x;
        v.y += w.y;
        v.z += w.z;
        v.w += w.w;
      }
      *at = v;
    }
  }
  // The expansion's chunks of 32 columns, as a lane holds them: y of its rows, and weights where they are few. AHEAD
  // of them are on their way, the first from here on.
  constexpr int YV = 8 / V;                     // 16-byte pieces of 8 columns
  constexpr int BLK = R < KB ? 1 : R / KB;      // weights: blocks of 16 bytes a lane,
  constexpr int PER = STEPS / BLK;              // of as many steps,
  constexpr int BW = R * (int)sizeof(T) >= 64 ? 4 : R * (int)sizeof(T) / 16;   // of as many words
  constexpr bool B_TOO = 4 * BLK * BW <= 32;
  constexpr int REGS = 2 * YV * 4 + (B_TOO ? 4 * BLK * BW : 0), ROOM = F32 ? 24 : 56;
  constexpr int AHEAD = ROOM / REGS < 1 ? 1 : ROOM / REGS > 3 ? 3 : ROOM / REGS;
  struct Chunk {
    uint4 y[2][YV];
    uint32_t b[B_TOO ? BLK : 1][4][BW];
  };
  auto load_b = [&](const T* b, int col0, int end, int blk, uint32_t (*bw)[BW]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // (columns behind the part's end read its last one's)
      const T* bc = b + (long long)min(col0 + (g >> 1) * 8 + 2 * j + (g & 1), end - 1) * R;
      if constexpr (BW == 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(bc + blk * KB) + q);
        bw[j][0] = v.x, bw[j][1] = v.y, bw[j][2] = v.z, bw[j][3] = v.w;
      } else if constexpr (BW == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(bc) + q);
        bw[j][0] = v.x, bw[j][1] = v.y;
      } else {
        bw[j][0] = __ldg(reinterpret_cast<const uint32_t*>(bc) + q);
      }
    }
  };
  auto load_chunk = [&](int h, Chunk& c) {
    const int s = part_of(h), col0 = p.starts[s] + (h - p.chunks[s]) * 32, end = p.starts[s + 1];
    const int mine = col0 + q * 8;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const T* from = y + s_from[8 * o + g] * p.y_rs;
#pragma unroll
      for (int w = 0; w < YV; ++w) c.y[o][w] = load16<T>(from, mine + w * V, end - mine - w * V, VEC ? 16 : p.y_unit);
    }
    if constexpr (B_TOO) {
#pragma unroll
      for (int blk = 0; blk < BLK; ++blk) load_b(b, col0, end, blk, c.b[blk]);
    }
  };
  Chunk chunk[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i)
    if (h0 + warp + i * kAdapterWarps < h1) load_chunk(h0 + warp + i * kAdapterWarps, chunk[i]);

  if (ranks > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }

  // ---- the sums over the cluster, of the parts that this CTA's columns lie in
  const int part0 = h0 < h1 ? part_of(h0) : 0, part1 = h0 < h1 ? part_of(h1 - 1) + 1 : 0;
  const int wide4 = (part1 - part0) * R / 4;
  for (int i = tid; i < M * wide4; i += kAdapterThreads) {
    const int m = i / wide4, n = part0 * R + (i - m * wide4) * 4;
    const float* at = s_part + (size_t)m * pitch + n;
    float4 v = *reinterpret_cast<const float4*>(at);
    if (ranks > 1) {
      float4 w[8];   // all on their way before the first is added
#pragma unroll
      for (int r = 0; r < 8; ++r) w[r] = r < ranks ? load_of_rank(at, r) : make_float4(0.f, 0.f, 0.f, 0.f);
      v = w[0];
#pragma unroll
      for (int r = 1; r < 8; ++r) {
        v.x += w[r].x;
        v.y += w[r].y;
        v.z += w[r].z;
        v.w += w[r].w;
      }
    }
    *reinterpret_cast<float4*>(s_sum + (size_t)m * pitch + n) = v;
  }
  if (ranks > 1) cluster_arrive();   // (waited for at the end: nobody leaves while its sums are read)
  __syncthreads();
  if constexpr (std::is_same<T, __half>::value) {
    // f16 ends at 65504: a row's numbers are taken by a power of two to below 2^8, and less than 2^-32 of the
    // largest is lost; the product is taken back by it.
    for (int i = warp; i < M * (part1 - part0); i += kAdapterWarps) {
      const int m = i / (part1 - part0), s = part0 + i - m * (part1 - part0);
      float most = 0.f;
      for (int n = lane; n < R; n += 32) most = most_finite(most, s_sum[(size_t)m * pitch + s * R + n]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      if (lane == 0) s_scale[m * kMaxParts + s] = low_rank_scale(most);
    }
    __syncthreads();
  }
  // as operands: what each lane holds of 16 rows and a step, the large parts and the small ones
  for (int i = tid; i < (part1 - part0) * STEPS * 32; i += kAdapterThreads) {
    const int l = i & 31, step = (i >> 5) % STEPS, s = part0 + (i >> 5) / STEPS;
    const int lg = l >> 2, lq = l & 3;
    const float* v0 = s_sum + (size_t)lg * pitch + s * R;
    const float* v1 = v0 + 8 * pitch;
    uint32_t hi[4], lo[4];
    if constexpr (F32) {
      const int k = R < 16 ? lq * 2 : (step >> 1) * 16 + lq * 4 + (step & 1) * 2;
      split_tf32<true>(v0[k], hi[0], lo[0]);
      split_tf32<true>(v1[k], hi[1], lo[1]);
      split_tf32<true>(v0[k + 1], hi[2], lo[2]);
      split_tf32<true>(v1[k + 1], hi[3], lo[3]);
    } else {
      float c0 = 1.f, c1 = 1.f;
      if constexpr (std::is_same<T, __half>::value) {
        c0 = s_scale[lg * kMaxParts + s];
        c1 = s_scale[(lg + 8) * kMaxParts + s];
      }
      if constexpr (R < 16) {
        split_pair<T>(v0[lq * 2] * c0, v0[lq * 2 + 1] * c0, hi[0], lo[0]);
        split_pair<T>(v1[lq * 2] * c1, v1[lq * 2 + 1] * c1, hi[1], lo[1]);
        hi[2] = hi[3] = lo[2] = lo[3] = 0u;
      } else {
        const int k = R < 32 ? lq * 4 : (step >> 1) * 32 + lq * 8 + (step & 1) * 4;
        split_pair<T>(v0[k] * c0, v0[k + 1] * c0, hi[0], lo[0]);
        split_pair<T>(v1[k] * c1, v1[k + 1] * c1, hi[1], lo[1]);
        split_pair<T>(v0[k + 2] * c0, v0[k + 3] * c0, hi[2], lo[2]);
        split_pair<T>(v1[k + 2] * c1, v1[k + 3] * c1, hi[3], lo[3]);
      }
    }
    uint4* to = s_frag + ((size_t)(s - part0) * STEPS + step) * 64 + l;
    to[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    to[32] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  __syncthreads();

  // ---- expansion: a warp 32 columns at once. Of 8-column tile j a lane holds columns 8 q + 2 j, 2 j + 1 of its
  // rows, so that its columns of the four tiles are neighbours.
  const float c_a = p.scales ? __ldg(p.scales + adapter) : 1.f;
  auto finish = [&](int h, const Chunk& now) {
    const int s = part_of(h), col0 = p.starts[s] + (h - p.chunks[s]) * 32, end = p.starts[s + 1];
    const int mine = col0 + q * 8, n_mine = min(end - mine, 8);   // (none there: below 1)
    float acc[4][4];
    const uint4* frag = s_frag + (size_t)(s - part0) * STEPS * 64 + lane;
    auto expand = [&](auto careful) {
      constexpr bool CAREFUL = decltype(careful)::value;
      const T* weights = b;
      const uint4* operand = frag;
      // (loaded again, then: kept from the first time they would fill the registers)
      if constexpr (CAREFUL) asm volatile("" : "+l"(weights), "+l"(operand));
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
      for (int blk = 0; blk < BLK; ++blk) {
        uint32_t bw[4][BW];
        if constexpr (!B_TOO) load_b(weights, col0, end, blk, bw);
        else memcpy(bw, now.b[blk], sizeof bw);
#pragma unroll
        for (int t = 0; t < PER; ++t) {
          uint32_t bh[4][2], bl[4][2];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t w = 2 * t + e < BW ? bw[j][2 * t + e] : 0u;
              if constexpr (F32) split_tf32<CAREFUL>(__uint_as_float(w), bh[j][e], bl[j][e]);
              else bh[j][e] = w;
            }
          const uint4* f = operand + (blk * PER + t) * 64;
          const uint4 fh = f[0], fl = f[32];
          const uint32_t hi[4] = {fh.x, fh.y, fh.z, fh.w}, lo[4] = {fl.x, fl.y, fl.z, fl.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (F32) {
              add_products<CAREFUL>(acc[j], hi, lo, bh[j], bl[j]);
            } else {
              mma16x8<T>(acc[j], lo, bh[j][0], bh[j][1]);
              mma16x8<T>(acc[j], hi, bh[j][0], bh[j][1]);
            }
          }
        }
      }
    };
    expand(std::false_type());
    if constexpr (F32) {
      if (any_not_finite<4>(acc)) expand(std::true_type());
    }
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const int m = 8 * o + g, r = s_row[m];
      if (r < 0 || n_mine <= 0) continue;
      float c = c_a;
      if constexpr (std::is_same<T, __half>::value) c = c_a / s_scale[m * kMaxParts + s];
      T* to = out + r * p.out_rs + mine;
      if constexpr (F32) {
        uint32_t v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint4 w = now.y[o][e / 4];
          v[e] = __float_as_uint(__uint_as_float(e % 4 == 0 ? w.x : e % 4 == 1 ? w.y : e % 4 == 2 ? w.z : w.w) +
                                 c * acc[e / 2][2 * o + (e & 1)]);
        }
        store16<T>(to, n_mine, VEC ? 16 : p.y_unit, v);
        store16<T>(to + 4, n_mine - 4, VEC ? 16 : p.y_unit, v + 4);
      } else {
        const uint32_t in[4] = {now.y[o][0].x, now.y[o][0].y, now.y[o][0].z, now.y[o][0].w};
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float y0, y1;
          if constexpr (std::is_same<T, __half>::value) {
            __half2 hv;
            memcpy(&hv, &in[j], 4);
            const float2 f = __half22float2(hv);
            y0 = f.x;
            y1 = f.y;
          } else {
            y0 = __uint_as_float(in[j] << 16);
            y1 = __uint_as_float(in[j] & 0xffff0000u);
          }
          w[j] = pack2(y0 + c * acc[j][2 * o], y1 + c * acc[j][2 * o + 1], T());
        }
        store16<T>(to, n_mine, VEC ? 16 : p.y_unit, w);
      }
    }
  };
#pragma unroll 1
  for (int h = h0 + warp; h < h1; h += AHEAD * kAdapterWarps) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int hh = h + i * kAdapterWarps;
      if (hh >= h1) break;
      const Chunk now = chunk[i];
      if (hh + AHEAD * kAdapterWarps < h1) load_chunk(hh + AHEAD * kAdapterWarps, chunk[i]);
      finish(hh, now);
    }
  }
  if (ranks > 1) cluster_wait();
}

// The 8-column tiles of a warp, of `columns` of them in all: the fewest built that take them with 1, 2, 4 or 8 warps
// side by side (`groups`).
inline int adapter_tiles(int columns, int& groups) {
  groups = 1;
  while ((columns + groups - 1) / groups > 8) groups *= 2;
  const int each = (columns + groups - 1) / groups;
  return each <= 4 ? 4 : each <= 6 ? 6 : 8;
}

// The kernel of a rank and of `tiles` 8-column tiles a warp.
template <typename T, int R, int NT>
const void* adapter_kernel_of(bool vec) {
  return vec ? reinterpret_cast<const void*>(&adapter_kernel<T, R, NT, true>)
             : reinterpret_cast<const void*>(&adapter_kernel<T, R, NT, false>);
}
template <typename T, int R>
const void* adapter_kernel_of(int tiles, bool vec) {
  if constexpr (R >= 16) {   // (rank 8: at most 4 tiles in all)
    if (tiles == 6) return adapter_kernel_of<T, R, 6>(vec);
    if (tiles == 8) return adapter_kernel_of<T, R, 8>(vec);
  }
  return adapter_kernel_of<T, R, 4>(vec);
}
template <typename T>
const void* adapter_kernel_for(int rank, int tiles, bool vec) {
  return rank == 8    ? adapter_kernel_of<T, 8>(tiles, vec)
         : rank == 16 ? adapter_kernel_of<T, 16>(tiles, vec)
         : rank == 32 ? adapter_kernel_of<T, 32>(tiles, vec)
         : rank == 64 ? adapter_kernel_of<T, 64>(tiles, vec)
                      : adapter_kernel_of<T, 128>(tiles, vec);
}

const void* adapter_kernel_bf16(int rank, int tiles, bool vec);
const void* adapter_kernel_f16(int rank, int tiles, bool vec);
const void* adapter_kernel_f32(int rank, int tiles, bool vec);

}  // namespace da
