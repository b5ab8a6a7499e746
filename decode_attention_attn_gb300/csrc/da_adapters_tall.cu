// da_adapters_tall.cu -- adapters of requests with many rows (prompts), 16-bit types, on the 5th-generation
// tensor cores: two launches over tiles of 128 rows of one request.
//
//   contract   low[r] = x[r] A_a^T: tcgen05.mma 128 x (parts * rank) x 64, x and A by TMA into a ring, an even run of
//              the tiles' widths a CTA; its fp32 sums into the workspace.
//   expand     out[r, c..c+127] = y + c_a low[r] B_a^T: the CTAs' sums as 16-bit operands in tensor memory (two
//              parts: at most 2^-17 of a number is lost in bf16, 2^-23 in f16), B and y by TMA. A CTA walks a run
//              of column blocks, tile by tile: one warp loads, one issues, four put the next rows' operand together,
//              and two teams of four finish blocks in turn (a thread a row) and write them row by row.
//
// Bound by HBM: x is read once, y once, out written once (the weights and the low-rank sums stay in L2). 8800 rows
// in 16 prompts, 4096 to 6144 columns, rank 64: the bytes are 47 us at a copy's rate.
// Rows behind a request's end in its last tile read others' (or zeros) and are not written.
#include <algorithm>
#include <climits>

#include "da_adapters.cuh"
#include "da_plan.h"
#include "da_tcgen05.cuh"

namespace da {
namespace {

constexpr int kTallTile = 128;
constexpr int kContractThreads = 256;
constexpr int kMaxTileList = 1024;    // tiles of a CTA's run

// Rows of request b, if they are many and it has an adapter; else 0.
__device__ __forceinline__ int tall_rows(const AdapterParams& p, int b, int& first) {
  const int n = rows_of(p, b, first);
  return n >= p.tall && adapter_of(p, b) < p.adapters ? n : 0;
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

struct TileInfo {
  int row0, rows, adapter;
};

// A CTA's run of `per_tile` items a tile, [i0, i1) of n_tiles * per_tile, and its tiles (from t0 on) in list; `ctas`
// share the items evenly, at most `spread` a tile (0: all of them). False: it has none. By every thread of a block
// whose first 256 look through the requests.
struct Run {
  long long i0, i1, items;
  int t0, n_tiles, ctas;
};
// (no more CTAs than items, so that each one between a tile's first and last has some of it)
__device__ __forceinline__ int ctas_of(long long items, int n_tiles, int spread) {
  return (int)min((long long)gridDim.x, min((long long)spread * n_tiles, items));
}
// a / b, short where both are
__device__ __forceinline__ long long divide(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}
template <int THREADS>
__device__ bool find_run(const AdapterParams& p, const TallParams& q, int per_tile, int spread, AdapterShared& scan,
                         TileInfo* list, Run& r) {
  const int tid = threadIdx.x;
  int first0 = 0, n0 = 0, a0 = 0, before0 = 0;   // of the request that is the thread's first
  r.n_tiles = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kAdapterThreads) {
    const int b = b0 + tid;
    int first = 0, n = 0;
    if (tid < kAdapterThreads && b < p.batch) {
      n = tall_rows(p, b, first);
      if (b0 == 0) a0 = adapter_of(p, b);
    }
    const int before = wide_prefix((n + kTallTile - 1) / kTallTile, scan);
    r.n_tiles += scan.chunk_total;
    __syncthreads();
    if (b0 == 0) first0 = first, n0 = n, before0 = before;
  }
  // (more than offsets in order allow: nothing is done)
  if (r.n_tiles < 0 || r.n_tiles > q.most_tiles) r.n_tiles = 0;
  r.items = (long long)r.n_tiles * per_tile;
  r.ctas = spread ? ctas_of(r.items, r.n_tiles, spread) : (int)gridDim.x;
  if ((int)blockIdx.x >= r.ctas) return false;
  r.i0 = divide(r.items * blockIdx.x, r.ctas);
  r.i1 = divide(r.items * (blockIdx.x + 1), r.ctas);
  if (r.i0 == r.i1) return false;
  r.t0 = (int)divide(r.i0, per_tile);
  const int t1 = (int)divide(r.i1 - 1, per_tile);   // t1 - t0 < kMaxTileList: tall_fits
  for (int t = tid; t <= t1 - r.t0; t += THREADS) list[t] = TileInfo{0, 0, 0};
  __syncthreads();
  for (int b0 = 0, base = 0; b0 < p.batch && base <= t1; b0 += kAdapterThreads) {
    const int b = b0 + tid;
    int first = first0, n = n0, adapter = a0, before = before0;
    if (p.batch > kAdapterThreads) {
      n = 0;
      if (tid < kAdapterThreads && b < p.batch) {
        n = tall_rows(p, b, first);
        adapter = adapter_of(p, b);
      }
      before = base + wide_prefix((n + kTallTile - 1) / kTallTile, scan);
      base += scan.chunk_total;
      __syncthreads();
    }
    const int end = before + (n + kTallTile - 1) / kTallTile;
    for (int t = max(before, r.t0); t <= t1 && t < end; ++t) {
      const int at = (t - before) * kTallTile;
      list[t - r.t0] = TileInfo{first + at, min(n - at, kTallTile), adapter};
    }
  }
  return true;
}

// The CTA whose run holds item u.
__device__ __forceinline__ int owner(const Run& r, long long u) {
  return (int)divide((u + 1) * r.ctas + r.items - 1, r.items) - 1;
}

// ---- contract ----------------------------------------------------------------------------------
// Runs of 64-wide blocks of the tiles' widths, evenly over the CTAs wherever a tile ends, so that a tile's sums come
// from up to kTallPieces of them. What bounds it is the way from L2: 40 KB a block of rank 64's three parts, of which 24
// are weights, at 87 GB/s an SM (13 TB/s in all); 8800 rows 24 us. (Whole tiles split in shares, two CTAs an SM: 25 us;
// 256 rows beside one tile of weights, 56 KB a block, three in flight: 27 us.)
constexpr int kContractSpread = 6;    // CTAs a tile at most: a tile then meets at most 6 + 2 runs
constexpr uint32_t kContractCols = 512;
static_assert(kContractSpread + 2 <= kTallPieces, "");

struct ContractShared {
  uint64_t full[8], empty[8], acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort_flag;
  AdapterShared scan;
  TileInfo tiles[kMaxTileList];
};

// Dynamic shared memory: stages of [128 rows | n columns] x 64, 1 KB aligned; more than half of an SM's, so that a
// CTA has its tensor memory to itself.
template <typename T>
__global__ void __launch_bounds__(kContractThreads, 1)
    contract_kernel(const __grid_constant__ AdapterParams p, const __grid_constant__ TallParams q,
                    const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tma) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ ContractShared sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  pdl_launch_dependents();
  if (tid == 0) {
    sh.abort_flag = 0;
    for (int i = 0; i < q.stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.acc_full[i], 1);
      mbar_init(&sh.acc_empty[i], 4);
    }
    mbar_init(&sh.done, 1);
    fence_mbar_init();
  }
  const int blocks = (p.width + 63) / 64;
  Run run;
  if (!find_run<kContractThreads>(p, q, blocks, kContractSpread, sh.scan, sh.tiles, run)) {
    pdl_wait();   // (its end stands for that of the launch ahead too)
    return;
  }
  if (warp == 5) tmem_alloc(&sh.tmem, kContractCols);
  if (tid == 0 && (smem_u32(smem) & 1023u)) {   // the swizzled tiles need it: nothing may run elsewhere
    sh.abort_flag = 1;
    atomicOr(q.status, kStatusTimeout);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int low = p.parts * q.rank;
  const uint32_t x_bytes = kTallTile * 128u, stage_bytes = x_bytes + (uint32_t)q.n * 128u;
  Waiter wait{&sh.abort_flag, q.status, kWaitLimitNs, sh.abort_flag != 0};
  const int units = (int)(run.i1 - run.i0);
  int k = (int)(run.i0 % blocks), tile = 0;          // of the unit at hand
  if (warp == 4) {
    const bool issuer = elect_one();
    int slot = 0, issued = 0;
    uint32_t par = 1;
    for (int u = 0; u < units; ++u) {
      wait(&sh.empty[slot], par);
      if (!wait.dead) {
        if (issuer) {
          const TileInfo t = sh.tiles[tile];
          uint8_t* at = smem + slot * stage_bytes;
          mbar_arrive_expect_tx(&sh.full[slot], stage_bytes);
          tma_load_2d(at, &tmx, &sh.full[slot], k * 64, t.row0);
          tma_load_2d(at + x_bytes, &tma, &sh.full[slot], k * 64, t.adapter * low);
        }
        ++issued;
      }
      __syncwarp();
      if (++slot == q.stages) slot = 0, par ^= 1;
      if (++k == blocks) k = 0, ++tile;
    }
    // never leave with copies in flight
    for (int i = max(issued - q.stages, 0); i < issued; ++i)
      mbar_wait(&sh.full[i % q.stages], (i / q.stages) & 1, kWaitLimitNs);
  } else if (warp == 5) {
    const bool issuer = elect_one();
    const uint32_t desc = mma_desc(std::is_same<T, __nv_bfloat16>::value, q.n, false);
    const uint64_t xd = tile_desc(smem_u32(smem), 16, 1024), ad = tile_desc(smem_u32(smem + x_bytes), 16, 1024);
    int slot = 0;
    uint32_t par = 0;
    bool fresh = true;
    for (int u = 0; u < units; ++u) {
      const uint32_t buf = tile & 1, bpar = (tile >> 1) & 1;
      if (fresh) wait(&sh.acc_empty[buf], bpar ^ 1);
      wait(&sh.full[slot], par);
      tc_fence_after();
      const bool last = k + 1 == blocks || u + 1 == units;
      if (!wait.dead && issuer) {
        const uint32_t off = slot * (stage_bytes >> 4);
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_ss(tmem + buf * 256u, xd + off + 2 * s, ad + off + 2 * s, desc, !fresh || s != 0);
        tc_commit(&sh.empty[slot]);
        if (last) tc_commit(&sh.acc_full[buf]);
      }
      __syncwarp();
      fresh = last;
      if (++slot == q.stages) slot = 0, par ^= 1;
      if (++k == blocks) k = 0, ++tile;
    }
    if (issuer) tc_commit(&sh.done);
    mbar_wait(&sh.done, 0, kWaitLimitNs);
  } else if (warp < 4) {
    const int row = warp * 32 + lane;
    const int n_tiles = (k + units + blocks - 1) / blocks;
    for (; tile < n_tiles; ++tile) {
      const TileInfo t = sh.tiles[tile];
      const uint32_t buf = tile & 1, bpar = (tile >> 1) & 1;
      // whose run the tile's first block is in says which piece this is
      const int piece = (int)blockIdx.x - owner(run, (long long)(run.t0 + tile) * blocks);
      wait(&sh.acc_full[buf], bpar);
      tc_fence_after();
      float4* to = q.sums + (long long)piece * (low / 4) * p.rows + t.row0 + row;
      const bool there = row < t.rows && !wait.dead && piece >= 0 && piece < kTallPieces;
#pragma unroll 1
      for (int c = 0; c < low; c += 32) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(tmem + ((uint32_t)warp << 21) + buf * 256u + c, v);
        tmem_ready(v);
        if (there) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + 4 * e < low)
              to[(long long)(c / 4 + e) * p.rows] =
                  make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]), __uint_as_float(v[4 * e + 2]),
                              __uint_as_float(v[4 * e + 3]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_free(tmem, kContractCols);
  pdl_wait();
}

// ---- expand --------------------------------------------------------------------------------------
constexpr int kExpandTeams = 2;                       // of 4 warps, that finish blocks in turn
constexpr int kExpandThreads = (kExpandTeams * 4 + 4 + 2) * 32;
constexpr uint32_t kExpandCols = 512, kColD = 0, kColV = 256;

struct ExpandShared {
  uint64_t y_full[4], y_empty[4], b_full[4], b_empty[4], d_full[2], d_empty[2], v_full[2], v_empty[2], drained;
  uint32_t tmem;
  int abort_flag;
  AdapterShared scan;
  float scale[4][kTallTile];    // f16: of a row's low-rank numbers, four segments
  TileInfo tiles[kMaxTileList];
};

// The blocks of a CTA's run: tile by tile, the column blocks of each part. A segment is a run of blocks of one
// tile and part, whose operand is the same.
struct BlockWalk {
  int item, end, tile, block, part, seg;
  __device__ __forceinline__ BlockWalk(const TallParams& q, long long i0, long long i1)
      : item(0), end((int)(i1 - i0)), tile(0), block((int)(i0 % q.blocks[kMaxParts])), part(0), seg(0) {
    settle(q);
  }
  __device__ __forceinline__ void settle(const TallParams& q) {
    part = 0;
    while (part + 1 < kMaxParts && block >= q.blocks[part + 1]) ++part;
  }
  __device__ __forceinline__ bool more() const { return item < end; }
  // to the next block; whether it begins a segment
  __device__ __forceinline__ bool next(const TallParams& q) {
    ++item;
    const int before = part;
    bool fresh = false;
    if (++block == q.blocks[kMaxParts]) {
      block = 0;
      ++tile;
      fresh = true;
    }
    settle(q);
    fresh |= part != before;
    seg += fresh;
    return fresh;
  }
  __device__ __forceinline__ int column(const AdapterParams& p, const TallParams& q) const {
    return p.starts[part] + (block - q.blocks[part]) * 128;
  }
};

template <typename T, int R>
__global__ void __launch_bounds__(kExpandThreads, 1)
    expand_kernel(const __grid_constant__ AdapterParams p, const __grid_constant__ TallParams q,
                  const __grid_constant__ CUtensorMap tmy, const __grid_constant__ CUtensorMap tmb) {
  constexpr int RB = R < 16 ? 16 : R;                  // depth that the instructions take
  constexpr int STEPS = RB / 16;
  constexpr uint32_t B_ROW = RB >= 64 ? 128u : RB * 2u;    // bytes of a row of B's tile (the swizzle's width)
  constexpr uint32_t B_BYTES = 128u * RB * 2u;
  constexpr uint32_t V_COLS = R < 32 ? 32u : (uint32_t)R;
  constexpr uint32_t Y_BYTES = 32768u;
  constexpr int YS = 4, BS = R == 128 ? 2 : 4;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ ExpandShared sh;
  uint8_t* const y_ring = smem;
  uint8_t* const b_ring = smem + YS * Y_BYTES;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    sh.abort_flag = 0;
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.y_full[i], 1);
      mbar_init(&sh.y_empty[i], 4);
      mbar_init(&sh.b_full[i], 1);
      mbar_init(&sh.b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.d_full[i], 1);
      mbar_init(&sh.d_empty[i], 4);
      mbar_init(&sh.v_full[i], 4);
      mbar_init(&sh.v_empty[i], 1);
    }
    mbar_init(&sh.drained, 1);
    fence_mbar_init();
  }
  // (the requests are no result of the launch ahead)
  Run run;
  if (!find_run<kExpandThreads>(p, q, q.blocks[kMaxParts], 0, sh.scan, sh.tiles, run)) {
    pdl_wait();
    return;
  }
  if (tid == 0 && (smem_u32(smem) & 1023u)) {
    sh.abort_flag = 1;
    atomicOr(q.status, kStatusTimeout);
  }
  __syncthreads();
  Waiter wait{&sh.abort_flag, q.status, kWaitLimitNs, sh.abort_flag != 0};
  BlockWalk w(q, run.i0, run.i1);
  const int low = p.parts * R;

  if (warp == 12) {
    // ---- loads of y and B: they need nothing of the launch ahead -------------------------------------
    const bool issuer = elect_one();
    int ys = 0, bs = 0, issued = 0;
    uint32_t yp = 1, bp = 1;
    for (; w.more(); w.next(q)) {
      const TileInfo t = sh.tiles[w.tile];
      const int col = w.column(p, q);
      wait(&sh.b_empty[bs], bp);
      wait(&sh.y_empty[ys], yp);
      if (!wait.dead) {
        if (issuer) {
          uint8_t* at = b_ring + bs * B_BYTES;
          mbar_arrive_expect_tx(&sh.b_full[bs], B_BYTES);
          tma_load_2d(at, &tmb, &sh.b_full[bs], 0, t.adapter * p.starts[p.parts] + col);
          if constexpr (R == 128)
            tma_load_2d(at + 16384, &tmb, &sh.b_full[bs], 64, t.adapter * p.starts[p.parts] + col);
          at = y_ring + ys * Y_BYTES;
          mbar_arrive_expect_tx(&sh.y_full[ys], Y_BYTES);
          tma_load_2d(at, &tmy, &sh.y_full[ys], col, t.row0);
          tma_load_2d(at + 16384, &tmy, &sh.y_full[ys], col + 64, t.row0);
        }
        ++issued;
      }
      __syncwarp();
      if (++ys == YS) ys = 0, yp ^= 1;
      if (++bs == BS) bs = 0, bp ^= 1;
    }
    // never leave with copies in flight
    for (int k = max(issued - YS, 0); k < issued; ++k) mbar_wait(&sh.y_full[k % YS], (k / YS) & 1, kWaitLimitNs);
    for (int k = max(issued - BS, 0); k < issued; ++k) mbar_wait(&sh.b_full[k % BS], (k / BS) & 1, kWaitLimitNs);
    pdl_wait();
    __syncthreads();
    return;
  }
  // Tensor memory only after the wait for the launch ahead, whose CTAs may need it on this SM.
  pdl_wait();
  if (warp == 13) tmem_alloc(&sh.tmem, kExpandCols);
  tc_fence_before();
  named_bar_sync(1, kExpandThreads - 32);
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  if (warp == 13) {
    // ---- products --------------------------------------------------------------------------------------
    const bool issuer = elect_one();
    const uint32_t desc = mma_desc(std::is_same<T, __nv_bfloat16>::value, 128, false);
    constexpr uint64_t kSwizzle = B_ROW == 128 ? 2ull : B_ROW == 64 ? 4ull : 6ull;   // of 128, 64 or 32 bytes
    const uint64_t bd = (uint64_t)((smem_u32(b_ring) & 0x3ffffu) >> 4) | 1ull << 16 |
                        (uint64_t)(8u * B_ROW >> 4) << 32 | 1ull << 46 | kSwizzle << 61;
    int bs = 0;
    uint32_t bp = 0;
    bool fresh = true;
    while (w.more()) {
      const uint32_t vb = w.seg & 1, vpar = (w.seg >> 1) & 1, db = w.item & 1, dpar = (w.item >> 1) & 1;
      if (fresh) wait(&sh.v_full[vb], vpar);
      wait(&sh.d_empty[db], dpar ^ 1);
      wait(&sh.b_full[bs], bp);
      tc_fence_after();
      const int seg = w.seg;
      fresh = w.next(q);
      const bool last = !w.more() || w.seg != seg;
      if (!wait.dead && issuer) {
        const uint64_t at = bd + bs * (B_BYTES >> 4);
        const uint32_t v = tmem + kColV + vb * V_COLS, d = tmem + kColD + db * 128u;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
          mma_ts(d, v + 8u * s, at + (uint32_t)(s / 4) * (16384u >> 4) + (uint32_t)(s % 4) * 2u, desc, s != 0);
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
          mma_ts(d, v + RB / 2u + 8u * s, at + (uint32_t)(s / 4) * (16384u >> 4) + (uint32_t)(s % 4) * 2u, desc, true);
        tc_commit(&sh.d_full[db]);
        tc_commit(&sh.b_empty[bs]);
        if (last) tc_commit(&sh.v_empty[vb]);
      }
      __syncwarp();
      if (++bs == BS) bs = 0, bp ^= 1;
    }
    if (issuer) tc_commit(&sh.drained);
    mbar_wait(&sh.drained, 0, kWaitLimitNs);
  } else if (warp >= 8) {
    // ---- the rows' operand: the contraction's sums, in two 16-bit parts, large ones first ---------------------
    const int row = (warp - 8) * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(warp - 8) << 21) + kColV;
    const int per_tile = (p.width + 63) / 64;      // the contraction's run, as its CTAs had it
    Run sums;
    sums.items = (long long)run.n_tiles * per_tile;
    sums.ctas = ctas_of(sums.items, run.n_tiles, kContractSpread);
    while (w.more()) {
      const TileInfo t = sh.tiles[w.tile];
      const uint32_t vb = w.seg & 1, vpar = (w.seg >> 1) & 1;
      // the tile's pieces, in order (one's numbers all on their way before the next is added)
      const long long u0 = (long long)(run.t0 + w.tile) * per_tile;
      const int pieces = min(owner(sums, u0 + per_tile - 1) - owner(sums, u0) + 1, kTallPieces);
      const float4* from = q.sums + (long long)(w.part * R / 4) * p.rows + t.row0 + row;
      float v[R] = {};
      if (row < t.rows) {
#pragma unroll 1
        for (int k = 0; k < pieces; ++k, from += (long long)(low / 4) * p.rows) {
          float4 m[R / 4];
#pragma unroll
          for (int c = 0; c < R / 4; ++c) m[c] = from[(long long)c * p.rows];
#pragma unroll
          for (int c = 0; c < R / 4; ++c) {
            v[4 * c] += m[c].x;
            v[4 * c + 1] += m[c].y;
            v[4 * c + 2] += m[c].z;
            v[4 * c + 3] += m[c].w;
          }
        }
      }
      __syncwarp();
      float s = 1.f;
      if constexpr (std::is_same<T, __half>::value) {
        // f16 ends at 65504: by a power of two to below 2^8, and back in the product
        float most = 0.f;
#pragma unroll
        for (int k = 0; k < R; ++k) most = most_finite(most, v[k]);
        s = low_rank_scale(most);
#pragma unroll
        for (int k = 0; k < R; ++k) v[k] *= s;
      }
      uint32_t o[V_COLS] = {};
#pragma unroll
      for (int k = 0; k < R / 2; ++k) split_pair<T>(v[2 * k], v[2 * k + 1], o[k], o[RB / 2 + k]);
      wait(&sh.v_empty[vb], vpar ^ 1);
      // The scale's place was segment seg - 4's, and is free only now: seg - 2's products are done, the last of them
      // two blocks or more behind seg - 4's last one, and a block's product waits (d_empty) until the block two before
      // it has been finished. Before the wait seg - 3's alone are known to be, which may be a single block, with
      // seg - 4's last one still waiting for its y.
      if constexpr (std::is_same<T, __half>::value) sh.scale[w.seg & 3][row] = s;
      tc_fence_after();
#pragma unroll
      for (uint32_t c = 0; c < V_COLS; c += 32) tmem_st32(lane_addr + vb * V_COLS + c, o + c);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.v_full[vb]);
      while (w.more() && !w.next(q)) {
      }
    }
  } else {
    // ---- a team finishes every other block ----------------------------------------------------------------
    const int team = warp >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)quarter << 21) + kColD;
    int ys = 0;
    uint32_t yp = 0;
    for (; w.more(); w.next(q)) {
      if ((w.item & 1) == team) {
        const TileInfo t = sh.tiles[w.tile];
        const uint32_t db = w.item & 1, dpar = (w.item >> 1) & 1;
        const int col = w.column(p, q), end = p.starts[w.part + 1];
        uint8_t* const ytile = y_ring + ys * Y_BYTES;
        float c = p.scales ? __ldg(p.scales + t.adapter) : 1.f;
        wait(&sh.d_full[db], dpar);
        tc_fence_after();
        wait(&sh.y_full[ys], yp);
        if constexpr (std::is_same<T, __half>::value) c /= sh.scale[w.seg & 3][row];
#pragma unroll 1
        for (int h = 0; h < 4; ++h) {
          uint32_t d[32];
          __syncwarp();
          tmem_ld32(lane_addr + db * 128u + h * 32, d);
          tmem_ready(d);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint4* at = reinterpret_cast<uint4*>(ytile + (h >> 1) * 16384 + row * 128 +
                                                 ((((h & 1) * 4 + k) ^ (row & 7)) << 4));
            const uint4 y = *at;
            const uint32_t in[4] = {y.x, y.y, y.z, y.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = unpack_pair<T>(in[e]);
              o[e] = pack_pair<T>(fmaf(c, __uint_as_float(d[8 * k + 2 * e]), f.x),
                                  fmaf(c, __uint_as_float(d[8 * k + 2 * e + 1]), f.y));
            }
            *at = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.d_empty[db]);
        // the warp's rows out, two to an instruction
        const int box = (lane >> 3) & 1, chunk = lane & 7;
        T* to = static_cast<T*>(p.out) + col + (lane & 15) * 8;
        const bool inside = col + (lane & 15) * 8 < end && !wait.dead;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          const int r = quarter * 32 + 2 * i + (lane >> 4);
          const uint4 v = *reinterpret_cast<const uint4*>(ytile + box * 16384 + r * 128 + ((chunk ^ (r & 7)) << 4));
          if (inside && r < t.rows) *reinterpret_cast<uint4*>(to + (t.row0 + r) * p.out_rs) = v;
        }
        fence_async_smem();   // (the slot is the loads' again)
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.y_empty[ys]);
      }
      if (++ys == YS) ys = 0, yp ^= 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 13) tmem_free(tmem, kExpandCols);
}

template <typename T>
const void* expand_for(int rank) {
  switch (rank) {
    case 8: return reinterpret_cast<const void*>(&expand_kernel<T, 8>);
    case 16: return reinterpret_cast<const void*>(&expand_kernel<T, 16>);
    case 32: return reinterpret_cast<const void*>(&expand_kernel<T, 32>);
    case 64: return reinterpret_cast<const void*>(&expand_kernel<T, 64>);
    case 128: return reinterpret_cast<const void*>(&expand_kernel<T, 128>);
    default: return nullptr;
  }
}

int map_2d(CUtensorMap* map, const void* base, long long inner, long long outer, long long stride_bytes, int box_inner,
           int box_outer, CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promote) {
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer}, strides[1] = {(cuuint64_t)stride_bytes};
  const cuuint32_t box[2] = {(cuuint32_t)box_inner, (cuuint32_t)box_outer};
  return encode_map(map, 2, 2, base, dims, strides, box, swizzle, promote);
}

int launch_with(const void* fn, int grid, int threads, size_t smem, bool dependent, cudaStream_t stream, void** args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = dependent ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  return e == cudaSuccess ? DA_OK : cuda_fail(e, "launching the tall adapter kernels");
}

}  // namespace

// Rows of a request fill tiles but for its last one; requests with fewer than kTallRows have none.
long long most_tall_tiles(const AdapterParams& p) {
  return p.rows / kTallTile + std::min(p.batch, p.rows / kTallRows);
}

size_t tall_workspace(int rows, int low) {
  return kTallStatusBytes + (size_t)kTallPieces * low * rows * sizeof(float);
}

int launch_tall(const AdapterParams& p, int rank, bool bf16, int sms, void* workspace, const cudaLaunchConfig_t& first,
                const void* fn) {
  const int low = p.parts * rank, columns = p.starts[p.parts];
  TallParams q = {};
  q.rank = rank;
  q.status = static_cast<int32_t*>(workspace);
  q.sums = reinterpret_cast<float4*>(static_cast<char*>(workspace) + kTallStatusBytes);
  q.n = (low + 15) / 16 * 16;
  const int stage = kTallTile * 128 + q.n * 128;
  q.stages = std::min(8, 200 * 1024 / stage);   // 147 KB and more
  for (int s = 0; s < kMaxParts; ++s)
    q.blocks[s + 1] = q.blocks[s] + (s < p.parts ? (p.starts[s + 1] - p.starts[s] + 127) / 128 : 0);
  for (int s = p.parts; s < kMaxParts; ++s) q.blocks[s] = q.blocks[kMaxParts];   // (no part begins there)
  CUtensorMap tmx, tma, tmy, tmb;
  const int rb = std::max(rank, 16);
  const CUtensorMapL2promotion next = CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
  int rc = map_2d(&tmx, p.x, p.width, p.rows, p.x_rs * 2, 64, kTallTile, CU_TENSOR_MAP_SWIZZLE_128B, next);
  if (rc == DA_OK)
    rc = map_2d(&tma, p.a, p.width, (long long)p.adapters * low, p.width * 2ll, 64, q.n, CU_TENSOR_MAP_SWIZZLE_128B,
                next);
  if (rc == DA_OK) rc = map_2d(&tmy, p.y, columns, p.rows, p.y_rs * 2, 64, kTallTile, CU_TENSOR_MAP_SWIZZLE_128B, next);
  if (rc == DA_OK)
    rc = map_2d(&tmb, p.b, rank, (long long)p.adapters * columns, rank * 2ll, std::min(rb, 64), 128,
                rb >= 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                : rb == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                           : CU_TENSOR_MAP_SWIZZLE_32B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
  if (rc != DA_OK) return rc;
  const void* contract = bf16 ? reinterpret_cast<const void*>(&contract_kernel<__nv_bfloat16>)
                              : reinterpret_cast<const void*>(&contract_kernel<__half>);
  const void* expand = bf16 ? expand_for<__nv_bfloat16>(rank) : expand_for<__half>(rank);
  const size_t contract_smem = (size_t)q.stages * stage;
  const size_t expand_smem = 4 * 32768 + (rank == 128 ? 2 : 4) * (size_t)128 * rb * 2;
  rc = raise_smem(contract, 200 * 1024, 0);
  if (rc == DA_OK) rc = raise_smem(expand, expand_smem, 0);
  if (rc != DA_OK) return rc;
  q.most_tiles = (int)most_tall_tiles(p);
  AdapterParams pp = p;
  // (nothing is enqueued before all that can fail has been prepared)
  void* fargs[1] = {&pp};
  const cudaError_t e = cudaLaunchKernelExC(&first, fn, fargs);
  if (e != cudaSuccess) return cuda_fail(e, "launching the adapter kernel");
  const cudaStream_t stream = first.stream;
  void* cargs[4] = {&pp, &q, &tmx, &tma};
  rc = launch_with(contract, sms, kContractThreads, contract_smem, true, stream, cargs);
  if (rc != DA_OK) return rc;
  void* eargs[4] = {&pp, &q, &tmy, &tmb};
  return launch_with(expand, sms, kExpandThreads, expand_smem, true, stream, eargs);
}

bool tall_fits(const AdapterParams& p, int rank, int sms) {
  const int low = p.parts * rank, columns = p.starts[p.parts];
  const long long tiles = most_tall_tiles(p);
  return low <= 256 && p.x_rs >= p.width && p.y_rs >= columns && p.x_rs < (1ll << 38) && p.y_rs < (1ll << 38) &&
         (long long)p.adapters * columns < INT_MAX - 256 && (long long)p.adapters * low < INT_MAX - 256 &&
         tiles < (1 << 24) && tiles / sms + 2 < kMaxTileList;
}

}  // namespace da
