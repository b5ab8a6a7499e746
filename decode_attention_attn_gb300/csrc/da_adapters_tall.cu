// da_adapters_tall.cu -- adapters of requests with many rows (prompts), 16-bit types, on the 5th-generation
// tensor cores: two launches over tiles of 128 rows of one request.
//
//   contract   low[r] = x[r] A_a^T: tcgen05.mma 128 x (parts * rank) x 64, x and A by TMA into a ring, a share of the
//              width a CTA; fp32 sums of every share into the workspace.
//   expand     out[r, c..c+127] = y + c_a low[r] B_a^T: the shares' sums as 16-bit operands in tensor memory (two
//              parts, so that nothing of fp32's order is lost), B and y by TMA. A CTA walks a run of column blocks,
//              tile by tile: one warp loads, one issues, four put the next rows' operand together, and two teams of
//              four finish blocks in turn (a thread a row) and write them row by row.
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

// Tiles of request b: as many as its rows fill, if they are many and it has an adapter.
__device__ __forceinline__ int tall_tiles(const AdapterParams& p, int b, int& first, int& n) {
  n = rows_of(p, b, first);
  return n >= p.tall && adapter_of(p, b) < p.adapters ? (n + kTallTile - 1) / kTallTile : 0;
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

// ---- contract ----------------------------------------------------------------------------------
struct ContractShared {
  uint64_t full[8], empty[8], done;
  uint32_t tmem;
  int abort_flag;
  int row0, rows, adapter;
  AdapterShared scan;
};

// grid: tile bound * shares. Dynamic shared memory: stages of [128 rows | n columns] x 64, 1 KB aligned.
template <typename T>
__global__ void __launch_bounds__(kContractThreads, 1)
    contract_kernel(const __grid_constant__ AdapterParams p, const __grid_constant__ TallParams q,
                    const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tma) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ ContractShared sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  pdl_launch_dependents();
  const int tile = blockIdx.x / q.shares, share = blockIdx.x % q.shares;
  if (tid == 0) {
    sh.adapter = -1;
    sh.abort_flag = 0;
    for (int i = 0; i < q.stages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.done, 1);
    fence_mbar_init();
  }
  __syncthreads();
  for (int b0 = 0, base = 0; b0 < p.batch; b0 += kContractThreads) {
    const int b = b0 + tid;
    int first = 0, n = 0;
    const int tiles = b < p.batch ? tall_tiles(p, b, first, n) : 0;
    const int before = base + block_prefix(tiles, sh.scan);
    if (before <= tile && tile < before + tiles) {
      sh.row0 = first + (tile - before) * kTallTile;
      sh.rows = min(n - (tile - before) * kTallTile, kTallTile);
      sh.adapter = adapter_of(p, b);
    }
    base += sh.scan.chunk_total;
    __syncthreads();
    if (base > tile) break;
  }
  const int adapter = sh.adapter;
  if (adapter < 0) {   // fewer tiles: nothing here may end before the launch ahead has
    pdl_wait();
    return;
  }
  if (warp == 5) tmem_alloc(&sh.tmem, q.tmem_cols);
  if (tid == 0 && (smem_u32(smem) & 1023u)) {   // the swizzled tiles need it: nothing may run elsewhere
    sh.abort_flag = 1;
    atomicOr(q.status, kStatusTimeout);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int low = p.parts * q.rank;
  const int blocks = (p.width + 63) / 64;
  const int k0 = (int)((long long)blocks * share / q.shares), k1 = (int)((long long)blocks * (share + 1) / q.shares);
  const uint32_t stage_bytes = 16384u + (uint32_t)q.n * 128u;
  Waiter wait{&sh.abort_flag, q.status, kWaitLimitNs, sh.abort_flag != 0};
  if (warp == 4) {
    const bool issuer = elect_one();
    int slot = 0, issued = 0;
    uint32_t par = 1;
    for (int k = k0; k < k1; ++k) {
      wait(&sh.empty[slot], par);
      if (!wait.dead) {
        if (issuer) {
          uint8_t* at = smem + slot * stage_bytes;
          mbar_arrive_expect_tx(&sh.full[slot], stage_bytes);
          tma_load_2d(at, &tmx, &sh.full[slot], k * 64, sh.row0);
          tma_load_2d(at + 16384, &tma, &sh.full[slot], k * 64, adapter * low);
        }
        ++issued;
      }
      __syncwarp();
      if (++slot == q.stages) slot = 0, par ^= 1;
    }
    // never leave with copies in flight
    for (int k = max(issued - q.stages, 0); k < issued; ++k)
      mbar_wait(&sh.full[k % q.stages], (k / q.stages) & 1, kWaitLimitNs);
  } else if (warp == 5) {
    const bool issuer = elect_one();
    const uint32_t desc = mma_desc(std::is_same<T, __nv_bfloat16>::value, q.n, false);
    const uint64_t xd = tile_desc(smem_u32(smem), 16, 1024), ad = tile_desc(smem_u32(smem + 16384), 16, 1024);
    int slot = 0;
    uint32_t par = 0;
    for (int k = k0; k < k1; ++k) {
      wait(&sh.full[slot], par);
      tc_fence_after();
      if (!wait.dead && issuer) {
        const uint32_t off = slot * (stage_bytes >> 4);
#pragma unroll
        for (int s = 0; s < 4; ++s) mma_ss(tmem, xd + off + 2 * s, ad + off + 2 * s, desc, k != k0 || s != 0);
        tc_commit(&sh.empty[slot]);
      }
      __syncwarp();
      if (++slot == q.stages) slot = 0, par ^= 1;
    }
    if (issuer) tc_commit(&sh.done);
    mbar_wait(&sh.done, 0, kWaitLimitNs);
  } else if (warp < 4) {
    wait(&sh.done, 0);
    tc_fence_after();
    const int row = warp * 32 + lane;
    float4* to = q.sums + (long long)share * (low / 4) * p.rows + sh.row0 + row;
#pragma unroll 1
    for (int c = 0; c < low; c += 32) {
      uint32_t v[32];
      __syncwarp();
      tmem_ld32(tmem + ((uint32_t)warp << 21) + c, v);
      tmem_ready(v);
      if (row < sh.rows && !wait.dead) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (c + 4 * k < low)
            to[(long long)(c / 4 + k) * p.rows] =
                make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]), __uint_as_float(v[4 * k + 2]),
                            __uint_as_float(v[4 * k + 3]));
      }
    }
    __syncwarp();
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_free(tmem, q.tmem_cols);
  pdl_wait();   // (its end stands for that of the launch ahead too)
}

// ---- expand --------------------------------------------------------------------------------------
constexpr int kExpandTeams = 2;                       // of 4 warps, that finish blocks in turn
constexpr int kExpandThreads = (kExpandTeams * 4 + 4 + 2) * 32;
constexpr uint32_t kExpandCols = 512, kColD = 0, kColV = 256;

struct TileInfo {
  int row0, rows, adapter;
};
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
  // how many tiles there are, and those of this CTA's run (inputs of the launches ahead, not theirs to write)
  int n_tiles = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kAdapterThreads) {   // (256 threads' prefix: the others bring nothing)
    const int b = b0 + tid;
    int first, n;
    const int tiles = tid < kAdapterThreads && b < p.batch ? tall_tiles(p, b, first, n) : 0;
    wide_prefix(tiles, sh.scan);
    n_tiles += sh.scan.chunk_total;
    __syncthreads();
  }
  // (more than offsets in order allow: nothing is done)
  const long long items = n_tiles < 0 || n_tiles > q.most_tiles ? 0 : (long long)n_tiles * q.blocks[kMaxParts];
  const long long i0 = items * blockIdx.x / gridDim.x, i1 = items * (blockIdx.x + 1) / gridDim.x;
  if (i0 == i1) {
    pdl_wait();
    return;
  }
  for (int t = tid; t < kMaxTileList; t += kExpandThreads) sh.tiles[t] = TileInfo{0, 0, 0};
  __syncthreads();
  const int t0 = (int)(i0 / q.blocks[kMaxParts]), t1 = (int)((i1 - 1) / q.blocks[kMaxParts]);
  for (int b0 = 0, base = 0; b0 < p.batch && base <= t1; b0 += kAdapterThreads) {
    const int b = b0 + tid;
    int first = 0, n = 0;
    const int tiles = tid < kAdapterThreads && b < p.batch ? tall_tiles(p, b, first, n) : 0;
    const int before = base + wide_prefix(tiles, sh.scan);
    for (int t = max(before, t0); t <= t1 && t < before + tiles; ++t)   // (t1 - t0 < kMaxTileList: tall_fits)
      sh.tiles[t - t0] = TileInfo{first + (t - before) * kTallTile, min(n - (t - before) * kTallTile, kTallTile),
                                  adapter_of(p, b)};
    base += sh.scan.chunk_total;
    __syncthreads();
  }
  if (tid == 0 && (smem_u32(smem) & 1023u)) {
    sh.abort_flag = 1;
    atomicOr(q.status, kStatusTimeout);
  }
  __syncthreads();
  Waiter wait{&sh.abort_flag, q.status, kWaitLimitNs, sh.abort_flag != 0};
  BlockWalk w(q, i0, i1);
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
    // ---- the rows' operand: the shares' sums, in two 16-bit parts, large ones first ---------------------
    const int row = (warp - 8) * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(warp - 8) << 21) + kColV;
    while (w.more()) {
      const TileInfo t = sh.tiles[w.tile];
      const uint32_t vb = w.seg & 1, vpar = (w.seg >> 1) & 1;
      const float4* from = q.sums + (long long)(w.part * R / 4) * p.rows + t.row0 + row;
      // (a share's numbers all on their way before the next is added)
      float v[R] = {};
      if (row < t.rows) {
#pragma unroll 1
        for (int k = 0; k < q.shares; ++k, from += (long long)(low / 4) * p.rows) {
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
      if constexpr (std::is_same<T, __half>::value) {
        // f16 ends at 65504: by a power of two to below 2^8, and back in the product
        float most = 0.f;
#pragma unroll
        for (int k = 0; k < R; ++k) most = fmaxf(most, fabsf(v[k]));
        const float s = low_rank_scale(most);
#pragma unroll
        for (int k = 0; k < R; ++k) v[k] *= s;
        sh.scale[w.seg & 3][row] = s;
      }
      uint32_t o[V_COLS] = {};
#pragma unroll
      for (int k = 0; k < R / 2; ++k) split_pair<T>(v[2 * k], v[2 * k + 1], o[k], o[RB / 2 + k]);
      wait(&sh.v_empty[vb], vpar ^ 1);
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

size_t tall_workspace(int rows, int low, int shares) {
  return kTallStatusBytes + (size_t)shares * low * rows * sizeof(float);
}

int tall_shares(int rows, int width, int sms) {
  // CTAs for two an SM, a share at least 4 blocks of the width
  const int tiles = std::max(1, rows / kTallTile);
  return std::max(1, std::min({2 * sms / tiles, 8, (width + 255) / 256}));
}

int launch_tall(const AdapterParams& p, int rank, bool bf16, int shares, int sms, void* workspace, cudaStream_t stream) {
  const int low = p.parts * rank, columns = p.starts[p.parts];
  TallParams q = {};
  q.rank = rank;
  q.shares = shares;
  q.status = static_cast<int32_t*>(workspace);
  q.sums = reinterpret_cast<float4*>(static_cast<char*>(workspace) + kTallStatusBytes);
  q.n = (low + 15) / 16 * 16;
  const int stage = 16384 + q.n * 128;
  q.stages = std::max(2, std::min(8, 106 * 1024 / stage));
  q.tmem_cols = 32;
  while ((int)q.tmem_cols < q.n) q.tmem_cols *= 2;
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
  rc = raise_smem(contract, 112 * 1024, 0);
  if (rc == DA_OK) rc = raise_smem(expand, expand_smem, 0);
  if (rc != DA_OK) return rc;
  const long long tiles = most_tall_tiles(p);
  q.most_tiles = (int)tiles;
  AdapterParams pp = p;
  void* cargs[4] = {&pp, &q, &tmx, &tma};
  rc = launch_with(contract, (int)(tiles * shares), kContractThreads, contract_smem, true, stream, cargs);
  if (rc != DA_OK) return rc;
  void* eargs[4] = {&pp, &q, &tmy, &tmb};
  return launch_with(expand, sms, kExpandThreads, expand_smem, true, stream, eargs);
}

bool tall_fits(const AdapterParams& p, int rank, int sms) {
  const int low = p.parts * rank, columns = p.starts[p.parts];
  long long blocks = 0;
  for (int s = 0; s < p.parts; ++s) blocks += (p.starts[s + 1] - p.starts[s] + 127) / 128;
  const long long tiles = most_tall_tiles(p);
  return low <= 256 && p.x_rs >= p.width && p.y_rs >= columns && p.x_rs < (1ll << 38) && p.y_rs < (1ll << 38) &&
         (long long)p.adapters * columns < INT_MAX - 256 && (long long)p.adapters * low < INT_MAX - 256 &&
         tiles * 8 < INT_MAX && tiles / sms + 2 < kMaxTileList && tiles * blocks < (1ll << 40);
}

}  // namespace da
