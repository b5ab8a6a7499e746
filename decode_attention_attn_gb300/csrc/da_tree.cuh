// da_tree.cuh -- what the tree-attention kernels share: launch parameters, the schedule that
// every CTA computes for itself from the lengths on the device, and the pieces' results.
//
// Work. The query heads of a KV head and the drafted tokens of a sequence are rows of one matrix:
// row r = i G + g is head g of drafted token i, so one read of a KV head serves T G rows. Rows are
// cut into row tiles, a sequence's tokens into KV tiles. The units of the schedule are the KV tiles
// of every (sequence, KV head), in that order; owner o of P takes units [o W / P, (o + 1) W / P).
// With R row tiles (the most that any sequence has) an owner is R CTAs that walk the same
// units, one row tile each, at about the same time, so that the second read of a KV tile hits L2.
//
// A (sequence, KV head) whose units lie with one owner is finished by it. One that spans owners
// leaves a partial with each (normalised rows and their log2 LSE), which the merge kernel joins: of
// an owner's pieces only the first and the last can be partial, so two slots an owner hold them.
#pragma once

#include "da_device.cuh"

namespace da {

struct TreeParams {
  Params c;                     // cache layout, block table, status (seq_lens unused)
  const void* q;                // [rows, hq, d]
  const int32_t* row_offsets;   // [B + 1]
  const int32_t* ctx_lens;      // [B]
  const unsigned long long* mask;   // [rows] or null (a chain)
  void* out;
  float* out_lse;
  int* head;                    // workspace: [0] units W, [1] owners P, [2] row tiles R
  int4* info;                   // [owners]: b, kvh, first unit's offset in its group, group tiles
  float* part_o;                // [2 owners][R][tile rows][d], 2 P R <= 2 CTAs
  float* part_l;                // [2 owners][R][tile rows]
  int rows, max_tree, group;
  int tile_rows, tile_tokens;
  int max_row_tiles;            // R's bound, from max_tree
  float qscale, v_scale;
};

struct TreeSeq {
  int row0;    // first row
  int T;       // drafted tokens
  int ctx;     // tokens before them
  int tiles;   // KV tiles of one KV head (0: no drafted tokens, nothing to do)
  int n;       // ctx + T
  bool bad;
};

// Sequence b's rows and lengths, clamped to what exists.
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int b) {
  TreeSeq s;
  const int lo = __ldg(p.row_offsets + b), hi = __ldg(p.row_offsets + b + 1);
  int ctx = __ldg(p.ctx_lens + b);
  s.row0 = min(max(lo, 0), p.rows);
  int T = min(max(hi, s.row0), p.rows) - s.row0;
  s.bad = ctx < 0 || T > p.max_tree || lo < 0;
  T = min(T, p.max_tree);
  if (T > 0 && (long long)ctx + T > p.c.capacity) s.bad = true;
  ctx = min(max(ctx, 0), p.c.capacity);
  T = min(T, p.c.capacity - ctx);
  s.T = T;
  s.ctx = ctx;
  s.n = ctx + T;
  s.tiles = T > 0 ? (s.n + p.tile_tokens - 1) / p.tile_tokens : 0;
  return s;
}

// The drafted tokens that row `row` (drafted token i of T) attends to.
__device__ __forceinline__ unsigned long long tree_word(const TreeParams& p, int row, int i,
                                                        int T) {
  const unsigned long long all = T >= 64 ? ~0ull : (1ull << T) - 1ull;
  return (p.mask ? __ldg(p.mask + row) : (2ull << i) - 1ull) & all;
}

// A CTA's part of the schedule.
// (units fit 32 bits: the plan refuses problems whose units might not)
struct TreeShare {
  int u0, u1;          // units
  int base;            // first unit of sequence b0
  int b0;              // the sequence that u0 lies in
  int row_tile, row_tiles, owner, owners;
};

struct TreeScratch {   // shared memory of tree_schedule
  int warp_sum[32];
  int warp_max[32];
  int base, b0;
};

__device__ __forceinline__ int tree_share_begin(int o, int W, int P) {
  return (int)((long long)o * W / P);
}
// The owner of unit u: the o with o W / P <= u < (o + 1) W / P (floor divisions).
__device__ __forceinline__ int tree_owner(int u, int W, int P) {
  return (int)((((long long)u + 1) * P - 1) / W);
}

// Every thread of the CTA calls this (NT threads). Each takes a run of sequences; a block scan of
// their tile counts gives the prefix, and the thread whose run holds u0 finds b0.
template <int NT>
__device__ __forceinline__ TreeShare tree_schedule(const TreeParams& p, TreeScratch& sc) {
  static_assert(NT % 32 == 0 && NT <= 1024, "");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.c.batch + NT - 1) / NT;
  const int first = min(tid * per, p.c.batch), last = min(first + per, p.c.batch);
  int sum = 0, most = 1;
  bool bad = false;
  for (int b = first; b < last; ++b) {
    const TreeSeq s = tree_seq(p, b);
    sum += s.tiles;
    most = max(most, (s.T * p.group + p.tile_rows - 1) / p.tile_rows);
    bad |= s.bad;
  }
  if (bad && blockIdx.x == 0) atomicOr(p.c.status, kStatusBadSeqLen);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  if (lane == 31) sc.warp_sum[warp] = inc;
  if (lane == 0) sc.warp_max[warp] = most;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += sc.warp_sum[w];
    total += sc.warp_sum[w];
    most = max(most, sc.warp_max[w]);
  }
  const int pre = before + inc - sum, units = total * p.c.hkv;
  TreeShare sh;
  sh.row_tiles = min(most, p.max_row_tiles);
  sh.owners = max(1, min((int)gridDim.x / sh.row_tiles, units));
  sh.owner = blockIdx.x / sh.row_tiles;
  sh.row_tile = blockIdx.x % sh.row_tiles;
  if (units == 0 || sh.owner >= sh.owners) {
    sh.u0 = sh.u1 = 0;
    sh.b0 = 0;
    sh.base = 0;
  } else {
    sh.u0 = tree_share_begin(sh.owner, units, sh.owners);
    sh.u1 = tree_share_begin(sh.owner + 1, units, sh.owners);
    if (pre * p.c.hkv <= sh.u0 && sh.u0 < (pre + sum) * p.c.hkv) {   // exactly one thread
      int at = pre;
      for (int b = first; b < last; ++b) {
        const int t = tree_seq(p, b).tiles;
        if (sh.u0 < (at + t) * p.c.hkv) {
          sc.b0 = b;
          sc.base = at * p.c.hkv;
          break;
        }
        at += t;
      }
    }
  }
  __syncthreads();
  if (sh.u1 > sh.u0) {
    sh.b0 = sc.b0;
    sh.base = sc.base;
  }
  if (tid == 0 && blockIdx.x == 0) {
    p.head[0] = units;
    p.head[1] = sh.owners;
    p.head[2] = sh.row_tiles;
  }
  return sh;
}

// Walks a share's pieces: units of one (sequence, KV head).
struct TreeWalk {
  int u;           // next unit
  int base;        // first unit of sequence b
  int b;
  TreeSeq s;
  // the current piece
  int kvh, t0, t1;      // KV tiles [t0, t1) of the sequence
  bool whole, head;     // covers all tiles; starts at the share's first unit

  __device__ __forceinline__ TreeWalk(const TreeParams& p, const TreeShare& sh)
      : u(sh.u0), base(sh.base), b(sh.b0) {
    if (sh.u1 > sh.u0) s = tree_seq(p, b);
  }
  __device__ __forceinline__ bool next(const TreeParams& p, const TreeShare& sh) {
    if (u >= sh.u1) return false;
    while (u >= base + s.tiles * p.c.hkv) {
      if (b + 1 >= p.c.batch) return false;   // (lengths that changed under way)
      base += s.tiles * p.c.hkv;
      s = tree_seq(p, ++b);
    }
    const int off = u - base;
    kvh = off / s.tiles;
    t0 = off - kvh * s.tiles;
    t1 = min(s.tiles, t0 + (sh.u1 - u));
    whole = t0 == 0 && t1 == s.tiles;
    head = u == sh.u0;
    u += t1 - t0;
    return true;
  }
};

// Slot of a partial: [2 owners][row tiles].
__device__ __forceinline__ long long tree_slot(int owner, bool head, int row_tile, int row_tiles) {
  return ((long long)owner * 2 + (head ? 0 : 1)) * row_tiles + row_tile;
}


}  // namespace da
