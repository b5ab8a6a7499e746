// da_tree.cuh -- what the tree-attention kernels share: launch parameters, the schedule that
// every CTA computes for itself from the lengths on the device, and the pieces' results.
//
// Work. The query heads of a KV head and the drafted tokens of a sequence are rows of one matrix:
// row r = i G + g is head g of drafted token i, so one read of a KV head serves T G rows. Rows are
// cut into row tiles, a sequence's tokens into KV tiles, the KV heads into blocks of `heads` heads. The
// units of the schedule are the KV tiles of every (sequence, block of heads), in that order; owner o of P
// takes units [o W / P, (o + 1) W / P). An owner is R x heads CTAs, for each of R row tiles (the most
// that any sequence has) and each head of a block, that walk the same units at about the same time: the
// second row tile's read of a KV tile then hits L2, and a token's rows of several heads, which lie side by
// side in the cache, are read together.
//
// A group, a (sequence, block of heads), whose units lie with one owner is finished by it. One that
// spans owners leaves a partial with each (normalised rows and their log2 LSE), which the merge kernel
// joins: of a CTA's pieces only the first and the last can be partial, so two slots a CTA hold them.
#pragma once

#include "da_device.cuh"

namespace da {

constexpr int kTreeMaxRowTiles = 16;   // 64 drafted tokens x 8 heads in tiles of 32 rows

struct TreeParams {
  Params c;                     // cache layout, block table, status (seq_lens unused)
  const void* q;                // [rows, hq, d]
  const int32_t* row_offsets;   // [B + 1]
  const int32_t* ctx_lens;      // [B]
  const unsigned long long* mask;   // [rows] or null (a chain)
  void* out;
  float* out_lse;
  int4* info;                   // [CTAs][2]: what the merge does for a CTA (tree_record)
  float* part_o;                // [owners][2][heads][R][tile rows][d]: 2 slots a CTA
  float* part_l;                // [owners][2][heads][R][tile rows]
  int rows, max_tree, group;
  int tile_rows, tile_tokens;
  int max_row_tiles;            // R's bound, from max_tree
  int narrow;                   // owners x units fits 32 bits: short divisions
  int stall;                    // test hook: 0, or 1 (2): CTA 0's loader of K (V) leaves out its second tile
  unsigned char heads[kTreeMaxRowTiles + 1];   // heads side by side, by R (tree_heads)
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

struct TreeRaw {   // a sequence's row range and length as they stand in memory
  int lo, hi, ctx;
};
__device__ __forceinline__ TreeRaw tree_raw(const TreeParams& p, int b) {
  return {__ldg(p.row_offsets + b), __ldg(p.row_offsets + b + 1), __ldg(p.ctx_lens + b)};
}

// A sequence's rows and lengths, clamped to what exists.
__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, const TreeRaw& raw) {
  TreeSeq s;
  const int lo = raw.lo, hi = raw.hi;
  int ctx = raw.ctx;
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

// The drafted tokens that drafted token i of T attends to, from its mask word (no mask: a chain).
__device__ __forceinline__ unsigned long long tree_clip(const TreeParams& p, unsigned long long word,
                                                        int i, int T) {
  const unsigned long long all = T >= 64 ? ~0ull : (1ull << T) - 1ull;
  return (p.mask ? word : (2ull << i) - 1ull) & all;
}

// A CTA's part of the schedule.
// (units fit 32 bits: the plan refuses problems whose units might not)
struct TreeShare {
  int u0, u1;          // units
  int base;            // first unit of sequence b0
  int b0;              // the sequence that u0 lies in
  int row_tile, row_tiles, head, heads, owner, owners, units;
  int blocks;          // blocks of heads
  TreeRaw raw;         // sequence b0
};

struct TreeScratch {   // shared memory of tree_schedule
  int warp_sum[32];
  int warp_max[32];
  int base, b0;
  TreeRaw raw;
};

__device__ __forceinline__ int tree_share_begin(int o, int W, int P, int narrow) {
  return narrow ? (int)((unsigned)o * (unsigned)W / (unsigned)P) : (int)((long long)o * W / P);
}
// The owner of unit u: the o with o W / P <= u < (o + 1) W / P (floor divisions).
__device__ __forceinline__ int tree_owner(int u, int W, int P, int narrow) {
  return narrow ? (int)((((unsigned)u + 1u) * (unsigned)P - 1u) / (unsigned)W)
                : (int)((((long long)u + 1) * P - 1) / W);
}

// Heads that an owner takes side by side: as many as leave at most 5 % of the CTAs without an owner (64
// sequences of 4350 FP8 tokens, 8 drafted: 168 us with 8 heads, 189 with one; bf16 the same within 1 %).
inline int tree_heads(int ctas, int row_tiles, int hkv) {
  for (int h = hkv; h > 1; --h)
    if (h < 256 && hkv % h == 0 && ctas / (row_tiles * h) * (row_tiles * h) * 20 >= ctas * 19)
      return h;
  return 1;
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
  TreeRaw raw{};   // of the run's last sequence, mostly its only one
  for (int b = first; b < last; ++b) {
    raw = tree_raw(p, b);
    const TreeSeq s = tree_seq(p, raw);
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
  TreeShare sh;
  sh.row_tiles = min(most, p.max_row_tiles);
  sh.heads = p.heads[sh.row_tiles];
  const unsigned lanes = sh.row_tiles * sh.heads;
  const int blocks = (unsigned)p.c.hkv / (unsigned)sh.heads;
  const int pre = before + inc - sum, units = total * blocks;
  sh.blocks = blocks;
  sh.owners = max(1, min((int)(gridDim.x / lanes), units));
  sh.owner = blockIdx.x / lanes;
  sh.head = (blockIdx.x - sh.owner * lanes) / (unsigned)sh.row_tiles;
  sh.row_tile = blockIdx.x - sh.owner * lanes - sh.head * sh.row_tiles;
  if (units == 0 || sh.owner >= sh.owners) {
    sh.u0 = sh.u1 = 0;
    sh.b0 = 0;
    sh.base = 0;
  } else {
    sh.u0 = tree_share_begin(sh.owner, units, sh.owners, p.narrow);
    sh.u1 = tree_share_begin(sh.owner + 1, units, sh.owners, p.narrow);
    if (pre * blocks <= sh.u0 && sh.u0 < (pre + sum) * blocks) {   // exactly one thread
      int at = pre;
      for (int b = first; b < last; ++b) {
        if (per > 1) raw = tree_raw(p, b);
        const int t = tree_seq(p, raw).tiles;
        if (sh.u0 < (at + t) * blocks) {
          sc.b0 = b;
          sc.base = at * blocks;
          sc.raw = raw;
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
    sh.raw = sc.raw;
  }
  sh.units = units;
  return sh;
}

// Walks a share's pieces: units of one group. The next sequence's lengths are loaded
// when a sequence is entered, a piece before they are needed: at a piece's end every role of the
// tensor-core kernel would otherwise wait for memory in turn.
struct TreeWalk {
  int u;           // next unit
  int base;        // first unit of sequence b
  int b;
  TreeSeq s;
  TreeRaw ahead;   // of sequence b + 1
  // the current piece
  int kvh, t0, t1;      // KV tiles [t0, t1) of the sequence
  bool whole, head;     // covers all tiles; starts at the share's first unit

  __device__ __forceinline__ TreeWalk(const TreeParams& p, const TreeShare& sh)
      : u(sh.u0), base(sh.base), b(sh.b0) {
    if (sh.u1 > sh.u0) {
      s = tree_seq(p, sh.raw);
      ahead = tree_raw(p, min(b + 1, p.c.batch - 1));
    }
  }
  __device__ __forceinline__ bool next(const TreeParams& p, const TreeShare& sh) {
    if (u >= sh.u1) return false;
    const int blocks = sh.blocks;
    while (u >= base + s.tiles * blocks) {
      if (b + 1 >= p.c.batch) return false;   // (lengths that changed under way)
      base += s.tiles * blocks;
      ++b;
      s = tree_seq(p, ahead);
      ahead = tree_raw(p, min(b + 1, p.c.batch - 1));
    }
    const int off = u - base;
    const int block = (unsigned)off / (unsigned)s.tiles;
    kvh = block * sh.heads + sh.head;
    t0 = off - block * s.tiles;
    t1 = min(s.tiles, t0 + (sh.u1 - u));
    whole = t0 == 0 && t1 == s.tiles;
    head = u == sh.u0;
    u += t1 - t0;
    return true;
  }
};

// Slot of a partial: [owners][2][heads][row tiles]; `lane` = head * row tiles + row tile.
__device__ __forceinline__ int tree_slot(int owner, bool head, int lanes, int lane) {
  return (owner * 2 + (head ? 0 : 1)) * lanes + lane;
}

// What the merge does for this CTA, written so that it learns it in one round trip to memory: the group
// whose units cross the start of this CTA's share, if the owner before is the first with units of it.
// {partials n (0: nothing), slot of the first, slot of the second less the first, slots from one to the
// next}, {first row, rows of a head left of this row tile, first row of it, head}. One thread calls this.
__device__ __forceinline__ void tree_record(const TreeParams& p, const TreeShare& sh, bool any,
                                            const TreeWalk& w) {
  int4 a = make_int4(0, 0, 0, 0), b = a;
  if (any && w.t0 > 0) {
    const int gs = sh.u0 - w.t0;   // the group's first unit
    const int o1 = tree_owner(gs, sh.units, sh.owners, p.narrow);
    if (o1 == sh.owner - 1) {
      const int o2 = tree_owner(gs + w.s.tiles - 1, sh.units, sh.owners, p.narrow);
      const int lanes = sh.row_tiles * sh.heads, lane = sh.head * sh.row_tiles + sh.row_tile;
      const bool whole = gs == tree_share_begin(o1, sh.units, sh.owners, p.narrow);
      const int first = tree_slot(o1, whole, lanes, lane);
      a = make_int4(o2 - o1 + 1, first, tree_slot(o1 + 1, true, lanes, lane) - first, 2 * lanes);
      b = make_int4(w.s.row0, w.s.T * p.group - sh.row_tile * p.tile_rows,
                    sh.row_tile * p.tile_rows, w.kvh);
    }
  }
  p.info[2 * blockIdx.x] = a;
  p.info[2 * blockIdx.x + 1] = b;
}

}  // namespace da
