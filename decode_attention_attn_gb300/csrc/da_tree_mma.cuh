// da_tree_mma.cuh -- shared-memory layout of the tensor-core tree kernel, known to host and device.
#pragma once

#include "da_tree.cuh"

namespace da {

constexpr int kTreeRows = 128;       // query rows per tile: the M of tcgen05.mma
constexpr int kTreeTokens = 128;     // KV tokens per tile

// Warps: 8 softmax (two teams of 4 that take the KV tiles in turn, a thread a row), then the loaders of K
// (with q, for 16-bit caches) and of V, the issuer of S, the issuer of O, and for FP8 caches 4 that
// convert codes to f16 tiles (and q). No register may spill: with all of L1 in use as shared memory a
// spilled one costs an L2 round trip.
constexpr int kTreeSoftmaxWarps = 8;
constexpr int kTreeConvertWarps = 4;
__host__ __device__ constexpr int tree_threads(bool fp8) {
  return (kTreeSoftmaxWarps + 4 + (fp8 ? kTreeConvertWarps : 0)) * 32;
}

// 16-bit caches: launched with kTreeLaunchRegs a thread; the softmax warps then take registers from the
// others. (FP8: 16 warps of 128 each.)
constexpr int kTreeLaunchRegs = 168, kTreeSoftmaxRegs = 192, kTreeOtherRegs = 120;
static_assert(kTreeSoftmaxWarps * kTreeSoftmaxRegs +
                      (tree_threads(false) / 32 - kTreeSoftmaxWarps) * kTreeOtherRegs <=
                  tree_threads(false) / 32 * kTreeLaunchRegs,
              "the register split must fit the launch allocation");

// A 16-bit tile of 128 rows (tokens or query rows) of D elements in shared memory, as tcgen05.mma
// reads it with the 128-byte swizzle: groups of 8 rows x 64 elements (1 KB), rows of 128 bytes. The
// groups of a 64-element block follow one another and the blocks too (q, contiguous caches, converted
// codes); a paged cache's tiles hold the D / 64 blocks of an 8-row group side by side, so that one TMA
// box brings whole rows of a page (half as many boxes: the loader's issue rate, about 100 cycles a box,
// is what 16-token pages run into).
__host__ __device__ constexpr uint32_t tree_tile_bytes(int D) { return 128u * D * 2u; }

struct TreeLayout {
  int nk, nv, nq;        // 16-bit K and V tiles; q tiles (16-bit caches: shared memory, FP8: TMEM)
  int raw;               // FP8: tiles of codes, for K and for V each
  uint32_t q_off, k_off, v_off, rawk_off, rawv_off, bar_off, exch_off, qexp_off, misc_off, total;
};
__host__ __device__ constexpr TreeLayout tree_layout(int D, bool fp8) {
  TreeLayout L{};
  const uint32_t tile = tree_tile_bytes(D), code = 128u * D;
  L.nq = 2;
  L.nk = fp8 || D == 128 ? 2 : 4;
  L.nv = fp8 ? 2 : D == 128 ? 3 : 5;
  L.raw = !fp8 ? 0 : D == 128 ? 3 : 4;
  uint32_t off = 0;
  L.q_off = off;
  if (!fp8) off += L.nq * tile;
  L.k_off = off;
  off += L.nk * tile;
  L.v_off = off;
  off += L.nv * tile;
  L.rawk_off = off;
  off += L.raw * code;
  L.rawv_off = off;
  off += L.raw * code;
  L.bar_off = off;
  off += 40 * 8;
  L.exch_off = off;           // row references of two pieces, row sums of the two teams
  off += 4 * 128 * 4;
  L.qexp_off = off;           // FP8: q's power of two per row
  off += 2 * 128;
  L.misc_off = off;           // TMEM address, abort flag, odd-token word, the CTA's share
  off += 16 + sizeof(TreeShare);
  // more than half of an SM's shared memory: one CTA an SM, so each has the SM's whole TMEM
  L.total = off > 120u * 1024 ? off : 120u * 1024;
  return L;
}
static_assert(tree_layout(128, false).total <= kSmemLimit, "");
static_assert(tree_layout(128, true).total <= kSmemLimit, "");
static_assert(tree_layout(64, false).total <= kSmemLimit, "");
static_assert(tree_layout(64, true).total <= kSmemLimit, "");
static_assert(sizeof(TreeScratch) <= 4 * 128 * 4, "the schedule's scratch lies there first");

// The kernel of a cache type (da_dtype, or FP8) and head_dim; null: not built.
const void* tree_mma_kernel(int dtype, bool fp8, int head_dim);

}  // namespace da
