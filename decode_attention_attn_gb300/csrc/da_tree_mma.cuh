// da_tree_mma.cuh -- shared-memory layout of the tensor-core tree kernel, known to host and device.
#pragma once

#include "da_tree.cuh"

namespace da {

constexpr int kTreeRows = 128;       // query rows per tile: the M of tcgen05.mma
constexpr int kTreeTokens = 128;     // KV tokens per tile

// Warps: 8 softmax, K producer, V producer, MMA issuer, q producer, and for FP8 caches 4 that
// convert codes to f16 tiles.
constexpr int kTreeSoftmaxWarps = 8;
constexpr int kTreeConvertWarps = 4;
__host__ __device__ constexpr int tree_threads(bool fp8) {
  return (kTreeSoftmaxWarps + 4 + (fp8 ? kTreeConvertWarps : 0)) * 32;
}

// A 16-bit tile of 128 rows (tokens or query rows) is D / 64 blocks of [128 rows][128 bytes], rows
// swizzled in groups of 8 (1 KB), as the TMA's 128-byte swizzle writes them and tcgen05.mma reads them.
__host__ __device__ constexpr uint32_t tree_tile_bytes(int D) { return 128u * D * 2u; }

struct TreeLayout {
  int nk, nv, nq;        // 16-bit K, V and q tiles
  int raw;               // FP8: tiles of codes, for K and for V each
  uint32_t q_off, k_off, v_off, rawk_off, rawv_off, bar_off, exch_off, qexp_off, misc_off, total;
};
__host__ __device__ constexpr TreeLayout tree_layout(int D, bool fp8) {
  TreeLayout L{};
  const uint32_t tile = tree_tile_bytes(D), code = 128u * D;
  L.nq = 2;
  if (!fp8) {
    // 160 KB (D = 128: 64 KB of K and V ahead of the softmax on average) or 144 KB
    L.nk = D == 128 ? 2 : 4;
    L.nv = D == 128 ? 3 : 5;
    L.raw = 0;
  } else {
    L.nk = 2;
    L.nv = D == 128 ? 1 : 2;
    L.raw = D == 128 ? 2 : 4;
  }
  uint32_t off = 0;
  L.q_off = off;
  off += L.nq * tile;
  L.k_off = off;
  off += L.nk * tile;
  L.v_off = off;
  off += L.nv * tile;
  L.rawk_off = off;
  off += L.raw * code;
  L.rawv_off = off;
  off += L.raw * code;
  L.bar_off = off;
  off += 48 * 8;
  L.exch_off = off;           // row maxima of the two column halves, two tiles; scratch of the schedule
  off += 2 * 2 * 128 * 4;
  L.qexp_off = off;           // FP8: q's power of two per row
  off += 2 * 128;
  L.misc_off = off;           // TMEM address, abort flag, odd-token word
  off += 32;
  L.total = off;
  return L;
}
static_assert(tree_layout(128, false).total <= kSmemLimit, "");
static_assert(tree_layout(128, true).total <= kSmemLimit, "");
static_assert(tree_layout(64, false).total <= kSmemLimit, "");
static_assert(tree_layout(64, true).total <= kSmemLimit, "");
// more than half of an SM's shared memory: one CTA an SM, so each has the SM's whole TMEM
static_assert(tree_layout(64, false).total > 116736 && tree_layout(64, true).total > 116736, "");
static_assert(sizeof(TreeScratch) <= 2 * 2 * 128 * 4, "the schedule's scratch lies in the exchange");

// The kernel of a cache type (da_dtype, or FP8), head_dim and output; null: not built.
// split: P enters as the sum of two 16-bit parts.
const void* tree_mma_kernel(int dtype, bool fp8, int head_dim, bool split);

}  // namespace da
