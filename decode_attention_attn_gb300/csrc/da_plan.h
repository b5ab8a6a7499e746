// da_plan.h -- the host-side plan object and the helpers that the translation units of the C
// ABI share: argument checks, error text, launch parameters, the tensor-map encoder.
#pragma once

#include <cudaTypedefs.h>

#include <cstddef>
#include <cstdint>
#include <string>

#include "da_device.cuh"
#include "decode_attn.h"

struct da_plan {
  da_problem prob;
  int num_sms;
  int group, es, unit, box_tokens, capacity, n_groups, piece_units;
  int kv_es;                    // K / V bytes per element (1: FP8 E4M3 cache; else es)
  int hp;                       // KV heads per split-kernel group (2: packed FP8 pairs)
  int sgroup;                   // query heads per split-kernel group (group * hp)
  int policy, num_splits;       // the plan's default split choice
  int narrow;                   // the device schedule's arithmetic fits 32 bits
  int grid;                     // balanced grid (or the default uniform grid)
  int recompute_splits, max_splits;
  int stages, batch_smem;
  size_t smem_bytes;
  long long slots;
  size_t off_counters, off_list, off_list_state, off_status, off_stats;
  size_t off_part_flags, off_part_l, off_part_o, zero_bytes, ws_bytes;
};

namespace da {

extern thread_local std::string g_cuda_error;   // text behind DA_ERR_CUDA

// Records the CUDA error's text for decode_attn_strerror and returns DA_ERR_CUDA. No exception leaves
// them: without memory for the text the last one stays.
int cuda_fail(cudaError_t e, const char* what) noexcept;
int text_fail(const char* text, const char* more = "") noexcept;

int validate_problem(const da_problem& p);

// Launch parameters of a plan's problem; the workspace's pointers when ws is given.
void fill_common(const da_plan& pl, Params& k, const int32_t* block_table,
                 const int32_t* seq_lens, void* ws);

// The DA_ERR_* code of a device status word.
int status_to_error(int s);

// The driver's cuTensorMapEncodeTiled, or null.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

inline size_t align256(size_t x) { return (x + 255) / 256 * 256; }

inline int elem_size(int dt) { return dt == DA_F32 ? 4 : 2; }

inline bool aligned(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

inline bool overlap(const void* a, long long na, const void* b, long long nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

}  // namespace da
