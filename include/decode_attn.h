/*
 * decode_attn.h -- C ABI of the GB300 (sm_103a) decode-attention library: single-query decode
 * attention over a KV cache, attention for trees of drafted tokens over the same cache, the
 * operators that fill and read it (rotary positions, quantising writes, reads), and what a serving
 * loop runs beside them: pages from lengths, norms, and requests' adapters.
 *
 * Computes, for every sequence b and query head h of a decode step,
 *     o[b,h] = softmax(scale * q[b,h] . K_b^T) V_b          (natural exp)
 *     lse[b,h] = ln sum_t exp(scale * q[b,h] . k_t)
 * over the first seq_lens[b] tokens of the sequence's KV cache. Sources (page, section):
 *   - "Flash-Decoding: Mathematical Foundations, Split-KV Parallelism, Online Softmax
 *     Reduction, and Serving Latency Optimization": "The Single-Token Generation
 *     Bottleneck" (the operation), "Mathematical Formulation of Split-KV Parallelism"
 *     (split partials O, m, l, L), "The Rescaling and Online Softmax Reduction Algorithm"
 *     (exact merge), "Production Implementation Guidelines" (split heuristics).
 *   - "FlashAttention and inference kernels": "PagedAttention" (block table), "A paged
 *     decode attention kernel (with GQA)" (cache layout, kernel signature, GQA mapping
 *     kv_head = h / (H_q / H_kv)), Exercise 3 (one read of a KV head serves its group).
 *   - "FlashDecoding++: Faster Large Language Model Inference on GPUs": "Asynchronized
 *     Softmax with Unified Max Value" (Eq. 3, Eq. 4) and "The Overflow Fallback:
 *     Recomputation" (Fig. 6: range check, synchronised recompute of flagged rows).
 *
 * Conventions for every entry point:
 *   - Device pointers are CUDA device (or managed) addresses on the device that is
 *     current when the call is made; host pointers are plain host memory.
 *   - The caller owns every buffer: inputs, outputs and the workspace. The library owns
 *     only the host-side plan object. decode_attn_run allocates nothing.
 *   - Return value: DA_OK (0) or a negative DA_ERR_* code; decode_attn_strerror gives a
 *     message (for DA_ERR_CUDA it includes the CUDA error text of the failing call on
 *     this thread). No exception crosses the ABI. Argument errors are detected on the
 *     host before anything is enqueued.
 *   - Work is enqueued on the given cudaStream_t (NULL = legacy default stream) and the
 *     call returns without synchronising, unless the problem's `validate` flag is set
 *     or a stats struct is requested: then the call synchronises the stream and reports
 *     device-side findings (bad block-table entries, bad lengths, pipeline timeouts).
 *   - Thread safety: plans are read-only after creation and may be shared between
 *     threads; one workspace must not be used by two runs that can overlap on the GPU.
 */
#ifndef DECODE_ATTN_H
#define DECODE_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DECODE_ATTN_ABI_VERSION 4

/* Largest bin count decode_attn_logit_histogram accepts. */
#define DECODE_ATTN_MAX_HIST_BINS 32768

typedef enum { DA_F32 = 0, DA_F16 = 1, DA_BF16 = 2 } da_dtype;

/* DA_SOFTMAX_SYNC: each split runs the online-softmax recurrence with its running
 *   maximum ("FlashAttention and inference kernels", "FlashAttention: tiling plus online
 *   softmax"; FlashDecoding++ Eq. 2).
 * DA_SOFTMAX_UNIFIED: every split exponentiates against the one constant phi =
 *   unified_max, with no maximum and no rescaling (FlashDecoding++ Eq. 3 and Eq. 4). A
 *   scaled logit x with x - phi < range_lo or x - phi > range_hi (the interval is
 *   closed: a value on a bound is in range, as in Fig. 6) flags its row; flagged rows are
 *   recomputed in DA_SOFTMAX_SYNC mode on the device, in the same call ("The Overflow
 *   Fallback: Recomputation").
 * DA_SOFTMAX_UNIFIED_LOCAL: as DA_SOFTMAX_UNIFIED, with the same row flags, but without the
 *   second pass: a unified partial whose logits were all in range is an exact online-softmax
 *   state with maximum phi, so on its first out-of-range logit each split rescales its state
 *   to the true maximum so far and continues with the synchronised recurrence, reading no
 *   KV twice. An extension of the FlashDecoding++ fallback (the outputs equal the plain
 *   softmax either way). */
typedef enum {
  DA_SOFTMAX_SYNC = 0,
  DA_SOFTMAX_UNIFIED = 1,
  DA_SOFTMAX_UNIFIED_LOCAL = 2
} da_softmax_mode;

enum {
  DA_OK = 0,
  DA_ERR_INVALID_ARG = -1,          /* a null, misaligned or inconsistent argument */
  DA_ERR_UNSUPPORTED = -2,          /* head_dim, dtype, group size or page size not built */
  DA_ERR_WORKSPACE_TOO_SMALL = -3,  /* workspace_bytes below the plan's requirement */
  DA_ERR_BAD_BLOCK_TABLE = -4,      /* validate: a used block-table entry outside the pool */
  DA_ERR_CUDA = -5,                 /* a CUDA runtime / driver call failed */
  DA_ERR_DEVICE_TIMEOUT = -6,       /* validate: a device pipeline wait ran out of time */
  DA_ERR_BAD_SEQ_LEN = -7,          /* validate: seq_lens[b] < 0 or above the capacity */
  DA_ERR_HISTOGRAM_RANGE = -8,      /* choose_phi: a coverage tail lies outside [lo, hi) */
  DA_ERR_RANGE_TOO_WIDE = -9,       /* choose_phi: covered range wider than max_width */
  DA_ERR_NO_PAGES = -10             /* validate: a step needs more pages than its pool has free */
};

typedef struct {
  int batch;                /* B >= 1 sequences */
  int num_q_heads;          /* H_q */
  int num_kv_heads;         /* H_kv; H_q % H_kv == 0; group G = H_q / H_kv in {1,2,4,8} */
  int head_dim;             /* d in {64, 128} */
  int paged;                /* 1: k/v caches are [num_physical_blocks, page_size, H_kv, d]
                               addressed through block_table (FlashAttention and inference
                               kernels, "PagedAttention");
                               0: k/v caches are [batch, max_seq_len, H_kv, d] */
  int page_size;            /* paged: tokens per physical block, a power of two in [8, 256] */
  int max_blocks_per_seq;   /* paged: block_table row length */
  int num_physical_blocks;  /* paged: pool size; num_physical_blocks * page_size < 2^31 */
  int max_seq_len;          /* contiguous: token capacity per sequence;
                               batch * max_seq_len < 2^31 */
  da_dtype qkv_dtype;       /* storage of q, k_cache and v_cache (q only when kv_fp8) */
  da_dtype out_dtype;       /* storage of out (rounded to nearest even from fp32) */
  da_softmax_mode mode;
  float unified_max;        /* phi (natural-log units of the scaled logits); UNIFIED modes */
  float range_lo;           /* closed in-range interval on x - phi; range_lo < range_hi */
  float range_hi;
  int validate;             /* 1: every run synchronises and reports device findings */
  int num_sms;              /* 0: plan for the current device's SM count; > 0: plan for
                               that many SMs without touching CUDA (host-side planning) */
  /* FP8 KV cache ("FlashAttention and inference kernels", "A paged decode attention kernel
   * (with GQA)": the cache is BF16 or FP8, converted to FP32 in registers on read).
   * kv_fp8 = 1: k_cache and v_cache hold one-byte E4M3 codes (sign, 4-bit exponent with
   * bias 7, 3-bit mantissa, no infinities, S.1111.111 = NaN; "E4M3FN"), element for element
   * in the layout above, and code c stands for c * k_scale (K) or c * v_scale (V), scales
   * finite and > 0; q stays qkv_dtype, which must be DA_BF16 (else DA_ERR_UNSUPPORTED).
   * With groups of 4 query heads over an even number of KV heads, the plan packs pairs of KV
   * heads into one group of the split kernel where the step is large (at least four packed
   * groups per SM, or a cache capacity of 128 MiB and more); da_plan_info reports it.
   * The codes convert exactly; k_scale enters the logits' FP32 scale factor and v_scale the
   * output's. P . V runs on f16, so in the unified modes each split keeps its p = exp(x - phi)
   * within f16's range by a power-of-two factor per head, which only changes when its largest
   * logit grows past the range (the outputs and flags are those of the unified softmax).
   * NaN codes are not detected (they read as finite values). kv_fp8 = 0: k_cache and v_cache
   * are qkv_dtype; the scales are not read. */
  int kv_fp8;
  float k_scale;
  float v_scale;
  /* Test hook, 0 in normal use. k > 0: in every run of the plan, CTA 0's copy producer neither
   * arms nor fills ring stage k - 1 (no copy is issued for it) and every pipeline wait gives up
   * after 2 ms instead of 2 s, so that the consumers waiting for that stage run out of time:
   * the device records DA_ERR_DEVICE_TIMEOUT, the producer issues nothing more and drains the
   * copies it issued, and the run ends with unspecified outputs (with validate set, the call
   * returns DA_ERR_DEVICE_TIMEOUT). This exercises the bounded-wait path without a fault. */
  int debug_stall_stage;
} da_problem;

typedef struct da_plan da_plan;   /* opaque, host-owned, immutable after creation */

/* What a plan chose (host-side, no CUDA call). */
typedef struct {
  int grid_ctas;            /* persistent CTAs per launch */
  int num_splits;           /* 0: balanced shares (one contiguous share per CTA);
                               > 0: uniform splits per sequence */
  int unit_tokens;          /* split boundaries fall on multiples of this many tokens */
  int stage_tokens;         /* tokens per shared-memory pipeline stage */
  int stages;               /* pipeline depth */
  int recompute_splits;     /* uniform splits per flagged group in the recompute pass */
  int max_splits;           /* largest num_splits a run may ask for with this workspace */
  size_t workspace_bytes;   /* device workspace the runs need */
  size_t smem_bytes;        /* dynamic shared memory per CTA */
  int split_tokens;         /* largest split (piece of one sequence's KV head, in tokens) of a
                               step whose sequences are all at capacity, under the plan's
                               default policy ("the split size" of Flash-Decoding) */
  int split_tokens_min;     /* smallest such split */
  int kv_heads_per_group;   /* KV heads one split-kernel group reads together: 2 where an FP8
                               cache's groups of 4 query heads are packed in pairs of KV heads
                               (8 query heads fill the tensor-core consumer; see kv_fp8), else
                               1. Splits, partials and the merge are then per pair. */
} da_plan_info;

/* Filled by decode_attn_run when requested (forces a stream synchronisation). */
typedef struct {
  int grid_ctas;
  int num_splits;           /* as in da_plan_info, for this run */
  long long rows_flagged;   /* UNIFIED: (b, h) rows whose range check failed */
  long long splits_flagged; /* UNIFIED: (split, h) partials whose range check failed */
  int recompute_launched;   /* 1 iff the recompute kernel was enqueued (DA_SOFTMAX_UNIFIED) */
  int split_tokens;         /* largest split of this run's first pass, in tokens (the split
                               the heuristic chose, as the device cut it from seq_lens) */
  int split_tokens_min;     /* smallest split of this run's first pass, in tokens */
} da_stats;

/* Validate a problem and choose the launch (grid, split policy, pipeline) for it.
 * num_splits: 0 = heuristic (one balanced share of the whole step's KV tokens per
 * persistent CTA, which splits a sequence exactly when the SMs would otherwise idle:
 * the Flash-Decoding rule of splitting only when B * H under-fills the GPU, applied to
 * the work itself); > 0 = exactly that many uniform splits per sequence, each of
 * roundup(ceil(N_b / num_splits), unit) tokens ("Mathematical Formulation of Split-KV
 * Parallelism"). *workspace_bytes_out receives the workspace size the runs need.
 * Owns: *plan_out (free with decode_attn_destroy). Errors: INVALID_ARG, UNSUPPORTED,
 * CUDA (only when num_sms == 0 and the device query fails). */
int decode_attn_plan(const da_problem* problem, int num_splits, da_plan** plan_out,
                     size_t* workspace_bytes_out);

/* Copy what the plan chose into *info. Errors: INVALID_ARG. */
int decode_attn_plan_info(const da_plan* plan, da_plan_info* info);

/* Zero the part of the workspace that runs expect at zero and leave at zero (counters and the
 * flagged list). Required once for a new workspace before its first run (a zero-filled
 * allocation needs no call), and again after a run reported DA_ERR_DEVICE_TIMEOUT. Enqueued
 * on `stream`.
 * Errors: INVALID_ARG, WORKSPACE_TOO_SMALL, CUDA. */
int decode_attn_workspace_init(const da_plan* plan, void* workspace, size_t workspace_bytes,
                               void* cuda_stream);

/* Run one decode step.
 *   q           device, [batch, H_q, d] in qkv_dtype, 16-byte aligned.
 *   k_cache,    device, layout per problem->paged (see da_problem), qkv_dtype (E4M3 codes
 *   v_cache     when kv_fp8), 16-byte aligned.
 *   block_table device int32 [batch, max_blocks_per_seq] when paged (entries for the
 *               pages a sequence uses must lie in [0, num_physical_blocks); the rest are
 *               ignored, -1 by convention); must be NULL when contiguous.
 *   seq_lens    device int32 [batch], 0 <= seq_lens[b] <= capacity (paged:
 *               max_blocks_per_seq * page_size; contiguous: max_seq_len).
 *   scale       multiplier of q . k (1/sqrt(d) for standard attention).
 *   num_splits  -1 = the plan's choice; 0 = balanced shares; > 0 = uniform splits
 *               (at most the plan's max_splits).
 *   out         device, [batch, H_q, d] in out_dtype. A sequence with seq_lens[b] == 0
 *               gets out = 0 ("FlashAttention and inference kernels", Exercise 2 skips
 *               empty segments; an empty row is this library's extension of it).
 *   out_lse     nullable device float [batch, H_q]: natural-log log-sum-exp of the
 *               scaled logits (-inf for an empty sequence).
 *   row_flags   nullable device uint8 [batch, H_q]: UNIFIED: 1 iff the row's range check
 *               failed (its out/out_lse then come from the synchronised recompute);
 *               SYNC: 0.
 *   workspace   device, at least the plan's workspace_bytes, 256-byte aligned, zeroed
 *               before first use (decode_attn_workspace_init); left reusable.
 *   cuda_stream cudaStream_t or NULL.
 *   stats       nullable; when given the call synchronises and fills it.
 * Errors: INVALID_ARG, WORKSPACE_TOO_SMALL, CUDA, and with validate (or stats):
 * BAD_BLOCK_TABLE, BAD_SEQ_LEN, DEVICE_TIMEOUT. A bad block-table entry never makes the
 * device read outside the cache: the page reads as zeros. */
int decode_attn_run(const da_plan* plan, const void* q, const void* k_cache,
                    const void* v_cache, const int32_t* block_table, const int32_t* seq_lens,
                    float scale, int num_splits, void* out, float* out_lse,
                    uint8_t* row_flags, void* workspace, size_t workspace_bytes,
                    void* cuda_stream, da_stats* stats);

/* All arguments of one run, for decode_attn_run_ex. Fields as for decode_attn_run, plus:
 *   split_event_begin, split_event_end: nullable cudaEvent_t handles recorded on the
 *   stream immediately before and immediately after the split kernel's launch (before the
 *   recompute kernel), so a caller can time the split kernel alone with
 *   cudaEventElapsedTime. Both or neither must be given. */
typedef struct {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_table;
  const int32_t* seq_lens;
  float scale;
  int num_splits;
  void* out;
  float* out_lse;
  uint8_t* row_flags;
  void* workspace;
  size_t workspace_bytes;
  void* cuda_stream;
  da_stats* stats;
  void* split_event_begin;
  void* split_event_end;
} da_run_args;

/* decode_attn_run with its arguments in a struct and optional timing events.
 * Errors: as decode_attn_run; INVALID_ARG also when only one event is given. */
int decode_attn_run_ex(const da_plan* plan, const da_run_args* args);

/* Size of the fixed scratch region that decode_attn_run_static uses (8 MiB per device). */
#define DECODE_ATTN_STATIC_SCRATCH_BYTES (8u << 20)

/* Run one decode step without a caller-provided workspace. The papers and pages this
 * library follows have no counterpart to this entry point; it exists for callers that
 * cannot allocate device memory for a workspace:
 *   - a server whose device memory is reserved up front for the KV-cache pool;
 *   - a process under a device-memory cap, where a new allocation can fail in mid-step;
 *   - a decode loop that cannot afford cudaMalloc / cudaFree, which may synchronise the
 *     whole device;
 *   - plain C code with no device allocator of its own.
 * In place of a workspace it uses one fixed region of DECODE_ATTN_STATIC_SCRATCH_BYTES per
 * device, which belongs to the library's device code and is reserved when that code is
 * loaded on the device. The call itself allocates nothing: no cudaMalloc, no cudaFree, no
 * allocating library routine.
 *   Arguments as for decode_attn_run, less workspace and workspace_bytes.
 *   First call in a CUDA context: it looks up the region's device address in the context
 *   current on the calling thread (which can load the library's device code there) and
 *   caches it under that context's unique ID; a device reset or a caller's own driver
 *   context therefore gets a lookup of its own. Make the first call in each context before
 *   any stream capture.
 *   Each call first clears, on `cuda_stream`, the part of the region the plan's run expects
 *   at zero (counters and the flagged list), so runs of different plans may follow one another
 *   on a stream.
 *   Overlapping calls race: all calls on one device share the one region, so two calls
 *   whose work can overlap on the GPU (other streams, other host threads, other plans)
 *   corrupt each other's results. Serialise them, or use decode_attn_run with separate
 *   workspaces.
 *   Device findings (bad block-table entries or lengths, pipeline timeouts) are reported
 *   only through `stats` or the problem's `validate` flag: the region's status word is
 *   cleared by the next call.
 * Errors: as decode_attn_run; WORKSPACE_TOO_SMALL also when the plan's workspace_bytes
 * exceeds DECODE_ATTN_STATIC_SCRATCH_BYTES (use decode_attn_run with a workspace of that
 * size instead). Argument errors, including a plan whose kernel is not built, are detected
 * before anything is enqueued. */
int decode_attn_run_static(const da_plan* plan, const void* q, const void* k_cache,
                           const void* v_cache, const int32_t* block_table,
                           const int32_t* seq_lens, float scale, int num_splits, void* out,
                           float* out_lse, uint8_t* row_flags, void* cuda_stream,
                           da_stats* stats);

/* Synchronise `stream`, then read and clear the device findings recorded in the
 * workspace by earlier runs. Returns DA_OK or the first finding's DA_ERR_* code. */
int decode_attn_check_status(const da_plan* plan, void* workspace, void* cuda_stream);

/* Test hook: the element offset (into k_cache / v_cache) from which the device reads
 * token t of (sequence b, KV head kvh), computed by the same device code the kernel's
 * loads use. offsets_out: device int64 [batch, H_kv, T] with T = max_blocks_per_seq *
 * page_size (paged) or max_seq_len (contiguous); -1 for t >= seq_lens[b] and for a
 * block-table entry outside the pool. Enqueued on `stream`. Errors: INVALID_ARG, CUDA. */
int decode_attn_debug_gather(const da_plan* plan, const int32_t* block_table,
                             const int32_t* seq_lens, int64_t* offsets_out, void* cuda_stream);

/* ---- Calibration: choosing phi from the logits of a step --------------------------------
 * "FlashDecoding++: Faster Large Language Model Inference on GPUs", "The Overflow and
 * Precision Problem: Choosing phi" and Fig. 5: the logits of a model's attention rows stay in
 * a narrow range, profiled as a histogram over many inputs; phi is set to the lower end of
 * the range that holds more than 99.99% of them, and where that range is too wide (OPT-6.7B
 * in Fig. 5) the unified max is not used. These two calls run that profile on the caller's
 * own steps: accumulate one histogram over as many steps as wanted, then read phi off it.
 * Neither is on the attention path. */

/* Histogram of the scaled logits x = scale * q[b,h] . k_t of one step, over every query head
 * h and every token t < seq_lens[b] of every sequence b, read through the plan's layout
 * (contiguous or block table, GQA mapping kv_head = h / G) as decode_attn_run reads them.
 *   plan: any plan of the problem shape; its softmax mode, phi and range are not used.
 *   q, k_cache, block_table, seq_lens, scale: as for decode_attn_run (device; k_cache
 *     16-byte aligned). v_cache is not read.
 *   lo, hi, nbins: nbins equal bins over [lo, hi), lo < hi finite, 1 <= nbins <=
 *     DECODE_ATTN_MAX_HIST_BINS. x falls in bin i = floor((x - lo) * (nbins / (hi - lo))),
 *     evaluated in fp32 from an fp32 dot product, so a logit within a few fp32 ulps of a bin
 *     edge may fall on either side of it.
 *   counts: device uint64 [nbins + 2], 8-byte aligned, ACCUMULATED into (zero it before the
 *     first step): counts[0] = values below lo, counts[1 + i] = bin i, counts[nbins + 1] =
 *     values at or above the top edge, and NaN.
 * A token whose block-table entry lies outside the pool, and tokens past the capacity, are
 * not counted: the counts then sum to less than H_q * sum_b min(seq_lens[b], capacity), which
 * the caller can check. Enqueued on `stream`; not synchronised.
 * For an FP8 cache (kv_fp8) the logits are scale * q . (code * k_scale), as decode_attn_run
 * forms them. Errors: INVALID_ARG (null or misaligned pointer, bad range or bin count),
 * UNSUPPORTED, CUDA. */
int decode_attn_logit_histogram(const da_plan* plan, const void* q, const void* k_cache,
                                const int32_t* block_table, const int32_t* seq_lens,
                                float scale, float lo, float hi, int nbins,
                                unsigned long long* counts, void* cuda_stream);

/* Host only: phi and the covered logit range from a histogram laid out as above.
 *   counts: HOST uint64 [nbins + 2]; nbins, lo, hi: those the histogram was taken with.
 *   coverage: the fraction of values the range must hold, in (0, 1] (0.9999 in Fig. 5).
 *     At most floor((1 - coverage) * total / 2) values are left out on each side, whole bins
 *     at a time, so the range is bin-aligned and holds at least that fraction.
 *   max_width: the widest covered range (x_hi - x_lo) for which the unified max is used.
 *   x_lo, x_hi (out): the covered range, bin edges rounded outwards to fp32.
 *   phi (out): x_lo, the pages' choice (the lower bound: a value below it underflows
 *     harmlessly, none in range overflows). With it, the in-range interval on x - phi of
 *     the covered values is [0, x_hi - x_lo]; da_problem's [range_lo, range_hi] may be set
 *     wider, to what fp32 tolerates, so that only values that would lose precision or
 *     overflow flag their rows.
 * Errors: INVALID_ARG (null pointer, empty histogram, bad coverage, range or max_width);
 * HISTOGRAM_RANGE (more than a tail's share of values lies below lo or at or above hi:
 * repeat the histogram over a wider [lo, hi); outputs not written); RANGE_TOO_WIDE (outputs
 * written, but x_hi - x_lo > max_width: the unified max does not apply to this data, use
 * DA_SOFTMAX_SYNC, as Fig. 5 does for OPT-6.7B). Touches no device. */
int decode_attn_choose_phi(const unsigned long long* counts, int nbins, float lo, float hi,
                           double coverage, float max_width, float* phi, float* x_lo,
                           float* x_hi);

/* ---- The rows around a step: rotary positions, writing the cache, reading it back ---------
 * A step's new rows are laid out one after another, sequence by sequence:
 *   row_offsets device int32 [batch + 1], non-decreasing: rows row_offsets[b] ..
 *               row_offsets[b + 1] - 1 belong to sequence b (none where they are equal). Rows
 *               before the first and behind the last sequence belong to none (a padded batch).
 *   start       device int32 [batch]: the cache position of sequence b's first row, >= 0; row r
 *               of sequence b stands for position start[b] + r - row_offsets[b]. To append to a
 *               cache that holds n tokens of b, start[b] = n.
 *   rows        the number of rows of the row tensors; row_offsets may reach past it, those rows
 *               do not exist. rows = 0: the call returns DA_OK and enqueues nothing.
 * Row tensors are [rows, heads, d]; where strides are taken, they count elements, between rows
 * and between heads, and the d elements of a head are contiguous. */

/* How a rotary embedding's frequencies theta_i = base^(-2 i / rotary_dim), i < rotary_dim / 2,
 * are scaled for contexts longer than those a model was trained on, s = factor,
 * L0 = original_max_position, rho_i = L0 theta_i / (2 pi) (turns over the original context):
 * DA_ROPE_NONE      as they are.
 * DA_ROPE_LINEAR    theta_i / s (position interpolation).
 * DA_ROPE_NTK       base replaced by base * s^(rotary_dim / (rotary_dim - 2)).
 * DA_ROPE_BY_PARTS  theta_i (keep + (1 - keep) / s), keep = clamp((rho_i - low) / (high - low),
 *                   0, 1): what turns more than `high` times is kept, less than `low` times
 *                   interpolated ("YaRN: Efficient Context Window Extension of Large Language
 *                   Models", "NTK-by-parts").
 * DA_ROPE_BY_INDEX  the same mix with a ramp that is linear in i: keep = 1 - clamp((i - first) /
 *                   max(last - first, 0.001), 0, 1), first = max(floor(at(high)), 0), last =
 *                   min(ceil(at(low)), rotary_dim - 1), at(n) = rotary_dim ln(L0 / (2 pi n)) /
 *                   (2 ln base), the index whose frequency turns n times. */
typedef enum {
  DA_ROPE_NONE = 0,
  DA_ROPE_LINEAR = 1,
  DA_ROPE_NTK = 2,
  DA_ROPE_BY_PARTS = 3,
  DA_ROPE_BY_INDEX = 4
} da_rope_scaling;

typedef struct {
  int head_dim;              /* d: even, 2 to 256 */
  int rotary_dim;            /* even, 2 to head_dim: elements [0, rotary_dim) of a head are rotated,
                                the rest pass unchanged */
  int interleaved;           /* 0: element i pairs with i + rotary_dim / 2; 1: 2 i with 2 i + 1 */
  da_rope_scaling scaling;
  double base;               /* > 1, finite */
  double factor;             /* s > 0, finite; every scaling but NONE */
  double original_max_position; /* L0 > 0; BY_PARTS, BY_INDEX */
  double low, high;          /* 0 < low < high; BY_PARTS, BY_INDEX */
  double attn_factor;        /* m, finite as a float: both elements of a rotated pair are multiplied by m */
} da_rope_config;

typedef struct da_rope da_rope;   /* opaque, host-owned, immutable after creation */

/* Compute the frequencies. Host only, touches no device. Owns: *rope_out (free with
 * decode_attn_rope_destroy). Errors: INVALID_ARG, UNSUPPORTED (head_dim or rotary_dim). */
int decode_attn_rope_create(const da_rope_config* config, da_rope** rope_out);

/* Copy the scaled frequencies (radians per position) into theta[rotary_dim / 2].
 * Errors: INVALID_ARG. */
int decode_attn_rope_frequencies(const da_rope* rope, double* theta);

void decode_attn_rope_destroy(da_rope* rope);

#define DECODE_ATTN_ROPE_MAX_HEADS (1 << 20)

/* Rotate rows: for every row r, head h and pair (a, b) with angle phi = positions[r] theta_i,
 *   out_a = m (x_a cos phi - x_b sin phi),  out_b = m (x_b cos phi + x_a sin phi);
 * transpose = 1: sin phi is negated, which is the transposed map, so the gradient with respect to
 * x of a forward call given the gradient with respect to its output (and, with m = 1, its
 * inverse). phi is reduced exactly in 64-bit fixed point whatever the position; the arithmetic is
 * fp32, rounded once to the storage type.
 *   x, out      device, [rows, heads, head_dim] of `dtype` with the given strides (elements; out's
 *               heads and rows must lie apart: overlapping strides are refused). out may be x
 *               with equal strides (in place), or other rows or heads of the same tensor; any
 *               other overlap is refused, and tensors of one memory that are interleaved some
 *               other way with it.
 *   positions   device int32 [rows]; negative positions rotate backwards.
 * Aligned to 16 bytes, with strides that are multiples of 16 bytes and rotary_dim and head_dim
 * multiples of 32 bytes, rows move 16 bytes a lane; any other case takes one pair a lane.
 * Enqueued on cuda_stream. Errors: INVALID_ARG, UNSUPPORTED (dtype; more than
 * DECODE_ATTN_ROPE_MAX_HEADS heads), CUDA. */
typedef struct {
  const void* x;
  void* out;
  da_dtype dtype;
  int rows;
  int heads;
  int64_t x_row_stride, x_head_stride;
  int64_t out_row_stride, out_head_stride;
  const int32_t* positions;
  int transpose;
  void* cuda_stream;
} da_rope_args;

int decode_attn_rope_apply(const da_rope* rope, const da_rope_args* args);

/* Write a step's K and V rows into the cache, in the layout and storage of the plan's problem,
 * and, with `rope`, rotate q and k on the way, all in one launch.
 *   plan: any plan of the problem shape; its softmax mode and split choice are not used.
 *   k, v        device, [rows, H_kv, d] in qkv_dtype with the given strides (parts of one
 *               projection's rows, for instance).
 *   k_cache,    device, as for decode_attn_run, apart (else refused); k and v must not lie where
 *   v_cache     rows are written. A 16-bit or fp32 cache takes the values as they are (a rotated k rounded once to nearest even). An FP8 cache takes E4M3
 *               codes of x / k_scale or x / v_scale, an fp32 quotient rounded to nearest
 *               even, values beyond +-448 to +-448, NaN to the NaN code; a rotated k is not
 *               rounded to qkv_dtype in between. (A scale whose reciprocal is no fp32 number
 *               is refused.)
 *   block_table as for decode_attn_run. Rows of two sequences must not fall on the same token
 *               of the pool (of two rows written to one token, either may stay, in parts).
 *   rope        nullable. With it k is rotated by its row's position, and q, when given, is
 *               rotated into q_out: [rows, H_q, d] in qkv_dtype, both with strides; q_out may be
 *               q with equal strides, and its heads and rows must lie apart, and apart from
 *               those of k and v (else refused, as in decode_attn_rope_apply).
 *               Without it q and q_out must be NULL. rope's head_dim must be the plan's.
 *   positions   nullable device int32 [rows]: the rotary positions where they are not the cache
 *               positions (drafted trees: a node's depth). Needs rope.
 *   amax        nullable device float [2]: amax[0] = max(amax[0], |k| as written before scaling),
 *               amax[1] likewise for v; initialise to 0. From them an FP8 cache's scales are
 *               chosen (amax / 448). NaNs are passed over; the result does not depend on order.
 *   workspace   nullable, the plan's workspace: device findings are recorded in its status word
 *               (decode_attn_check_status). Required when the problem's validate is set: the call
 *               then synchronises and returns them.
 * A row whose position lies outside [0, capacity) (BAD_SEQ_LEN) or on a block-table entry outside
 * the pool (BAD_BLOCK_TABLE) is not written; its q is still rotated. Rows of no sequence leave
 * the cache and q_out as they were. Enqueued on cuda_stream.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE_TOO_SMALL, CUDA; with validate the findings. */
typedef struct {
  const void* k;
  const void* v;
  int64_t k_row_stride, k_head_stride;
  int64_t v_row_stride, v_head_stride;
  int rows;
  void* k_cache;
  void* v_cache;
  const int32_t* block_table;
  const int32_t* row_offsets;
  const int32_t* start;
  const da_rope* rope;
  const int32_t* positions;
  const void* q;
  void* q_out;
  int64_t q_row_stride, q_head_stride;
  int64_t q_out_row_stride, q_out_head_stride;
  float* amax;
  void* workspace;
  size_t workspace_bytes;
  void* cuda_stream;
} da_kv_write_args;

int decode_attn_kv_write(const da_plan* plan, const da_kv_write_args* args);

/* Read rows back from the cache: k_out[r], v_out[r] = the K and V of row r's position, codes of an
 * FP8 cache times k_scale or v_scale, rounded once to qkv_dtype (to nearest even).
 *   k_out, v_out  device, [rows, H_kv, d] contiguous, qkv_dtype, 16-byte aligned, apart (else
 *                 refused), and not where rows are read; either may be NULL (not both), and its
 *                 cache then too.
 * Rows at a position outside [0, capacity) or on a bad block-table entry read as zeros and are
 * recorded as in decode_attn_kv_write; rows of no sequence are left as they were.
 * Writing rows read from an FP8 cache back with the same scales reproduces their codes (a NaN
 * code's sign excepted) as long as the products are normal numbers of qkv_dtype. Enqueued on
 * cuda_stream. Errors: as kv_write. */
typedef struct {
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_table;
  const int32_t* row_offsets;
  const int32_t* start;
  int rows;
  void* k_out;
  void* v_out;
  void* workspace;
  size_t workspace_bytes;
  void* cuda_stream;
} da_kv_read_args;

int decode_attn_kv_read(const da_plan* plan, const da_kv_read_args* args);

/* ---- Attention for a tree of drafted tokens ------------------------------------------------
 * Verification of drafted tokens: sequence b holds ctx_lens[b] tokens, and T_b drafted tokens'
 * K and V follow them in the cache, at positions ctx_lens[b] + j, j < T_b (decode_attn_kv_write
 * with start = ctx_lens puts them there). Every drafted token i has H_q queries, which attend to
 * the whole context and to the drafted tokens that tree_mask names:
 *     o[i,h] = softmax over t in S_i of (scale q[i,h] . k_t) applied to v_t,
 *     S_i = [0, ctx_lens[b]) and { ctx_lens[b] + j : bit j of tree_mask[i], j < T_b },
 * with the GQA mapping of decode_attn_run. Rows are laid out by row_offsets as above, T_b =
 * row_offsets[b + 1] - row_offsets[b] <= max_tree. */

#define DECODE_ATTN_MAX_TREE 64

typedef struct da_tree_plan da_tree_plan;   /* opaque, host-owned, immutable after creation */

typedef struct {
  int grid_ctas;            /* CTAs of the attention launch */
  int row_tiles;            /* tiles of query rows (T * G rows of one KV head) a sequence takes */
  int tile_rows;            /* query rows per tile */
  int tile_tokens;          /* KV tokens per tile */
  int stages;               /* K or V tiles in flight (0: the fp32 kernel, which has no ring) */
  int max_tree;
  size_t workspace_bytes;
  size_t smem_bytes;
} da_tree_plan_info;

/* Plan for the problem's cache and up to max_tree (1 to DECODE_ATTN_MAX_TREE) drafted tokens a
 * sequence. problem->mode must be DA_SOFTMAX_SYNC (a unified maximum has no counterpart here:
 * UNSUPPORTED); debug_stall_stage must be 0. Errors: as decode_attn_plan. */
int decode_attn_tree_plan(const da_problem* problem, int max_tree, da_tree_plan** plan_out,
                          size_t* workspace_bytes_out);

int decode_attn_tree_plan_info(const da_tree_plan* plan, da_tree_plan_info* info);

/* Test hook, 0 in normal use. tensor = 1 (2): in the plan's later runs CTA 0 leaves out its second
 * load of K (V) and every pipeline wait gives up after 2 ms instead of 2 s, so that the warps waiting
 * for it run out of time: the device records DA_ERR_DEVICE_TIMEOUT, nothing more is issued, copies in
 * flight are waited for, and the run ends with unspecified results (with validate set, the call returns
 * DA_ERR_DEVICE_TIMEOUT). This exercises the bounded-wait path without a fault. Not to be called while
 * another thread runs the plan. Errors: INVALID_ARG, UNSUPPORTED (fp32 caches, whose kernel has no such
 * wait). */
int decode_attn_tree_debug_stall(da_tree_plan* plan, int tensor);

/* Clear a new workspace's status word (a zero-filled allocation needs no call). Enqueued on
 * cuda_stream. Errors: INVALID_ARG, WORKSPACE_TOO_SMALL, CUDA. */
int decode_attn_tree_workspace_init(const da_tree_plan* plan, void* workspace,
                                    size_t workspace_bytes, void* cuda_stream);

/* Run one verification step.
 *   q           device, [rows, H_q, d] in qkv_dtype, contiguous, 16-byte aligned.
 *   k_cache, v_cache, block_table, scale: as for decode_attn_run.
 *   row_offsets, ctx_lens: device int32 [batch + 1] and [batch]. ctx_lens[b] + T_b above the
 *               capacity, T_b above max_tree or a negative length is recorded (BAD_SEQ_LEN) and
 *               clamped; rows past the clamped T_b are left as they were.
 *   tree_mask   nullable device uint64 [rows]: bit j of row i's word is set iff drafted token i
 *               attends to drafted token j of its sequence (its own bit too, where it should
 *               see itself). Bits at or past T_b are ignored. NULL: a chain, j <= i.
 *   out         device, [rows, H_q, d] in out_dtype, 16-byte aligned. A row that attends to
 *               nothing (no context, mask 0) gets 0. out that overlaps q is refused.
 *   out_lse     nullable device float [rows, H_q]: natural-log log-sum-exp (-inf: nothing).
 *   workspace   device, 256-byte aligned, at least the plan's workspace_bytes.
 * Masked drafted tokens and cache slots past a sequence's end add nothing, whatever they hold
 * (NaN and infinities included). Rows of no sequence are left as they were. Results do not depend
 * on launch order. Enqueued on cuda_stream; with the problem's validate set the call
 * synchronises and returns the device's findings.
 * Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE_TOO_SMALL, CUDA, and the findings. */
typedef struct {
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_table;
  const int32_t* row_offsets;
  const int32_t* ctx_lens;
  const uint64_t* tree_mask;
  int rows;
  float scale;
  void* out;
  float* out_lse;
  void* workspace;
  size_t workspace_bytes;
  void* cuda_stream;
} da_tree_args;

int decode_attn_tree_run(const da_tree_plan* plan, const da_tree_args* args);

/* decode_attn_check_status for a tree plan's workspace. */
int decode_attn_tree_check_status(const da_tree_plan* plan, void* workspace, void* cuda_stream);

void decode_attn_tree_destroy(da_tree_plan* plan);

/* ---- Pages: block tables and slots from the sequences' lengths --------------------------------
 * A pool is a device array of DECODE_ATTN_POOL_HEAD + num_physical_blocks int32, 16-byte aligned:
 *   pool[0]  the number of free pages, F (taken as 0 .. num_physical_blocks where it lies outside);
 *   pool[1]  the pages that the last reservation lacked (0: it had them);
 *   pool[2]  the library's, pool[3] unused; both 0 at the start;
 *   pool[DECODE_ATTN_POOL_HEAD + i], i < F: the free pages, a stack whose top is the last.
 * The caller may fill it by itself (in any order of pages), or by decode_attn_pages_init. Each page is on the
 * stack or in one place of one sequence's row of the block table; a page that sequences share is the caller's
 * to keep out. Calls on one pool must not overlap on the GPU; they may be captured into a graph.
 * `plan` is any plan of the (paged) problem shape; batch may be at most DECODE_ATTN_MAX_PAGED_BATCH
 * (else UNSUPPORTED). Results must lie apart from inputs and from one another (else INVALID_ARG). */

#define DECODE_ATTN_POOL_HEAD 4
#define DECODE_ATTN_MAX_PAGED_BATCH 16384

/* Every page free, page 0 on top. Enqueued on cuda_stream. Errors: INVALID_ARG, UNSUPPORTED (not paged), CUDA. */
int decode_attn_pages_init(const da_plan* plan, int32_t* pool, void* cuda_stream);

/* Pages for a step's rows, and where each row goes. Sequence b holds ctx_lens[b] tokens, in the first
 * ceil(ctx_lens[b] / page_size) entries of its block-table row, and gets T_b rows (row_offsets as above; those
 * past `rows` do not count), so it takes ceil((ctx_lens[b] + T_b) / page_size) - ceil(ctx_lens[b] / page_size)
 * pages. They come off the top of the stack, sequence by sequence, and are entered in block_table, whose other
 * entries stay as they are.
 *   seq_lens    nullable device int32 [batch]: ctx_lens[b] + T_b (what decode_attn_run takes). May be ctx_lens.
 *   slots       nullable device int32 [rows]: the cache row block_table[b][t / page_size] * page_size +
 *               t % page_size of each row's position t = ctx_lens[b] + r - row_offsets[b] (row z of a cache
 *               seen as [tokens, H_kv, d]); -1 for a row without a place: one of no sequence, one at a
 *               position outside [0, capacity), one on an entry outside the pool.
 *   positions   nullable device int32 [rows]: t; 0 for rows of no sequence.
 * The pool has fewer pages than the step takes: it takes none. The tables and the stack stay as they are, every
 * slot is -1, seq_lens[b] = ctx_lens[b], pool[1] says how many pages were missing (0 otherwise), and NO_PAGES
 * is recorded. Nor does it where row_offsets fall anywhere up to `rows`: every slot is -1 and every position 0 then,
 * pool[1] is 0, and BAD_SEQ_LEN is recorded. A length that is negative or would pass the capacity is recorded
 * (BAD_SEQ_LEN) and clamped, as are entries outside the pool (BAD_BLOCK_TABLE; one of the stack is entered as -1).
 *   workspace   nullable, the plan's workspace: takes the findings (decode_attn_check_status); required when
 *               the problem's validate is set: the call then synchronises and returns them.
 * Enqueued on cuda_stream. Errors: INVALID_ARG, UNSUPPORTED, WORKSPACE_TOO_SMALL, CUDA; with validate the
 * findings. */
typedef struct {
  int32_t* pool;
  int32_t* block_table;
  const int32_t* row_offsets;
  const int32_t* ctx_lens;
  int rows;
  int32_t* seq_lens;
  int32_t* slots;
  int32_t* positions;
  void* workspace;
  size_t workspace_bytes;
  void* cuda_stream;
} da_pages_reserve_args;

int decode_attn_pages_reserve(const da_plan* plan, const da_pages_reserve_args* args);

/* Cut sequences back from seq_lens[b] to keep_lens[b] tokens (0: the sequence has ended; a step's drafted tokens
 * that were turned down): pages past ceil(keep_lens[b] / page_size) go onto the stack, and their entries of
 * block_table become -1. The last sequence's last page goes first, so that a reservation given back whole leaves
 * the stack as it was. keep_lens[b] outside [0, seq_lens[b]], and seq_lens[b] outside [0, capacity], are
 * recorded (BAD_SEQ_LEN) and clamped. An entry outside the pool is pushed as -1 and recorded (BAD_BLOCK_TABLE).
 * More pages than the pool has room for (some come back twice): none is taken back, and BAD_BLOCK_TABLE is
 * recorded. keep_lens may be seq_lens. workspace, errors: as above. */
typedef struct {
  int32_t* pool;
  int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* keep_lens;
  void* workspace;
  size_t workspace_bytes;
  void* cuda_stream;
} da_pages_release_args;

int decode_attn_pages_release(const da_plan* plan, const da_pages_release_args* args);

/* ---- Root-mean-square norm ----------------------------------------------------------------------
 * Of every row r and head h of x, over its n elements:
 *     u = x + residual, rounded to the type (u = x without a residual),
 *     y = u (weight + weight_offset) / sqrt(mean(u^2) + eps),
 * hidden rows (heads = 1) with the residual's addition, or q and k heads ahead of a rotary. Statistics, products
 * and y are fp32; each result is rounded once. y goes out in x's type, as E4M3 codes of y / scale (an fp32
 * quotient, rounded to nearest even, values beyond +-448 to +-448, NaN to the NaN code), or both. */

/* Where the codes' scales come from. Found ones are s = max(max |y| / 448, 2^-126), NaNs passed over:
 * DA_SCALE_NONE    no codes.
 * DA_SCALE_TENSOR  scales[0], read by the call (a device float, finite and > 0).
 * DA_SCALE_ROW     one for each row and head: scales [rows, heads], written.
 * DA_SCALE_GROUP   one for each `group` (32, 64 or 128) neighbouring elements, the last group of a row as long
 *                  as n leaves it: scales [rows, heads, ceil(n / group)], written. */
typedef enum { DA_SCALE_NONE = 0, DA_SCALE_TENSOR = 1, DA_SCALE_ROW = 2, DA_SCALE_GROUP = 3 } da_scaling;

#define DECODE_ATTN_NORM_MAX 32768

typedef struct {
  int n;                    /* 1 to DECODE_ATTN_NORM_MAX (else UNSUPPORTED) */
  float eps;                /* finite, >= 0 (0: a row of zeros gives NaN; fp32 and bf16 below 2^-80: slower) */
  float weight_offset;      /* finite; 1 for weights stored as their distance from 1 */
} da_norm_config;

/* One call.
 *   x             device, [rows, heads, n] of `dtype` with strides in elements (any, 0 among them).
 *   residual      nullable, likewise. residual_out: nullable, takes u; needs a residual; may be x or
 *                 residual with its strides.
 *   weight        nullable device [n] (null: y = u / sqrt(...), weight_offset is not used), of `dtype`, or
 *                 fp32 where weight_f32 is set.
 *   out           nullable, takes y in `dtype`; may be x or residual with its strides.
 *   codes, scales nullable, one byte an element, and as da_scaling says (contiguous); given where scaling is
 *                 not NONE. out or codes must be given.
 * Results' rows and heads must lie apart from one another, from other results and from inputs, except as said
 * (else INVALID_ARG). Rows of 32-byte multiples on 32-byte boundaries (codes: 16 or, for fp32, 8) move 32 bytes
 * a lane, others an element a lane. rows = 0: nothing is enqueued. Enqueued on cuda_stream.
 * Errors: INVALID_ARG, UNSUPPORTED (dtype, n, group, more than DECODE_ATTN_ROPE_MAX_HEADS heads), CUDA. */
typedef struct {
  const void* x;
  const void* residual;
  const void* weight;
  void* residual_out;
  void* out;
  void* codes;
  float* scales;
  da_dtype dtype;
  int weight_f32;
  da_scaling scaling;
  int group;
  int rows;
  int heads;
  int64_t x_row_stride, x_head_stride;
  int64_t residual_row_stride, residual_head_stride;
  int64_t residual_out_row_stride, residual_out_head_stride;
  int64_t out_row_stride, out_head_stride;
  int64_t codes_row_stride, codes_head_stride;
  void* cuda_stream;
} da_norm_args;

int decode_attn_norm_apply(const da_norm_config* config, const da_norm_args* args);

/* ---- Low-rank adapters of many requests beside a shared projection -------------------------------
 * Rows x [rows, width] of a batch of requests went through one projection, to y [rows, columns]; the columns
 * are `parts` side by side (q, k and v). Request b's rows (row_offsets as above) take adapter a =
 * adapter_ids[b]:
 *     out[r, part s] = y[r, part s] + scales[a] (x[r] A_{a,s}^T) B_{a,s}^T,
 * A_{a,s} [rank, width], B_{a,s} [out_sizes[s], rank]. A request whose id lies outside [0, adapters) (-1 by
 * convention) has none: out = y. An adapter of a smaller rank has zeros in the rest.
 * Sums are fp32, and the low-rank numbers x A^T are not rounded to the type in between: they enter the second
 * product as two parts, which keep all but 2^-17 (bf16) or 2^-23 (f16, and 2^-32 of the row's largest) of them. fp32
 * products are formed of two tf32 parts of each factor, within 2^-20. out is rounded once. An infinite number gives
 * what the formula gives, but that one of b in 16 bits may come out as NaN. */

#define DECODE_ATTN_ADAPTER_PARTS 4
#define DECODE_ATTN_ADAPTER_MAX_WIDTH (1 << 20)
#define DECODE_ATTN_MAX_ADAPTERS 8192

typedef struct {
  da_dtype dtype;           /* of x, y, a, b and out */
  int width;                /* 1 to DECODE_ATTN_ADAPTER_MAX_WIDTH */
  int parts;                /* 1 to DECODE_ATTN_ADAPTER_PARTS */
  int out_sizes[DECODE_ATTN_ADAPTER_PARTS];   /* columns of each part, 1 to DECODE_ATTN_ADAPTER_MAX_WIDTH */
  int rank;                 /* 8, 16, 32, 64 or 128 */
} da_adapter_config;

/* One call.
 *   x, y, out     device, rows with strides in elements (x's and y's any, 0 among them); out may be y with its
 *                 stride, and lies apart from everything else (else INVALID_ARG).
 *   a             device [adapters, parts, rank, width], contiguous, 16-byte aligned.
 *   b             device [adapters, columns, rank], contiguous, 16-byte aligned (column by column, the parts
 *                 one after another).
 *   scales        nullable device float [adapters] (null: 1).
 *   row_offsets, adapter_ids   device int32 [batch + 1] and [batch].
 *   workspace     nullable device memory, 256-byte aligned, of decode_attn_adapters_workspace bytes, which lies
 *                 apart from everything else (else INVALID_ARG): 16-bit steps of 1024 rows and more then take
 *                 requests of 64 rows and more in two further launches on the tensor cores (tcgen05). Its first
 *                 word takes DEVICE_TIMEOUT, cleared by the caller ahead of the first call; the rest need not be.
 *                 Two calls that can overlap on the GPU need workspaces of their own.
 * Rows of no request are left as they were. Results do not depend on the order of execution. Rows and parts of
 * 16-byte multiples on 16-byte boundaries move 16 bytes a lane, others 8, 4 or an element. Enqueued on
 * cuda_stream. Errors: INVALID_ARG, WORKSPACE_TOO_SMALL, UNSUPPORTED (dtype, rank, parts, sizes; more than
 * DECODE_ATTN_MAX_ADAPTERS adapters or DECODE_ATTN_MAX_PAGED_BATCH requests), CUDA. */
typedef struct {
  const void* x;
  const void* y;
  void* out;
  const void* a;
  const void* b;
  const float* scales;
  const int32_t* row_offsets;
  const int32_t* adapter_ids;
  int rows;
  int batch;
  int adapters;
  int64_t x_row_stride;
  int64_t y_row_stride;
  int64_t out_row_stride;
  void* workspace;
  size_t workspace_bytes;
  void* cuda_stream;
} da_adapter_args;

/* The workspace with which a call over `rows` rows is fastest (0: without one; the size depends on rows, parts and rank
 * alone, whether there is one on the widths too: none for fp32, for few rows or weights, nor where parts * rank passes
 * 256). Host only. Errors: INVALID_ARG. */
int decode_attn_adapters_workspace(const da_adapter_config* config, int rows, size_t* bytes);

/* Synchronise `stream`, then read and clear the finding that calls with this workspace left in its first word:
 * DA_OK or DEVICE_TIMEOUT. */
int decode_attn_adapters_check_status(void* workspace, void* cuda_stream);

int decode_attn_adapters_apply(const da_adapter_config* config, const da_adapter_args* args);

void decode_attn_destroy(da_plan* plan);

const char* decode_attn_strerror(int code);

int decode_attn_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DECODE_ATTN_H */
