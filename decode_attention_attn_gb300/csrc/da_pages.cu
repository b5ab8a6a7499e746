// da_pages.cu -- pages of a paged cache from the lengths of its sequences: what a step needs is taken off a
// stack of free pages and entered in the block table, with each new row's slot; what sequences lose goes back.
//
// Everything is whole numbers and little of it: 4 to 8 bytes a row, a table entry a page. A call is a launch and
// a chain of dependent loads (lengths, then a stack or table entry); only admissions of a million tokens write
// enough to notice. So each CTA takes the prefix sums over all sequences for itself, from lengths that are a few
// KB, where a launch of their own (or a wait between CTAs) would cost more than the rest.
#include <algorithm>
#include <climits>

#include "da_plan.h"

using namespace da;

namespace {

constexpr int kPageThreads = 512;
constexpr int kPageRows = 4;        // rows (or entries) a thread has in flight
constexpr size_t kMostSmem = 4 * (3 * (size_t)DECODE_ATTN_MAX_PAGED_BATCH + 1);   // of any plan's call
static_assert(kMostSmem + 1024 <= kSmemLimit, "the lengths fit shared memory");

struct PageParams {
  int32_t* pool;                // head, then the stack
  int32_t* table;
  const int32_t* row_offsets;   // reserve
  const int32_t* ctx_lens;      // reserve: tokens held; release: tokens held
  const int32_t* keep_lens;     // release
  int32_t* seq_lens;
  int32_t* slots;
  int32_t* positions;
  int32_t* status;
  int batch, rows, max_blocks, num_blocks, capacity;
  int page_shift;               // a page is 2^page_shift tokens
};

struct PageShared {
  int warp_sums[kPageThreads / 32];
  int total;
  int last;
};

__device__ __forceinline__ int clamp_len(long long n, int capacity) {
  return (int)max(0ll, min(n, (long long)capacity));
}
__device__ __forceinline__ int pages_of(int tokens, int shift) {
  return (int)(((unsigned)tokens + (1u << shift) - 1) >> shift);
}
__device__ __forceinline__ void find(const PageParams& p, int bits) {
  if (bits && p.status) atomicOr(p.status, bits);
}

// Sums of pages end here, so that lengths that no pool can hold do not pass 32 bits (a pool is below 2^28 pages).
constexpr int kMostPages = 1 << 29;
__device__ __forceinline__ int add_pages(int a, int b) { return min(a + b, kMostPages); }

// s_count[b] -> the sum over the sequences before b, in place (as long as it is below kMostPages); returns the sum
// over all. A thread adds up a run of sequences (of odd length, so that the threads' places fall on different banks).
__device__ int prefix_sums(int32_t* s_count, int batch, PageShared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = ((batch + kPageThreads - 1) / kPageThreads) | 1;
  const int b0 = min(tid * per, batch), b1 = min(b0 + per, batch);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine = add_pages(mine, s_count[b]);
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int below = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto = add_pages(upto, below);
  }
  if (lane == 31) sh.warp_sums[warp] = upto;
  __syncthreads();
  if (warp == 0) {
    int w = lane < kPageThreads / 32 ? sh.warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int below = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w = add_pages(w, below);
    }
    if (lane < kPageThreads / 32) sh.warp_sums[lane] = w;
    if (lane == 31) sh.total = w;
  }
  __syncthreads();
  int at = upto - mine + (warp ? sh.warp_sums[warp - 1] : 0);
  for (int b = b0; b < b1; ++b) {
    const int n = s_count[b];
    s_count[b] = at;
    at = add_pages(at, n);
  }
  __syncthreads();
  return sh.total;
}

// Whether this CTA is the last of the launch to come here (the pool's ticket counts, and is left at zero). Every
// CTA has read the pool's head and the lengths by then, so the last one may write over them.
__device__ bool last_of_launch(const PageParams& p, PageShared& sh) {
  __syncthreads();
  if (threadIdx.x == 0) {
    bool last = true;
    if (gridDim.x > 1) {
      __threadfence();
      last = atomicAdd(p.pool + 2, 1) == (int)gridDim.x - 1;
      if (last) p.pool[2] = 0;
    }
    sh.last = last;
  }
  __syncthreads();
  return sh.last != 0;
}

// The last i in [lo, n) with first[i] <= x, where first[lo] <= x.
__device__ __forceinline__ int last_at_or_below(const int32_t* first, int lo, int n, int x) {
  int hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// What a sequence holds before and after its rows, and the pages that lie between.
struct Growth {
  int first, need, len;   // pages held, pages to come, tokens then
};
__device__ __forceinline__ Growth growth(const PageParams& p, int ctx, int t) {
  const int held = clamp_len(ctx, p.capacity);
  Growth g;
  g.len = max(clamp_len((long long)ctx + t, p.capacity), held);
  g.first = pages_of(held, p.page_shift);
  g.need = pages_of(g.len, p.page_shift) - g.first;
  return g;
}

// A thread a row (rows in runs, a run a warp): its sequence by a search of the offsets in shared memory, begun
// where the warp's last rows were. The row that is a page's first enters the page in the table: a new page's first
// token is always one of the step's rows. 1M rows of 256 prompts, 65k pages: 8.4 MB written.
__global__ void __launch_bounds__(kPageThreads) reserve_kernel(const __grid_constant__ PageParams p) {
  extern __shared__ int32_t s_lens[];   // offsets [batch + 1], ctx [batch], pages before [batch]
  __shared__ PageShared sh;
  int32_t *s_off = s_lens, *s_ctx = s_off + p.batch + 1, *s_before = s_ctx + p.batch;
  const int tid = threadIdx.x, lane = tid & 31;
  const int free = min(max(p.pool[0], 0), p.num_blocks);
  // offsets clipped to the rows there are
  for (int b = tid; b <= p.batch; b += kPageThreads)
    s_off[b] = min(max(__ldg(p.row_offsets + b), 0), p.rows);
  for (int b = tid; b < p.batch; b += kPageThreads) s_ctx[b] = p.ctx_lens[b];
  __syncthreads();
  int found = 0;
  bool falls = false;
  for (int b = tid; b < p.batch; b += kPageThreads) {
    const int t = max(s_off[b + 1] - s_off[b], 0), ctx = s_ctx[b];
    falls |= s_off[b + 1] < s_off[b];
    if (ctx < 0 || (long long)ctx + t > p.capacity) found = kStatusBadSeqLen;
    s_before[b] = growth(p, ctx, t).need;
  }
  // Where offsets fall, rows are two sequences' at once, and pages would be counted for both that one of them enters:
  // no row is anybody's then, and nothing is taken.
  const bool in_order = !__syncthreads_or(falls);
  const int total = prefix_sums(s_before, p.batch, sh);
  const bool fits = in_order && total <= free;
  if (blockIdx.x == 0)
    find(p, found | (falls ? kStatusBadSeqLen : 0) | (in_order && !fits && tid == 0 ? kStatusNoPages : 0));
  found = 0;

  const int warps = gridDim.x * (kPageThreads / 32), warp = blockIdx.x * (kPageThreads / 32) + (tid >> 5);
  const int run = (int)(((long long)p.rows + warps - 1) / warps);
  const long long r0 = (long long)warp * run;
  const int r1 = (int)min((long long)p.rows, r0 + run);
  int b = 0;
  const int first_row = s_off[0], end_row = s_off[p.batch];
  for (long long rr = r0 + lane; rr < r1; rr += 32 * kPageRows) {
    const int32_t* from[kPageRows];   // where the row's page is read: the table, or the stack
    long long to[kPageRows];          // where it is entered (-1: it is there)
    int entry[kPageRows], in_page[kPageRows], pos[kPageRows];
#pragma unroll
    for (int k = 0; k < kPageRows; ++k) {
      from[k] = nullptr;
      to[k] = -1;
      in_page[k] = pos[k] = 0;
      const int r = (int)min(rr + 32 * k, (long long)INT_MAX);
      if (r >= r1 || r < first_row || r >= end_row || !in_order) continue;
      if (!(s_off[b] <= r && r < s_off[b + 1])) b = last_at_or_below(s_off, s_off[b] <= r ? b : 0, p.batch, r);
      const long long t = (long long)s_ctx[b] + (r - s_off[b]);
      pos[k] = (int)min(t, (long long)INT_MAX);
      if (!fits || t < 0 || t >= p.capacity) continue;
      const Growth g = growth(p, s_ctx[b], max(s_off[b + 1] - s_off[b], 0));
      const int page = (int)t >> p.page_shift, more = page - g.first;
      in_page[k] = (int)t & ((1 << p.page_shift) - 1);
      const long long place = (long long)b * p.max_blocks + page;
      if (more < 0) {
        from[k] = p.table + place;
      } else if (more < g.need) {
        from[k] = p.pool + DECODE_ATTN_POOL_HEAD + (free - 1 - s_before[b] - more);
        if (in_page[k] == 0) to[k] = place;
      }
    }
#pragma unroll
    for (int k = 0; k < kPageRows; ++k) entry[k] = from[k] ? *from[k] : -1;
#pragma unroll
    for (int k = 0; k < kPageRows; ++k) {
      const long long r = rr + 32 * k;
      if (r >= r1) break;
      const bool good = entry[k] >= 0 && entry[k] < p.num_blocks;
      if (from[k] && !good) found = kStatusBadBlockTable;
      if (to[k] >= 0) p.table[to[k]] = good ? entry[k] : -1;
      if (p.slots) p.slots[r] = good ? (entry[k] << p.page_shift) + in_page[k] : -1;
      if (p.positions) p.positions[r] = pos[k];
    }
  }
  find(p, found);
  if (!last_of_launch(p, sh)) return;
  if (p.seq_lens)
    for (int i = tid; i < p.batch; i += kPageThreads)
      p.seq_lens[i] = fits ? growth(p, s_ctx[i], max(s_off[i + 1] - s_off[i], 0)).len
                           : clamp_len(s_ctx[i], p.capacity);
  if (tid == 0) {
    p.pool[0] = fits ? free - total : free;
    p.pool[1] = fits || !in_order ? 0 : total - free;
  }
}

// A thread an entry: the pages past what each sequence keeps go onto the stack, the last sequence's last one
// first, so that a reservation given back whole leaves the stack as it was.
__global__ void __launch_bounds__(kPageThreads) release_kernel(const __grid_constant__ PageParams p) {
  extern __shared__ int32_t s_lens[];   // first page lost [batch], pages lost before [batch]
  __shared__ PageShared sh;
  int32_t *s_first = s_lens, *s_before = s_first + p.batch;
  const int tid = threadIdx.x;
  const int free = min(max(p.pool[0], 0), p.num_blocks);
  int found = 0;
  for (int b = tid; b < p.batch; b += kPageThreads) {
    const int raw = __ldg(p.ctx_lens + b), keep = __ldg(p.keep_lens + b);
    if (raw < 0 || raw > p.capacity || keep < 0 || keep > raw) found = kStatusBadSeqLen;
    const int len = clamp_len(raw, p.capacity);
    s_first[b] = pages_of(min(max(keep, 0), len), p.page_shift);
    s_before[b] = pages_of(len, p.page_shift) - s_first[b];
  }
  __syncthreads();
  const int total = prefix_sums(s_before, p.batch, sh);
  const bool room = free + (long long)total <= p.num_blocks;   // not so where pages come back twice
  if (!room) found |= kStatusBadBlockTable;
  if (blockIdx.x == 0) find(p, found);
  found = 0;
  const int threads = gridDim.x * kPageThreads;
  for (long long i0 = (long long)blockIdx.x * kPageThreads + tid; room && i0 < total;
       i0 += (long long)threads * kPageRows) {
    long long place[kPageRows];
    int entry[kPageRows];
#pragma unroll
    for (int k = 0; k < kPageRows; ++k) {
      const long long i = i0 + (long long)threads * k;
      place[k] = -1;
      if (i >= total) continue;
      const int b = last_at_or_below(s_before, 0, p.batch, (int)i);
      place[k] = (long long)b * p.max_blocks + s_first[b] + ((int)i - s_before[b]);
    }
#pragma unroll
    for (int k = 0; k < kPageRows; ++k) entry[k] = place[k] >= 0 ? p.table[place[k]] : -1;
#pragma unroll
    for (int k = 0; k < kPageRows; ++k) {
      if (place[k] < 0) continue;
      const bool good = entry[k] >= 0 && entry[k] < p.num_blocks;
      if (!good) found = kStatusBadBlockTable;
      p.pool[DECODE_ATTN_POOL_HEAD + free + (total - 1 - (i0 + (long long)threads * k))] = good ? entry[k] : -1;
      p.table[place[k]] = -1;
    }
  }
  find(p, found);
  if (last_of_launch(p, sh) && tid == 0) p.pool[0] = room ? free + total : free;
}

__global__ void pool_init_kernel(int32_t* pool, int num_blocks) {
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < DECODE_ATTN_POOL_HEAD + num_blocks;
       i += gridDim.x * blockDim.x)
    pool[i] = i >= DECODE_ATTN_POOL_HEAD ? num_blocks - 1 - (i - DECODE_ATTN_POOL_HEAD) : i == 0 ? num_blocks : 0;
}

int checks(const da_plan* plan, const void* pool, const void* table, const void* workspace,
           size_t workspace_bytes) {
  if (!plan) return DA_ERR_INVALID_ARG;
  if (!plan->prob.paged || plan->prob.batch > DECODE_ATTN_MAX_PAGED_BATCH) return DA_ERR_UNSUPPORTED;
  if (!pool || !table || !aligned(pool, 16) || !aligned(table, 4)) return DA_ERR_INVALID_ARG;
  if (workspace ? !aligned(workspace, 256) : plan->prob.validate != 0) return DA_ERR_INVALID_ARG;
  if (workspace && workspace_bytes < plan->ws_bytes) return DA_ERR_WORKSPACE_TOO_SMALL;
  return DA_OK;
}

// A buffer of a call: results lie apart from each other and from every input (but one that may be itself).
struct Buffer {
  const void* p;
  long long words;
  bool result;
};
bool lie_well(const Buffer* v, int n) {
  for (int i = 0; i < n; ++i)
    for (int j = i + 1; j < n; ++j)
      if ((v[i].result || v[j].result) && overlap(v[i].p, 4 * v[i].words, v[j].p, 4 * v[j].words)) return false;
  return true;
}

PageParams page_params(const da_plan& pl, int32_t* pool, int32_t* table, void* workspace) {
  Params c;
  fill_common(pl, c, table, nullptr, workspace);
  PageParams p = {};
  p.pool = pool;
  p.table = table;
  p.status = c.status;
  p.batch = c.batch;
  p.max_blocks = c.max_blocks;
  p.num_blocks = c.num_blocks;
  p.capacity = c.capacity;
  while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
  return p;
}

int launch(const da_plan& pl, const PageParams& p, const void* fn, long long items, size_t smem, void* workspace,
           void* cuda_stream) {
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t e = cudaSuccess;
  if (pl.prob.validate)
    e = cudaMemsetAsync(static_cast<char*>(workspace) + pl.off_status, 0, 4, stream);
  if (e != cudaSuccess) return cuda_fail(e, "preparing the page kernel");
  if (smem > 40 * 1024) {   // to the most that any call takes: the limit is the kernel's, which other threads launch too
    const int rc = raise_smem(fn, kMostSmem, 0);
    if (rc != DA_OK) return rc;
  }
  const long long per = (long long)kPageThreads * kPageRows;
  const int grid = (int)std::max(1ll, std::min((items + per - 1) / per, 2ll * pl.num_sms));
  void* args[1] = {const_cast<PageParams*>(&p)};
  e = cudaLaunchKernel(fn, dim3((unsigned)grid), dim3(kPageThreads), args, smem, stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the page kernel");
  return pl.prob.validate ? decode_attn_check_status(&pl, workspace, cuda_stream) : DA_OK;
}

}  // namespace

extern "C" {

int decode_attn_pages_init(const da_plan* plan, int32_t* pool, void* cuda_stream) {
  if (!plan) return DA_ERR_INVALID_ARG;
  if (!plan->prob.paged) return DA_ERR_UNSUPPORTED;
  if (!pool || !aligned(pool, 16)) return DA_ERR_INVALID_ARG;
  const int n = plan->prob.num_physical_blocks;
  pool_init_kernel<<<std::min(n / 1024 + 1, plan->num_sms), 256, 0, static_cast<cudaStream_t>(cuda_stream)>>>(pool, n);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? DA_OK : cuda_fail(e, "launching the pool's initialisation");
}

int decode_attn_pages_reserve(const da_plan* plan, const da_pages_reserve_args* args) {
  if (!plan || !args) return DA_ERR_INVALID_ARG;
  const da_pages_reserve_args& a = *args;
  const int rc = checks(plan, a.pool, a.block_table, a.workspace, a.workspace_bytes);
  if (rc != DA_OK) return rc;
  if (a.rows < 0 || !a.row_offsets || !a.ctx_lens || !aligned(a.row_offsets, 4) || !aligned(a.ctx_lens, 4) ||
      !aligned(a.seq_lens, 4) || !aligned(a.slots, 4) || !aligned(a.positions, 4))
    return DA_ERR_INVALID_ARG;
  const da_problem& pr = plan->prob;
  const bool in_place = a.seq_lens == a.ctx_lens;
  const Buffer all[] = {{a.pool, DECODE_ATTN_POOL_HEAD + (long long)pr.num_physical_blocks, true},
                        {a.block_table, (long long)pr.batch * pr.max_blocks_per_seq, true},
                        {a.row_offsets, pr.batch + 1ll, false},
                        {a.ctx_lens, pr.batch, in_place},
                        {in_place ? nullptr : a.seq_lens, pr.batch, true},
                        {a.slots, a.rows, true},
                        {a.positions, a.rows, true}};
  if (!lie_well(all, 7)) return DA_ERR_INVALID_ARG;
  PageParams p = page_params(*plan, a.pool, a.block_table, a.workspace);
  p.row_offsets = a.row_offsets;
  p.ctx_lens = a.ctx_lens;
  p.seq_lens = a.seq_lens;
  p.slots = a.slots;
  p.positions = a.positions;
  p.rows = a.rows;
  return launch(*plan, p, reinterpret_cast<const void*>(&reserve_kernel), a.rows, 4 * (3 * (size_t)pr.batch + 1),
                a.workspace, a.cuda_stream);
}

int decode_attn_pages_release(const da_plan* plan, const da_pages_release_args* args) {
  if (!plan || !args) return DA_ERR_INVALID_ARG;
  const da_pages_release_args& a = *args;
  const int rc = checks(plan, a.pool, a.block_table, a.workspace, a.workspace_bytes);
  if (rc != DA_OK) return rc;
  if (!a.seq_lens || !a.keep_lens || !aligned(a.seq_lens, 4) || !aligned(a.keep_lens, 4)) return DA_ERR_INVALID_ARG;
  const da_problem& pr = plan->prob;
  const long long entries = (long long)pr.batch * pr.max_blocks_per_seq;
  const Buffer all[] = {{a.pool, DECODE_ATTN_POOL_HEAD + (long long)pr.num_physical_blocks, true},
                        {a.block_table, entries, true},
                        {a.seq_lens, pr.batch, false},
                        {a.keep_lens, pr.batch, false}};
  if (!lie_well(all, 4)) return DA_ERR_INVALID_ARG;
  PageParams p = page_params(*plan, a.pool, a.block_table, a.workspace);
  p.ctx_lens = a.seq_lens;
  p.keep_lens = a.keep_lens;
  // How many entries go back the device alone knows: threads for every second one, which
  // take them 4 at a time.
  return launch(*plan, p, reinterpret_cast<const void*>(&release_kernel), entries / 2, 4 * (2 * (size_t)pr.batch),
                a.workspace, a.cuda_stream);
}

}  // extern "C"
