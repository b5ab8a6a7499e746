// da_adapters.cu -- low-rank adapters of many requests beside a shared projection: checks and launch.
#include <algorithm>
#include <climits>
#include <initializer_list>

#include "da_adapters.cuh"
#include "da_plan.h"

using namespace da;

namespace {

// Rows of a step from which the tall kernels may be launched.
constexpr int kTallStep = 1024;

// Whether they are worth it. The short kernel takes, in effect, x, y and out at 4 TB/s and an adapter's weights once
// for 16 rows at 12 (they come from L2); the tall ones x, y and out at 4.6, with 11 us more of launches and first
// operands (rank 64: 17, as the products weigh; rank 128: 47, as its operands fill the registers). bf16, 4096 wide,
// short and tall in us: to 6144 columns, 8000 rows of rank 64 183 and 83, of rank 16 95 and 71, 2000 rows 50 and 36, 24
// and 26; to 4096 columns, 2000 rows of rank 64 23 and 27, 3200 of rank 128 71 and 81, 8000 147 and 102.
bool tall_pays(const da_adapter_config& c, long long rows, long long columns) {
  const long long low = (long long)c.parts * c.rank;
  const double weights = 2.0 * (rows / kAdapterTile) * (low * c.width + columns * c.rank);
  const double others = 2.0 * rows * (c.width + 2 * columns);
  return weights + 0.4 * others > 130e6 + (c.rank < 64 ? 0.0 : c.rank == 64 ? 72e6 : 432e6);
}

// The most of 16, 8 and 4 bytes (fp32: 16) that all of v are multiples of, else an element's.
int unit_of(std::initializer_list<long long> v, int es) {
  unsigned long long bits = 0;
  for (long long x : v) bits |= (unsigned long long)x;
  return bits % 16 == 0 ? 16 : es == 4 ? 4 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : es;
}

}  // namespace

extern "C" {

int decode_attn_adapters_apply(const da_adapter_config* config, const da_adapter_args* args) {
  if (!config || !args) return DA_ERR_INVALID_ARG;
  const da_adapter_config& c = *config;
  const da_adapter_args& a = *args;
  if (c.width < 1 || c.parts < 1 || a.rows < 0 || a.batch < 1 || a.adapters < 1) return DA_ERR_INVALID_ARG;
  if (c.dtype < DA_F32 || c.dtype > DA_BF16 || c.parts > DECODE_ATTN_ADAPTER_PARTS ||
      (c.rank != 8 && c.rank != 16 && c.rank != 32 && c.rank != 64 && c.rank != 128) ||
      c.width > DECODE_ATTN_ADAPTER_MAX_WIDTH || a.adapters > DECODE_ATTN_MAX_ADAPTERS ||
      a.batch > DECODE_ATTN_MAX_PAGED_BATCH)
    return DA_ERR_UNSUPPORTED;
  AdapterParams p = {};
  long long columns = 0;
  for (int s = 0; s < c.parts; ++s) {
    if (c.out_sizes[s] < 1) return DA_ERR_INVALID_ARG;
    if (c.out_sizes[s] > DECODE_ATTN_ADAPTER_MAX_WIDTH) return DA_ERR_UNSUPPORTED;
    p.starts[s] = (int)columns;
    columns += c.out_sizes[s];
    p.chunks[s + 1] = p.chunks[s] + (c.out_sizes[s] + 31) / 32;
  }
  p.starts[c.parts] = (int)columns;
  if (a.rows == 0) return DA_OK;
  const int es = elem_size(c.dtype);
  if (!a.x || !a.y || !a.out || !a.a || !a.b || !a.row_offsets || !a.adapter_ids || !aligned(a.x, es) ||
      !aligned(a.y, es) || !aligned(a.out, es) || !aligned(a.a, 16) || !aligned(a.b, 16) || !aligned(a.scales, 4) ||
      !aligned(a.row_offsets, 4) || !aligned(a.adapter_ids, 4))
    return DA_ERR_INVALID_ARG;
  const int low = c.parts * c.rank;
  const RowRuns x = runs(a.x, a.rows, a.x_row_stride, 1, 0, c.width, es);
  const RowRuns y = runs(a.y, a.rows, a.y_row_stride, 1, 0, (int)columns, es);
  const RowRuns out = runs(a.out, a.rows, a.out_row_stride, 1, 0, (int)columns, es);
  auto flat = [](const void* at, long long bytes) { return RowRuns{(uint64_t)(uintptr_t)at, 1, 0, 1, 0, bytes}; };
  if (!lie_apart(out) || !result_ok(y, out) || may_share(x, out) ||
      may_share(flat(a.a, (long long)a.adapters * low * c.width * es), out) ||
      may_share(flat(a.b, (long long)a.adapters * columns * c.rank * es), out) ||
      (a.scales && may_share(flat(a.scales, 4ll * a.adapters), out)) ||
      may_share(flat(a.row_offsets, 4ll * (a.batch + 1)), out) || may_share(flat(a.adapter_ids, 4ll * a.batch), out) ||
      !aligned(a.workspace, 256))
    return DA_ERR_INVALID_ARG;
  if (a.workspace && a.workspace_bytes) {   // the sums are results too
    const RowRuns ws = flat(a.workspace, (long long)a.workspace_bytes);
    if (may_share(ws, out) || may_share(ws, x) || may_share(ws, y) ||
        may_share(ws, flat(a.a, (long long)a.adapters * low * c.width * es)) ||
        may_share(ws, flat(a.b, (long long)a.adapters * columns * c.rank * es)) ||
        (a.scales && may_share(ws, flat(a.scales, 4ll * a.adapters))) ||
        may_share(ws, flat(a.row_offsets, 4ll * (a.batch + 1))) || may_share(ws, flat(a.adapter_ids, 4ll * a.batch)))
      return DA_ERR_INVALID_ARG;
  }
  p.x = a.x;
  p.y = a.y;
  p.out = a.out;
  p.a = a.a;
  p.b = a.b;
  p.scales = a.scales;
  p.row_offsets = a.row_offsets;
  p.ids = a.adapter_ids;
  p.x_rs = a.x_row_stride;
  p.y_rs = a.y_row_stride;
  p.out_rs = a.out_row_stride;
  p.rows = a.rows;
  p.batch = a.batch;
  p.adapters = a.adapters;
  p.width = c.width;
  p.parts = c.parts;
  p.copy = a.out != a.y;
  // What x (and A, whose rows are as wide) and y and out move by, 16 bytes in a kernel of its own. (500 rows of 5196
  // bf16 to 3436: 14.2 us by 8 bytes, of 5198 to 3442 15.6 by 4, 27 by elements.)
  p.x_unit = unit_of({(long long)(uintptr_t)a.x, (long long)a.x_row_stride * es, (long long)c.width * es}, es);
  p.y_unit = unit_of({(long long)(uintptr_t)a.y, (long long)a.y_row_stride * es, (long long)(uintptr_t)a.out,
                      (long long)a.out_row_stride * es}, es);
  for (int s = 0; s <= c.parts; ++s) p.y_unit = std::min(p.y_unit, unit_of({(long long)p.starts[s] * es}, es));
  const bool vec = p.x_unit == 16 && p.y_unit == 16;
  const int sms = device_sms();
  if (sms <= 0) return DA_ERR_CUDA;

  // Requests of many rows go to the tensor cores' two launches, where the step has enough of them to be worth it
  // and a workspace for their sums is there.
  const bool tall = vec && c.dtype != DA_F32 && a.rows >= kTallStep && a.workspace && tall_fits(p, c.rank, sms);
  p.tall = tall ? kTallRows : INT_MAX;
  if (tall && a.workspace_bytes < tall_workspace(a.rows, low)) return DA_ERR_WORKSPACE_TOO_SMALL;

  const int groups = std::min(a.batch, a.adapters);
  const long long most_rows = tall ? std::min((long long)a.rows, (kTallRows - 1ll) * a.batch) : a.rows;
  const int tiles_of_warp = adapter_tiles(low / 8, p.n_groups);
  p.pitch = low + ((8 - low) & 31);   // (8 mod 32: the accumulators' pairs of eight rows on different banks)
  // CTAs a tile: as many as run at once, two an SM (by a count of tiles that is the same in place, as the sums'
  // order is then), by the tiles that are likely: a half full one an adapter; beside the tall kernels few. More
  // than run at once begin over: 26 requests of 33 rows 15.9 us with 4 a tile, 25 with 8; 62 of 2 rows, 2176 wide, 12.1
  // with 4 and 21.7 with 8. (Beside the tall kernels 4 at most, as their tiles may be many all the same: 4 requests of
  // 900 rows and 60 of one 60 us with 8, 68 with 4, 122 with 1; 64 of 20 to 40 rows 85, 63 and 83.)
  p.log_ranks = tall ? 2 : 3;
  const long long likely = tall ? std::max(groups, a.batch / 4)
                                : std::max((long long)groups, most_rows / kAdapterTile + groups / 2);
  while (p.log_ranks > 0 && likely << p.log_ranks > 2ll * sms) --p.log_ranks;
  const int ranks = 1 << p.log_ranks;
  // one cluster for each tile there can be, and what copies rows without an adapter (however many)
  const int copiers = p.copy ? std::min(a.rows / kAdapterTile + 1, std::max(2 * sms >> p.log_ranks, 1)) : 0;
  const long long tiles = most_rows / kAdapterTile + std::min(groups, a.rows) + copiers;
  const size_t smem = adapter_smem(a.adapters, c.parts, c.rank, es, p.n_groups, p.pitch);
  if (smem + 4096 > kSmemLimit || tiles * ranks > INT_MAX) return DA_ERR_UNSUPPORTED;
  const void* fn = c.dtype == DA_F32   ? adapter_kernel_f32(c.rank, tiles_of_warp, vec)
                   : c.dtype == DA_F16 ? adapter_kernel_f16(c.rank, tiles_of_warp, vec)
                                       : adapter_kernel_bf16(c.rank, tiles_of_warp, vec);
  if (smem > 40 * 1024) {
    const int rc = raise_smem(fn, kSmemLimit - 4096, 0);
    if (rc != DA_OK) return rc;
  }
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ranks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * ranks));
  cfg.blockDim = dim3(kAdapterThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(a.cuda_stream);
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (tall) return launch_tall(p, c.rank, c.dtype == DA_BF16, sms, a.workspace, cfg, fn);
  void* kargs[1] = {&p};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, kargs);
  return e == cudaSuccess ? DA_OK : cuda_fail(e, "launching the adapter kernel");
}

int decode_attn_adapters_workspace(const da_adapter_config* config, int rows, size_t* bytes) {
  if (!config || !bytes || rows < 0 || config->width < 1 || config->parts < 1 || config->rank < 1 ||
      config->parts > DECODE_ATTN_ADAPTER_PARTS)
    return DA_ERR_INVALID_ARG;
  *bytes = 0;
  if (rows < kTallStep || config->dtype == DA_F32) return DA_OK;
  const long long low = (long long)config->parts * config->rank;
  long long columns = 0;
  for (int s = 0; s < config->parts; ++s) columns += config->out_sizes[s];
  if (low <= 256 && tall_pays(*config, rows, columns)) *bytes = tall_workspace(rows, (int)low);
  return DA_OK;
}

int decode_attn_adapters_check_status(void* workspace, void* cuda_stream) {
  if (!workspace) return DA_ERR_INVALID_ARG;
  cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
  int32_t st = 0;
  cudaError_t e = cudaMemcpyAsync(&st, workspace, 4, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemsetAsync(workspace, 0, 4, stream);
  if (e != cudaSuccess) return cuda_fail(e, "reading the device status");
  return status_to_error(st);
}

}  // extern "C"
