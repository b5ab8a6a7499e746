// da_adapters.cu -- low-rank adapters of many requests beside a shared projection: checks and launch.
#include <algorithm>
#include <climits>

#include "da_adapters.cuh"
#include "da_plan.h"

using namespace da;

namespace {

// Rows of a step from which the tall kernels are launched. They cost two launches where no request is long (4 us),
// and a request of 1024 rows 60 us without them.
constexpr int kTallStep = 1024;

bool begins_on_16(const void* p, long long stride, int es) { return aligned(p, 16) && stride * es % 16 == 0; }

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
        may_share(ws, flat(a.b, (long long)a.adapters * columns * c.rank * es)))
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
  p.x_wide = begins_on_16(a.x, a.x_row_stride, es) && (long long)c.width * es % 16 == 0;
  p.y_wide = begins_on_16(a.y, a.y_row_stride, es) && begins_on_16(a.out, a.out_row_stride, es);
  for (int s = 0; s <= c.parts; ++s) p.y_wide = p.y_wide && (long long)p.starts[s] * es % 16 == 0;
  const bool vec = p.x_wide && p.y_wide;
  const int sms = device_sms();
  if (sms <= 0) return DA_ERR_CUDA;

  // Requests of many rows go to the tensor cores' two launches, where the step has enough of them to be worth it
  // and a workspace for their sums is there.
  const bool tall = vec && c.dtype != DA_F32 && a.rows >= kTallStep && a.workspace && tall_fits(p, c.rank, sms);
  p.tall = tall ? kTallRows : INT_MAX;
  if (tall && a.workspace_bytes < tall_workspace(a.rows, low)) return DA_ERR_WORKSPACE_TOO_SMALL;

  // Tiles of 16 rows where an adapter has few, of 64 where it has many (the weights come from L2 once a tile).
  const int groups = std::min(a.batch, a.adapters);
  const long long most_rows = tall ? std::min((long long)a.rows, (kTallRows - 1ll) * a.batch) : a.rows;
  const long long each = most_rows / groups;
  int mt = !vec || c.dtype == DA_F32 || each < 40 ? 1 : each < 64 ? 2 : 4;
  const int column_tiles = low / 8;
  if (mt == 4 && column_tiles > 32) mt = 2;
  if (mt == 2 && column_tiles > 48) mt = 1;
  const int tiles_of_warp = adapter_tiles(mt, column_tiles, p.n_groups);
  p.pitch = low + ((8 - low) & 31);   // (8 mod 32: the accumulators' pairs of eight rows on different banks)
  const int m = 16 * mt;
  // (rows without an adapter are copied whatever their number)
  const long long tiles = (p.copy ? a.rows : most_rows) / m +
                          std::min({(long long)a.batch, (long long)a.adapters + p.copy, (long long)a.rows});
  // CTAs a tile, where an SM holds two at once (by a count that is the same in place, as the sums' order is then;
  // it is a bound, so that up to three an SM are let in).
  p.log_ranks = 3;
  while (p.log_ranks > 0 && (a.rows / m + groups) << p.log_ranks > 3ll * sms) --p.log_ranks;
  const int ranks = 1 << p.log_ranks;
  const size_t smem = adapter_smem(a.adapters, mt, c.parts, c.rank, es, p.n_groups, p.pitch);
  if (smem + 4096 > kSmemLimit || tiles * ranks > INT_MAX) return DA_ERR_UNSUPPORTED;
  const void* fn = c.dtype == DA_F32   ? adapter_kernel_f32(c.rank, mt, tiles_of_warp, vec)
                   : c.dtype == DA_F16 ? adapter_kernel_f16(c.rank, mt, tiles_of_warp, vec)
                                       : adapter_kernel_bf16(c.rank, mt, tiles_of_warp, vec);
  if (!fn) return DA_ERR_UNSUPPORTED;
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
  void* kargs[1] = {&p};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, kargs);
  if (e != cudaSuccess) return cuda_fail(e, "launching the adapter kernel");
  return tall ? launch_tall(p, c.rank, c.dtype == DA_BF16, sms, a.workspace, cfg.stream) : DA_OK;
}

int decode_attn_adapters_workspace(const da_adapter_config* config, int rows, size_t* bytes) {
  if (!config || !bytes || rows < 0 || config->width < 1 || config->parts < 1) return DA_ERR_INVALID_ARG;
  *bytes = 0;
  if (rows < kTallStep || config->dtype == DA_F32) return DA_OK;
  const long long low = (long long)config->parts * config->rank;
  if (low <= 256) *bytes = tall_workspace(rows, (int)low);
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
