// da_norm.cu -- root-mean-square norms: checks and launch.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <map>
#include <mutex>
#include <tuple>

#include "da_norm.cuh"
#include "da_plan.h"

using namespace da;

namespace {

// Whether a row tensor's runs begin on multiples of `bytes`.
bool begins_on(const void* p, long long rs, long long hs, int es, int bytes) {
  return !p || (aligned(p, bytes) && rs * es % bytes == 0 && hs * es % bytes == 0);
}

// Blocks of `fn` that an SM holds, asked for once a device.
int resident_blocks(const void* fn, int threads, int& count) {
  static std::mutex mu;
  static std::map<std::tuple<int, const void*, int>, int> known;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  std::lock_guard<std::mutex> lk(mu);
  const auto key = std::make_tuple(dev, fn, threads);
  const auto at = known.find(key);
  if (at != known.end()) {
    count = at->second;
    return DA_OK;
  }
  e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&count, fn, threads, 0);
  if (e != cudaSuccess) return cuda_fail(e, "asking for the norm kernel's occupancy");
  if (count < 1) return text_fail("the norm kernel does not fit an SM");
  try {
    known.emplace(key, count);
  } catch (...) {   // (asked again next time)
  }
  return DA_OK;
}

}  // namespace

extern "C" {

int decode_attn_norm_apply(const da_norm_config* config, const da_norm_args* args) {
  if (!config || !args) return DA_ERR_INVALID_ARG;
  const da_norm_config& c = *config;
  const da_norm_args& a = *args;
  if (c.n < 1 || !std::isfinite(c.eps) || c.eps < 0.f || !std::isfinite(c.weight_offset)) return DA_ERR_INVALID_ARG;
  if (c.n > DECODE_ATTN_NORM_MAX || a.dtype < DA_F32 || a.dtype > DA_BF16 ||
      a.heads > DECODE_ATTN_ROPE_MAX_HEADS)
    return DA_ERR_UNSUPPORTED;
  if (a.rows < 0 || a.heads < 1 || (a.weight_f32 != 0 && a.weight_f32 != 1) || a.scaling < DA_SCALE_NONE ||
      a.scaling > DA_SCALE_GROUP)
    return DA_ERR_INVALID_ARG;
  if (a.scaling == DA_SCALE_GROUP && a.group != 32 && a.group != 64 && a.group != 128) return DA_ERR_UNSUPPORTED;
  if (a.rows == 0) return DA_OK;
  const int es = elem_size(a.dtype);
  if (!a.x || (!a.out && !a.codes) || (a.residual_out && !a.residual) ||
      (a.codes != nullptr) != (a.scaling != DA_SCALE_NONE) || (a.scales != nullptr) != (a.scaling != DA_SCALE_NONE))
    return DA_ERR_INVALID_ARG;
  if (!aligned(a.x, es) || !aligned(a.residual, es) || !aligned(a.residual_out, es) || !aligned(a.out, es) ||
      !aligned(a.weight, a.weight_f32 ? 4 : es) || !aligned(a.scales, 4))
    return DA_ERR_INVALID_ARG;
  const long long items = (long long)a.rows * a.heads;
  const int groups = a.scaling == DA_SCALE_GROUP ? (c.n + a.group - 1) / a.group : 1;
  // where everything lies: results apart from one another and from inputs (but x or the residual itself)
  const long long scale_count = a.scaling == DA_SCALE_TENSOR ? 1 : items * groups;
  const RowRuns in[4] = {
      runs(a.x, a.rows, a.x_row_stride, a.heads, a.x_head_stride, c.n, es),
      runs(a.residual, a.rows, a.residual_row_stride, a.heads, a.residual_head_stride, c.n, es),
      runs(a.weight, 1, 0, 1, 0, c.n, a.weight_f32 ? 4 : es),
      {(uint64_t)(uintptr_t)a.scales, 1, 0, 1, 0, 4 * scale_count}};
  const bool in_there[4] = {true, a.residual != nullptr, a.weight != nullptr, a.scales != nullptr};
  const RowRuns res[3] = {
      runs(a.residual_out, a.rows, a.residual_out_row_stride, a.heads, a.residual_out_head_stride, c.n, es),
      runs(a.out, a.rows, a.out_row_stride, a.heads, a.out_head_stride, c.n, es),
      runs(a.codes, a.rows, a.codes_row_stride, a.heads, a.codes_head_stride, c.n, 1)};
  const bool there[3] = {a.residual_out != nullptr, a.out != nullptr, a.codes != nullptr};
  for (int i = 0; i < 3; ++i) {
    if (!there[i]) continue;
    if (!lie_apart(res[i])) return DA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (there[j] && may_share(res[i], res[j])) return DA_ERR_INVALID_ARG;
    for (int j = 0; j < 4; ++j)
      if (in_there[j] && (j < 2 && i < 2 ? !result_ok(in[j], res[i]) : may_share(in[j], res[i])))
        return DA_ERR_INVALID_ARG;
  }
  if (a.scales && a.scaling != DA_SCALE_TENSOR)   // the scales are results then
    for (int j = 0; j < 3; ++j)
      if (in_there[j] && may_share(in[j], in[3])) return DA_ERR_INVALID_ARG;
  NormParams p;
  std::memset(&p, 0, sizeof p);
  p.x = a.x;
  p.residual = a.residual;
  p.weight = a.weight;
  p.total = a.residual_out;
  p.out = a.out;
  p.codes = static_cast<uint8_t*>(a.codes);
  p.scales = a.scales;
  p.x_rs = a.x_row_stride;
  p.x_hs = a.x_head_stride;
  p.res_rs = a.residual_row_stride;
  p.res_hs = a.residual_head_stride;
  p.tot_rs = a.residual_out_row_stride;
  p.tot_hs = a.residual_out_head_stride;
  p.out_rs = a.out_row_stride;
  p.out_hs = a.out_head_stride;
  p.code_rs = a.codes_row_stride;
  p.code_hs = a.codes_head_stride;
  p.items = items;
  p.heads = a.heads;
  p.n = c.n;
  p.weight_f32 = a.weight_f32;
  p.scaling = a.scaling;
  p.group = a.group;
  p.groups = groups;
  p.eps = c.eps;
  p.offset = c.weight_offset;
  const int E = 32 / es;
  const bool vec = c.n % E == 0 && begins_on(a.x, p.x_rs, p.x_hs, es, 32) &&
                   begins_on(a.residual, p.res_rs, p.res_hs, es, 32) &&
                   begins_on(a.residual_out, p.tot_rs, p.tot_hs, es, 32) &&
                   begins_on(a.out, p.out_rs, p.out_hs, es, 32) && begins_on(a.codes, p.code_rs, p.code_hs, 1, E) &&
                   aligned(a.weight, 32);
  const int sms = device_sms();
  if (sms <= 0) return DA_ERR_CUDA;
  if (c.eps < kLeastEps && a.dtype != DA_F16) {   // (f16's squares are 2^-48 and more)
    const int threads = std::min(kCarefulThreads, (c.n + 31) / 32 * 32);
    const void* fn = a.dtype == DA_F32 ? careful_norm_kernel_f32() : careful_norm_kernel_bf16();
    void* kargs[1] = {&p};
    const cudaError_t e = cudaLaunchKernel(fn, dim3((unsigned)std::min(items, 8ll * sms)), dim3(threads), kargs, 0,
                                           static_cast<cudaStream_t>(a.cuda_stream));
    return e == cudaSuccess ? DA_OK : cuda_fail(e, "launching the norm kernel");
  }
  // Rows that begin anywhere, but alike in every tensor (see NormLayout), where a row takes a block.
  const int V = E / 2;
  auto alike = [&](const void* at, long long rs, int bytes) {
    return !at || (aligned(at, bytes) && (((unsigned long long)rs - (unsigned long long)p.x_rs) & (V - 1)) == 0);
  };
  const bool shifted = !vec && a.heads == 1 && a.scaling != DA_SCALE_GROUP && c.n > 32 * E &&
                       c.n <= DECODE_ATTN_NORM_MAX - V && alike(a.x, p.x_rs, 16) &&
                       alike(a.residual, p.res_rs, 16) && alike(a.residual_out, p.tot_rs, 16) &&
                       alike(a.out, p.out_rs, 16) && alike(a.codes, p.code_rs, V);
  const int layout = vec ? kWide : shifted ? kShifted : kScattered;
  // Threads of a row: one for each of its units up to a warp; then whole warps, of two units a thread where there
  // are more than 256. (A scattered row's: whole warps throughout.)
  const int units = vec ? c.n / E : shifted ? (c.n + V - 1 + E - 1) / E : (c.n + 32 * E - 1) / (32 * E);
  p.units = units;
  int threads, per = 1, items_each;
  bool block = false;
  if (vec && units <= 32) {
    p.lanes = 1;
    while (p.lanes < units) p.lanes *= 2;
    threads = 128;
    per = threads / p.lanes;
    items_each = 1;
  } else if (!vec && !shifted && units <= 1) {
    p.lanes = 32;
    threads = 128;
    per = 4;
    items_each = 1;
  } else {
    block = true;
    const int warps = vec || shifted ? (units + 31) / 32 : units;   // at a unit a thread
    // kWide, many rows: two units a thread from 4 warps on, as that has more on its way for the registers (8192 rows
    // of 4096 bf16 with residual and groups: 56 us with one, 44 with two; 620 rows 7.3 and 5.5). kScattered: one as
    // long as a block holds it (4000 rows of 4107 bf16 with residual and groups: 59 us with one, 181 with two).
    const int ones = vec ? (items >= 4ll * sms ? 3 : 8) : shifted ? 8 : 16;
    items_each = warps <= ones ? 1 : warps <= 32 ? 2 : warps <= 64 ? 4 : 8;
    threads = 32 * ((warps + items_each - 1) / items_each);
    p.lanes = threads;
  }
  const bool residual = a.residual != nullptr;
  const void* fn = a.dtype == DA_F32   ? norm_kernel_f32(layout, items_each, block, residual)
                   : a.dtype == DA_F16 ? norm_kernel_f16(layout, items_each, block, residual)
                                       : norm_kernel_bf16(layout, items_each, block, residual);
  // as many blocks as run at once: a thread loads its next row's share while it works on one
  int resident = 0;
  const int rc = resident_blocks(fn, threads, resident);
  if (rc != DA_OK) return rc;
  long long blocks = std::min((items + per - 1) / per, (long long)sms * resident);
  if (shifted && blocks < items) blocks = std::max<long long>(V, blocks / V * V);   // (a block's rows begin alike)
  void* kargs[1] = {&p};
  const cudaError_t e = cudaLaunchKernel(fn, dim3((unsigned)blocks), dim3(threads), kargs, 0,
                                         static_cast<cudaStream_t>(a.cuda_stream));
  return e == cudaSuccess ? DA_OK : cuda_fail(e, "launching the norm kernel");
}

}  // extern "C"
