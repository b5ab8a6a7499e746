// da_norm.cu -- root-mean-square norm of rows, with the residual's addition ahead of it and an output in 8 bits
// behind it:
//     h = x + residual (rounded to the type: what the next block adds to),
//     y = h (w + o) / sqrt(mean(h^2) + eps),   code = E4M3(y / scale),
// scale given, or max |y| / 448 over the row or over groups of 32, 64 or 128 elements.
//
// Bound by HBM: every element is read once and written once, about 10 operations between. A row stays in registers
// from the loads to the stores; what the row's threads exchange is one sum and one maximum, together. The maximum
// needs no second pass over y: rounding is monotone, so max |y| = round(max |h (w + o)| r) with y = round(h (w + o) r).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "da_plan.h"
#include "da_rowvec.cuh"

using namespace da;

namespace {

constexpr float kE4M3Max = 448.f;
constexpr float kFarScale = 5.421010862e-20f;    // 2^-64
constexpr float kLeastScale = 1.17549435e-38f;   // 2^-126: of a row of zeros; no scale is subnormal

struct NormParams {
  const void *x, *residual, *weight;
  void *total, *out;
  uint8_t* codes;
  float* scales;
  // strides in elements, of rows and heads
  long long x_rs, x_hs, res_rs, res_hs, tot_rs, tot_hs, out_rs, out_hs, code_rs, code_hs;
  long long items;              // rows * heads
  int heads, n, units;          // units: of E elements, or (not VEC) of 32 E elements a warp
  int lanes;                    // lanes a row takes (a power of two; a warp's or more: BLOCK)
  int weight_f32, scaling, group, groups;
  float eps, offset;
};

template <typename T>
struct Unit {   // elements a lane holds of a row, side by side: 32 bytes
  static constexpr int E = 32 / (int)sizeof(T);
};

template <typename T>
__device__ __forceinline__ float widen(T x) {
  if constexpr (std::is_same<T, float>::value) return x;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
  else return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T narrow(float x) {
  if constexpr (std::is_same<T, float>::value) return x;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// 8 words of T as floats, and back (rounded to nearest even).
template <typename T>
__device__ __forceinline__ void unpack(const uint32_t* w, float* f) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (std::is_same<T, float>::value) {
      f[i] = __uint_as_float(w[i]);
    } else if constexpr (std::is_same<T, __half>::value) {
      __half2 h;
      memcpy(&h, &w[i], 4);
      const float2 g = __half22float2(h);
      f[2 * i] = g.x;
      f[2 * i + 1] = g.y;
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <typename T>
__device__ __forceinline__ void pack(const float* f, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (std::is_same<T, float>::value) w[i] = __float_as_uint(f[i]);
    else w[i] = pack2(f[2 * i], f[2 * i + 1], T());
  }
}
__device__ __forceinline__ void load8(const void* p, uint32_t* w) {
  uint4 a, b;
  load32(p, a, b);
  w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
}
__device__ __forceinline__ void store8(void* p, const uint32_t* w) {
  store32(p, make_uint4(w[0], w[1], w[2], w[3]), make_uint4(w[4], w[5], w[6], w[7]));
}

// The sum of v over a row's threads, by its block or `lanes` lanes.
template <bool BLOCK>
__device__ __forceinline__ float row_sum(float v, int lanes, float* s_part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (!BLOCK && o >= lanes) continue;
    v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  if constexpr (BLOCK) {
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < warps; ++w) v += s_part[w];
    __syncthreads();
  }
  return v;
}

// A row's threads: a block (BLOCK), or `lanes` lanes of a warp, several rows a warp. A thread holds ITEMS units of E
// elements. VEC: a unit is 32 bytes of the row, loaded at once, and the row's units go round the threads. Otherwise
// (an odd width, rows that lie anywhere) a warp holds 32 E elements, a lane every 32nd of them, so that each
// load of a warp is of neighbours. In both a group's elements are in one warp: in VEC, neighbouring lanes' units;
// else, group / 32 of each lane's elements.
template <typename T, int ITEMS, bool VEC, bool BLOCK>
__global__ void __launch_bounds__(512) norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int E = Unit<T>::E;
  __shared__ float2 s_part[2][16];
  __shared__ float s_far[16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lanes = BLOCK ? (int)blockDim.x : p.lanes;
  const int me = BLOCK ? tid : tid & (lanes - 1);
  const int per_block = BLOCK ? 1 : (int)blockDim.x / lanes;
  // the element e of item i
  auto place = [&](int i, int e) {
    return VEC ? (i * lanes + me) * E + e : (i * (lanes / 32) + (BLOCK ? warp : 0)) * 32 * E + e * 32 + lane;
  };
  auto there = [&](int i) { return VEC ? i * lanes + me < p.units : true; };

  int flip = 0;
  for (long long item0 = (long long)blockIdx.x * per_block; item0 < p.items;
       item0 += (long long)gridDim.x * per_block, flip ^= 1) {
    const long long item = item0 + (BLOCK ? 0 : tid / lanes);
    const bool live = item < p.items;
    const long long row = p.heads == 1 ? item : item / p.heads, head = p.heads == 1 ? 0 : item - row * p.heads;
    const T* x = static_cast<const T*>(p.x) + row * p.x_rs + head * p.x_hs;
    const T* res = static_cast<const T*>(p.residual) + row * p.res_rs + head * p.res_hs;
    T* tot = static_cast<T*>(p.total) + row * p.tot_rs + head * p.tot_hs;
    T* out = static_cast<T*>(p.out) + row * p.out_rs + head * p.out_hs;
    uint8_t* codes = p.codes + row * p.code_rs + head * p.code_hs;

    // everything read ahead of its use
    uint32_t wx[VEC ? ITEMS : 1][8], wr[VEC ? ITEMS : 1][8];
    float h[ITEMS][E];
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) wx[i][j] = wr[i][j] = 0u;
        if (live && there(i)) {
          load8(x + place(i, 0), wx[i]);
          if (p.residual) load8(res + place(i, 0), wr[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        unpack<T>(wx[i], h[i]);
        if (p.residual) {
          float r[E];
          unpack<T>(wr[i], r);
#pragma unroll
          for (int e = 0; e < E; ++e) h[i][e] += r[e];
          pack<T>(h[i], wr[i]);
          unpack<T>(wr[i], h[i]);
          if (p.total && live && there(i)) store8(tot + place(i, 0), wr[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int at = place(i, e);
          h[i][e] = live && at < p.n ? widen(x[at]) : 0.f;
        }
      }
      if (p.residual) {
        float r[ITEMS][E];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int at = place(i, e);
            r[i][e] = live && at < p.n ? widen(res[at]) : 0.f;
          }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int at = place(i, e);
            const T sum = narrow<T>(h[i][e] + r[i][e]);
            h[i][e] = widen(sum);
            if (p.total && live && at < p.n) tot[at] = sum;
          }
      }
    }

    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      float part = 0.f;   // (shorter chains, and sums of like size)
#pragma unroll
      for (int e = 0; e < E; ++e) part = fmaf(h[i][e], h[i][e], part);
      sum += part;
    }
    // The same of h 2^-64, for rows whose squares pass fp32: a thread whose own do not adds what is left of them.
    float far = sum * kFarScale * kFarScale;
    if (!(sum <= 1.2676506e30f)) {   // 2^100
      far = 0.f;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) far = fmaf(h[i][e] * kFarScale, h[i][e] * kFarScale, far);
    }
    // h becomes h (w + o)
    if (p.weight) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        float w[E];
        if constexpr (VEC) {
          if (!there(i)) continue;
          if (std::is_same<T, float>::value || !p.weight_f32) {
            uint32_t u[8];
            load8(static_cast<const T*>(p.weight) + place(i, 0), u);
            unpack<T>(u, w);
          } else {
            uint32_t u[8];
#pragma unroll
            for (int k = 0; k < E / 8; ++k) {
              load8(static_cast<const float*>(p.weight) + place(i, 8 * k), u);
#pragma unroll
              for (int e = 0; e < 8; ++e) w[8 * k + e] = __uint_as_float(u[e]);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int at = place(i, e);
            w[e] = at >= p.n      ? 0.f
                   : p.weight_f32 ? __ldg(static_cast<const float*>(p.weight) + at)
                                  : widen(static_cast<const T*>(p.weight)[at]);
          }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) h[i][e] *= w[e] + p.offset;
      }
    }
    float most = 0.f;
    if (p.scaling == DA_SCALE_ROW) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) most = fmaxf(most, fabsf(h[i][e]));   // NaN passes over
    }
    // the row's sum and maximum, in an order that the width alone sets
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (!BLOCK && o >= lanes) continue;
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    if constexpr (BLOCK) {
      // (two places in turn: a warp may be a row ahead, not two)
      if (lane == 0) s_part[flip][warp] = make_float2(sum, most);
      __syncthreads();
      const int warps = blockDim.x >> 5;
      const float2 v = lane < warps ? s_part[flip][lane] : make_float2(0.f, 0.f);
      sum = v.x;
      most = v.y;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      }
      sum = __shfl_sync(0xffffffffu, sum, 0);
      most = __shfl_sync(0xffffffffu, most, 0);
    }
    const float n = (float)p.n;
    float r = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(sum, n) + p.eps));
    const bool passed = sum > 3.4028235e38f;
    if (BLOCK ? passed : __any_sync(0xffffffffu, passed)) {
      far = row_sum<BLOCK>(far, lanes, s_far);
      if (passed) r = __fdiv_rn(kFarScale, __fsqrt_rn(__fdiv_rn(far, n) + p.eps * kFarScale * kFarScale));
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) h[i][e] *= r;

    if (p.out) {
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          uint32_t w[8];
          pack<T>(h[i], w);
          if (live && there(i)) store8(out + place(i, 0), w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int at = place(i, e);
            if (live && at < p.n) out[at] = narrow<T>(h[i][e]);
          }
      }
    }
    if (!p.codes) continue;
    float scale = 1.f;
    if (p.scaling == DA_SCALE_TENSOR) scale = __ldg(p.scales);
    if (p.scaling == DA_SCALE_ROW) {
      scale = fmaxf(__fdiv_rn(most * r, kE4M3Max), kLeastScale);
      if (me == 0 && live) p.scales[item] = scale;
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if constexpr (VEC) {
        float s = scale;
        if (p.scaling == DA_SCALE_GROUP) {
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) m = fmaxf(m, fabsf(h[i][e]));
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) {
            const float other = __shfl_xor_sync(0xffffffffu, m, o);
            if (o * E < p.group && (BLOCK || o < lanes)) m = fmaxf(m, other);
          }
          s = fmaxf(__fdiv_rn(m, kE4M3Max), kLeastScale);
          const int at = place(i, 0);
          if (live && there(i) && (at & (p.group - 1)) == 0) p.scales[item * p.groups + at / p.group] = s;
        }
        uint32_t w[E / 4];
#pragma unroll
        for (int k = 0; k < E / 4; ++k)
          w[k] = pack_e4m3x2(__fdiv_rn(h[i][4 * k], s), __fdiv_rn(h[i][4 * k + 1], s)) |
                 pack_e4m3x2(__fdiv_rn(h[i][4 * k + 2], s), __fdiv_rn(h[i][4 * k + 3], s)) << 16;
        if (live && there(i)) {
          if constexpr (E == 16)
            *reinterpret_cast<uint4*>(codes + place(i, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
          else
            *reinterpret_cast<uint2*>(codes + place(i, 0)) = make_uint2(w[0], w[1]);
        }
      } else {
        float m[E];
#pragma unroll
        for (int e = 0; e < E; ++e) m[e] = scale;
        if (p.scaling == DA_SCALE_GROUP) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            m[e] = fabsf(h[i][e]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], o));
          }
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            const float a = fmaxf(m[e], m[e + 1]), b = fmaxf(m[e + 2], m[e + 3]), c = fmaxf(a, b);
            if (p.group == 64) {
              m[e] = m[e + 1] = a;
              m[e + 2] = m[e + 3] = b;
            } else if (p.group == 128) {
              m[e] = m[e + 1] = m[e + 2] = m[e + 3] = c;
            }
          }
#pragma unroll
          for (int e = 0; e < E; ++e) {
            m[e] = fmaxf(__fdiv_rn(m[e], kE4M3Max), kLeastScale);
            const int at = place(i, e);
            if (live && lane == 0 && at < p.n && (at & (p.group - 1)) == 0)
              p.scales[item * p.groups + at / p.group] = m[e];
          }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int at = place(i, e);
          if (live && at < p.n) codes[at] = (uint8_t)pack_e4m3x2(__fdiv_rn(h[i][e], m[e]), 0.f);
        }
      }
    }
  }
}

template <typename T, bool VEC>
const void* kernel_of(int items, bool block) {
  if (!block) return reinterpret_cast<const void*>(&norm_kernel<T, 1, VEC, false>);
  return items <= 1   ? reinterpret_cast<const void*>(&norm_kernel<T, 1, VEC, true>)
         : items <= 2 ? reinterpret_cast<const void*>(&norm_kernel<T, 2, VEC, true>)
         : items <= 4 ? reinterpret_cast<const void*>(&norm_kernel<T, 4, VEC, true>)
                      : reinterpret_cast<const void*>(&norm_kernel<T, std::is_same<T, float>::value ? 8 : 4, VEC, true>);
}
template <typename T>
const void* kernel_of(int items, bool vec, bool block) {
  return vec ? kernel_of<T, true>(items, block) : kernel_of<T, false>(items, block);
}

// Whether a row tensor's runs begin on multiples of `bytes`.
bool begins_on(const void* p, long long rs, long long hs, int es, int bytes) {
  return !p || (aligned(p, bytes) && rs * es % bytes == 0 && hs * es % bytes == 0);
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
  const bool vec = c.n % E == 0 && begins_on(a.x, p.x_rs, p.x_hs, es, 32) && begins_on(a.residual, p.res_rs, p.res_hs, es, 32) &&
                   begins_on(a.residual_out, p.tot_rs, p.tot_hs, es, 32) && begins_on(a.out, p.out_rs, p.out_hs, es, 32) &&
                   begins_on(a.codes, p.code_rs, p.code_hs, 1, E) && aligned(a.weight, 32);
  const int sms = device_sms();
  if (sms <= 0) return DA_ERR_CUDA;
  // Threads of a row: one for each of its units up to a warp; then whole warps, of two units a thread where there
  // are more than 256.
  p.units = vec ? c.n / E : (c.n + 32 * E - 1) / (32 * E);
  int threads, per = 1, items_each;
  bool block = false;
  if (vec && p.units <= 32) {
    p.lanes = 1;
    while (p.lanes < p.units) p.lanes *= 2;
    threads = 128;
    per = threads / p.lanes;
    items_each = 1;
  } else if (!vec && p.units <= 1) {
    p.lanes = 32;
    threads = 128;
    per = 4;
    items_each = 1;
  } else {
    block = true;
    const int warps = vec ? (p.units + 31) / 32 : p.units;   // at a unit a thread
    items_each = warps <= 8 ? 1 : warps <= 16 ? 2 : warps <= 32 ? 2 : warps <= 64 ? 4 : 8;
    threads = 32 * ((warps + items_each - 1) / items_each);
    p.lanes = threads;
  }
  const void* fn = a.dtype == DA_F32   ? kernel_of<float>(items_each, vec, block)
                   : a.dtype == DA_F16 ? kernel_of<__half>(items_each, vec, block)
                                       : kernel_of<__nv_bfloat16>(items_each, vec, block);
  const long long blocks = std::min((items + per - 1) / per, (1ll << 31) - 1);
  void* kargs[1] = {&p};
  const cudaError_t e = cudaLaunchKernel(fn, dim3((unsigned)blocks), dim3(threads), kargs, 0,
                                         static_cast<cudaStream_t>(a.cuda_stream));
  return e == cudaSuccess ? DA_OK : cuda_fail(e, "launching the norm kernel");
}

}  // extern "C"
