// da_norm.cuh -- root-mean-square norm of rows, with the residual's addition ahead of it and an output in 8 bits
// behind it: the kernel.
//     h = x + residual (rounded to the type: what the next block adds to),
//     y = h (w + o) / sqrt(mean(h^2) + eps),   code = E4M3(y / scale),
// scale given, or max |y| / 448 over the row or over groups of 32, 64 or 128 elements.
//
// Bound by HBM: every element is read once and written once, about 10 operations between. A row stays in registers
// from the loads to the stores (past 16384 elements not all of it: kWide with a residual spills 0.5 KB a thread in 16
// bits and 1.4 KB in fp32, kShifted 0.8 and 2.3); what the row's threads exchange is one sum and one maximum,
// together. The maximum needs no second pass over y: rounding is monotone, so max |y| = round(max |h (w + o)| r) with
// y = round(h (w + o) r).
#pragma once

#include <cstring>
#include <type_traits>

#include "da_device.cuh"
#include "da_rowvec.cuh"
#include "decode_attn.h"

namespace da {

constexpr float kE4M3Max = 448.f;
constexpr float kFarSum = 1.2676506e30f;         // 2^100: larger sums of squares are formed again,
constexpr float kFarScale = 8.2718061e-25f;      // 2^-80: of h taken by that
constexpr float kLeastScale = 1.17549435e-38f;   // 2^-126: of a row of zeros; no scale is subnormal

struct NormParams {
  const void *x, *residual, *weight;
  void *total, *out;
  uint8_t* codes;
  float* scales;
  // strides in elements, of rows and heads
  long long x_rs, x_hs, res_rs, res_hs, tot_rs, tot_hs, out_rs, out_hs, code_rs, code_hs;
  long long items;              // rows * heads
  int heads, n, units;          // units: of a row
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

// Pairs of floats, two of them to an instruction: what bounds the kernel beside HBM is the instructions it issues
// (8192 rows of 8192 bf16 with groups: 17 an element 122 us, 8 an element 91).
__device__ __forceinline__ float2 both(f32x2 x) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(x));
  return f;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// max(m, |x|, |y|); a NaN passes over
__device__ __forceinline__ float most_of(float m, f32x2 x) {
  const float2 f = both(x);
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(f.x)), "f"(fabsf(f.y)));
  return r;
}

// the largest of the warp's m >= 0; a NaN passes over
__device__ __forceinline__ float warp_most(float m) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(m));
  return r;
}

// 8 words of T as floats, and back (rounded to nearest even).
template <typename T>
__device__ __forceinline__ void unpack(const uint32_t* w, f32x2* f) {
  if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2_pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (std::is_same<T, __half>::value) {
        __half2 h;
        memcpy(&h, &w[i], 4);
        const float2 g = __half22float2(h);
        f[i] = f2_pack(g.x, g.y);
      } else {
        f[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      }
    }
  }
}
template <typename T>
__device__ __forceinline__ void pack(const f32x2* f, uint32_t* w) {
  if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 g = both(f[i]);
      w[2 * i] = __float_as_uint(g.x);
      w[2 * i + 1] = __float_as_uint(g.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 g = both(f[i]);
      w[i] = pack2(g.x, g.y, T());
    }
  }
}
// 8 words of x + residual, rounded once. (fp32 has 24 bits, at least 2 p + 2 of a type of p: the sum rounded to fp32
// and then to the type is the same.)
template <typename T>
__device__ __forceinline__ void add_words(uint32_t* x, const uint32_t* r) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (std::is_same<T, float>::value)
      x[i] = __float_as_uint(__uint_as_float(x[i]) + __uint_as_float(r[i]));
    else if constexpr (std::is_same<T, __half>::value)
      asm("add.rn.f16x2 %0, %1, %2;" : "=r"(x[i]) : "r"(x[i]), "r"(r[i]));
    else
      asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(x[i]) : "r"(x[i]), "r"(r[i]));
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

// y / s by s's reciprocal, and that corrected.
__device__ __forceinline__ f32x2 divided(f32x2 y, f32x2 minus_s, f32x2 inverse) {
  const f32x2 q = f2_mul(y, inverse);
  return fma2(fma2(q, minus_s, y), inverse, q);
}

// y / s rounded to nearest, for a scale that the row shares: the product with the reciprocal, corrected once by
// its remainder (Markstein 1990: correctly rounded where the reciprocal is, short of under- and overflow), and the
// plain division for scales near the ends of the range. `given`: a scale that was not found from y, whose
// quotients may be infinite or far past E4M3's largest: those stay as they are.
struct Divider {
  float s;
  f32x2 inverse, minus;
  bool middling, given;
  __device__ __forceinline__ Divider(float scale, bool from_caller) {
    s = scale;
    given = from_caller;
    const float r = __fdiv_rn(1.f, scale);
    inverse = f2_pack(r, r);
    minus = f2_pack(-scale, -scale);
    middling = scale > 8.2718061e-25f && scale < 1.2089258e24f;   // 2^+-80
  }
  __device__ __forceinline__ float2 operator()(f32x2 y) const {
    if (!middling) {
      const float2 f = both(y);
      return make_float2(__fdiv_rn(f.x, s), __fdiv_rn(f.y, s));
    }
    float2 better = both(divided(y, minus, inverse));
    if (given) {
      const float2 f = both(f2_mul(y, inverse));
      if (!(fabsf(f.x) < 1048576.f)) better.x = f.x;
      if (!(fabsf(f.y) < 1048576.f)) better.y = f.y;
    }
    return better;
  }
};

// The sum (MOST: the largest) of v over a row's threads, by its block or `lanes` lanes. Of rows that hardly ever come,
// but what it is made of is felt in all: with a loop over the warps' values in place of the shuffles (STRAIGHT), what
// is loaded ahead is waited for too early (8192 rows of 6464 bf16 with residual and groups: 109 us in place of 85);
// where several units a thread are not loaded ahead, the loop leaves more registers (4000 rows of 4107 fp32: 79 us
// without it, 49 with).
template <bool BLOCK, bool MOST, bool STRAIGHT>
__device__ __forceinline__ float over_row(float v, int lanes, float* s_part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (!BLOCK && o >= lanes) continue;
    const float other = __shfl_xor_sync(0xffffffffu, v, o);
    v = MOST ? fmaxf(v, other) : v + other;
  }
  if constexpr (BLOCK) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) s_part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    if constexpr (STRAIGHT) {
      if (lane < warps) v = s_part[lane];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        const float other = __shfl_xor_sync(0xffffffffu, v, o);
        v = MOST ? fmaxf(v, other) : v + other;
      }
      v = __shfl_sync(0xffffffffu, v, 0);
    } else {
#pragma unroll 1
      for (int w = 0; w < warps; ++w) v = MOST ? fmaxf(v, s_part[w]) : v + s_part[w];
    }
    __syncthreads();
  }
  return v;
}

// How a row's elements lie with its threads. A thread holds ITEMS units of E elements:
// kWide     a unit is 32 bytes of the row, loaded at once, and the row's units go round the threads.
// kShifted  the same for rows of any width that begin anywhere, but all tensors' alike (one block a row): units lie on
//           16-byte boundaries, so a row begins and ends inside one, whose elements are moved one by one. Rows that are
//           a multiple of 8 (fp32: 4) apart begin alike, so a block keeps to such rows, with its weights in registers.
//           (2002 rows of 5119 bf16 to 8 bits: 34 us element by element, 30 so; 1001 of fp32 19 both ways.)
// kScattered a warp holds 32 E elements, a lane every 32nd of them, so that each load of a warp is of neighbours.
// A group's elements are in one warp: in kWide, neighbouring lanes' units; in kScattered, group / 32 of each lane's
// elements; kShifted has none.
enum NormLayout { kScattered = 0, kWide = 1, kShifted = 2 };

// Registers of a block's thread: 128; with a residual and at most two units 96 (by 640 threads), for 5 blocks an SM of
// 4 warps in place of 4 (8192 rows of bf16 with groups: width 4096 47 to 44 us, 6144 80 to 65, 8192 alike; without
// groups alike). kScattered with one unit 64, for two blocks an SM or more, as it loads nothing ahead (4000 rows of
// 4107 bf16 with residual and groups: 147 to 59 us).
template <int ITEMS, int LAYOUT, bool BLOCK, bool RES>
constexpr int kMostThreads = !BLOCK ? 128 : LAYOUT == kWide && RES && ITEMS <= 2 ? 640 : 512;

// A row's threads: a block (BLOCK), or `lanes` lanes of a warp, several rows a warp.
template <typename T, int ITEMS, int LAYOUT, bool BLOCK, bool RES>
__global__ void __launch_bounds__(kMostThreads<ITEMS, LAYOUT, BLOCK, RES>,
                                  !BLOCK                               ? (RES ? 6 : 8)
                                  : LAYOUT == kScattered && ITEMS == 1 ? 2
                                                                       : 1)
    norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int E = Unit<T>::E, V = E / 2;
  constexpr bool VEC = LAYOUT != kScattered, SHIFTED = LAYOUT == kShifted, STRAIGHT = VEC || ITEMS == 1;
  static_assert(BLOCK || !SHIFTED, "");
  __shared__ float2 s_part[2][16];
  __shared__ float s_far[16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int lanes = BLOCK ? (int)blockDim.x : p.lanes;
  const int me = BLOCK ? tid : tid & (lanes - 1);
  const int per_block = BLOCK ? 1 : (int)blockDim.x / lanes;
  // how far into its first unit the block's rows begin
  const int shift = SHIFTED ? (int)((unsigned long long)blockIdx.x * (unsigned long long)p.x_rs & (V - 1)) : 0;
  // the element e of item i
  auto place = [&](int i, int e) {
    return VEC ? (i * lanes + me) * E + e - shift : (i * (lanes / 32) + (BLOCK ? warp : 0)) * 32 * E + e * 32 + lane;
  };
  auto there = [&](int i) { return !VEC || (i * lanes + me < p.units && (!SHIFTED || place(i, 0) < p.n)); };
  auto whole = [&](int i) { return !SHIFTED || (place(i, 0) >= 0 && place(i, E) <= p.n); };
  auto load_unit = [&](const T* row, int i, uint32_t* w) {
    if (!SHIFTED) {
      load8(row + place(i, 0), w);
    } else if (whole(i)) {
      const uint4 a = *reinterpret_cast<const uint4*>(row + place(i, 0));
      const uint4 b = *reinterpret_cast<const uint4*>(row + place(i, V));
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int at = place(i, e);
        const bool in = at >= 0 && at < p.n;
        if constexpr (E == 8) {
          w[e] = in ? reinterpret_cast<const uint32_t*>(row)[at] : 0u;
        } else {
          const uint32_t u = in ? (uint32_t)reinterpret_cast<const uint16_t*>(row)[at] : 0u;
          w[e / 2] = e & 1 ? w[e / 2] | u << 16 : u;
        }
      }
    }
  };
  auto store_unit = [&](T* row, int i, const uint32_t* w) {
    if (!SHIFTED) {
      store8(row + place(i, 0), w);
    } else if (whole(i)) {
      *reinterpret_cast<uint4*>(row + place(i, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(row + place(i, V)) = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int at = place(i, e);
        if (at < 0 || at >= p.n) continue;
        if constexpr (E == 8) reinterpret_cast<uint32_t*>(row)[at] = w[e];
        else reinterpret_cast<uint16_t*>(row)[at] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
      }
    }
  };

  // where an item (a row's head) lies
  auto find = [&](long long item, long long& row, long long& head) {
    row = p.heads == 1            ? item
          : p.items < (1ll << 31) ? (unsigned)item / (unsigned)p.heads
                                  : item / p.heads;
    head = item - row * p.heads;
  };
  uint32_t wx[VEC ? ITEMS : 1][8], wr[VEC ? ITEMS : 1][8];
  auto load = [&](long long item) {   // VEC
    if (item >= p.items) return;
    long long row, head;
    find(item, row, head);
    const T* x = static_cast<const T*>(p.x) + row * p.x_rs + head * p.x_hs;
    const T* res = static_cast<const T*>(p.residual) + row * p.res_rs + head * p.res_hs;
#pragma unroll
    for (int i = 0; i < (VEC ? ITEMS : 1); ++i) {
      if (!there(i)) continue;
      load_unit(x, i, wx[i]);
      if constexpr (RES) load_unit(res, i, wr[i]);
    }
  };
  const long long step = (long long)gridDim.x * per_block;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) wx[i][j] = wr[i][j] = 0u;
    load((long long)blockIdx.x * per_block + (BLOCK ? 0 : tid / lanes));
  }

  // the weights that a block's rows have alike
  f32x2 ws[SHIFTED ? ITEMS : 1][E / 2];
  if constexpr (SHIFTED) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        float v[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int at = place(i, e + k);
          v[k] = !p.weight || at < 0 || at >= p.n ? 0.f
                 : p.weight_f32 ? __ldg(static_cast<const float*>(p.weight) + at)
                                : widen(static_cast<const T*>(p.weight)[at]);
          v[k] += p.offset;
        }
        ws[i][e / 2] = f2_pack(v[0], v[1]);
      }
  }

  int flip = 0;
  for (long long item0 = (long long)blockIdx.x * per_block; item0 < p.items; item0 += step, flip ^= 1) {
    const long long item = item0 + (BLOCK ? 0 : tid / lanes);
    const bool live = item < p.items;
    long long row, head;
    find(item, row, head);
    T* tot = static_cast<T*>(p.total) + row * p.tot_rs + head * p.tot_hs;
    T* out = static_cast<T*>(p.out) + row * p.out_rs + head * p.out_hs;
    uint8_t* codes = p.codes + row * p.code_rs + head * p.code_hs;

    f32x2 h[ITEMS][E / 2];
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        if constexpr (RES) {
          add_words<T>(wx[i], wr[i]);
          if (p.total && live && there(i)) store_unit(tot, i, wx[i]);
        }
        unpack<T>(wx[i], h[i]);
      }
      load(item + step);   // the next row's, on their way while this one is worked on
    } else {
      const T* x = static_cast<const T*>(p.x) + row * p.x_rs + head * p.x_hs;
      const T* res = static_cast<const T*>(p.residual) + row * p.res_rs + head * p.res_hs;
      float v[ITEMS][E];
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int at = place(i, e);
          v[i][e] = live && at < p.n ? widen(x[at]) : 0.f;
        }
      if constexpr (RES) {
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
            const T sum = narrow<T>(v[i][e] + r[i][e]);
            v[i][e] = widen(sum);
            if (p.total && live && at < p.n) tot[at] = sum;
          }
      }
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int e = 0; e < E / 2; ++e) h[i][e] = f2_pack(v[i][2 * e], v[i][2 * e + 1]);
    }

    f32x2 sum2 = f2_pack(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      f32x2 part = f2_mul(h[i][0], h[i][0]);   // (shorter chains, and sums of like size)
#pragma unroll
      for (int e = 1; e < E / 2; ++e) part = fma2(h[i][e], h[i][e], part);
      sum2 = add2(sum2, part);
    }
    float sum = both(sum2).x + both(sum2).y;
    // Squares, and products with the weights, pass fp32 where h does not. A thread whose sum is that large takes its h
    // by a power of two and sums again; where a row's is, the others add what is left of theirs.
    float far = sum * kFarScale * kFarScale;
    const bool taken = !(sum <= kFarSum);
    if (taken) {
      const f32x2 c = f2_pack(kFarScale, kFarScale);
      f32x2 part = f2_pack(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          h[i][e] = f2_mul(h[i][e], c);
          part = fma2(h[i][e], h[i][e], part);
        }
      far = both(part).x + both(part).y;
    }
    // h becomes h (w + o)
    if (p.weight) {
      const f32x2 o = f2_pack(p.offset, p.offset);
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        f32x2 w[E / 2];
        if constexpr (SHIFTED) {
#pragma unroll
          for (int e = 0; e < E / 2; ++e) w[e] = ws[i][e];
        } else if constexpr (VEC) {
          if (!there(i)) continue;
          if (std::is_same<T, float>::value || !p.weight_f32) {
            uint32_t u[8];
            load8(static_cast<const T*>(p.weight) + place(i, 0), u);
            unpack<T>(u, w);
          } else {
#pragma unroll
            for (int k = 0; k < E / 8; ++k) {
              uint32_t u[8];
              load8(static_cast<const float*>(p.weight) + place(i, 8 * k), u);
              unpack<float>(u, w + 4 * k);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            float v[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int at = place(i, e + k);
              v[k] = at >= p.n      ? 0.f
                     : p.weight_f32 ? __ldg(static_cast<const float*>(p.weight) + at)
                                    : widen(static_cast<const T*>(p.weight)[at]);
            }
            w[e / 2] = f2_pack(v[0], v[1]);
          }
        }
        if (!SHIFTED && p.offset != 0.f) {
#pragma unroll
          for (int e = 0; e < E / 2; ++e) w[e] = add2(w[e], o);
        }
#pragma unroll
        for (int e = 0; e < E / 2; ++e) h[i][e] = f2_mul(h[i][e], w[e]);
      }
    }
    float most = 0.f;
    if (p.scaling == DA_SCALE_ROW) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int e = 0; e < E / 2; ++e) most = most_of(most, h[i][e]);
    }
    // the row's sum and maximum, in an order that goes by the threads a row has (its width, and whether rows are many)
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
    const bool passed = sum > kFarSum;
    if (BLOCK ? passed : __any_sync(0xffffffffu, passed)) {
      far = over_row<BLOCK, false, STRAIGHT>(far, lanes, s_far);
      if (passed)
        r = __fdiv_rn(taken ? 1.f : kFarScale, __fsqrt_rn(__fdiv_rn(far, n) + p.eps * kFarScale * kFarScale));
    }
    const f32x2 r2 = f2_pack(r, r);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int e = 0; e < E / 2; ++e) h[i][e] = f2_mul(h[i][e], r2);
    auto value = [&](int i, int e) { return e & 1 ? both(h[i][e / 2]).y : both(h[i][e / 2]).x; };

    if (p.out) {
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
          uint32_t w[8];
          pack<T>(h[i], w);
          if (live && there(i)) store_unit(out, i, w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int at = place(i, e);
            if (live && at < p.n) out[at] = narrow<T>(value(i, e));
          }
      }
    }
    if (!p.codes) continue;
    float scale = 1.f;
    if (p.scaling == DA_SCALE_TENSOR) scale = __ldg(p.scales);
    if (p.scaling == DA_SCALE_ROW) {
      most *= r;
      if (BLOCK ? passed : __any_sync(0xffffffffu, passed)) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
#pragma unroll
          for (int e = 0; e < E / 2; ++e) y = most_of(y, h[i][e]);
        y = over_row<BLOCK, true, STRAIGHT>(y, lanes, s_far);
        if (passed) most = y;   // (its threads' products are not alike: y itself)
      }
      scale = fmaxf(__fdiv_rn(most, kE4M3Max), kLeastScale);
      if (me == 0 && live) p.scales[item] = scale;
    }
    Divider over(scale, p.scaling == DA_SCALE_TENSOR);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if constexpr (VEC) {
        if (p.scaling == DA_SCALE_GROUP) {
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < E / 2; ++e) m = most_of(m, h[i][e]);
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) {
            if (o * E >= p.group) continue;
            const float other = __shfl_xor_sync(0xffffffffu, m, o);
            if (BLOCK || o < lanes) m = fmaxf(m, other);
          }
          // (lanes without a unit: no scale that would take the warp to the plain division)
          const float s = there(i) ? fmaxf(__fdiv_rn(m, kE4M3Max), kLeastScale) : 1.f;
          const int at = place(i, 0);
          if (live && there(i) && (at & (p.group - 1)) == 0) p.scales[item * p.groups + at / p.group] = s;
          over = Divider(s, false);
        }
        uint32_t w[E / 4];
#pragma unroll
        for (int k = 0; k < E / 4; ++k) {
          const float2 a = over(h[i][2 * k]), b = over(h[i][2 * k + 1]);
          w[k] = pack_e4m3x2(a.x, a.y) | pack_e4m3x2(b.x, b.y) << 16;
        }
        if (SHIFTED && live && there(i)) {
          if (whole(i)) {
            if constexpr (E == 16) {
              *reinterpret_cast<uint2*>(codes + place(i, 0)) = make_uint2(w[0], w[1]);
              *reinterpret_cast<uint2*>(codes + place(i, V)) = make_uint2(w[2], w[3]);
            } else {
              *reinterpret_cast<uint32_t*>(codes + place(i, 0)) = w[0];
              *reinterpret_cast<uint32_t*>(codes + place(i, V)) = w[1];
            }
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const int at = place(i, e);
              if (at >= 0 && at < p.n) codes[at] = (uint8_t)(w[e / 4] >> (8 * (e & 3)));
            }
          }
        } else if (live && there(i)) {
          if constexpr (E == 16)
            *reinterpret_cast<uint4*>(codes + place(i, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
          else
            *reinterpret_cast<uint2*>(codes + place(i, 0)) = make_uint2(w[0], w[1]);
        }
      } else if (p.scaling != DA_SCALE_GROUP) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 q = over(h[i][e / 2]);
          const uint32_t w = pack_e4m3x2(q.x, q.y);
          const int a0 = place(i, e), a1 = place(i, e + 1);
          if (live && a0 < p.n) codes[a0] = (uint8_t)w;
          if (live && a1 < p.n) codes[a1] = (uint8_t)(w >> 8);
        }
      } else {
        // A group is K = group / 32 of every lane's elements; lane g finds the scale of the unit's group g and its
        // reciprocal, for all (4000 rows of 4107 fp32, groups of 64: 86 us with every lane finding every scale
        // and dividing by it, 49 so).
        auto groups_of = [&](auto k) {
          constexpr int K = decltype(k)::value, G = E / K;
          float mine = 0.f;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            float m = 0.f;
#pragma unroll
            for (int e = 0; e < K; ++e) m = fmaxf(m, fabsf(value(i, g * K + e)));
            m = warp_most(m);
            if (lane == g) mine = m;
          }
          const int first = place(i, 0) - lane + lane * 32 * K;   // of lane's group
          const bool has = lane < G && first < p.n;
          const float s = has ? fmaxf(__fdiv_rn(mine, kE4M3Max), kLeastScale) : 1.f;
          if (live && has) p.scales[item * p.groups + first / (32 * K)] = s;
          const Divider by(s, false);
          const bool middling = !__any_sync(0xffffffffu, !by.middling);
          const float inverse = both(by.inverse).x;
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const f32x2 y = h[i][e / 2];
            const float2 t = make_float2(__shfl_sync(0xffffffffu, s, e / K), __shfl_sync(0xffffffffu, s, (e + 1) / K));
            float2 q;
            if (middling) {
              const f32x2 r2 = f2_pack(__shfl_sync(0xffffffffu, inverse, e / K),
                                       __shfl_sync(0xffffffffu, inverse, (e + 1) / K));
              q = both(divided(y, f2_pack(-t.x, -t.y), r2));
            } else {
              q = make_float2(__fdiv_rn(both(y).x, t.x), __fdiv_rn(both(y).y, t.y));
            }
            const uint32_t w = pack_e4m3x2(q.x, q.y);
            const int a0 = place(i, e), a1 = place(i, e + 1);
            if (live && a0 < p.n) codes[a0] = (uint8_t)w;
            if (live && a1 < p.n) codes[a1] = (uint8_t)(w >> 8);
          }
        };
        if (p.group == 32) groups_of(std::integral_constant<int, 1>());
        else if (p.group == 64) groups_of(std::integral_constant<int, 2>());
        else groups_of(std::integral_constant<int, 4>());
      }
    }
  }
}

// ---- an eps that small rows' squares do not reach --------------------------------------------------------------
// Squares of numbers below 2^-63 vanish in fp32, and with them a row's size, unless eps covers it. Under an eps of less
// than kLeastEps rows are taken by a power of two that brings their largest number to 1, which takes another reading of
// them: a block a row, an element a lane, three times over the row (the last two from L1 or L2). Zero is the only such
// eps that is met, and rarely, so this is not made fast: 8192 rows of 8192 bf16 with a residual and codes by rows 511
// us, where the kernel above takes 77.
constexpr float kLeastEps = 8.2718061e-25f;   // 2^-80
constexpr int kCarefulThreads = 256;

// The sum (MOST: the largest) of v over the block.
template <bool MOST, typename V>
__device__ __forceinline__ V over_block(V v, V* s_part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const V other = __shfl_xor_sync(0xffffffffu, v, o);
    v = MOST ? max(v, other) : v + other;
  }
  __syncthreads();   // (what was there has been read)
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = s_part[0];
  for (int w = 1; w < (int)(blockDim.x >> 5); ++w) v = MOST ? max(v, s_part[w]) : v + s_part[w];
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kCarefulThreads) careful_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float s_most[kCarefulThreads / 32];
  __shared__ double s_sum[kCarefulThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
  for (long long item = blockIdx.x; item < p.items; item += gridDim.x) {
    const long long row = item / p.heads, head = item - row * p.heads;
    const T* x = static_cast<const T*>(p.x) + row * p.x_rs + head * p.x_hs;
    const T* res = static_cast<const T*>(p.residual) + row * p.res_rs + head * p.res_hs;
    T* tot = static_cast<T*>(p.total) + row * p.tot_rs + head * p.tot_hs;
    T* out = static_cast<T*>(p.out) + row * p.out_rs + head * p.out_hs;
    uint8_t* codes = p.codes + row * p.code_rs + head * p.code_hs;
    auto sum_at = [&](int e) { return p.residual ? narrow<T>(widen(x[e]) + widen(res[e])) : x[e]; };
    auto weight = [&](int e) {
      if (!p.weight) return 1.f;
      const float w = p.weight_f32 ? static_cast<const float*>(p.weight)[e] : widen(static_cast<const T*>(p.weight)[e]);
      return w + p.offset;
    };
    float most = 0.f;
    for (int e = tid; e < p.n; e += threads) {
      const T h = sum_at(e);
      if (p.total) tot[e] = h;
      most = fmaxf(most, fabsf(widen(h)));
    }
    most = over_block<true>(most, s_most);
    // 2^-e of the largest number's 2^e (of a subnormal one 2^126, which brings it above 2^-24; else 1)
    const int bits = (int)(__float_as_uint(most) >> 23);
    const int up = most > 0.f && bits < 255 ? min(127 - bits, 126) : 0;
    const float c0 = __uint_as_float((uint32_t)(127 + up / 2) << 23);                // (2^-127 is not normal)
    const float c1 = __uint_as_float((uint32_t)(127 + up - up / 2) << 23);
    auto taken = [&](int e) { return (p.total ? widen(tot[e]) : widen(sum_at(e))) * c0 * c1; };
    double sum = 0.;
    most = 0.f;
    for (int e0 = tid; e0 < p.n; e0 += 16 * threads) {
      float part = 0.f;
      for (int k = 0; k < 16 && e0 + k * threads < p.n; ++k) {
        const float h = taken(e0 + k * threads);
        part = fmaf(h, h, part);
        most = fmaxf(most, fabsf(h * weight(e0 + k * threads)));
      }
      sum += part;
    }
    sum = over_block<false>(sum, s_sum);
    // (eps taken as the squares are, which fp32 may not hold; the quotient it does)
    const double c = (double)c0 * c1;
    const float r = (float)(1. / sqrt(sum / p.n + p.eps * c * c));
    float scale = p.scaling == DA_SCALE_TENSOR ? __ldg(p.scales) : 1.f;
    if (p.scaling == DA_SCALE_ROW) {
      scale = fmaxf(__fdiv_rn(over_block<true>(most, s_most) * r, kE4M3Max), kLeastScale);
      if (tid == 0) p.scales[item] = scale;
    }
    // A warp takes a group (or 128 elements); out may be x, whose elements only their own lane reads from here on.
    const int size = p.scaling == DA_SCALE_GROUP ? p.group : 128;
    for (int g = tid >> 5; g * size < p.n; g += threads >> 5) {
      const int end = min(p.n, (g + 1) * size);
      if (p.scaling == DA_SCALE_GROUP) {
        float m = 0.f;
        for (int e = g * size + lane; e < end; e += 32) m = fmaxf(m, fabsf(taken(e) * weight(e) * r));
        scale = fmaxf(__fdiv_rn(warp_most(m), kE4M3Max), kLeastScale);
        if (lane == 0) p.scales[item * p.groups + g] = scale;
      }
      for (int e = g * size + lane; e < end; e += 32) {
        const float y = taken(e) * weight(e) * r;
        if (p.out) out[e] = narrow<T>(y);
        if (p.codes) codes[e] = (uint8_t)pack_e4m3x2(__fdiv_rn(y, scale), 0.f);
      }
    }
    __syncthreads();   // (the next row's sums may go where this one's are read)
  }
}

// The kernel of a layout: ITEMS units a thread (1, 2, 4 or, fp32, 8), a block a row or not.
template <typename T, int LAYOUT, bool RES>
const void* norm_kernel_of(int items, bool block) {
  if constexpr (LAYOUT != kShifted)
    if (!block) return reinterpret_cast<const void*>(&norm_kernel<T, 1, LAYOUT, false, RES>);
  constexpr int MOST = std::is_same<T, float>::value ? 8 : 4;
  return items <= 1   ? reinterpret_cast<const void*>(&norm_kernel<T, 1, LAYOUT, true, RES>)
         : items <= 2 ? reinterpret_cast<const void*>(&norm_kernel<T, 2, LAYOUT, true, RES>)
         : items <= 4 ? reinterpret_cast<const void*>(&norm_kernel<T, 4, LAYOUT, true, RES>)
                      : reinterpret_cast<const void*>(&norm_kernel<T, MOST, LAYOUT, true, RES>);
}
template <typename T>
const void* norm_kernel_for(int layout, int items, bool block, bool residual) {
  if (layout == kWide)
    return residual ? norm_kernel_of<T, kWide, true>(items, block) : norm_kernel_of<T, kWide, false>(items, block);
  if (layout == kShifted)
    return residual ? norm_kernel_of<T, kShifted, true>(items, block) : norm_kernel_of<T, kShifted, false>(items, block);
  return residual ? norm_kernel_of<T, kScattered, true>(items, block)
                  : norm_kernel_of<T, kScattered, false>(items, block);
}

const void* norm_kernel_f32(int layout, int items, bool block, bool residual);
const void* norm_kernel_f16(int layout, int items, bool block, bool residual);
const void* norm_kernel_bf16(int layout, int items, bool block, bool residual);
const void* careful_norm_kernel_f32();
const void* careful_norm_kernel_bf16();

}  // namespace da
