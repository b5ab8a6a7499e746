// da_cache.cu -- the operators around a step: rotary positions, the quantising write of new
// rows into the cache (rotary fused in), and the read of rows back out of it.
//
// All three are bound by memory: every row element is read once and written once, and the
// arithmetic (two products and an add per element, a conversion) is small beside it. At a decode
// step's size (one row a sequence) the time is the launch and a chain of dependent loads.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstring>
#include <new>
#include <type_traits>
#include <utility>

#include "da_plan.h"
#include "da_rows.h"

using namespace da;

struct da_rope {
  da_rope_config cfg;
  double theta[128];        // radians per position
  unsigned long long turn[128];   // turns per position, 0.64 fixed point (mod 1)
};

namespace {

constexpr int kRowThreads = 128;
constexpr int kMaxPairs = 128;   // rotary_dim / 2 <= 128

// ---- rows kernel: rotary and the quantising write ------------------------------------------
struct RowParams {
  Params cache;                 // layout of the cache, block table, status
  const void* q;                // [rows, hq, d] or null
  const void* k;                // [rows, hkv, d] or null (plain rotary)
  const void* v;
  void* q_out;
  void* k_cache;
  void* v_cache;
  long long q_rs, q_hs, k_rs, k_hs, v_rs, v_hs, qo_rs, qo_hs;   // strides, elements
  const int32_t* row_offsets;   // null: plain rotary, every row has a position of its own
  const int32_t* start;
  const int32_t* positions;     // null: the cache positions
  float* amax;
  int rows, hq, hkv;
  int units, head_lanes;        // a head is `units` lanes wide; head_lanes heads a block pass
  int wide_in, wide_out;        // rows read (written) lie on 32-byte boundaries
  int rotary, interleaved, transpose;
  float m;                      // attn_factor
  float k_scale, v_scale;       // of an FP8 cache
  unsigned long long turn[kMaxPairs];
};

// 32 bytes a lane (aligned to 32): neighbouring lanes then fill whole sectors in one instruction,
// where two 16-byte accesses 32 bytes apart touch each sector twice (1.7 GB read back from FP8, 8 items a lane:
// 266 us, 340 with 16-byte stores; a rotary gradient 26.7, 27.4; a plain write of 134 MB 23.1, 24.0).
__device__ __forceinline__ void load32(const void* p, uint4& a, uint4& b) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                 "=r"(b.w)
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
               "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// The sequence whose rows hold row r: the last b with offsets[b] <= r, or -1 where r lies
// before the first row or behind the last one.
__device__ __forceinline__ int find_sequence(const int32_t* offsets, int batch, int r) {
  int lo = 0, hi = batch;   // offsets[lo] <= r < offsets[hi], once both ends are checked
  if (r < __ldg(offsets) || r >= __ldg(offsets + batch)) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(offsets + mid) <= r) lo = mid; else hi = mid;
  }
  return lo;
}

// Where row r goes: its cache position (pos) and cache row (z; -1: none, recorded).
// Returns false for a row of no sequence.
__device__ __forceinline__ bool locate_row(const Params& c, const int32_t* offsets,
                                           const int32_t* start, int r, long long& pos, int& z) {
  const int b = find_sequence(offsets, c.batch, r);
  if (b < 0) return false;
  const long long t = (long long)__ldg(start + b) + ((long long)r - __ldg(offsets + b));
  pos = t;
  z = -1;
  if (t < 0 || t >= c.capacity) {
    if (c.status) atomicOr(c.status, kStatusBadSeqLen);
    return true;
  }
  const int entry =
      c.paged ? __ldg(c.block_table + (long long)b * c.max_blocks + (int)t / c.page_size) : 0;
  z = token_row(c, b, (int)t, entry);
  if (z < 0 && c.status) atomicOr(c.status, kStatusBadBlockTable);
  return true;
}

// VEC elements of T as a lane holds them: 16 bytes (VEC = 16 / sizeof(T)), or one element.
template <typename T, int VEC>
struct RowVec {
  using Raw = uint4;
  __device__ __forceinline__ static void to_f32(const Raw& r, float* f) {
    Elem<T>::to_f32(r, f);
  }
};
template <typename T>
struct RowVec<T, 1> {
  using Raw = T;
  __device__ __forceinline__ static void to_f32(const Raw& r, float* f) {
    if constexpr (std::is_same<T, float>::value) f[0] = r;
    else if constexpr (std::is_same<T, __half>::value) f[0] = __half2float(r);
    else f[0] = __bfloat162float(r);
  }
};

__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
// Two E4M3 codes, nearest even, |x| > 448 to +-448; `a` in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float a, float b) {
  uint32_t u;
  asm("{\n\t.reg .b16 c;\n\tcvt.rn.satfinite.e4m3x2.f32 c, %2, %1;\n\tcvt.u32.u16 %0, c;\n\t}"
      : "=r"(u)
      : "f"(a), "f"(b));
  return u;
}

// VEC floats as VEC stored elements of C: 16 bytes (8 for E4M3), or one element.
template <typename C, int VEC>
struct Packed;
template <typename C>
struct Packed<C, 8> {
  using type = uint4;
  __device__ __forceinline__ static uint4 pack(const float* f) {
    return make_uint4(pack2(f[0], f[1], C()), pack2(f[2], f[3], C()), pack2(f[4], f[5], C()),
                      pack2(f[6], f[7], C()));
  }
};
template <>
struct Packed<float, 4> {
  using type = uint4;
  __device__ __forceinline__ static uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};
template <>
struct Packed<fp8e4m3, 8> {
  using type = uint2;
  __device__ __forceinline__ static uint2 pack(const float* f) {
    return make_uint2(pack_e4m3x2(f[0], f[1]) | pack_e4m3x2(f[2], f[3]) << 16,
                      pack_e4m3x2(f[4], f[5]) | pack_e4m3x2(f[6], f[7]) << 16);
  }
};
template <typename C>
struct Packed<C, 1> {
  using type = C;
  __device__ __forceinline__ static C pack(const float* f) {
    if constexpr (std::is_same<C, float>::value) return f[0];
    else if constexpr (std::is_same<C, __half>::value) return __float2half_rn(f[0]);
    else if constexpr (std::is_same<C, __nv_bfloat16>::value) return __float2bfloat16_rn(f[0]);
    else return C{(uint8_t)pack_e4m3x2(f[0], 0.f)};
  }
};

// A unit's two vectors to dst + a0 and dst + b0 (elements of C); `joined`: they are neighbours, and (16-byte
// vectors) the row is aligned for one 32-byte access.
template <typename C, typename V>
__device__ __forceinline__ void store_unit(C* dst, int a0, int b0, bool joined, const V& a, const V& b) {
  if constexpr (sizeof(V) == 16) {
    if (joined) {
      store32(dst + a0, a, b);
      return;
    }
  } else if constexpr (sizeof(V) == 8) {
    if (joined) {
      *reinterpret_cast<uint4*>(dst + a0) = make_uint4(a.x, a.y, b.x, b.y);
      return;
    }
  }
  *reinterpret_cast<V*>(dst + a0) = a;
  *reinterpret_cast<V*>(dst + b0) = b;
}

// One block per row (and slice of its heads). A head of d elements is d / (2 VEC) units; a unit is
// two vectors of VEC elements, so VEC rotated pairs: with half pairs the vectors at u VEC and
// u VEC + rotary / 2, else 2 VEC neighbours (also where nothing is rotated). A thread keeps one
// unit position u and walks over heads.
//
// The angle of position t is t * turn mod 1 in 64-bit fixed point: exact for any t, with
// no 64-bit float arithmetic (an fp32 angle at t = 10^6 would be off by 0.06). Its top 32 bits,
// as a signed half-turn count, go through sincospif.
//
// The first two heads' vectors are loaded before the row's place in the cache is looked up, so that the
// lookup chain (offsets, start, table) and the loads run side by side.
//
// Bound by HBM: the rotary of q and k with the FP8 write of 64 prompts (19k rows of 32 + 2 x 8 heads, 441 MB)
// 86 us, 5.1 TB/s; a plain f16 write of 4096 rows of 32 heads 24.6 us, 5.5 TB/s; half-rotated interleaved
// f16 in a gradient (8191 x 32 heads) 26.8 us, 5.0 TB/s, where 134 MB are still short beside the ramp. With
// one row a sequence (64 rows) it is a launch: 4 to 6 us back to back.
template <typename T, typename C, int VEC>
__global__ void __launch_bounds__(kRowThreads, 7)
    rows_kernel(const __grid_constant__ RowParams p) {
  __shared__ __align__(16) float s_cos[kMaxPairs], s_sin[kMaxPairs];
  __shared__ int s_info[4];   // member, position (its low 32 bits, signed; 2^32 more?), cache row
  using V = RowVec<T, VEC>;
  using Raw = typename V::Raw;
  using PT = Packed<T, VEC>;
  using PC = Packed<C, VEC>;
  const int row = blockIdx.x, tid = threadIdx.x;
  const int u = tid % p.units, lane_head = tid / p.units;
  const int heads = p.hq + 2 * p.hkv;
  const int step = p.head_lanes * gridDim.y;
  const int d = p.units * 2 * VEC;
  const bool turned = u * 2 * VEC < p.rotary;
  const bool apart = turned && !p.interleaved;   // the two vectors lie rotary / 2 apart
  const int a0 = apart ? u * VEC : u * 2 * VEC;
  const int b0 = apart ? a0 + p.rotary / 2 : a0 + VEC;
  int h = lane_head < p.head_lanes ? lane_head + p.head_lanes * blockIdx.y : heads;

  auto load = [&](int hh, Raw& a, Raw& b) {
    const T* x;
    if (hh < p.hq) x = static_cast<const T*>(p.q) + row * p.q_rs + hh * p.q_hs;
    else if (hh < p.hq + p.hkv) x = static_cast<const T*>(p.k) + row * p.k_rs + (hh - p.hq) * p.k_hs;
    else x = static_cast<const T*>(p.v) + row * p.v_rs + (hh - p.hq - p.hkv) * p.v_hs;
    if constexpr (VEC > 1) {
      if (!apart && p.wide_in) {
        load32(x + a0, a, b);
        return;
      }
    }
    a = *reinterpret_cast<const Raw*>(x + a0);
    b = *reinterpret_cast<const Raw*>(x + b0);
  };
  // two heads ahead of the one in hand
  Raw ra[2]{}, rb[2]{};
  if (h < heads) load(h, ra[0], rb[0]);
  if (h + step < heads) load(h + step, ra[1], rb[1]);

  long long z = -1;
  int pos = 0;
  bool far = false;   // past 2^31, where a row lies far behind its cache: its q is rotated all the same
  if (p.row_offsets) {
    if (tid == 0) {
      long long at = 0;
      int zz = -1;
      const bool member = locate_row(p.cache, p.row_offsets, p.start, row, at, zz);
      if (member && p.positions) at = __ldg(p.positions + row);
      s_info[0] = member;
      s_info[1] = (int)at;
      s_info[2] = at > INT_MAX;
      s_info[3] = zz;
    }
    __syncthreads();
    if (!s_info[0]) return;
    pos = s_info[1];
    far = s_info[2];
    z = s_info[3];
  } else {
    pos = __ldg(p.positions + row);
  }
  if (p.rotary) {
    for (int i = tid; i < p.rotary / 2; i += kRowThreads) {
      unsigned long long a = (unsigned long long)(long long)pos * p.turn[i];
      if (far) a += p.turn[i] << 32;
      float s, c;
      sincospif((float)(int)(unsigned)(a >> 32) * 4.656612873077393e-10f, &s, &c);   // 2^-31
      s_cos[i] = c * p.m;
      s_sin[i] = (p.transpose ? -s : s) * p.m;
    }
    __syncthreads();
  }

  float most_k = 0.f, most_v = 0.f;
  const bool out_joined = VEC > 1 && !apart && p.wide_out;
  auto put = [&](int cur, const Raw& xa, const Raw& xb) {
    const bool is_q = cur < p.hq, is_k = !is_q && cur < p.hq + p.hkv;
    if (!is_q && z < 0) return;   // no place in the cache
    const bool rot = turned && (is_q || is_k);
    const int kvh = is_k ? cur - p.hq : cur - p.hq - p.hkv;
    const long long at = is_q ? row * p.qo_rs + cur * p.qo_hs
                              : (z * p.hkv + kvh) * (long long)d;
    // elements that pass unchanged move as they are
    if (!rot && !p.amax && (is_q || std::is_same<T, C>::value)) {
      T* dst = static_cast<T*>(is_q ? p.q_out : is_k ? p.k_cache : p.v_cache) + at;
      store_unit(dst, a0, b0, out_joined, xa, xb);
      return;
    }
    float e[2 * VEC];
    V::to_f32(xa, e);
    V::to_f32(xb, e + VEC);
    if (rot) {
      const float* cs = s_cos + u * VEC;   // (kept in shared memory: registers bound the blocks an SM)
      const float* sn = s_sin + u * VEC;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        if (p.interleaved) {
          const float a = e[2 * i], b = e[2 * i + 1];
          e[2 * i] = __fmaf_rn(a, cs[i], -__fmul_rn(b, sn[i]));   // the same in every instantiation
          e[2 * i + 1] = __fmaf_rn(b, cs[i], __fmul_rn(a, sn[i]));
        } else {
          const float a = e[i], b = e[VEC + i];
          e[i] = __fmaf_rn(a, cs[i], -__fmul_rn(b, sn[i]));
          e[VEC + i] = __fmaf_rn(b, cs[i], __fmul_rn(a, sn[i]));
        }
      }
    }
    if (is_q) {
      store_unit(static_cast<T*>(p.q_out) + at, a0, b0, out_joined, PT::pack(e), PT::pack(e + VEC));
      return;
    }
    if (p.amax) {
      float& most = is_k ? most_k : most_v;
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i) most = fmaxf(most, fabsf(e[i]));   // NaN passes over
    }
    if constexpr (std::is_same<C, fp8e4m3>::value) {
      // A division: next to a tie between two codes a product with 1 / scale, rounded twice, falls to the
      // other side (30 of the 65280 bf16 values at scale 0.0075). It costs 8 of the 86 us of 64 prompts. (Products,
      // and a division only where one lies within its error of a tie: 89 us.)
      const float scale = is_k ? p.k_scale : p.v_scale;
#pragma unroll
      for (int i = 0; i < 2 * VEC; ++i) e[i] = __fdiv_rn(e[i], scale);
    }
    store_unit(static_cast<C*>(is_k ? p.k_cache : p.v_cache) + at, a0, b0,
               std::is_same<C, fp8e4m3>::value ? VEC > 1 && !apart : out_joined, PC::pack(e),
               PC::pack(e + VEC));
  };
  while (h < heads) {
    {
      const Raw xa = ra[0], xb = rb[0];
      if (h + 2 * step < heads) load(h + 2 * step, ra[0], rb[0]);
      put(h, xa, xb);
    }
    h += step;
    if (h >= heads) break;
    const Raw xa = ra[1], xb = rb[1];
    if (h + 2 * step < heads) load(h + 2 * step, ra[1], rb[1]);
    put(h, xa, xb);
    h += step;
  }
  if (p.amax) {
    __syncwarp();
    for (int o = 16; o > 0; o >>= 1) {
      most_k = fmaxf(most_k, __shfl_xor_sync(0xffffffffu, most_k, o));
      most_v = fmaxf(most_v, __shfl_xor_sync(0xffffffffu, most_v, o));
    }
    // non-negative floats order as their bits; a maximum does not depend on order (64 prompts of 300 rows into
    // FP8 pages, rotary: 92.5 us with the maxima, 88.4 without)
    if ((tid & 31) == 0) {
      if (most_k > 0.f) atomicMax(reinterpret_cast<int*>(p.amax), __float_as_int(most_k));
      if (most_v > 0.f) atomicMax(reinterpret_cast<int*>(p.amax) + 1, __float_as_int(most_v));
    }
  }
}

template <typename T, typename C>
const void* rows_kernel_for(bool vec) {
  return vec ? reinterpret_cast<const void*>(&rows_kernel<T, C, 16 / (int)sizeof(T)>)
             : reinterpret_cast<const void*>(&rows_kernel<T, C, 1>);
}

// Whether a row tensor can move `bytes` (16 or 32) a lane.
bool vector_ok(const void* p, long long rs, long long hs, int es, int bytes = 16) {
  return !p || (aligned(p, bytes) && rs * es % bytes == 0 && hs * es % bytes == 0);
}

// A row tensor's places in memory, from its strides in elements (of which a byte's are a few bits more: larger
// ones than memory has are as good as the largest).
RowRuns runs(const void* p, long long rows, long long rs, long long heads, long long hs, int d, int es) {
  auto bytes = [es](long long s) {
    const long long most = INT64_MAX / 8;
    return std::min(std::max(s, -most), most) * es;
  };
  return {(uint64_t)(uintptr_t)p, rows, bytes(rs), heads, bytes(hs), (int64_t)d * es};
}

// SMs of the current device, asked for once; 0: not known (cuda_fail has the reason).
int device_sms() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0, n = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < kDevices && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) {
    cuda_fail(e, "asking for the device's SMs");
    return 0;
  }
  if (dev < kDevices) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

int launch_rows(RowParams& p, int head_dim, int es, bool vec, int sms, const void* fn,
                cudaStream_t stream) {
  const int v = vec ? 16 / es : 1;
  p.units = head_dim / (2 * v);
  p.head_lanes = kRowThreads / p.units;
  const int heads = p.hq + 2 * p.hkv;
  // A block per row, or several (64 rows of 64 heads, or 1 of 128: 4.1 us, one block a row 6.2).
  const int passes = (heads + p.head_lanes - 1) / p.head_lanes;
  const int slices = row_slices(p.rows, passes, sms);
  void* args[1] = {&p};
  const cudaError_t e = cudaLaunchKernel(fn, dim3((unsigned)p.rows, (unsigned)slices),
                                         dim3(kRowThreads), args, 0, stream);
  return e == cudaSuccess ? DA_OK : cuda_fail(e, "launching the rows kernel");
}

void set_rope(RowParams& p, const da_rope* rope) {
  if (!rope) return;
  p.rotary = rope->cfg.rotary_dim;
  p.interleaved = rope->cfg.interleaved;
  p.m = (float)rope->cfg.attn_factor;
  std::memcpy(p.turn, rope->turn, sizeof p.turn);
}

// ---- read kernel ----------------------------------------------------------------------------
struct ReadParams {
  Params cache;
  const void* src[2];           // the caches read (K, V, or one of them)
  void* dst[2];
  float scale[2];
  const int32_t* row_offsets;
  const int32_t* start;
  int rows;
  int chunks;                   // 16-byte chunks of a cache row of one tensor
  int row_items;                // chunks * tensors
  unsigned row_magic, chunk_magic;   // ceil(2^32 / row_items), ceil(2^32 / chunks)
  long long items;              // rows * row_items
  int wide;                     // the outputs lie on 32-byte boundaries
};

constexpr int kReadThreads = 256, kReadItems = 4;

// The step's rows as one line of items (row, tensor, 16-byte chunk of the cache row). A warp takes
// 128 neighbouring items, 4 a lane with all their loads in flight; its lanes look up the
// rows these touch, one row a lane, and pass the cache rows on by shuffles. They are at most 32: a
// row has a multiple of 4 items, and one of 4 (one tensor, one head of 64 codes) starts where a
// warp does. (8 a lane: up to 4 % slower below 2e6 items, the same above, bf16 and fp32; for FP8, whose results take
// twice the registers, 266 us instead of 244 below.)
// Bound by HBM: 64 sequences of 512 to 8192 FP8 tokens to bf16 (1.7 GB) 244 us, 7.0 TB/s (a plain
// copy: 6.7); a warp a row, with its lookup ahead of its loads, took 346.
template <typename T, typename C>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ ReadParams p) {
  constexpr int PER = kReadItems;
  constexpr bool kFp8 = std::is_same<C, fp8e4m3>::value;
  const int lane = threadIdx.x & 31;
  const long long i0 =
      ((long long)blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5)) * (32 * PER);
  if (i0 >= p.items) return;   // the whole warp
  const int row0 = (int)(i0 / p.row_items);
  const int off0 = (int)(i0 - (long long)row0 * p.row_items);
  // rows row0 + lane: -2 none or of no sequence, -1 no place, else the cache row
  int z = -2;
  if (lane * p.row_items < off0 + 32 * PER && row0 + lane < p.rows) {
    long long pos;
    if (!locate_row(p.cache, p.row_offsets, p.start, row0 + lane, pos, z)) z = -2;
  }
  uint4 c[PER];
  int zr[PER], dr[PER], ch[PER];
  unsigned t[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const unsigned i = (unsigned)(off0 + k * 32 + lane);
    dr[k] = (int)__umulhi(i, p.row_magic);                    // i / row_items
    const unsigned in_row = i - (unsigned)dr[k] * p.row_items;
    t[k] = __umulhi(in_row, p.chunk_magic);                   // 0: the first tensor, 1: the second
    ch[k] = (int)(in_row - t[k] * p.chunks);
    zr[k] = __shfl_sync(0xffffffffu, z, dr[k] & 31);
    c[k] = make_uint4(0u, 0u, 0u, 0u);
    if (zr[k] >= 0)
      c[k] = __ldg(reinterpret_cast<const uint4*>(p.src[t[k] & 1]) +
                   (long long)zr[k] * p.chunks + ch[k]);
  }
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    if (zr[k] == -2) continue;
    const long long at = (long long)(row0 + dr[k]) * p.chunks + ch[k];
    if constexpr (!kFp8) {
      static_cast<uint4*>(p.dst[t[k] & 1])[at] = c[k];
    } else {
      const float s = p.scale[t[k] & 1];
      const uint32_t w[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t lo, hi;
        e4m3x4_to_f16x2(w[j], lo, hi);
        __half2 h;
        memcpy(&h, &lo, 4);
        const float2 f = __half22float2(h);
        memcpy(&h, &hi, 4);
        const float2 g = __half22float2(h);
        o[2 * j] = pack2(f.x * s, f.y * s, T());
        o[2 * j + 1] = pack2(g.x * s, g.y * s, T());
      }
      uint4* d = static_cast<uint4*>(p.dst[t[k] & 1]) + 2 * at;
      const uint4 lo4 = make_uint4(o[0], o[1], o[2], o[3]), hi4 = make_uint4(o[4], o[5], o[6], o[7]);
      if (p.wide) {
        store32(d, lo4, hi4);
      } else {
        d[0] = lo4;
        d[1] = hi4;
      }
    }
  }
}

// Checks that the write and the read share; the status word when a workspace is given.
int common_checks(const da_plan& pl, const int32_t* block_table, const int32_t* row_offsets,
                  const int32_t* start, int rows, const void* workspace, size_t workspace_bytes) {
  if (rows < 0 || !row_offsets || !start) return DA_ERR_INVALID_ARG;
  if (pl.prob.paged ? !block_table : block_table != nullptr) return DA_ERR_INVALID_ARG;
  if (!aligned(row_offsets, 4) || !aligned(start, 4) || (block_table && !aligned(block_table, 4)))
    return DA_ERR_INVALID_ARG;
  if (workspace ? !aligned(workspace, 256) : pl.prob.validate != 0) return DA_ERR_INVALID_ARG;
  if (workspace && workspace_bytes < pl.ws_bytes) return DA_ERR_WORKSPACE_TOO_SMALL;
  return DA_OK;
}

int clear_status(const da_plan& pl, void* workspace, cudaStream_t stream) {
  if (!pl.prob.validate) return DA_OK;
  const cudaError_t e = cudaMemsetAsync(static_cast<char*>(workspace) + pl.off_status, 0, 4, stream);
  return e == cudaSuccess ? DA_OK : cuda_fail(e, "cudaMemsetAsync(status)");
}

}  // namespace

extern "C" {

int decode_attn_rope_create(const da_rope_config* config, da_rope** rope_out) {
  if (!config || !rope_out) return DA_ERR_INVALID_ARG;
  *rope_out = nullptr;
  const da_rope_config& c = *config;
  if (c.head_dim < 2 || c.head_dim > 2 * kMaxPairs || c.head_dim % 2) return DA_ERR_UNSUPPORTED;
  if (c.rotary_dim < 2 || c.rotary_dim > c.head_dim || c.rotary_dim % 2) return DA_ERR_UNSUPPORTED;
  if (c.interleaved != 0 && c.interleaved != 1) return DA_ERR_INVALID_ARG;
  if (!std::isfinite(c.base) || !(c.base > 1.0) || !std::isfinite((float)c.attn_factor))
    return DA_ERR_INVALID_ARG;
  const bool ramp = c.scaling == DA_ROPE_BY_PARTS || c.scaling == DA_ROPE_BY_INDEX;
  if (c.scaling < DA_ROPE_NONE || c.scaling > DA_ROPE_BY_INDEX) return DA_ERR_INVALID_ARG;
  if (c.scaling != DA_ROPE_NONE && (!std::isfinite(c.factor) || !(c.factor > 0.0)))
    return DA_ERR_INVALID_ARG;
  if (ramp && (!std::isfinite(c.original_max_position) || !(c.original_max_position > 0.0) ||
               !std::isfinite(c.low) || !std::isfinite(c.high) || !(c.low > 0.0) ||
               !(c.low < c.high)))
    return DA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  const int n = c.rotary_dim;
  double base = c.base;
  if (c.scaling == DA_ROPE_NTK && n > 2) base *= std::pow(c.factor, (double)n / (n - 2));
  if (!std::isfinite(base) || !(base > 0.0)) return DA_ERR_INVALID_ARG;
  double first = 0.0, last = 0.0;
  if (c.scaling == DA_ROPE_BY_INDEX) {
    auto at = [&](double turns) {
      return n * std::log(c.original_max_position / (turns * two_pi)) / (2.0 * std::log(c.base));
    };
    first = std::max(std::floor(at(c.high)), 0.0);
    last = std::min(std::ceil(at(c.low)), (double)n - 1.0);
  }
  da_rope* r = new (std::nothrow) da_rope();
  if (!r) return DA_ERR_INVALID_ARG;
  r->cfg = c;
  for (int i = 0; i < n / 2; ++i) {
    double theta = std::pow(base, -2.0 * i / n);
    double keep = 1.0;
    if (c.scaling == DA_ROPE_LINEAR) keep = 0.0;
    if (c.scaling == DA_ROPE_BY_PARTS) {
      const double turns = c.original_max_position * theta / two_pi;
      keep = std::min(std::max((turns - c.low) / (c.high - c.low), 0.0), 1.0);
    }
    if (c.scaling == DA_ROPE_BY_INDEX)
      keep = 1.0 - std::min(std::max((i - first) / std::max(last - first, 0.001), 0.0), 1.0);
    if (keep < 1.0) theta = theta / c.factor * (1.0 - keep) + theta * keep;
    if (!std::isfinite(theta)) {
      delete r;
      return DA_ERR_INVALID_ARG;
    }
    r->theta[i] = theta;
    // whole turns per position leave every integer position where it is
    const double turns = theta / two_pi;
    const double frac = turns - std::floor(turns);
    // 64 fraction bits in two halves, each exact in a double
    const double hi = std::floor(frac * 4294967296.0);
    const double lo = std::floor((frac * 4294967296.0 - hi) * 4294967296.0 + 0.5);
    r->turn[i] = ((unsigned long long)hi << 32) + (unsigned long long)lo;
  }
  *rope_out = r;
  return DA_OK;
}

int decode_attn_rope_frequencies(const da_rope* rope, double* theta) {
  if (!rope || !theta) return DA_ERR_INVALID_ARG;
  std::memcpy(theta, rope->theta, sizeof(double) * (rope->cfg.rotary_dim / 2));
  return DA_OK;
}

void decode_attn_rope_destroy(da_rope* rope) { delete rope; }

int decode_attn_rope_apply(const da_rope* rope, const da_rope_args* args) {
  if (!rope || !args) return DA_ERR_INVALID_ARG;
  const da_rope_args& a = *args;
  if (a.rows < 0 || a.heads < 1 || (a.transpose != 0 && a.transpose != 1))
    return DA_ERR_INVALID_ARG;
  if (a.dtype < DA_F32 || a.dtype > DA_BF16 || a.heads > DECODE_ATTN_ROPE_MAX_HEADS)
    return DA_ERR_UNSUPPORTED;
  if (a.rows == 0) return DA_OK;
  const int es = elem_size(a.dtype);
  if (!a.x || !a.out || !a.positions || !aligned(a.x, es) || !aligned(a.out, es) ||
      !aligned(a.positions, 4))
    return DA_ERR_INVALID_ARG;
  const int d = rope->cfg.head_dim;
  const RowRuns in = runs(a.x, a.rows, a.x_row_stride, a.heads, a.x_head_stride, d, es);
  const RowRuns result = runs(a.out, a.rows, a.out_row_stride, a.heads, a.out_head_stride, d, es);
  if (!lie_apart(result) || !result_ok(in, result)) return DA_ERR_INVALID_ARG;
  RowParams p;
  std::memset(&p, 0, sizeof p);
  set_rope(p, rope);
  p.q = a.x;
  p.q_out = a.out;
  p.q_rs = a.x_row_stride;
  p.q_hs = a.x_head_stride;
  p.qo_rs = a.out_row_stride;
  p.qo_hs = a.out_head_stride;
  p.positions = a.positions;
  p.rows = a.rows;
  p.hq = a.heads;
  p.transpose = a.transpose;
  const int pair = 32 / es;   // elements of one unit
  const bool vec = rope->cfg.head_dim % pair == 0 && rope->cfg.rotary_dim % pair == 0 &&
                   vector_ok(a.x, a.x_row_stride, a.x_head_stride, es) &&
                   vector_ok(a.out, a.out_row_stride, a.out_head_stride, es);
  p.wide_in = vector_ok(a.x, a.x_row_stride, a.x_head_stride, es, 32);
  p.wide_out = vector_ok(a.out, a.out_row_stride, a.out_head_stride, es, 32);
  const void* fn = a.dtype == DA_F32   ? rows_kernel_for<float, float>(vec)
                   : a.dtype == DA_F16 ? rows_kernel_for<__half, __half>(vec)
                                       : rows_kernel_for<__nv_bfloat16, __nv_bfloat16>(vec);
  const int sms = device_sms();
  if (sms <= 0) return DA_ERR_CUDA;
  return launch_rows(p, rope->cfg.head_dim, es, vec, sms, fn, static_cast<cudaStream_t>(a.cuda_stream));
}

int decode_attn_kv_write(const da_plan* plan, const da_kv_write_args* args) {
  if (!plan || !args) return DA_ERR_INVALID_ARG;
  const da_plan& pl = *plan;
  const da_kv_write_args& a = *args;
  const da_problem& pr = pl.prob;
  int rc = common_checks(pl, a.block_table, a.row_offsets, a.start, a.rows, a.workspace,
                         a.workspace_bytes);
  if (rc != DA_OK) return rc;
  if (!a.rope && (a.positions || a.q || a.q_out)) return DA_ERR_INVALID_ARG;
  if ((a.q == nullptr) != (a.q_out == nullptr) && a.rows > 0) return DA_ERR_INVALID_ARG;
  if (a.rope && a.rope->cfg.head_dim != pr.head_dim) return DA_ERR_INVALID_ARG;
  if (a.rows == 0) return DA_OK;
  const int es = pl.es;
  if (!a.k || !a.v || !a.k_cache || !a.v_cache || !aligned(a.k, es) || !aligned(a.v, es) ||
      !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !aligned(a.positions, 4) ||
      !aligned(a.q, es) || !aligned(a.q_out, es) || !aligned(a.amax, 4))
    return DA_ERR_INVALID_ARG;
  const int d = pr.head_dim;
  if (a.q) {
    const RowRuns q = runs(a.q, a.rows, a.q_row_stride, pr.num_q_heads, a.q_head_stride, d, es);
    const RowRuns k = runs(a.k, a.rows, a.k_row_stride, pr.num_kv_heads, a.k_head_stride, d, es);
    const RowRuns v = runs(a.v, a.rows, a.v_row_stride, pr.num_kv_heads, a.v_head_stride, d, es);
    const RowRuns out = runs(a.q_out, a.rows, a.q_out_row_stride, pr.num_q_heads, a.q_out_head_stride, d, es);
    if (!lie_apart(out) || !result_ok(q, out) || may_share(k, out) || may_share(v, out))
      return DA_ERR_INVALID_ARG;
  }
  const long long tokens = pr.paged ? (long long)pr.num_physical_blocks * pr.page_size
                                    : (long long)pr.batch * pr.max_seq_len;
  const long long cache_bytes = tokens * pr.num_kv_heads * d * pl.kv_es;
  if (overlap(a.k_cache, cache_bytes, a.v_cache, cache_bytes)) return DA_ERR_INVALID_ARG;
  RowParams p;
  std::memset(&p, 0, sizeof p);
  fill_common(pl, p.cache, a.block_table, nullptr, a.workspace);
  set_rope(p, a.rope);
  p.q = a.q;
  p.q_out = a.q_out;
  p.k = a.k;
  p.v = a.v;
  p.k_cache = a.k_cache;
  p.v_cache = a.v_cache;
  p.q_rs = a.q_row_stride;
  p.q_hs = a.q_head_stride;
  p.qo_rs = a.q_out_row_stride;
  p.qo_hs = a.q_out_head_stride;
  p.k_rs = a.k_row_stride;
  p.k_hs = a.k_head_stride;
  p.v_rs = a.v_row_stride;
  p.v_hs = a.v_head_stride;
  p.row_offsets = a.row_offsets;
  p.start = a.start;
  p.positions = a.positions;
  p.amax = a.amax;
  p.rows = a.rows;
  p.hq = a.q ? pr.num_q_heads : 0;
  p.hkv = pr.num_kv_heads;
  if (pr.kv_fp8) {
    p.k_scale = pr.k_scale;
    p.v_scale = pr.v_scale;
    // (so small a scale stands for no stored row: its codes end below fp32's normal range)
    if (!std::isfinite((float)(1.0 / (double)pr.k_scale)) ||
        !std::isfinite((float)(1.0 / (double)pr.v_scale)))
      return DA_ERR_INVALID_ARG;
  }
  const bool vec = (!a.rope || a.rope->cfg.rotary_dim % (32 / es) == 0) &&
                   vector_ok(a.q, a.q_row_stride, a.q_head_stride, es) &&
                   vector_ok(a.q_out, a.q_out_row_stride, a.q_out_head_stride, es) &&
                   vector_ok(a.k, a.k_row_stride, a.k_head_stride, es) &&
                   vector_ok(a.v, a.v_row_stride, a.v_head_stride, es);
  p.wide_in = vector_ok(a.q, a.q_row_stride, a.q_head_stride, es, 32) &&
              vector_ok(a.k, a.k_row_stride, a.k_head_stride, es, 32) &&
              vector_ok(a.v, a.v_row_stride, a.v_head_stride, es, 32);
  p.wide_out = vector_ok(a.q_out, a.q_out_row_stride, a.q_out_head_stride, es, 32) &&
               aligned(a.k_cache, 32) && aligned(a.v_cache, 32);
  const void* fn = pr.kv_fp8                ? rows_kernel_for<__nv_bfloat16, fp8e4m3>(vec)
                   : pr.qkv_dtype == DA_F32 ? rows_kernel_for<float, float>(vec)
                   : pr.qkv_dtype == DA_F16 ? rows_kernel_for<__half, __half>(vec)
                                            : rows_kernel_for<__nv_bfloat16, __nv_bfloat16>(vec);
  cudaStream_t stream = static_cast<cudaStream_t>(a.cuda_stream);
  rc = clear_status(pl, a.workspace, stream);
  if (rc == DA_OK) rc = launch_rows(p, pr.head_dim, es, vec, pl.num_sms, fn, stream);
  if (rc == DA_OK && pr.validate) rc = decode_attn_check_status(plan, a.workspace, stream);
  return rc;
}

int decode_attn_kv_read(const da_plan* plan, const da_kv_read_args* args) {
  if (!plan || !args) return DA_ERR_INVALID_ARG;
  const da_plan& pl = *plan;
  const da_kv_read_args& a = *args;
  const da_problem& pr = pl.prob;
  int rc = common_checks(pl, a.block_table, a.row_offsets, a.start, a.rows, a.workspace,
                         a.workspace_bytes);
  if (rc != DA_OK) return rc;
  if (a.rows == 0) return DA_OK;
  if ((a.k_out == nullptr) != (a.k_cache == nullptr) ||
      (a.v_out == nullptr) != (a.v_cache == nullptr) || (!a.k_out && !a.v_out))
    return DA_ERR_INVALID_ARG;
  if (!aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) || !aligned(a.k_out, 16) ||
      !aligned(a.v_out, 16))
    return DA_ERR_INVALID_ARG;
  const long long bytes = (long long)a.rows * pr.num_kv_heads * pr.head_dim * pl.es;
  if (overlap(a.k_out, bytes, a.v_out, bytes)) return DA_ERR_INVALID_ARG;
  ReadParams p;
  std::memset(&p, 0, sizeof p);
  fill_common(pl, p.cache, a.block_table, nullptr, a.workspace);
  int nt = 0;
  if (a.k_out) {
    p.src[nt] = a.k_cache;
    p.dst[nt] = a.k_out;
    p.scale[nt++] = pr.k_scale;
  }
  if (a.v_out) {
    p.src[nt] = a.v_cache;
    p.dst[nt] = a.v_out;
    p.scale[nt++] = pr.v_scale;
  }
  p.row_offsets = a.row_offsets;
  p.start = a.start;
  p.rows = a.rows;
  p.chunks = pr.num_kv_heads * pr.head_dim * pl.kv_es / 16;
  p.row_items = p.chunks * nt;
  // i / n = umulhi(i, ceil(2^32 / n)) for i n < 2^32: here i < row_items + 128 and n = row_items,
  // or i < row_items and n = chunks, which caps row_items at 2^15
  if (p.row_items > (1 << 15)) return DA_ERR_UNSUPPORTED;
  p.row_magic = (unsigned)(((1ull << 32) + p.row_items - 1) / p.row_items);
  p.chunk_magic = (unsigned)(((1ull << 32) + p.chunks - 1) / p.chunks);
  p.items = (long long)p.rows * p.row_items;
  p.wide = aligned(a.k_out, 32) && aligned(a.v_out, 32);
  const long long per_block = (long long)kReadThreads * kReadItems;
  const long long blocks = (p.items + per_block - 1) / per_block;
  if (blocks >= (1ll << 31)) return DA_ERR_UNSUPPORTED;
  const void* fn = pr.kv_fp8 ? reinterpret_cast<const void*>(&read_kernel<__nv_bfloat16, fp8e4m3>)
                   : pr.qkv_dtype == DA_F32
                       ? reinterpret_cast<const void*>(&read_kernel<float, float>)
                       : reinterpret_cast<const void*>(&read_kernel<__half, __half>);   // moved as bits
  cudaStream_t stream = static_cast<cudaStream_t>(a.cuda_stream);
  rc = clear_status(pl, a.workspace, stream);
  if (rc != DA_OK) return rc;
  void* kargs[1] = {&p};
  const cudaError_t e = cudaLaunchKernel(fn, dim3((unsigned)blocks), dim3(kReadThreads), kargs, 0,
                                         stream);
  if (e != cudaSuccess) return cuda_fail(e, "launching the read kernel");
  return pr.validate ? decode_attn_check_status(plan, a.workspace, stream) : DA_OK;
}

}  // extern "C"
