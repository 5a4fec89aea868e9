// Writing rows of K and V into the 4-bit paged cache, and reading them back.
//
// A group of 32 values x is held as codes c and a pair (lo, step):
//   lo = min x (down to bf16), step = (max x - lo) / 15 (up to bf16),
//   c = rint((x - lo) / step) in 0..15,   value = lo + step c.
// Both are bound by the rows' bytes (2 or 4 a value, against 5 bits in the
// cache).  A warp takes the rows of one tile (16 positions of one sequence and
// head) of K or of V, so that what it touches is contiguous on both sides: the
// tile's rows, and its codes and pairs.
//
// Measured on GB300 (CUDA graph, back to back; of the measured copy rate of
// 6.80 TB/s): 8 x 4096 rows of 8 heads, d = 128, bf16, written and read back,
// 63 us for 352 MB (82 %): writing about 37 us (176 MB, 70 %; with two lanes a
// group 40 us, 16.5 instructions a value issued in 74 % of the cycles, the
// logic pipe 64 % busy), reading about 26 us, at the copy rate.  One token of
// each of 64 sequences, written and read, 4.6 us: two launches' latency.
// A thread per group took 520 us for the first of these (its lanes' addresses
// lie apart), a warp per tile 133, one pass of loads in flight ahead of the
// other 88, two lanes a group instead of four 82, codes without a branch for
// exact halves 67, streaming loads 65.7, one lane a group 63.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "plsh_internal.h"
#include "q4.cuh"

namespace plsh {
namespace {

using namespace q4;
using namespace ptx;

constexpr int kWarps = 4;
constexpr unsigned FULL = 0xffffffffu;

// The warp's tile and the rows of it that the call names.
struct TileRows {
  uint8_t* tile;
  int64_t row0;        // row of [B, H, m] that position 0 of the tile would be
  int r0, r1;          // positions [r0, r1) of the tile
  bool value;          // V's part
};

// Tiles that m consecutive positions can touch.
__host__ __device__ __forceinline__ int64_t tiles_of(int64_t m) { return (m + 2 * (kTile - 1)) / kTile; }

template <int D>
__device__ __forceinline__ bool tile_rows(const Q4RowsArgs& a, TileRows& w) {
  const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  // (fewer than 2^31 tiles in a call)
  const uint32_t tiles = (uint32_t)tiles_of(a.m), unit = (uint32_t)(id >> 1);
  w.value = id & 1;
  const uint32_t bh = unit / tiles;
  if (bh >= (uint32_t)a.c.B * (uint32_t)a.c.H) return false;
  const int b = (int)(bh / (uint32_t)a.c.H), h = (int)(bh - (uint32_t)b * a.c.H);
  const int64_t len = a.len == nullptr ? a.m : min((int64_t)a.len[b], a.m);
  const int64_t p0 = a.pos[b], start = ((p0 >> 4) + (int64_t)(unit - bh * tiles)) * kTile;   // the tile's first position
  w.r0 = (int)max((int64_t)0, p0 - start);
  w.r1 = (int)min((int64_t)kTile, p0 + len - start);
  if (w.r0 >= w.r1) return false;
  w.row0 = (int64_t)bh * a.m + (start - p0);
  w.tile = tile_of<D>(a.c, b, h, start, a.err);
  return w.tile != nullptr;
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float reciprocal(float x) {      // within an ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Eight consecutive values of a row: 16 bytes of bf16, 32 of fp32; read once.
template <typename T> struct Eight {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) w[k] = __ldcs(reinterpret_cast<const uint4*>(p) + k);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
      const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (sizeof(T) == 4) {
          v[4 * k + e] = __uint_as_float(x[e]);
        } else {
          v[2 * e] = __uint_as_float(x[e] << 16);
          v[2 * e + 1] = __uint_as_float(x[e] & 0xffff0000u);
        }
      }
    }
  }
  // smallest and largest of the eight; NaN if one is NaN
  __device__ __forceinline__ void range(const float (&v)[8], float& mn, float& mx) const {
    if constexpr (sizeof(T) == 4) {
      mn = mx = v[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) {
        mn = min_nan(mn, v[e]);
        mx = max_nan(mx, v[e]);
      }
    } else {
      const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&w[0]);
      const __nv_bfloat162 lo = __hmin2_nan(__hmin2_nan(x[0], x[1]), __hmin2_nan(x[2], x[3]));
      const __nv_bfloat162 hi = __hmax2_nan(__hmax2_nan(x[0], x[1]), __hmax2_nan(x[2], x[3]));
      mn = min_nan(__low2float(lo), __high2float(lo));
      mx = max_nan(__low2float(hi), __high2float(hi));
    }
  }
};

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r, x, y, z;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }

// A code c is left as the bits of 1.5 2^23 + c, that is kMagicBits + c.
constexpr float kMagic = 12582912.f;
constexpr uint32_t kMagicBits = 0x4b400000u;

// The word of eight codes, c0 + 16 c1 + ... + 16^7 c7, from such bits; their
// constants add up to a constant (modulo 2^32).
__device__ __forceinline__ uint32_t eight_codes(const float (&c)[8]) {
  uint32_t w = __float_as_uint(c[0]) - kMagicBits * 0x11111111u;
#pragma unroll
  for (int e = 1; e < 8; ++e) w += __float_as_uint(c[e]) << (4 * e);
  return w;
}

// Eight codes from the definition: the quotient rounded to fp32, then to the
// nearest integer.
__device__ __noinline__ uint32_t codes_by_division(float d0, float d1, float d2, float d3, float d4, float d5,
                                                   float d6, float d7, float step) {
  const float c[8] = {__fdiv_rn(d0, step) + kMagic, __fdiv_rn(d1, step) + kMagic, __fdiv_rn(d2, step) + kMagic,
                      __fdiv_rn(d3, step) + kMagic, __fdiv_rn(d4, step) + kMagic, __fdiv_rn(d5, step) + kMagic,
                      __fdiv_rn(d6, step) + kMagic, __fdiv_rn(d7, step) + kMagic};
  return eight_codes(c);
}

// The same without a division (Markstein, 1990): q0 = d inv, with inv the
// reciprocal of step within an ulp, is within three ulp of Q = d / step; the
// remainder r = d - q0 step is exact (step has eight bits, so r has at most
// eleven); and q0 + r inv, rounded once, is Q's rounding.  For its unrounded
// value is within 3 2^-22 ulp of Q, and Q, unless it is an fp32 number itself,
// is no nearer than 2^-9 ulp to a midpoint m of two of them: d - m step is a
// multiple of half an ulp of Q times step's last bit, not zero (m step has 25
// bits or more, d 24), and step is less than 256 of its last bits.  A step
// whose reciprocal or products leave fp32's normal range is `rare` and takes
// the division.
// A pass of 32 lanes met an exact half (bf16 values: one in some hundreds)
// nearly always, so settling halves in a branch cost every warp that branch;
// this costs two packed products a pair of values.
__device__ __forceinline__ uint32_t codes_of(const float (&v)[8], float lo, float step, float inv, bool rare) {
  float d[8], c[8];
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 x = fma2(make_float2(v[e], v[e + 1]), two(1.f), two(-lo));
    const float2 q0 = fma2(x, two(inv), two(0.f));
    const float2 r = fma2(q0, two(-step), x);
    const float2 q = fma2(r, two(inv), q0);
    const float2 k = fma2(q, two(1.f), two(kMagic));
    d[e] = x.x, d[e + 1] = x.y;
    c[e] = k.x, c[e + 1] = k.y;
  }
  if (rare) return codes_by_division(d[0], d[1], d[2], d[3], d[4], d[5], d[6], d[7], step);
  return eight_codes(c);
}

// G lanes a group, 32 / G values each (eights t, t + G, ...): what a group costs
// beside its values (range, pair, reciprocal, addresses) is shared by more of
// them where one lane has a group, and a row is done sooner where two have it
// (launch_rows).
template <typename T, int D, int G>
__global__ void __launch_bounds__(32 * kWarps) q4_write_kernel(const __grid_constant__ Q4RowsArgs a) {
  using L = Layout<D>;
  constexpr int kLanes = D / 32 * G;              // lanes of a row
  constexpr int kEights = 4 / G;                  // eights t, t + G, ... of a group
  constexpr int kRows = 32 / kLanes;              // rows of a pass
  __shared__ alignas(16) uint8_t stage_s[kWarps][10 * D];    // a whole tile's codes and pairs
  grid_dep_wait();
  TileRows w;
  if (!tile_rows<D>(a, w)) return;
  const int lane = threadIdx.x & 31, t = lane % G, y = lane % kLanes / G, sub = lane / kLanes;
  const T* src = static_cast<const T*>(w.value ? a.V : a.K) + w.row0 * D + 32 * y + 8 * t;
  uint8_t* stage = stage_s[threadIdx.x >> 5];
  const bool whole = w.r0 == 0 && w.r1 == kTile;
  uint8_t* codes = w.tile + (w.value ? L::kV : 0);
  uint8_t* pairs = w.tile + (w.value ? L::kVPairs : L::kKPairs);
  uint8_t* c_at = whole ? stage : codes;
  uint8_t* p_at = whole ? stage + 8 * D : pairs;
  const int first = w.r0 / kRows * kRows;
  Eight<T> raw[kEights];                          // of the pass ahead
  auto load = [&](int r) {
    if (r >= w.r0 && r < w.r1) {
#pragma unroll
      for (int k = 0; k < kEights; ++k) raw[k].load(src + (int64_t)r * D + 8 * G * k);
    }
  };
  load(first + sub);
  // (not unrolled: its passes would not stay in the instruction cache)
#pragma unroll 1
  for (int r = first + sub; r - sub < w.r1; r += kRows) {
    float v[kEights][8], mn, mx;
#pragma unroll
    for (int k = 0; k < kEights; ++k) {
      float mn1, mx1;
      raw[k].get(v[k]);
      raw[k].range(v[k], mn1, mx1);
      mn = k == 0 ? mn1 : min_nan(mn, mn1);
      mx = k == 0 ? mx1 : max_nan(mx, mx1);
    }
    load(r + kRows);
    if (G == 2) {
      mn = min_nan(mn, __shfl_xor_sync(FULL, mn, 1));
      mx = max_nan(mx, __shfl_xor_sync(FULL, mx, 1));
    }
    if (r < w.r0 || r >= w.r1) continue;
    const uint32_t pair = make_pair(mn, mx);
    const float lo = pair_lo(pair), step = pair_step(pair);
    const float inv = step > 0.f ? reciprocal(step) : 0.f;
    const bool rare = !(step > 0x1p-100f && step < 0x1p100f) && step != 0.f;
    const uint32_t keep = step > 0.f ? 0xffffffffu : 0u;
#pragma unroll
    for (int k = 0; k < kEights; ++k) {
      const uint32_t w8 = codes_of(v[k], lo, step, inv, rare) & keep;
      if (!w.value) {
        *reinterpret_cast<uint32_t*>(c_at + L::k_code(r, y, 8 * (t + G * k))) = w8;
      } else {
        uint16_t* out = reinterpret_cast<uint16_t*>(c_at + L::v_code(r, y, 8 * (t + G * k)) - L::kV);
        out[0] = (uint16_t)w8;
        out[32] = (uint16_t)(w8 >> 16);           // the next four values: 64 bytes on
      }
    }
    if (t == 0) *reinterpret_cast<uint32_t*>(p_at + L::pair(r, y)) = pair;
  }
  if (whole) {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
      reinterpret_cast<uint4*>(codes)[32 * k + lane] = reinterpret_cast<const uint4*>(stage)[32 * k + lane];
    if (lane < D / 8)
      reinterpret_cast<uint4*>(pairs)[lane] = reinterpret_cast<const uint4*>(stage + 8 * D)[lane];
  }
}

__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
// the values of the codes in bits 16 half .. 16 half + 15 of w
__device__ __forceinline__ void four_values(uint32_t w, int half, uint32_t pair, float (&v)[4]) {
  const float lo = pair_lo(pair), step = pair_step(pair);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t c = (w >> (16 * half + 4 * e)) & 15u;
    v[e] = fmaf(step, __uint_as_float(c | 0x4b000000u) - 8388608.f, lo);
  }
}

template <int N> struct Words { uint32_t w[N]; };
template <int N>
__device__ __forceinline__ Words<N> load_words(const uint8_t* p) {
  Words<N> r;
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r.w[0] = v.x, r.w[1] = v.y, r.w[2] = v.z, r.w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  }
  return r;
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) q4_read_kernel(const __grid_constant__ Q4RowsArgs a) {
  using L = Layout<D>;
  constexpr int Y = L::kGroups;
  grid_dep_wait();
  TileRows w;
  if (!tile_rows<D>(a, w)) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  T* dst = static_cast<T*>(const_cast<void*>(w.value ? a.V : a.K)) + w.row0 * D;
  auto in = [&](int r) { return r >= w.r0 && r < w.r1; };
  if (!w.value) {
    // lane (g, t): values 8 t .. 8 t + 7 of every group of positions g, g + 8
    Words<Y> c[2], p[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      c[k] = load_words<Y>(w.tile + L::k_code(g + 8 * k, 0, 8 * t));
      p[k] = load_words<Y>(w.tile + L::kKPairs + L::pair(g + 8 * k, 0));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int y = 0; y < Y; ++y) {
        float v[2][4];
        four_values(c[k].w[y], 0, p[k].w[y], v[0]);
        four_values(c[k].w[y], 1, p[k].w[y], v[1]);
        if (!in(g + 8 * k)) continue;
        T* out = dst + (int64_t)(g + 8 * k) * D + 32 * y + 8 * t;
        if constexpr (sizeof(T) == 2) {
          uint32_t b[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v[e >> 1][2 * (e & 1)], v[e >> 1][2 * (e & 1) + 1]);
            b[e] = *reinterpret_cast<const uint32_t*>(&x);
          }
          *reinterpret_cast<uint4*>(out) = make_uint4(b[0], b[1], b[2], b[3]);
        } else {
          store4(out, v[0]);
          store4(out + 4, v[1]);
        }
      }
  } else {
    // lane (g, t): values 4 g .. 4 g + 3 of every group of positions 2 t,
    // 2 t + 1, 2 t + 8, 2 t + 9
    uint4 c[Y / 2];
#pragma unroll
    for (int k = 0; k < Y / 2; ++k) c[k] = *reinterpret_cast<const uint4*>(w.tile + L::kV + 512 * k + 16 * lane);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 2 * t + (k & 1) + 8 * (k >> 1);
      const Words<Y> p = load_words<Y>(w.tile + L::kVPairs + L::pair(r, 0));
#pragma unroll
      for (int y = 0; y < Y; ++y) {
        const uint4& q = c[y >> 1];
        const uint32_t word = (y & 1) ? ((k >> 1) ? q.w : q.z) : ((k >> 1) ? q.y : q.x);
        float v[4];
        four_values(word, k & 1, p.w[y], v);
        if (in(r)) store4(dst + (int64_t)r * D + 32 * y + 4 * g, v);
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_rows(const Q4RowsArgs& a, bool write, cudaStream_t st) {
  const int64_t warps = 2 * (int64_t)a.c.B * a.c.H * tiles_of(a.m);
  const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps);
  // writing: one lane a group where there are warps enough to be bound by
  // instructions (8 x 4096 rows, written and read back: 65.7 -> 63.4 us; the
  // 333 rows of 5 fp32 sequences: 4.8 -> 5.6)
  const bool many = warps >= 32 * (int64_t)a.num_sms;
  return launch_dependent(!write ? q4_read_kernel<T, D> : many ? q4_write_kernel<T, D, 1> : q4_write_kernel<T, D, 2>,
                          dim3(grid), 32 * kWarps, 0, st, a);
}

cudaError_t launch_any(const Q4RowsArgs& a, bool write, cudaStream_t st) {
  if (a.dtype == PLSH_BF16)
    return a.c.d == 64 ? launch_rows<__nv_bfloat16, 64>(a, write, st)
                       : launch_rows<__nv_bfloat16, 128>(a, write, st);
  return a.c.d == 64 ? launch_rows<float, 64>(a, write, st) : launch_rows<float, 128>(a, write, st);
}

}  // namespace

cudaError_t launch_q4_write(const Q4RowsArgs& a, cudaStream_t st) { return launch_any(a, true, st); }
cudaError_t launch_q4_read(const Q4RowsArgs& a, cudaStream_t st) { return launch_any(a, false, st); }

}  // namespace plsh
