// Layout of the 4-bit paged K/V cache (the format stands in plsh.h).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "plsh_internal.h"
#include "tc_ptx.cuh"

namespace plsh {
namespace q4 {

constexpr int kTile = 16;     // positions of a tile
constexpr int kGroup = 32;    // values that share (lo, step)

template <int D>
struct Layout {
  static constexpr int kGroups = D / kGroup;         // groups of a row
  static constexpr int kV = 8 * D;                   // offset of V's codes in a tile
  static constexpr int kKPairs = 16 * D;             // of K's pairs
  static constexpr int kVPairs = 18 * D;             // of V's pairs
  static constexpr int kTileBytes = 20 * D;
  // byte of the code of value i (even) of group y of position r
  __host__ __device__ static constexpr int k_code(int r, int y, int i) {
    return r * (D / 2) + (i >> 3) * (D / 8) + 4 * y + ((i & 7) >> 1);
  }
  __host__ __device__ static constexpr int v_code(int r, int y, int i) {
    return kV + (y >> 1) * 512 + (4 * (i >> 2) + ((r & 7) >> 1)) * 16 + (y & 1) * 8 +
           4 * (r >> 3) + 2 * (r & 1) + ((i & 3) >> 1);
  }
  __host__ __device__ static constexpr int pair(int r, int y) { return (r * kGroups + y) * 4; }
};

// Tile of position p of sequence b (head h), or null when p or its page index
// is out of range, which raises kErrCachePlace.
template <int D>
__device__ __forceinline__ uint8_t* tile_of(const Q4Cache& c, int b, int h, int64_t p, int* err) {
  if (p >= 0 && p < (c.max_pages << c.page_shift)) {
    const int64_t pg = c.table[(int64_t)b * c.max_pages + (p >> c.page_shift)];
    if (pg >= 0 && pg < c.pages) {
      const int in_page = (int)(p & ((1 << c.page_shift) - 1));
      return c.data + (((pg * c.H + h) << (c.page_shift - 4)) + (in_page >> 4)) *
                          (int64_t)Layout<D>::kTileBytes;
    }
  }
  atomicOr(err, kErrCachePlace);
  return nullptr;
}

// A group's pair as stored: lo in the low half, step in the high half.
__device__ __forceinline__ float pair_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float pair_step(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The pair of a group with smallest and largest values mn and mx (either is
// NaN if one of the values is).  spread / 15 is correctly rounded: from
// q = spread y with y = 1 / 15 rounded, the remainder r = spread - 15 q is exact
// and q + r y rounds to the quotient (Markstein's theorem on division by a
// number whose reciprocal is known correctly rounded; checked over every
// significand).  Spreads near the ends of fp32's range take the division.
__device__ __forceinline__ uint32_t make_pair(float mn, float mx) {
  // mn rounded down, the quotient rounded up, to the upper 16 bits
  const uint32_t m = __float_as_uint(mn);
  const uint32_t lo = (m & 0xffff0000u) + ((m & 0xffffu) && (m >> 31) ? 0x10000u : 0u);
  const float spread = mx - __uint_as_float(lo);
  constexpr float y = 1.f / 15.f;
  float q = spread * y;
  q = fmaf(fmaf(-15.f, q, spread), y, q);
  if (!(spread >= 0x1p-100f && spread <= 3.402823466e38f)) {      // a constant group among them
    if (!(mn == mn && spread <= 3.402823466e38f)) return 0x7fc00000u;       // lo 0, step NaN
    q = __fdiv_rn(spread, 15.f);
  }
  return (lo >> 16) | ((__float_as_uint(q) + 0xffffu) & 0xffff0000u);
}

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  __device__ static float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  __device__ static __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <> struct Elem<float> {
  __device__ static float get(float v) { return v; }
  __device__ static float put(float v) { return v; }
};

// Launches a kernel as a programmatic dependent of the one before it on the
// stream: its launch overlaps that one's tail, and it waits for its end
// (grid_dep_wait) before any access.  `cluster` CTAs form a cluster.
template <typename... P, typename... A>
cudaError_t launch_clusters(unsigned cluster, void (*kern)(P...), dim3 grid, int threads, size_t smem,
                            cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, size_t smem,
                             cudaStream_t st, const A&... args) {
  return launch_clusters(1, kern, grid, threads, smem, st, args...);
}

}  // namespace q4
}  // namespace plsh
