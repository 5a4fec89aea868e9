// Writing rows of K and V into the 4-bit paged cache, and reading them back.
//
// A group of 32 values x is held as codes c and a pair (lo, step):
//   lo = min x (down to bf16), step = (max x - lo) / 15 (up to bf16),
//   c = rint((x - lo) / step) in 0..15,   value = lo + step c.
// A thread per group.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "plsh_internal.h"
#include "q4.cuh"

namespace plsh {
namespace {

using namespace q4;

constexpr int kThreads = 128;

struct RowGroup {
  uint8_t* tile;
  int64_t at;      // first value of the group in K / V
  int r, y;
};

template <int D>
__device__ bool row_group(const Q4RowsArgs& a, RowGroup& g) {
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = id / Layout<D>::kGroups;
  if (row >= (int64_t)a.c.B * a.c.H * a.m) return false;
  const int64_t i = row % a.m;
  const int b = (int)(row / a.m / a.c.H), h = (int)(row / a.m % a.c.H);
  if (a.len != nullptr && i >= a.len[b]) return false;
  const int64_t p = (int64_t)a.pos[b] + i;
  g.y = (int)(id % Layout<D>::kGroups);
  g.at = row * D + g.y * kGroup;
  g.r = (int)(p & 15);
  g.tile = tile_of<D>(a.c, b, h, p, a.err);
  return g.tile != nullptr;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) q4_write_kernel(Q4RowsArgs a) {
  using L = Layout<D>;
  RowGroup g;
  if (!row_group<D>(a, g)) return;
  for (int which = 0; which < 2; ++which) {
    const T* x = static_cast<const T*>(which ? a.V : a.K) + g.at;
    float v[kGroup];
    float mn = INFINITY, mx = -INFINITY;
    bool nan = false;
    for (int i = 0; i < kGroup; ++i) {
      v[i] = Elem<T>::get(x[i]);
      nan |= v[i] != v[i];
      mn = fminf(mn, v[i]);
      mx = fmaxf(mx, v[i]);
    }
    const uint32_t w = make_pair(nan ? NAN : mn, mx);
    const float lo = pair_lo(w), step = pair_step(w);
    *reinterpret_cast<uint32_t*>(g.tile + (which ? L::kVPairs : L::kKPairs) + L::pair(g.r, g.y)) = w;
    for (int i = 0; i < kGroup; i += 2) {
      uint32_t c[2];
      for (int e = 0; e < 2; ++e)
        c[e] = step > 0.f ? (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(v[i + e] - lo, step)), 0.f), 15.f) : 0u;
      g.tile[which ? L::v_code(g.r, g.y, i) : L::k_code(g.r, g.y, i)] = (uint8_t)(c[0] | (c[1] << 4));
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(Q4RowsArgs a) {
  using L = Layout<D>;
  RowGroup g;
  if (!row_group<D>(a, g)) return;
  for (int which = 0; which < 2; ++which) {
    T* x = static_cast<T*>(const_cast<void*>(which ? a.V : a.K)) + g.at;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(
        g.tile + (which ? L::kVPairs : L::kKPairs) + L::pair(g.r, g.y));
    const float lo = pair_lo(w), step = pair_step(w);
    for (int i = 0; i < kGroup; i += 2) {
      const uint32_t c = g.tile[which ? L::v_code(g.r, g.y, i) : L::k_code(g.r, g.y, i)];
      x[i] = Elem<T>::put(fmaf(step, (float)(c & 15u), lo));
      x[i + 1] = Elem<T>::put(fmaf(step, (float)(c >> 4), lo));
    }
  }
}

template <typename T, int D>
cudaError_t launch_rows(const Q4RowsArgs& a, bool write, cudaStream_t st) {
  const int64_t groups = (int64_t)a.c.B * a.c.H * a.m * Layout<D>::kGroups;
  const unsigned grid = (unsigned)((groups + kThreads - 1) / kThreads);
  if (write)
    q4_write_kernel<T, D><<<grid, kThreads, 0, st>>>(a);
  else
    q4_read_kernel<T, D><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
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
