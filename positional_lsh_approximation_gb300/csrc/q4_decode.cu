// One decode step over the 4-bit paged cache, approximate and exact ALiBi.
//
// Per sequence b and query head h, with pos = pos[b] and the cached values
// k_j, v_j (value = lo + step c of each group of 32):
//   o = sum_j w_j e^{x_j} v_j / sum_j w_j e^{x_j},  x_j = q . k_j / sqrt(d),
//   approximate:  w_j = c_j = #{t : lo_t(pos) <= j},  j <= pos
//   exact:        w_j = e^{-(pos - j) / sigma_h},     j <= pos
// (Positional LSH, technical summary, Methodology 1 and 3, for one row.)
// A CTA per (sequence, query head): a key per thread for the scores of 128
// keys at a time, a running maximum and sum, then a value per thread for P V.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bins_dev.cuh"
#include "plsh_internal.h"
#include "q4.cuh"

namespace plsh {
namespace {

using namespace q4;

constexpr int kThreads = 128;
constexpr float kLog2e = 1.4426950408889634f;

struct DecodeParams {
  Q4Cache c;
  const void* q;
  void* o;
  const int32_t* pos;
  int Hq;
  const BinRecord* rec;
  int s;
  int64_t W, bins_n;
  int* err;
  float slope[kMaxExactHeads];
};

template <typename T, int D, bool EXACT>
__global__ void __launch_bounds__(kThreads) q4_decode_kernel(const __grid_constant__ DecodeParams p) {
  using L = Layout<D>;
  __shared__ float qs[D], w_s[kThreads], red[4];
  __shared__ int lo_s[kMaxS];
  __shared__ const uint8_t* tile_s[kThreads / kTile];
  const int b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  T* o = static_cast<T*>(p.o) + (int64_t)blockIdx.x * D;
  const int pos = p.pos[b];
  const bool over = pos >= (p.c.max_pages << p.c.page_shift) || (!EXACT && pos >= p.bins_n);
  if (pos < 0 || over) {
    if (over && tid == 0) atomicOr(p.err, kErrCachePlace);
    if (tid < D) o[tid] = Elem<T>::put(0.f);
    return;
  }
  int first = 0;
  if (!EXACT) {
    if (tid < p.s)
      lo_s[tid] = bin_lo(load_record(p.rec, ((int64_t)h * p.s + tid) * p.W + (pos >> 5)), pos);
    __syncthreads();
    first = pos;
    for (int t = 0; t < p.s; ++t) first = min(first, lo_s[t]);
  }
  const float scale = kLog2e / sqrtf((float)D);
  if (tid < D) qs[tid] = Elem<T>::get(static_cast<const T*>(p.q)[(int64_t)blockIdx.x * D + tid]) * scale;
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int j0 = first & ~15; j0 <= pos; j0 += kThreads) {
    __syncthreads();
    if (tid < kThreads / kTile)
      tile_s[tid] = j0 + tid * kTile <= pos ? tile_of<D>(p.c, b, h / (p.Hq / p.c.H), j0 + tid * kTile, p.err)
                                            : nullptr;
    __syncthreads();
    const int j = j0 + tid, r = tid & 15;
    const uint8_t* tile = tile_s[tid >> 4];
    int c = j >= first && j <= pos && tile != nullptr;
    if (!EXACT && c) {
      c = 0;
      for (int t = 0; t < p.s; ++t) c += lo_s[t] <= j;
    }
    float x = -INFINITY;
    if (c > 0) {
      x = 0.f;
      for (int y = 0; y < L::kGroups; ++y) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + L::kKPairs + L::pair(r, y));
        float dot = 0.f, sum = 0.f;
        for (int i = 0; i < kGroup; i += 2) {
          const uint32_t k = tile[L::k_code(r, y, i)];
          const float q0 = qs[y * kGroup + i], q1 = qs[y * kGroup + i + 1];
          dot = fmaf(q0, (float)(k & 15u), fmaf(q1, (float)(k >> 4), dot));
          sum += q0 + q1;
        }
        x = fmaf(pair_step(w), dot, fmaf(pair_lo(w), sum, x));
      }
      if (EXACT) x = fmaf(-(float)(pos - j), p.slope[h], x);
    }
    float mx = x;
    for (int e = 16; e > 0; e >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, e));
    if (lane == 0) red[warp] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    // every score NaN leaves the maximum at -inf: the weights come out NaN
    const float ref = mx == -INFINITY ? 0.f : mx;
    w_s[tid] = c > 0 ? (float)c * exp2f(x - ref) : 0.f;
    __syncthreads();
    const float f = m == -INFINITY ? 1.f : exp2f(m - ref);
    l *= f;
    acc *= f;
    m = mx;
    const int y = tid / kGroup, i = tid & 31;
    for (int k = 0; k < kThreads && j0 + k <= pos; ++k) {
      const float w = w_s[k];
      if (w == 0.f) continue;
      l += w;
      if (tid < D) {
        const uint8_t* tl = tile_s[k >> 4];
        const uint32_t pr = *reinterpret_cast<const uint32_t*>(tl + L::kVPairs + L::pair(k & 15, y));
        const uint32_t v = tl[L::v_code(k & 15, y, i & ~1)] >> (4 * (i & 1));
        acc = fmaf(w, fmaf(pair_step(pr), (float)(v & 15u), pair_lo(pr)), acc);
      }
    }
  }
  if (tid < D) o[tid] = Elem<T>::put(l == 0.f ? 0.f : acc / l);
}

template <typename T, int D>
cudaError_t launch_typed(const DecodeParams& p, bool exact, cudaStream_t st) {
  const unsigned grid = (unsigned)(p.c.B * p.Hq);
  if (exact)
    q4_decode_kernel<T, D, true><<<grid, kThreads, 0, st>>>(p);
  else
    q4_decode_kernel<T, D, false><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

int64_t q4_decode_work_bytes(int, int, int, int, int) { return 16; }

cudaError_t launch_q4_decode(const Q4DecodeArgs& a, cudaStream_t st) {
  DecodeParams p;
  p.c = a.c;
  p.q = a.q;
  p.o = a.o;
  p.pos = a.pos;
  p.Hq = a.Hq;
  p.rec = a.rec;
  p.s = a.s;
  p.W = a.W;
  p.bins_n = a.bins_n;
  p.err = a.err;
  for (int h = 0; h < kMaxExactHeads; ++h) p.slope[h] = a.slope_log2 && h < a.Hq ? a.slope_log2[h] : 0.f;
  const bool exact = a.rec == nullptr;
  if (a.dtype == PLSH_BF16)
    return a.c.d == 64 ? launch_typed<__nv_bfloat16, 64>(p, exact, st)
                       : launch_typed<__nv_bfloat16, 128>(p, exact, st);
  return a.c.d == 64 ? launch_typed<float, 64>(p, exact, st) : launch_typed<float, 128>(p, exact, st);
}

}  // namespace plsh
