// Page tables of the 4-bit paged cache, kept on the GPU from the lengths that
// requests ask for, and the slots that their new rows go to.
//
// Sequence b asks for need[b] positions and holds held[b] pages, the first S of
// every row that holds anything being a shared prefix's.  It wants
//   w = 0 where need <= 0, else max(ceil(need / page), S),
// of which max(w - S, 0) come from the stack of free pages.  First the pages held
// beyond w are pushed, from the last sequence's last page to the first one's
// first; then, from the first sequence on, the missing ones are popped, first
// entry first, while they fit.  With back_b and take_b the pages that b gives
// and takes, F = sum back, and c the free pages before:
//   page i of b goes to place  c + sum_{b' > b} back_b' + (held_b - 1 - i),
//   entry i of b comes from    c + F - 1 - sum_{b' < b} take_b' - (i - first_b),
//   b is granted iff           sum_{b' <= b} take_b' <= c + F,
// two prefix sums over the sequences (64 bits: a request may be any number), so
// that no step waits for the one before it.  Growing and then releasing leaves
// the stack as it was.
//
// Bound by latency: what changes hands is a few bytes a sequence.  One cluster of
// 1 to 8 CTAs, so that one launch does it all: every CTA makes the prefix sums for
// itself, the cluster's warps move the pages of a sequence each, and the cluster's
// barrier stands between what is read and what is written over it.  Measured with the
// slots of the new rows (requests taken back, made again, slots: three launches): 64
// sequences growing by a token 8.8 us, 256 of which a quarter finish and a quarter
// bring prompts of up to 2048 tokens 19.6 (4 MB of slots).  There each trip of the loops
// that move a request's pages waits for the one before, as table and pool might be one
// memory: 15 trips for a request of 460 pages.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "plsh_internal.h"
#include "q4.cuh"
#include "tc_ptx.cuh"

namespace plsh {
namespace {

using namespace q4;
using namespace ptx;

constexpr int kThreads = 1024, kWarps = kThreads / 32, kMaxCluster = 8;
constexpr unsigned FULL = 0xffffffffu;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// Inclusive sums over the CTA's threads, and the total; all threads call it.
__device__ __forceinline__ int64_t block_sums(int64_t v, int64_t* scratch, int64_t& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(FULL, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();                      // the scratch of the call before has been read
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  int64_t all = scratch[lane], upto = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(FULL, upto, o);
    if (lane >= o) upto += u;
  }
  total = __shfl_sync(FULL, upto, 31);
  const int64_t before = __shfl_sync(FULL, upto - all, warp);
  return v + before;
}
static_assert(kWarps == 32, "a warp sums the warps' sums");

// What a sequence does, held for the warp that moves its pages.
struct Move {
  int held, want;        // want as granted
  int64_t place;         // of its last page given back, or of its first one taken
};

__global__ void __launch_bounds__(kThreads) q4_reserve_kernel(const __grid_constant__ Q4ReserveArgs a) {
  __shared__ int64_t scratch[kWarps];
  __shared__ Move moves[kThreads];
  grid_dep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), size = (int)cluster_size();
  const int S = a.prefix_pages, batches = (a.c.B + kThreads - 1) / kThreads;
  int32_t* table = const_cast<int32_t*>(a.c.table);
  int64_t count = a.pool[0];
  bool bad = count < 0 || count > a.pool_pages;
  count = max((int64_t)0, min(count, a.pool_pages));
  auto mine = [&](int64_t x) { return max((int64_t)0, x - S); };
  // a sequence's pages, held and wanted (it asks for more than its row has
  // entries, or holds more: it wants what it has)
  auto ask = [&](int b, int& h, int& w) {
    h = w = 0;
    if (b >= a.c.B) return;
    const int64_t need = a.need[b];
    h = a.held[b];
    const int64_t want = need <= 0 ? 0 : max((need + (1 << a.c.page_shift) - 1) >> a.c.page_shift, (int64_t)S);
    const bool wrong = h < 0 || h > a.c.max_pages || want > a.c.max_pages;
    bad = bad || wrong;
    h = max(0, (int)min((int64_t)h, a.c.max_pages));
    w = wrong ? h : (int)want;
  };
  int h = 0, w = 0;
  int64_t given = 0, total = 0;
  for (int k = 0; k < batches; ++k) {
    ask(k * kThreads + tid, h, w);
    int64_t t;
    block_sums(max((int64_t)0, mine(h) - mine(w)), scratch, t);
    given += t;
  }
  // ---- pages given back
  int64_t behind = given;               // by the sequences from this batch on
  for (int k = 0; k < batches && given > 0; ++k) {
    if (batches > 1) ask(k * kThreads + tid, h, w);
    const int64_t back = max((int64_t)0, mine(h) - mine(w));
    const int64_t upto = block_sums(back, scratch, total);
    moves[tid] = Move{h, w, count + behind - upto};
    behind -= total;
    __syncthreads();
    for (int s = rank * kWarps + warp; s < kThreads && k * kThreads + s < a.c.B; s += size * kWarps) {
      const Move m = moves[s];
      const int32_t* row = table + (int64_t)(k * kThreads + s) * a.c.max_pages;
      for (int i = max(m.want, S) + lane; i < m.held; i += 32) {
        const int64_t to = m.place + (m.held - 1 - i);
        if (to < a.pool_pages)
          a.pool[1 + to] = row[i];
        else
          bad = true;
      }
    }
    __syncthreads();
  }
  // (pops read what any CTA pushed; entries are cleared behind the pushes)
  cluster_sync();
  const int64_t free_pages = min(count + given, a.pool_pages);
  // ---- pages taken
  int64_t before = 0, taken = 0;
  for (int k = 0; k < batches; ++k) {
    const int b = k * kThreads + tid;
    if (batches > 1) ask(b, h, w);
    const int64_t take = w > h ? mine(w) - mine(h) : 0;
    const int64_t upto = before + block_sums(take, scratch, total);
    const bool granted = upto <= free_pages;
    const int now = w > h && !granted ? h : w;
    moves[tid] = Move{h, now, free_pages - 1 - (upto - take)};
    // granted ones come first: the last of them has taken all that are taken
    int64_t t = granted ? upto : 0;
    before += total;
    __syncthreads();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(FULL, t, o));
    if (lane == 0) scratch[warp] = t;
    __syncthreads();
    t = scratch[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(FULL, t, o));
    taken = max(taken, t);
    // every CTA has read this batch's held, and pool[0]
    if (size > 1) cluster_sync();
    if (rank == 0 && b < a.c.B && now != h) a.held[b] = now;
    for (int s = rank * kWarps + warp; s < kThreads && k * kThreads + s < a.c.B; s += size * kWarps) {
      const Move m = moves[s];
      int32_t* row = table + (int64_t)(k * kThreads + s) * a.c.max_pages;
      for (int i = m.want + lane; i < m.held; i += 32) row[i] = -1;
      if (m.want > m.held) {
        for (int i = m.held + lane; i < min(S, m.want); i += 32) row[i] = a.prefix[i];
        const int first = max(m.held, S);
        for (int i = first + lane; i < m.want; i += 32) row[i] = a.pool[1 + m.place - (i - first)];
      }
    }
    __syncthreads();
  }
  if (rank == 0 && tid == 0) a.pool[0] = (int32_t)(free_pages - taken);
  if (__any_sync(FULL, bad) && lane == 0) atomicOr(a.err, kErrCachePlace);
}

// Slots of rows: position p of sequence b is row p % page of page table[b, p / page].
// Two rows a thread, so that a store is 16 bytes wide.
__global__ void __launch_bounds__(256) q4_slots_kernel(const __grid_constant__ Q4SlotsArgs a) {
  grid_dep_wait();
  // (fewer than 2^31 rows in a call)
  const uint32_t at = 2 * (blockIdx.x * 256u + threadIdx.x), all = (uint32_t)a.c.B * (uint32_t)a.m;
  if (at >= all) return;
  int64_t slot[2] = {-1, -1};
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (at + k >= all) break;
    const uint32_t b = (at + k) / (uint32_t)a.m;
    const int64_t i = at + k - b * (uint32_t)a.m, p = (int64_t)a.pos[b] + i;
    if (i >= (a.len == nullptr ? a.m : (int64_t)a.len[b])) continue;
    if (p < 0 || p >= (a.c.max_pages << a.c.page_shift)) {
      bad = bad || p >= 0;
      continue;
    }
    const int64_t pg = a.c.table[(int64_t)b * a.c.max_pages + (p >> a.c.page_shift)];
    if (pg >= 0 && pg < a.c.pages) slot[k] = (pg << a.c.page_shift) + (p & ((1 << a.c.page_shift) - 1));
  }
  if (bad) atomicOr(a.err, kErrCachePlace);
  if (at + 1 < all)
    *reinterpret_cast<longlong2*>(a.slots + at) = make_longlong2(slot[0], slot[1]);
  else
    a.slots[at] = slot[0];
}

}  // namespace

cudaError_t launch_q4_reserve(const Q4ReserveArgs& a, cudaStream_t st) {
  // a CTA's 32 warps take a sequence each at a time; more CTAs where rows are
  // many and long enough to pay for the cluster's barriers (two calls and the slots in a
  // graph: 256 rows of 512, a quarter coming and going: 8 CTAs 24.6 us, 4 26.7, 2 30.7,
  // 1 34.9; 64 rows of 128 growing by a token: 1 CTA 10.3, 2 to 8 12.3)
  const int64_t pages = (int64_t)a.c.B * a.c.max_pages;
  unsigned cluster = 1;
  while (cluster < kMaxCluster && pages > (int64_t)cluster * 8192 && a.c.B > (int)cluster * kWarps) cluster *= 2;
  return launch_clusters(cluster, q4_reserve_kernel, dim3(cluster), kThreads, 0, st, a);
}

cudaError_t launch_q4_slots(const Q4SlotsArgs& a, cudaStream_t st) {
  const int64_t grid = ((int64_t)a.c.B * a.m + 511) / 512;
  return launch_dependent(q4_slots_kernel, dim3((unsigned)grid), 256, 0, st, a);
}

}  // namespace plsh
