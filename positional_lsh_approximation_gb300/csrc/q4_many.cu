// Exact ALiBi attention of many query rows over the 4-bit paged cache: a chunk of
// new tokens of every sequence (row i at position p = pos[b] + i), and the part of
// a decode step that lies in a prefix which all sequences share (one row a
// sequence, p = pos[b], keys below the prefix's end):
//   o = sum_j e^{q.k_j / sqrt(d) - (p - j) / sigma_h} v_j / sum_j (the weights), j <= p.
//
// The rows of all query heads of a KV head see the same keys, so an item is 256
// such rows (two tiles of 128) and the keys up to the last of their positions, in
// steps of 128.  A step's codes (20 d bytes for 16 positions) are taken apart once
// for the 256 rows, into f16 tiles in shared memory, and the products run on the
// tensor cores (tcgen05): S = Q K^T from shared memory, P V with P in tensor
// memory.  Next to the products' 2048 cycles a step (at 4096 multiply-adds a cycle)
// stand about 1900 issue slots a scheduler of softmax and of taking codes apart.
//
// Numbers.  Codes are exact in f16, so a value lo + step c is rounded once, in one
// f16 multiply-add: a code in the low bits of an f16 is the subnormal c 2^-24 (or
// 16 c 2^-24, or 2^6 c 2^-24 behind a shift), and the power of two goes into step.
// Powers of two keep everything within f16's range:
//   q  times one per tile of 128 rows, the largest magnitude in [2^14, 2^15);
//   K  times one per position, largest below 2^-6: undone in the fp32 scores
//      (cs_j, times q's and log2(e) / sqrt(d));
//   V  times one per group of 32 values, R_y, by the first step of a piece, and one
//      per step, ev, by how far any group exceeds that: largest below 1.  2^ev goes
//      into the step's weights, P = 2^{x + ev - M} with M the running maximum of
//      x + ev, so that a large value takes precision from others of its own step
//      alone; the row sum takes P 2^-ev in fp32.
// P and V are rounded to f16 (2^-11 of themselves): bf16's 2^-8 would show beside
// the output's own rounding.  Scores, sums and maxima are fp32.
//
// Warps of a CTA (one per SM): 0-3 and 4-7 softmax of the two tiles, a thread a
// row; 8-11 take codes apart; 12 issues the products, PV_A(g-1) S_A(g) PV_B(g-1)
// S_B(g), so that the tensor cores work on one tile while the other's scores become
// weights; 13 lists the items and copies the codes.  The flat list (KV head, item,
// step), each item preceded by kItemCost entries for its beginning and end, is cut
// into equal shares of the CTAs; items cut by a CTA's edge are joined by a second
// kernel, in a fixed order.  Every wait is bounded; on expiry the CTA raises the
// error flag, lets its copies and products drain, frees its tensor memory and exits.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "plsh_internal.h"
#include "q4.cuh"
#include "tc_ptx.cuh"

namespace plsh {
namespace {

using namespace q4;
using namespace ptx;

constexpr int BM = 128, BN = 128;       // rows of a tile, keys of a step
constexpr int kItemRows = 2 * BM;
constexpr int kDeqWarp = 8, kDeqWarps = 4, kMmaWarp = 12, kProdWarp = 13, kWarps = 14;
constexpr int kThreads = 32 * kWarps, kDeqThreads = 32 * kDeqWarps;
constexpr int kTiles = BN / kTile;      // tiles of 16 positions of a step
constexpr uint32_t kHalf = BM * 128;    // 128 rows of 64 f16 values, 128-byte swizzle
constexpr int kItemCost = 2;            // steps that beginning and ending an item costs
constexpr int kMinSteps = 4;            // steps of a CTA at least
constexpr uint32_t kTmemCols = 512;     // S_A | S_B | O_A | O_B; P over S
constexpr uint32_t kColP = 64, kColO = 256;
constexpr float kRescaleLog2 = 8.f;     // a maximum that grew by more moves the reference
constexpr float kGrowLog2 = 15.f;       // largest weight 2^15
constexpr float kNothing = -3.402823466e38f;
constexpr unsigned FULL = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kErrTimeout = 1, kErrRange = 2;

template <int D>
struct Sizes {
  static constexpr int Y = D / kGroup;
  static constexpr uint32_t kTileB = BM * D * 2;               // an f16 tile
  static constexpr uint32_t kRaw = kTiles * Layout<D>::kTileBytes;
  static constexpr int kRawStages = D == 128 ? 2 : 4;
  static constexpr uint32_t kQ = 0, kK = 2 * kTileB, kV = 4 * kTileB, kRawAt = 5 * kTileB,
                            kEnd = kRawAt + kRawStages * kRaw;
};

enum {
  B_IFULL = 0, B_IEMPTY = 2, B_RAWFULL = 4, B_RAWEMPTY = 8, B_KREADY = 12, B_KEMPTY = 14, B_VREADY = 16,
  B_VEMPTY, B_QFULL, B_SFULL = 20, B_PFULL = 22, B_ODONE = 24, B_DRAIN = 26, NUM_BARS
};

// Rows [row0, row1) of a sequence's (or the batch's) rows of one KV head against the
// key steps [k0, k1), of which positions up to `last` count.
struct Item {
  int valid, b, kvh, row0, row1, k0, k1, pos, last, slot;      // slot < 0: the whole item
};

template <int D>
struct Ctl {
  static constexpr int Y = Sizes<D>::Y;
  uint64_t bars[NUM_BARS];
  Item ring[2];
  alignas(16) uint2 kq[BN][Y];          // per position and group: step, lo as f16 pairs
  alignas(16) uint2 vq[Y][BN];
  alignas(16) float cs[2][2][BN];       // per step and tile: a position's factor of the scores
  uint32_t mask[2][4];                  // per step: positions that count
  uint32_t vnan[2][Y][4];               // positions whose group of V is no number
  int ev[2], any_nan[2];
  int vr[2][Y];                         // per item slot: V's exponents R_y + 1
  uint32_t vmax[kDeqWarps][Y];
  uint32_t qmax[2][4];
  float qs[2];
  int present[4];                       // per raw stage: tiles that were copied
  int64_t sums[kWarps], found[2];
  uint32_t tmem_base;
  int abort;
};

struct ManyParams {
  Q4Cache c;
  const void* q;
  void* o;
  const int32_t* pos;
  const int32_t* len;                   // chunk
  const int32_t* prefix;                // prefix: its pages
  int Hq, G, m;                         // chunk: m rows a sequence
  int tiles;                            // items of a sequence and KV head, at most
  int limit;                            // positions below this may be asked for
  int keys;                             // prefix: its positions
  int4* ends;                           // chunk: per CTA {item, first CTA, first piece} that ends in it
  float* part;                          // pieces: o [D / 4][256][4], maximum [256], sum [256]
  int* err;
  uint64_t wait_ns;
  float slope[kMaxExactHeads];          // log2(e) / sigma_h
};

template <int D>
__host__ __device__ constexpr int64_t part_floats() { return kItemRows * (D + 2); }

__device__ __forceinline__ float pow2(int e) { return e < -126 ? 0.f : __int_as_float((min(e, 127) + 127) << 23); }

// A barrier of `n` threads that tells all of them whether all say ok.
__device__ __forceinline__ bool barrier_and(int id, int n, bool ok) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((int)ok)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Bit e set when key jc + e is at or before position jc + eb.
__device__ __forceinline__ uint32_t upto_mask(int eb) {
  return eb < 0 ? 0u : eb >= 31 ? 0xffffffffu : (2u << eb) - 1u;
}

template <int N>
__device__ __forceinline__ Item read_item(const Item (&ring)[N], int slot) {
  const volatile int* v = reinterpret_cast<const volatile int*>(&ring[slot]);
  return Item{v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[8], v[9]};
}

// New tokens of sequence b that have a position (chunk).
__device__ __forceinline__ int tokens_of(const ManyParams& p, int b, int& pos) {
  pos = p.pos[b];
  const int n = p.len == nullptr ? p.m : max(0, min(p.len[b], p.m));
  return pos < 0 ? 0 : max(0, min(n, p.limit - pos));
}

// Item t of entry e = (sequence, t): its rows, steps and last position.
template <bool PREFIX>
__device__ __forceinline__ int item_steps(const ManyParams& p, int b, int t, int& pos, int& rows, int& last) {
  if constexpr (PREFIX) {
    pos = 0;
    rows = p.c.B * p.G;
    last = p.keys - 1;
  } else {
    rows = tokens_of(p, b, pos) * p.G;
    last = pos + (min(rows, kItemRows * (t + 1)) - 1) / p.G;
  }
  return kItemRows * t < rows ? (last >> 7) + 1 : 0;
}

// Offset (in elements) of row r of a KV head's rows in q and o, its query head and
// position.
template <bool PREFIX, int D>
__device__ __forceinline__ int64_t row_at(const ManyParams& p, int b, int kvh, int pos0, int r, int& h, int& pos) {
  const int i = r / p.G;                       // token of the sequence, or sequence
  h = kvh * p.G + (r - i * p.G);
  if constexpr (PREFIX) {
    pos = p.pos[i];
    if (pos >= p.limit) pos = -1;
    return ((int64_t)i * p.Hq + h) * D;
  }
  pos = pos0 + i;
  return (((int64_t)b * p.Hq + h) * p.m + i) * D;
}

// Value of the row that column x of O stands for: columns 8 c .. 8 c + 7 are values
// 4 g .. 4 g + 3 of groups y and y + 1, c = 4 y + g, in the order 0, 2, 1, 3.

template <int D, bool PREFIX>
__global__ void __launch_bounds__(kThreads, 1) q4_many_kernel(const __grid_constant__ ManyParams p) {
  extern __shared__ uint8_t smem_raw[];
  using S = Sizes<D>;
  constexpr int Y = S::Y;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t sbase = (raw_u32 + 1023u) & ~1023u;
  Ctl<D>* ctl = reinterpret_cast<Ctl<D>*>(smem_raw + (sbase - raw_u32) + S::kEnd);
  auto bar = [&](int k) { return smem_u32(&ctl->bars[k]); };
  volatile int* abort = &ctl->abort;
  const uint64_t lim = p.wait_ns;

  if (tid == 0) {
    for (int k = 0; k < 2; ++k) {
      mbar_init(bar(B_IFULL + k), 1);
      mbar_init(bar(B_IEMPTY + k), 8 + kDeqWarps + 1);
      mbar_init(bar(B_KREADY + k), kDeqWarps);
      mbar_init(bar(B_KEMPTY + k), 1);
      mbar_init(bar(B_QFULL + k), BM);
      mbar_init(bar(B_SFULL + k), 1);
      mbar_init(bar(B_PFULL + k), BM);
      mbar_init(bar(B_ODONE + k), 1);
    }
    for (int k = 0; k < 4; ++k) {
      mbar_init(bar(B_RAWFULL + k), 1);
      mbar_init(bar(B_RAWEMPTY + k), kDeqWarps);
    }
    mbar_init(bar(B_VREADY), kDeqWarps);
    mbar_init(bar(B_VEMPTY), 1);
    mbar_init(bar(B_DRAIN), 1);
    ctl->abort = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&ctl->tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();
  const uint32_t tmem = ctl->tmem_base;

  // ---- the CTA's share of the flat list
  const int entries = PREFIX ? p.tiles : p.c.B * p.tiles;       // of one KV head
  int64_t total = 0, begin, end, per;
  {
    auto cost = [&](int e) -> int {
      int pos, rows, last;
      const int b = e / p.tiles, n = item_steps<PREFIX>(p, b, e - b * p.tiles, pos, rows, last);
      return n == 0 ? 0 : n + kItemCost;
    };
    const int each = (entries + kThreads - 1) / kThreads;
    const int e0 = min(entries, tid * each), e1 = min(entries, e0 + each);
    int64_t mine = 0;
    for (int e = e0; e < e1; ++e) mine += cost(e);
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(FULL, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) ctl->sums[warp] = upto;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) upto += ctl->sums[w];
      total += ctl->sums[w];
    }
    const int64_t all = total * p.c.H, fair = (all + gridDim.x - 1) / gridDim.x;
    per = fair < kMinSteps + kItemCost ? kMinSteps + kItemCost : fair;
    begin = blockIdx.x * per;
    end = min(all, begin + per);
    if (begin < end) {
      const int64_t rel = begin % total;
      if (rel >= upto - mine && rel < upto) {
        int64_t at = upto - mine;
        int e = e0;
        for (;; ++e) {
          const int n = cost(e);
          if (rel < at + n) break;
          at += n;
        }
        ctl->found[0] = e;
        ctl->found[1] = at;
      }
    }
    if (!PREFIX && tid == 0) p.ends[blockIdx.x].x = -1;
    if constexpr (!PREFIX) {
      // rows without a position: idle sequences', and those past the limit
      for (int b = blockIdx.x; b < p.c.B; b += gridDim.x) {
        int pos;
        const int n = tokens_of(p, b, pos);
        const int rows = p.len == nullptr ? p.m : max(0, min(p.len[b], p.m));
        if (n == rows) continue;
        if (pos >= 0 && tid == 0) atomicOr(p.err, kErrCachePlace);
        const int vecs = (rows - n) * (D / 8);               // of a head
        for (int64_t x = tid; x < (int64_t)vecs * p.Hq; x += kThreads) {
          const int h = (int)(x / vecs), v = (int)(x - (int64_t)h * vecs);
          reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) +
                                   (((int64_t)b * p.Hq + h) * p.m + n) * D)[v] = make_uint4(0, 0, 0, 0);
        }
      }
    }
    __syncthreads();
  }

  if (warp == kProdWarp) {
    // ---------------------------------------------------- items, copies of codes
    bool ok = true;
    int seq = 0, g = 0, slot = 2 * blockIdx.x;
    int issued[4] = {0, 0, 0, 0};
    auto publish = [&](const Item& it) {
      const int s = seq & 1;
      ok = __all_sync(FULL, mbar_wait(bar(B_IEMPTY + s), ((uint32_t)(seq >> 1) & 1u) ^ 1u, abort, lim));
      if (ok && lane == 0) {
        volatile int* v = reinterpret_cast<volatile int*>(&ctl->ring[s]);
        v[0] = it.valid; v[1] = it.b; v[2] = it.kvh; v[3] = it.row0; v[4] = it.row1;
        v[5] = it.k0; v[6] = it.k1; v[7] = it.pos; v[8] = it.last; v[9] = it.slot;
        mbar_arrive(bar(B_IFULL + s));
      }
      __syncwarp();
      ++seq;
    };
    if (begin < end) {
      int e = (int)ctl->found[0], kvh = (int)(begin / total);
      int64_t base = (int64_t)kvh * total + ctl->found[1];
      for (int64_t f = begin; ok && f < end;) {
        const int b = e / p.tiles, t = e - b * p.tiles;
        int pos, rows, last;
        const int n = item_steps<PREFIX>(p, b, t, pos, rows, last);
        const int cost = n == 0 ? 0 : n + kItemCost;
        if (f >= base + cost) {
          base += cost;
          e = n == 0 ? (b + 1) * p.tiles : e + 1;
          if (e >= entries) {
            e = 0;
            ++kvh;
          }
          continue;
        }
        const int64_t till = min(end, base + cost);
        const int t0 = (int)max((int64_t)0, f - base - kItemCost), t1 = (int)(till - base - kItemCost);
        f = till;
        if (t1 <= t0) continue;
        const bool closes = till == base + cost, whole = !PREFIX && t0 == 0 && closes;
        if (!PREFIX && closes && !whole && lane == 0) {
          const int i0 = (int)((base + kItemCost) / per);          // the CTA of its first step
          p.ends[blockIdx.x] = make_int4(kvh * entries + e, i0, base <= i0 * per ? 2 * i0 : 2 * i0 + 1, 0);
        }
        publish(Item{1, b, kvh, kItemRows * t, min(rows, kItemRows * (t + 1)), t0, t1, pos, last,
                     whole ? -1 : slot});
        slot = 2 * blockIdx.x + 1;
        // a lane of the first eight a tile of 16 positions; the table entries of a
        // step are read while the step before waits for its room
        const int32_t* table = PREFIX ? p.prefix : p.c.table + (int64_t)b * p.c.max_pages;
        auto entry = [&](int s) -> int32_t {
          const int at = BN * s + kTile * lane;
          return lane < kTiles && s >= t0 && at <= last ? table[at >> p.c.page_shift] : -1;
        };
        int32_t next = entry(t1 - 1);
        for (int s = t1 - 1; ok && s >= t0; --s, ++g) {
          const int32_t pg = next;
          next = entry(s - 1);
          const int st = g % S::kRawStages;
          ok = __all_sync(FULL, mbar_wait(bar(B_RAWEMPTY + st), ((uint32_t)(g / S::kRawStages) & 1u) ^ 1u, abort, lim));
          if (!ok) break;
          const int at = BN * s + kTile * lane;
          const bool want = lane < kTiles && at <= last, here = want && pg >= 0 && pg < p.c.pages;
          if (want && !here) atomicOr(p.err, kErrCachePlace);
          const unsigned got = __ballot_sync(FULL, here);
          if (lane == 0) {
            *reinterpret_cast<volatile int*>(&ctl->present[st]) = (int)got;
            mbar_arrive_expect_tx(bar(B_RAWFULL + st), __popc(got) * Layout<D>::kTileBytes);
          }
          ++issued[st];
          __syncwarp();
          if (here) {
            const int in_page = at & ((1 << p.c.page_shift) - 1);
            const uint8_t* src = p.c.data + (((int64_t)pg * p.c.H + kvh) * (1 << (p.c.page_shift - 4)) + (in_page >> 4)) *
                                                (int64_t)Layout<D>::kTileBytes;
            bulk_load(sbase + S::kRawAt + st * S::kRaw + lane * Layout<D>::kTileBytes, src, Layout<D>::kTileBytes,
                      bar(B_RAWFULL + st));
          }
        }
      }
    }
    if (ok) publish(Item{});
    if (!ok && lane == 0) {
      *abort = 1;
      atomicOr(p.err, kErrTimeout);
    }
    // every copy this warp started lands before the CTA can exit
#pragma unroll
    for (int st = 0; st < S::kRawStages; ++st)
      if (issued[st]) mbar_wait(bar(B_RAWFULL + st), (uint32_t)(issued[st] - 1) & 1u, nullptr, lim);
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ the products
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_f16_f32(BM, BN, 0, 0), id_pv = idesc_f16_f32(BM, D, 0, 1);
      const uint64_t dq0 = desc_sw128(sbase + S::kQ, 16, 1024);
      const uint64_t dk0 = desc_sw128(sbase + S::kK, 16, 1024);
      const uint64_t dv0 = desc_sw128(sbase + S::kV, kHalf, 1024);
      auto issue_s = [&](int tile, int kb) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          mma_bf16_ss(tmem + tile * BN, desc_add(dq0, tile * (S::kTileB >> 4) + off),
                      desc_add(dk0, kb * (S::kTileB >> 4) + off), id_s, kk > 0 ? 1u : 0u);
        }
        mma_commit(bar(B_SFULL + tile));
      };
      auto issue_pv = [&](int tile, bool first) {
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          mma_f16kind_ts(tmem + kColO + tile * 128, tmem + tile * BN + kColP + kk * 8,
                         desc_add(dv0, kk * (2048 >> 4)), id_pv, first && kk == 0 ? 0u : 1u);
      };
      bool ok = true;
      int g = 0, gb = 0, seq = 0, jj = 0;        // steps, steps with both tiles, items, step of the item
      bool have = false, pfirst = false, plast = false, ptwo = false;
      int pslot = 0;
      Item it{};
      auto next_item = [&]() {
        ok = mbar_wait(bar(B_IFULL + (seq & 1)), (uint32_t)(seq >> 1) & 1u, abort, lim);
        it = ok ? read_item(ctl->ring, seq & 1) : Item{};
        jj = 0;
      };
      // P V of the step before, tile A or B
      auto close_a = [&]() -> bool {
        if (!mbar_wait(bar(B_PFULL), (uint32_t)(g - 1) & 1u, abort, lim) ||
            !mbar_wait(bar(B_VREADY), (uint32_t)(g - 1) & 1u, abort, lim))
          return false;
        tc_fence_after();
        issue_pv(0, pfirst);
        if (plast) mma_commit(bar(B_ODONE));
        if (!ptwo) mma_commit(bar(B_VEMPTY));
        return true;
      };
      auto close_b = [&](int steps) -> bool {
        if (ptwo) {
          if (!mbar_wait(bar(B_PFULL + 1), (uint32_t)(steps - 1) & 1u, abort, lim)) return false;
          tc_fence_after();
          issue_pv(1, pfirst);
          mma_commit(bar(B_VEMPTY));
          if (plast) mma_commit(bar(B_ODONE + 1));
        }
        if (plast) mbar_arrive(bar(B_IEMPTY + pslot));
        return true;
      };
      next_item();
      while (ok && it.valid) {
        const bool two = it.row1 - it.row0 > BM;
        const int kb = g & 1;
        if (have && !(ok = close_a())) break;
        ok = mbar_wait(bar(B_KREADY + kb), (uint32_t)(g >> 1) & 1u, abort, lim) &&
             (jj > 0 || mbar_wait(bar(B_QFULL), (uint32_t)seq & 1u, abort, lim));
        if (!ok) break;
        tc_fence_after();
        issue_s(0, kb);
        if (!two) mma_commit(bar(B_KEMPTY + kb));
        if (have && !(ok = close_b(gb))) break;
        if (two) {
          ok = jj > 0 || mbar_wait(bar(B_QFULL + 1), (uint32_t)seq & 1u, abort, lim);
          if (!ok) break;
          tc_fence_after();
          issue_s(1, kb);
          mma_commit(bar(B_KEMPTY + kb));
          ++gb;
        }
        have = true;
        pfirst = jj == 0;
        plast = jj == it.k1 - it.k0 - 1;
        ptwo = two;
        pslot = seq & 1;
        ++g;
        ++jj;
        if (plast) {
          ++seq;
          next_item();
        }
      }
      if (ok && have) ok = close_a() && close_b(gb);
      if (!ok) {
        *abort = 1;
        atomicOr(p.err, kErrTimeout);
      }
      // every product of this thread has completed once this arrives
      mma_commit(bar(B_DRAIN));
      mbar_wait(bar(B_DRAIN), 0, nullptr, lim);
    }
    __syncwarp();
  } else if (warp >= kDeqWarp) {
    // ------------------------------------------------- codes into f16 tiles
    const int dw = warp - kDeqWarp, t = tid - 32 * kDeqWarp;     // t: a position of the step
    bool ok = true, range = false;
    int g = 0;
    int vr[Y];
    for (int seq = 0; ok; ++seq) {
      const int islot = seq & 1;
      ok = __all_sync(FULL, mbar_wait(bar(B_IFULL + islot), (uint32_t)(seq >> 1) & 1u, abort, lim));
      ok = barrier_and(1, kDeqThreads, ok);
      if (!ok) break;
      const Item it = read_item(ctl->ring, islot);
      if (!it.valid) break;
      const bool two = it.row1 - it.row0 > BM;
      for (int s = it.k1 - 1; s >= it.k0; --s, ++g) {
        const int st = g % S::kRawStages, kb = g & 1;
        const uint32_t raw = sbase + S::kRawAt + st * S::kRaw;
        ok = ok && mbar_wait(bar(B_RAWFULL + st), (uint32_t)(g / S::kRawStages) & 1u, abort, lim);
        // -- this position's pairs of K and V
        const bool counts = ok && ((*reinterpret_cast<volatile int*>(&ctl->present[st]) >> (t >> 4)) & 1) &&
                            BN * s + t <= it.last;
        const uint32_t pairs = raw + (t >> 4) * Layout<D>::kTileBytes + Layout<D>::pair(t & 15, 0);
        uint32_t kw[Y], vw[Y];
        if constexpr (Y == 4) {
          const uint4 a = ld_shared_v4(pairs + Layout<D>::kKPairs), b = ld_shared_v4(pairs + Layout<D>::kVPairs);
          kw[0] = a.x, kw[1] = a.y, kw[2] = a.z, kw[3] = a.w;
          vw[0] = b.x, vw[1] = b.y, vw[2] = b.z, vw[3] = b.w;
        } else {
#pragma unroll
          for (int y = 0; y < Y; ++y) {
            kw[y] = ld_shared_u32(pairs + Layout<D>::kKPairs + 4 * y);
            vw[y] = ld_shared_u32(pairs + Layout<D>::kVPairs + 4 * y);
          }
        }
        float kmax = 0.f;
        int bad = 0;
#pragma unroll
        for (int y = 0; y < Y; ++y) {
          if (!counts) kw[y] = vw[y] = 0;
          // the largest magnitude of a group is at one of its ends
          const float k = fmaxf(fabsf(pair_lo(kw[y])), fabsf(fmaf(15.f, pair_step(kw[y]), pair_lo(kw[y]))));
          if (k <= 3.402823466e38f) kmax = fmaxf(kmax, k);
          const float a = fabsf(pair_lo(vw[y])), b = fabsf(fmaf(15.f, pair_step(vw[y]), pair_lo(vw[y])));
          const bool fine = a <= 3.402823466e38f && b <= 3.402823466e38f;
          if (!fine) {
            bad |= 1 << y;
            vw[y] = 0;
          }
          const uint32_t top = __reduce_max_sync(FULL, fine ? __float_as_uint(fmaxf(a, b)) : 0u);
          if (lane == 0) ctl->vmax[dw][y] = top;
        }
        const uint32_t there = __ballot_sync(FULL, counts);
        if (lane == 0) ctl->mask[kb][dw] = there;
#pragma unroll
        for (int y = 0; y < Y; ++y) {
          const uint32_t w = __ballot_sync(FULL, (bad >> y) & 1);
          if (lane == 0) ctl->vnan[kb][y][dw] = w;
        }
        // The queries' scale goes into the positions' factors: by the softmax warps in
        // the item's first step (to wait for it here would hold up that step's K,
        // behind which the item before ends), from here on later.
        const bool first = s == it.k1 - 1;
        if (s == it.k1 - 2 && ok)
          ok = mbar_wait(bar(B_QFULL), (uint32_t)seq & 1u, abort, lim) &&
               (!two || mbar_wait(bar(B_QFULL + 1), (uint32_t)seq & 1u, abort, lim));
        ok = barrier_and(1, kDeqThreads, ok);
        if (!ok) break;
        // -- scales
        int ev = -1000;
        {
          int top[Y], base = -1000;
#pragma unroll
          for (int y = 0; y < Y; ++y) {
            uint32_t v = 0;
#pragma unroll
            for (int w = 0; w < kDeqWarps; ++w) v = max(v, ctl->vmax[w][y]);
            top[y] = v == 0 ? -1000 : max((int)(v >> 23) - 127, -100);
            base = max(base, top[y]);
          }
          if (first) {
#pragma unroll
            for (int y = 0; y < Y; ++y) {
              vr[y] = base == -1000 ? 0 : top[y] == -1000 ? base : max(top[y], base - 48);
              vr[y] = min(vr[y], 110);
              if (t == 0) ctl->vr[islot][y] = vr[y] + 1;
            }
          }
#pragma unroll
          for (int y = 0; y < Y; ++y)
            if (top[y] != -1000) ev = max(ev, top[y] - vr[y]);
          if (ev == -1000) ev = 0;
          ev = max(-48, min(48, ev));
#pragma unroll
          for (int y = 0; y < Y; ++y) range = range || top[y] - vr[y] - ev > 14;
        }
        {
          const int e = min(max((int)(__float_as_uint(kmax) >> 23) - 127, -100), 118);
          const float f = pow2(-(e + 7));
#pragma unroll
          for (int y = 0; y < Y; ++y) {
            const float step = pair_step(kw[y]) * (f * 0x1p24f), lo = pair_lo(kw[y]) * f;
            ctl->kq[t][y] = make_uint2(pack_f16(step, step), pack_f16(lo, lo));
            const float fv = pow2(-(vr[y] + ev + 1)), sv = pow2(18 - (vr[y] + ev + 1));
            const float vs = pair_step(vw[y]) * sv, vl = pair_lo(vw[y]) * fv;
            ctl->vq[y][t] = make_uint2(pack_f16(vs, vs), pack_f16(vl, vl));
          }
          const float back = pow2(e + 7);
          ctl->cs[kb][0][t] = first ? back : fminf(back * ctl->qs[0], 3.402823466e38f);
          if (two) ctl->cs[kb][1][t] = first ? back : fminf(back * ctl->qs[1], 3.402823466e38f);
        }
        if (t == 0) ctl->ev[kb] = ev;
        ok = mbar_wait(bar(B_KEMPTY + kb), ((uint32_t)(g >> 1) & 1u) ^ 1u, abort, lim);
        ok = barrier_and(1, kDeqThreads, ok);
        if (!ok) break;
        if (t == 0) {
          uint32_t any = 0;
#pragma unroll
          for (int y = 0; y < Y; ++y)
#pragma unroll
            for (int w = 0; w < 4; ++w) any |= ctl->vnan[kb][y][w];
          ctl->any_nan[kb] = any != 0;
        }
        // -- K: a lane a position and a quarter of each group; eight positions a
        // warp and turn, bit 2 of the position in bit 2 of the lane, so that eight
        // lanes' stores lie in eight different banks
        {
          const uint32_t dst = sbase + S::kK + kb * S::kTileB;
          const int u = lane & 3, r8 = (lane & 4) | ((lane >> 3) & 3);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = dw * 32 + i * 8 + r8;
            const uint32_t at = raw + (row >> 4) * Layout<D>::kTileBytes + (row & 15) * (D / 2) + u * (D / 8);
            uint32_t w[Y];
            if constexpr (Y == 4) {
              const uint4 a = ld_shared_v4(at);
              w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
            } else {
#pragma unroll
              for (int y = 0; y < Y; ++y) w[y] = ld_shared_u32(at + 4 * y);
            }
#pragma unroll
            for (int y = 0; y < Y; ++y) {
              const uint2 k = ctl->kq[row][y];
              const uint32_t s24 = k.x, s20 = hmul2(k.x, 0x2c002c00u), hi = w[y] >> 8;    // 2^-4
              st_shared_v4(dst + (y >> 1) * kHalf + row * 128 + ((((y & 1) * 4 + u) ^ (row & 7)) << 4),
                           hfma2(w[y] & 0x000f000fu, s24, k.y), hfma2(w[y] & 0x00f000f0u, s20, k.y),
                           hfma2(hi & 0x000f000fu, s24, k.y), hfma2(hi & 0x00f000f0u, s20, k.y));
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_KREADY + kb));
        // -- V: a lane a quarter group of two neighbouring groups, four positions
        ok = mbar_wait(bar(B_VEMPTY), ((uint32_t)g & 1u) ^ 1u, abort, lim);
        ok = __all_sync(FULL, ok);
        if (ok) {
          const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int tile = dw * 2 + i;
#pragma unroll
            for (int yy = 0; yy < Y / 2; ++yy) {
              const uint4 a = ld_shared_v4(raw + tile * Layout<D>::kTileBytes + Layout<D>::kV + yy * 512 + lane * 16);
              const uint32_t w[2][2] = {{a.x, a.y}, {a.z, a.w}};
#pragma unroll
              for (int blk = 0; blk < 2; ++blk) {
                const int key = tile * 16 + blk * 8 + 2 * tq;
                const uint4 q0 = ld_shared_v4(smem_u32(&ctl->vq[2 * yy][key]));
                const uint4 q1 = ld_shared_v4(smem_u32(&ctl->vq[2 * yy + 1][key]));
#pragma unroll
                for (int par = 0; par < 2; ++par) {
                  const uint32_t x0 = __byte_perm(w[0][blk], 0, par ? 0x4342 : 0x4140);
                  const uint32_t x1 = __byte_perm(w[1][blk], 0, par ? 0x4342 : 0x4140);
                  const uint32_t s0 = par ? q0.z : q0.x, l0 = par ? q0.w : q0.y;
                  const uint32_t s1 = par ? q1.z : q1.x, l1 = par ? q1.w : q1.y;
                  const int row = key + par;
                  st_shared_v4(sbase + S::kV + yy * kHalf + row * 128 + ((gq ^ (row & 7)) << 4),
                               hfma2((x0 << 6) & 0x03c003c0u, s0, l0), hfma2((x0 << 2) & 0x03c003c0u, s0, l0),
                               hfma2((x1 << 6) & 0x03c003c0u, s1, l1), hfma2((x1 << 2) & 0x03c003c0u, s1, l1));
                }
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(B_VREADY));
            mbar_arrive(bar(B_RAWEMPTY + st));
          }
        }
        // (a wait that ran out is told to the others at the next barrier)
        if (!ok && lane == 0) *abort = 1;
      }
      ok = barrier_and(1, kDeqThreads, ok);
      if (!ok) break;
      if (lane == 0) mbar_arrive(bar(B_IEMPTY + islot));
    }
    if (lane == 0) {
      if (!ok) {
        *abort = 1;
        atomicOr(p.err, kErrTimeout);
      }
      if (range) atomicOr(p.err, kErrRange);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------ softmax, epilogue
    const int tile = warp >> 2, r = tid & (BM - 1);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + tile * BN, o_col = tmem + lane_base + kColO + tile * 128;
    const float norm = kLog2e * (D == 64 ? 0.125f : 0.08838834764831845f);
    bool ok = true;
    int g = 0, gt = 0, items = 0;        // steps, this tile's steps and items
    for (int seq = 0; ok; ++seq) {
      const int islot = seq & 1;
      ok = __all_sync(FULL, mbar_wait(bar(B_IFULL + islot), (uint32_t)(seq >> 1) & 1u, abort, lim));
      if (!ok) break;
      const Item it = read_item(ctl->ring, islot);
      if (!it.valid) break;
      const int steps = it.k1 - it.k0, row = it.row0 + tile * BM + r;
      if (tile == 1 && it.row1 - it.row0 <= BM) {
        mbar_arrive(bar(B_QFULL + 1));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_IEMPTY + islot));
        g += steps;
        continue;
      }
      // -- the row's query
      bool row_ok = row < it.row1, row_bad = false;
      int h = 0, pos = -1;
      int64_t at = 0;
      float slope = 0.f;
      if (row_ok) {
        at = row_at<PREFIX, D>(p, it.b, it.kvh, it.pos, row, h, pos);
        slope = p.slope[h];
        row_ok = pos >= 0;
      }
      {
        uint4 qv[D / 8];
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + at);
        uint32_t mx = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          qv[c] = row_ok ? src[c] : make_uint4(0, 0, 0, 0);
          mx = __vmaxu2(mx, qv[c].x & 0x7fff7fffu);
          mx = __vmaxu2(mx, qv[c].y & 0x7fff7fffu);
          mx = __vmaxu2(mx, qv[c].z & 0x7fff7fffu);
          mx = __vmaxu2(mx, qv[c].w & 0x7fff7fffu);
        }
        mx = max(mx & 0xffff0000u, mx << 16);
        row_bad = mx >= (110u + 127u) << 23;             // 2^110, infinities, NaN
        const uint32_t top = __reduce_max_sync(FULL, row_bad ? 0u : mx);
        if (lane == 0) ctl->qmax[tile][warp & 3] = top;
        ok = barrier_and(2 + tile, BM, ok);
        uint32_t all = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) all = max(all, ctl->qmax[tile][w]);
        const int e = min(max((int)(all >> 23) - 127, -100), 110);
        const float up = row_bad ? 0.f : pow2(14 - e);
        if (r == 0) ctl->qs[tile] = pow2(e - 14) * norm;
        const uint32_t dst = sbase + S::kQ + tile * S::kTileB + r * 128;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t w[4] = {qv[c].x, qv[c].y, qv[c].z, qv[c].w};
          float v[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[2 * k] = row_bad ? 0.f : __uint_as_float(w[k] << 16) * up;
            v[2 * k + 1] = row_bad ? 0.f : __uint_as_float(w[k] & 0xffff0000u) * up;
          }
          // values in the order that K's codes come in: 0, 4, 1, 5, 2, 6, 3, 7
          st_shared_v4(dst + (c >> 3) * kHalf + (((c & 7) ^ (r & 7)) << 4), pack_f16(v[0], v[4]), pack_f16(v[1], v[5]),
                       pack_f16(v[2], v[6]), pack_f16(v[3], v[7]));
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(B_QFULL + tile));
      }
      if (!ok) break;
      uint64_t eslope[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) eslope[e] = f2_pack((float)(2 * e) * slope, (float)(2 * e + 1) * slope);
      float m_ref = -INFINITY, l = 0.f;
      int nan_groups = 0;
      for (int s = it.k1 - 1; s >= it.k0; --s, ++g, ++gt) {
        const int kb = g & 1, jt = s * BN;
        // (the step's scales, then its scores)
        ok = mbar_wait(bar(B_KREADY + kb), (uint32_t)(g >> 1) & 1u, abort, lim);
        if (s == it.k1 - 1) {
          ctl->cs[kb][tile][r] = fminf(ctl->cs[kb][tile][r] * ctl->qs[tile], 3.402823466e38f);
          ok = barrier_and(2 + tile, BM, ok);
        }
        ok = ok && mbar_wait(bar(B_SFULL + tile), (uint32_t)gt & 1u, abort, lim);
        ok = __all_sync(FULL, ok);
        if (!ok) break;
        tc_fence_after();
        const int ev = ctl->ev[kb];
        const uint32_t cs = smem_u32(&ctl->cs[kb][tile][0]);
        auto mask = [&](int q) { return row_ok ? upto_mask(pos - jt - 32 * q) & ctl->mask[kb][q] : 0u; };
        // exponents of a chunk of 32 keys: x + ev - mu, -inf where masked
        auto exponents = [&](int q, float mu, const uint32_t (&rr)[32], uint32_t vm, float (&x)[32]) {
          const float off = fmaf((float)(jt + 32 * q - pos), slope, (float)ev - mu);
          const uint64_t off2 = f2_pack(off, off);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const uint4 c4 = ld_shared_v4(cs + 128 * q + 4 * e);
            f2_unpack(f2_fma(f2_pack(__uint_as_float(rr[e]), __uint_as_float(rr[e + 1])),
                             f2_pack(__uint_as_float(c4.x), __uint_as_float(c4.y)), f2_add(eslope[e >> 1], off2)),
                      x[e], x[e + 1]);
            f2_unpack(f2_fma(f2_pack(__uint_as_float(rr[e + 2]), __uint_as_float(rr[e + 3])),
                             f2_pack(__uint_as_float(c4.z), __uint_as_float(c4.w)),
                             f2_add(eslope[(e >> 1) + 1], off2)),
                      x[e + 2], x[e + 3]);
          }
          if (__any_sync(FULL, vm != 0xffffffffu)) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(vm & (1u << e))) x[e] = -INFINITY;
          }
        };
        // The first step of a row finds its maximum first; later ones take their
        // weights against the maximum as it stands and watch for growth.
        const bool one_pass = s < it.k1 - 1 && !__any_sync(FULL, row_ok && m_ref == -INFINITY);
        float m_use = m_ref, alpha = 1.f;
        bool resc = false;
        if (!one_pass) {
          float mt = -INFINITY;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            const uint32_t vm = mask(q);
            if (!__any_sync(FULL, vm != 0u)) continue;
            uint32_t rr[32];
            tmem_ld32(s_col + q * 32, rr);
            tmem_wait_ld();
            float x[32];
            exponents(q, 0.f, rr, vm, x);
#pragma unroll
            for (int e = 0; e < 32; e += 2) mt = max3(mt, x[e], x[e + 1]);
          }
          const float m_new = fmaxf(m_ref, mt);
          resc = m_new > m_ref + kRescaleLog2;
          m_use = resc ? m_new : m_ref;
          alpha = resc ? ex2(m_ref - m_new) : 1.f;
        }
        float mu = m_use == -INFINITY ? 0.f : m_use;
        if (s < it.k1 - 1 && __any_sync(FULL, resc)) {
          // (the commit behind these scores proves that P V of the step before is done)
          const float f = resc ? alpha : 1.f;
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(o_col + q * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(o_col + q * 32, o);
          }
        }
        uint64_t lsum = f2_pack(0.f, 0.f);
#pragma unroll 1
        for (int q = 3; q >= 0; --q) {
          const uint32_t vm = mask(q);
          if (!__any_sync(FULL, vm != 0u)) {
            const uint32_t z[16] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
            tmem_st16(s_col + kColP + q * 16, z);
            continue;
          }
          uint32_t rr[32];
          tmem_ld32(s_col + q * 32, rr);
          tmem_wait_ld();
          float x[32];
          exponents(q, mu, rr, vm, x);
          if (one_pass) {
            float c0 = -INFINITY, c1 = -INFINITY;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              c0 = max3(c0, x[e], x[e + 1]);
              c1 = max3(c1, x[e + 2], x[e + 3]);
            }
            const float cm = fmaxf(c0, c1);
            if (__any_sync(FULL, cm > kGrowLog2)) {
              // a jump of the scores: O, l and the weights of this step written so
              // far are scaled to the new maximum
              const float d = cm > kGrowLog2 ? cm : 0.f, f = ex2(-d);
              mu += d;
              if (row_ok) m_use = mu;
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] -= d;
              l *= f;
              lsum = f2_mul(lsum, f2_pack(f, f));
#pragma unroll 1
              for (int q3 = 0; q3 < D / 32; ++q3) {
                uint32_t o[32];
                tmem_ld32(o_col + q3 * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(o_col + q3 * 32, o);
              }
#pragma unroll 1
              for (int q3 = 3; q3 > q; --q3) {
                uint32_t w[16];
                tmem_ld16(s_col + kColP + q3 * 16, w);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
                  w[e] = pack_f16(v.x * f, v.y * f);
                }
                tmem_st16(s_col + kColP + q3 * 16, w);
              }
            }
          }
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float a = ex2(x[2 * e]), b = ex2(x[2 * e + 1]);
            lsum = f2_add(lsum, f2_pack(a, b));
            pk[e] = pack_f16(a, b);
          }
          tmem_st16(s_col + kColP + q * 16, pk);
        }
        float ls0, ls1;
        f2_unpack(lsum, ls0, ls1);
        l = fmaf(ls0 + ls1, pow2(-ev), l * alpha);
        m_ref = m_use;
        if (ctl->any_nan[kb]) {
          for (int q = 0; q < 4; ++q) {
            const uint32_t vm = mask(q);
#pragma unroll
            for (int y = 0; y < Y; ++y)
              if (ctl->vnan[kb][y][q] & vm) nan_groups |= 1 << y;
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(B_PFULL + tile));
      }
      if (!ok) break;
      // -- the row
      ok = __all_sync(FULL, mbar_wait(bar(B_ODONE + tile), (uint32_t)items & 1u, abort, lim));
      if (!ok) break;
      ++items;
      tc_fence_after();
      if (row_bad) l = NAN;
      const bool whole = it.slot < 0;
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      float* part = p.part + (int64_t)it.slot * part_floats<D>();
      const int pr = tile * BM + r;                        // row of the piece
      float up[Y];
#pragma unroll
      for (int y = 0; y < Y; ++y) up[y] = (nan_groups >> y) & 1 ? NAN : pow2(ctl->vr[islot][y]) * inv;
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        uint32_t o[32];
        tmem_ld32(o_col + q * 32, o);
        tmem_wait_ld();
        // four quarter groups of groups y and y + 1
        const int y = 2 * (q >> 1), g0 = 4 * (q & 1);
        float u0 = up[0], u1 = up[1];
        if constexpr (Y == 4) {
          if (y == 2) u0 = up[2], u1 = up[3];
        }
        if (whole) {
          if (row_ok) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + at + 32 * y + 4 * g0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float u = k ? u1 : u0;
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint32_t* a = &o[16 * c + 4 * k];
                auto v = [&](int i) { return __uint_as_float(a[i]) * u; };
                reinterpret_cast<uint4*>(dst + 32 * k)[c] =
                    make_uint4(pack_bf16(v(0), v(2)), pack_bf16(v(1), v(3)), pack_bf16(v(8), v(10)), pack_bf16(v(9), v(11)));
              }
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float u = c & 1 ? u1 : u0;
            reinterpret_cast<float4*>(part)[(8 * q + c) * kItemRows + pr] =
                make_float4(__uint_as_float(o[4 * c]) * u, __uint_as_float(o[4 * c + 1]) * u,
                            __uint_as_float(o[4 * c + 2]) * u, __uint_as_float(o[4 * c + 3]) * u);
          }
        }
      }
      if (!whole) {
        part[kItemRows * D + pr] = m_ref == -INFINITY ? kNothing : m_ref;
        part[kItemRows * (D + 1) + pr] = row_ok ? l : 0.f;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_IEMPTY + islot));
    }
    if (!ok && lane == 0) {
      *abort = 1;
      atomicOr(p.err, kErrTimeout);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------- joining
// A lane a row, a warp every eighth of the columns' quads; 32 rows of an item a CTA.
constexpr int kJoinThreads = 256;

template <int D>
__device__ __forceinline__ void store4(__nv_bfloat16* o, int quad, const float4& a) {
  // quad c: values 4 g .. 4 g + 3 of group y, in the order 0, 2, 1, 3
  const int c = quad >> 1, y = 2 * (c >> 3) + (quad & 1), g = c & 7;
  *reinterpret_cast<uint2*>(o + 32 * y + 4 * g) = make_uint2(pack_bf16(a.x, a.z), pack_bf16(a.y, a.w));
}

template <int D>
__global__ void __launch_bounds__(kJoinThreads) q4_many_join_kernel(const __grid_constant__ ManyParams p) {
  grid_dep_wait();
  const int4 end = p.ends[blockIdx.x];
  if (end.x < 0) return;
  const int entries = p.c.B * p.tiles, kvh = end.x / entries, e = end.x - kvh * entries, b = e / p.tiles;
  int pos0, rows, last;
  item_steps<false>(p, b, e - b * p.tiles, pos0, rows, last);
  const int pr = blockIdx.y * 32 + (threadIdx.x & 31), row = kItemRows * (e - b * p.tiles) + pr;
  if (row >= rows) return;
  int h, pos;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + row_at<false, D>(p, b, kvh, pos0, row, h, pos);
  const int n = (int)blockIdx.x - end.y + 1;
  auto piece = [&](int k) { return p.part + (int64_t)(k == 0 ? end.z : 2 * (end.y + k)) * part_floats<D>(); };
  float mm = kNothing, sum = 0.f;
  for (int k = 0; k < n; ++k) mm = fmaxf(mm, piece(k)[kItemRows * D + pr]);
  float4 acc[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < n; ++k) {
    const float* pt = piece(k);
    const float l = pt[kItemRows * (D + 1) + pr];
    if (l == 0.f) continue;
    const float f = ex2(pt[kItemRows * D + pr] - mm);
    sum = fmaf(f, l, sum);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const float4 v = reinterpret_cast<const float4*>(pt)[((threadIdx.x >> 5) + 8 * c) * kItemRows + pr];
      acc[c].x = fmaf(f, v.x, acc[c].x);
      acc[c].y = fmaf(f, v.y, acc[c].y);
      acc[c].z = fmaf(f, v.z, acc[c].z);
      acc[c].w = fmaf(f, v.w, acc[c].w);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    store4<D>(o, (threadIdx.x >> 5) + 8 * c,
              make_float4(acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv));
}

// A decode step's rows: the prefix's pieces and those of the sequences' own keys.
struct PrefixJoin {
  int64_t total, per;                 // of the prefix's list: entries of a KV head, of a CTA
  const int4* rows;                   // own keys: per row {first piece, second, pieces, 0}
  const float* own;                   // their pieces: o [8][D], maximum [8], sum [8]
  int chunks, per_chunk;
};

template <int D>
__global__ void __launch_bounds__(kJoinThreads)
q4_prefix_join_kernel(const __grid_constant__ ManyParams p, const __grid_constant__ PrefixJoin j) {
  grid_dep_wait();
  constexpr int kOwn = 8 * (D + 2);
  const int kvh = blockIdx.x / p.tiles, t = blockIdx.x - kvh * p.tiles;
  const int pr = blockIdx.y * 32 + (threadIdx.x & 31), row = kItemRows * t + pr;
  if (row >= p.c.B * p.G) return;
  int h, pos;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + row_at<true, D>(p, 0, kvh, 0, row, h, pos);
  // the item's entries [base, base + cost): its pieces' CTAs
  const int64_t cost = ((p.keys + BN - 1) / BN) + kItemCost, base = kvh * j.total + t * cost;
  const int i0 = (int)((base + kItemCost) / j.per), i1 = (int)((base + cost - 1) / j.per);
  const int slot0 = base <= i0 * j.per ? 2 * i0 : 2 * i0 + 1, n = i1 - i0 + 1;
  auto piece = [&](int k) { return p.part + (int64_t)(k == 0 ? slot0 : 2 * (i0 + k)) * part_floats<D>(); };
  const int b = row / p.G, hh = row - b * p.G, ch = hh / j.per_chunk, hc = hh - ch * j.per_chunk;
  const int4 own = j.rows[((int64_t)b * p.c.H + kvh) * j.chunks + ch];
  auto own_piece = [&](int k) { return j.own + (int64_t)(k == 0 ? own.x : own.y + 2 * (k - 1)) * kOwn; };
  float mm = kNothing, sum = 0.f;
  for (int k = 0; k < n; ++k) mm = fmaxf(mm, piece(k)[kItemRows * D + pr]);
  for (int k = 0; k < own.z; ++k) mm = fmaxf(mm, own_piece(k)[8 * D + hc]);
  float4 acc[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < n; ++k) {
    const float* pt = piece(k);
    const float l = pt[kItemRows * (D + 1) + pr];
    if (l == 0.f) continue;
    const float f = ex2(pt[kItemRows * D + pr] - mm);
    sum = fmaf(f, l, sum);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const float4 v = reinterpret_cast<const float4*>(pt)[((threadIdx.x >> 5) + 8 * c) * kItemRows + pr];
      acc[c].x = fmaf(f, v.x, acc[c].x);
      acc[c].y = fmaf(f, v.y, acc[c].y);
      acc[c].z = fmaf(f, v.z, acc[c].z);
      acc[c].w = fmaf(f, v.w, acc[c].w);
    }
  }
  for (int k = 0; k < own.z; ++k) {
    const float* pt = own_piece(k);
    const float l = pt[8 * D + 8 + hc];
    if (l == 0.f) continue;
    const float f = ex2(pt[8 * D + hc] - mm);
    sum = fmaf(f, l, sum);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const int quad = (threadIdx.x >> 5) + 8 * c, x = quad >> 1;
      const float4 v = *reinterpret_cast<const float4*>(pt + hc * D + 32 * (2 * (x >> 3) + (quad & 1)) + 4 * (x & 7));
      acc[c].x = fmaf(f, v.x, acc[c].x);
      acc[c].y = fmaf(f, v.z, acc[c].y);
      acc[c].z = fmaf(f, v.y, acc[c].z);
      acc[c].w = fmaf(f, v.w, acc[c].w);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    store4<D>(o, (threadIdx.x >> 5) + 8 * c,
              make_float4(acc[c].x * inv, acc[c].y * inv, acc[c].z * inv, acc[c].w * inv));
}

template <int D>
constexpr size_t smem_bytes() { return 1024 + Sizes<D>::kEnd + sizeof(Ctl<D>); }
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory");

void fill(ManyParams& p, const Q4DecodeArgs& a, void* work) {
  p.c = a.c;
  p.q = a.q;
  p.o = a.o;
  p.pos = a.pos;
  p.len = a.len;
  p.prefix = a.prefix;
  p.Hq = a.Hq;
  p.G = a.Hq / a.c.H;
  p.m = a.m;
  p.limit = (int)(a.c.max_pages << a.c.page_shift);
  p.keys = a.prefix_pages << a.c.page_shift;
  p.ends = static_cast<int4*>(work);
  p.part = reinterpret_cast<float*>(p.ends + a.num_sms);
  p.err = a.err;
  p.wait_ns = a.wait_ns;
  for (int h = 0; h < a.Hq; ++h) p.slope[h] = a.slope_log2[h];
}

template <int D>
cudaError_t launch_chunk(const Q4DecodeArgs& a, cudaStream_t st) {
  ManyParams p;
  fill(p, a, a.work);
  p.tiles = (int)(((int64_t)p.m * p.G + kItemRows - 1) / kItemRows);
  auto kern = q4_many_kernel<D, false>;
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kern), (int)smem_bytes<D>());
  if (e == cudaSuccess) e = launch_dependent(kern, dim3(a.num_sms), kThreads, smem_bytes<D>(), st, p);
  if (e == cudaSuccess)
    e = launch_dependent(q4_many_join_kernel<D>, dim3(a.num_sms, kItemRows / 32), kJoinThreads, 0, st, p);
  return e;
}

template <int D>
cudaError_t launch_prefix(const Q4DecodeArgs& a, cudaStream_t st) {
  ManyParams p;
  const int64_t own = q4_own_work_bytes(D, a.num_sms, a.c.B, a.c.H, a.Hq / a.c.H);
  fill(p, a, static_cast<uint8_t*>(a.work) + own);
  p.tiles = (int)(((int64_t)a.c.B * p.G + kItemRows - 1) / kItemRows);
  PrefixJoin j;
  j.chunks = (p.G + 7) / 8;
  j.per_chunk = (p.G + j.chunks - 1) / j.chunks;
  // (as the kernel finds them)
  j.total = (int64_t)p.tiles * ((p.keys + BN - 1) / BN + kItemCost);
  const int64_t all = j.total * a.c.H;
  j.per = std::max<int64_t>((all + a.num_sms - 1) / a.num_sms, kMinSteps + kItemCost);
  // the sequences' own keys, then the prefix's, then both together
  Q4DecodeArgs b = a;
  uint8_t* w = static_cast<uint8_t*>(a.work);
  b.rows = reinterpret_cast<int4*>(w + own) - (int64_t)a.c.B * a.c.H * j.chunks;
  j.rows = b.rows;
  j.own = q4_own_pieces(a.work, a.num_sms);
  cudaError_t e = launch_q4_decode(b, st);
  auto kern = q4_many_kernel<D, true>;
  if (e == cudaSuccess) e = set_smem_limit(reinterpret_cast<const void*>(kern), (int)smem_bytes<D>());
  if (e == cudaSuccess) e = launch_dependent(kern, dim3(a.num_sms), kThreads, smem_bytes<D>(), st, p);
  if (e == cudaSuccess)
    e = launch_dependent(q4_prefix_join_kernel<D>, dim3(a.c.H * p.tiles, kItemRows / 32), kJoinThreads, 0, st, p, j);
  return e;
}

}  // namespace

int64_t q4_many_work_bytes(int d, int num_sms) {
  return (int64_t)num_sms * (sizeof(int4) + 2 * sizeof(float) * kItemRows * (d + 2));
}

cudaError_t launch_q4_chunk(const Q4DecodeArgs& a, cudaStream_t st) {
  return a.c.d == 64 ? launch_chunk<64>(a, st) : launch_chunk<128>(a, st);
}
cudaError_t launch_q4_prefix(const Q4DecodeArgs& a, cudaStream_t st) {
  return a.c.d == 64 ? launch_prefix<64>(a, st) : launch_prefix<128>(a, st);
}

}  // namespace plsh
