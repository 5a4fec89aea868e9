// Exact ALiBi attention of many query rows over the 4-bit paged cache: a chunk of
// new tokens of every sequence (row i at position p = pos[b] + i), and the part of
// a decode step that lies in a prefix which all sequences share (one row a
// sequence, p = pos[b], keys below the prefix's end):
//   o = sum_j e^{q.k_j / sqrt(d) - (p - j) / sigma_h} v_j / sum_j (the weights), j <= p.
//
// The rows of all query heads of a KV head see the same keys, so an item is 256
// such rows (two tiles of 128) and the keys up to the last of their positions, in
// steps of 128, last step first.  A step's codes (20 d bytes for 16 positions) are
// taken apart once for the 256 rows, into f16 tiles in shared memory, and the products
// run on the tensor cores (tcgen05): S = Q K^T from shared memory, P V with P in
// tensor memory.
//
// Numbers.  Codes are exact in f16, so a value lo + step c is rounded once, in one
// f16 multiply-add (c is taken from the low bits of 1024 + c or 64 + c, exactly).
// Powers of two keep everything within f16's range:
//   q  times one per row, the largest magnitude in [2^14, 2^15);
//   K  times one per 32 positions, likewise: undone in the fp32 scores (with q's, and
//      log2(e) / sqrt(d));
//   V  times one per group of 32 values, 2^-R_y, by the step's largest in that group
//      (undone in the epilogue), and one per 32 positions, 2^-ev, by how far all their
//      groups stay below that (or one exceeds it): likewise.  R_y stays while every
//      group of every 32 positions is near it; else it moves, and O's columns of that
//      group with it, as a row's O does with its reference: what is large in one
//      group moves little of the others.  2^ev goes into these positions' weights,
//      P = 2^{x + ev - M} with M near the maximum of x + ev so far; the row sum takes
//      P 2^-ev in fp32.  ev is below 10 (values from 2^111 on aside), so a weight keeps
//      2^-14 of the row's largest (2^-25 where ev is 0 throughout); where a group is far
//      above the item's others, ev is 8 there, and these positions' weights keep 2^-8
//      of that.  A value of V keeps 2^-24 of the largest of its group in its 32
//      positions; where a group of 32 positions keeps no 2^-14 of itself, the call is
//      reported.
// P and V are rounded to f16 (2^-11 of themselves): bf16's 2^-8 would show beside
// the output's own rounding.  Scores, sums and maxima are fp32.
//
// Warps of a CTA (one per SM): 0-7 and 8-15 softmax of the two tiles, two threads a
// row with 64 of a step's keys each; 16-19 take K's codes apart and 20-23 V's, up to
// two steps ahead; 24 issues the products, PV_A(g-1) S_A(g) PV_B(g-1) S_B(g), so that
// the tensor cores work on one tile while the other's scores become weights; 25 lists
// the items.  The flat list (KV head, item, step), each item preceded by kItemCost
// entries for its beginning and end, is cut into equal shares of the CTAs; items cut
// by a CTA's edge are joined by a second kernel, in a fixed order.  Every wait is
// bounded; on expiry the CTA raises the error flag, lets its copies and products
// drain, frees its tensor memory and exits.
//
// What bounds it.  The products of a step (two tiles) take 2048 cycles at 4096
// multiply-adds a cycle.  Measured (CUDA graph, back to back; shares of the measured
// GEMM rate of 1918 TFLOP/s): 2048 tokens behind 63488, 40/8 heads, 2395 us (1130
// TFLOP/s, 59 %), 2.25 us a step; 512 tokens behind 7680, 32/8 heads, 91 us (26 steps
// a CTA); a batch of eight ragged chunks 236 us; 128 sequences behind a prefix of
// 65536, 40/8 heads, 220 us, 64 behind 8192, 32/8 heads, 50 us (four steps a CTA).
// Neither the tensor cores nor the schedulers are full (512 behind 7680: pipe 36 %,
// issue slots 55 %): a tile's steps follow one another through its scores (1000
// cycles with P V before them), its softmax (2100 of weights, 500 until they are in
// tensor memory) and the products' barriers, as P stands where its scores stood (with
// steps of 128 keys S and O of two tiles fill the tensor memory; steps of 64 with two
// buffers of scores a tile would fit, and are not tried), and the two tiles' chains
// fill each other's gaps in part.  Beginning an item costs more: 12000 cycles from its
// listing to the first scores, where table, pages and queries come one after another
// from memory not touched before, and 7000 for the first step, whose weights are taken
// twice.  (Cycles as stamped when a step took 4600; it takes 4400 now.)
//
// What it took (2048 behind 63488): one thread's product issue from a branch of its
// own 3311 us, the whole warp's with a predicate 2835 (operands stay in uniform
// registers); softmax by sixteen columns with the next ones' load in flight, V's
// exponents from one reduction 2550; whether anything is masked decided once a step,
// and registers given to the codes 2430; V's exponents moving with the step (a barrier
// of V's warps a step) 2360, q's by row 2465, the exponents by a lane a group 2280, part
// of a large group's excess left in its weights 2395.
// Slower, and dropped: one thread a row (3100), 80 registers for softmax (2770), scalar
// instead of paired fp32 multiply-adds (+6 %), the first step's weights not tried
// before its maximum is known (+14 %, the loop's code suffers), K's and V's next codes
// loaded while these are taken apart (2415 to 2480, shorter items lose more), O
// following V's exponents by V's warps behind the softmax (2590 to 2780) or at a step's
// start (2590), the row's largest weight at 2^10 instead of 1, which would hold small
// weights of large values without V's part in them (heads of flat slopes and scores of
// sigma 3 move their references 40 % longer), the bias from positions instead of added up (2700), and for items of one
// tile the other tile on every second step of the same keys (64 rows of 131072 keys:
// 146 -> 166 us).  The softmax's 88 registers spill 84 to 132 bytes a thread (0.8 % of
// the instructions of 512 behind 7680); which values, and with them 5 % of the time,
// changes with the code around the loop.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "plsh_internal.h"
#include "q4.cuh"
#include "tc_ptx.cuh"

namespace plsh {
namespace {

using namespace q4;
using namespace ptx;

constexpr int BM = 128, BN = 128;       // rows of a tile, keys of a step
constexpr int kItemRows = 2 * BM;
constexpr int kSoftWarps = 16, kKWarp = 16, kVWarp = 20, kDeqWarps = 4, kMmaWarp = 24, kProdWarp = 25, kWarps = 28;
constexpr int kThreads = 32 * kWarps, kDeqThreads = 32 * kDeqWarps, kTileThreads = 256;
// of 896 threads' 72 at launch: 512 x 88 + 256 x 64 + 128 x 24 = 64512, all of them
constexpr int kRegsSoftmax = 88, kRegsDeq = 64, kRegsRest = 24;
enum { BAR_V = 1, BAR_PAIR = 2, BAR_CODES = 10 };      // named barriers: V's warps, two warps of a row, K's and V's
constexpr uint32_t kHalf = BM * 128;    // 128 rows of 64 f16 values, 128-byte swizzle
// Steps that beginning and ending an item costs (a batch of eight ragged chunks: 2 ->
// 293 us, 4 -> 266, 6 -> 248, 12 -> 250; 512 tokens behind 7680: 104, 100, 101, 107),
// and entries of a CTA at least (64 sequences behind a prefix of 8192: 3 -> 52 us, 6 ->
// 53, 9 -> 60).
constexpr int kItemCost = 6, kMinShare = 3;
constexpr uint32_t kTmemCols = 512;     // S_A | S_B | O_A | O_B; P over S
constexpr uint32_t kColP = 64, kColO = 256;
// A wait for an item to begin or end may last as long as one (a step's does not), and
// ends when a step's wait ran out: its limit is this many of theirs.
constexpr uint64_t kItemWaits = 64;
constexpr float kGrowLog2 = 15.f;       // largest weight 2^15: above, the reference moves
// V's groups within 2^-5 and 2^10 of R_y leave it where it is.  A group 2^7 above the
// item's smallest and more gets an R_y up to 2^8 below itself, so that ev raises the
// weights of its positions: as large as they are, they may count where their weights are
// below what f16 holds beside the row's largest.  R_y comes down to 2^-72 of an item's
// largest at most (O, below 2^30 of each key, goes up with it, and has to stay a number
// for 2^24 keys); 32 positions' group more than 2^24 below where f16 has them (its half
// step is 2^-39 of that) no longer keeps 2^-14 of itself, and is reported.
constexpr float kVBelow = 0x1p-5f;
constexpr int kVAbove = 10, kVRise = 7, kVRiseMost = 8, kVSpan = 72, kVLost = 24, kNoGroup = -1000;
constexpr float kNothing = -3.402823466e38f;
constexpr unsigned FULL = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kErrTimeout = 1, kErrRange = 2;

template <int D>
struct Sizes {
  static constexpr int Y = D / kGroup;
  static constexpr uint32_t kTileB = BM * D * 2;               // an f16 tile
  static constexpr uint32_t kQ = 0, kK = 2 * kTileB, kV = 4 * kTileB, kEnd = 6 * kTileB;      // two of each
};

enum {
  B_IFULL = 0, B_IEMPTY = 2, B_VEMPTY = 4, B_VREADY = 6, B_INFO = 8, B_KREADY = 12,
  B_KEMPTY = 16, B_QFULL = 18, B_SFULL = 20, B_PFULL = 22, B_ODONE = 24,
  B_DRAIN = 26, NUM_BARS = 27
};

// Rows [row0, row1) of a sequence's (or the batch's) rows of one KV head against the
// key steps [k0, k1), of which positions up to `last` count.  slot: the piece it
// leaves; a CTA's first piece 2 i, its last 2 i + 1, and, behind all of these, a
// prefix's item that lies in one CTA, of which a CTA may have many.
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
  // K and V run up to two steps ahead of the products, the softmax up to one behind
  alignas(16) uint2 kinfo[4][4];        // per step and 32 positions: K's factor, to be undone; positions that count
  // V's exponent beyond R_y; 2^-that, negative for a step with either of:
  alignas(16) uint2 vinfo[4][4];
  uint32_t vnan[4][Y][4];               // positions whose group of V is no number
  int vmoved[4][4];                     // R_y moved: O's columns follow by these factors
  float vscale[4][Y];
  int vr[2][Y];                         // per item slot: V's exponents R_y, less 14
  int vmax[kDeqWarps][Y];               // a step's exponents by 32 positions
  int vhigh[Y], vlow[Y];                // an item's largest R_y, and smallest group of 32 positions
  alignas(16) int tops[2 * kDeqWarps];  // prefix: the furthest positions of any row
  float pair[2][2][BM];                 // per tile and half: what the two threads of a row tell each other
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
  uint64_t wait_ns, item_wait_ns;       // of a step's waits, of an item's
  int stall;                            // fault injection: no item is listed
  float slope[kMaxExactHeads];          // log2(e) / sigma_h
};

template <int N>
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void leave_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <int D>
__host__ __device__ constexpr int64_t part_floats() { return kItemRows * (D + 2); }

__device__ __forceinline__ float pow2(int e) { return e < -126 ? 0.f : __int_as_float((min(e, 127) + 127) << 23); }

// A barrier of `n` threads that tells all of them whether any says so, or all do.
__device__ __forceinline__ bool barrier_or(int id, int n, bool any) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((int)any)
      : "memory");
  return r != 0;
}
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

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Two codes of a word as f16 numbers: bits 0-3 of each half (1024 + c, less 1024),
// or 4-7 (64 + c, less 64).
__device__ __forceinline__ uint32_t low_codes(uint32_t w) {
  return hsub2((w & 0x000f000fu) | 0x64006400u, 0x64006400u);
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w) {
  return hsub2((w & 0x00f000f0u) | 0x54005400u, 0x54005400u);
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}
// The products and the commit of tc_ptx.cuh, by the lane whose `lead` is set.
__device__ __forceinline__ void product_ss(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void product_ts(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}

// A 128-byte swizzled operand's descriptor from its lower word; rows 1024 bytes apart
// by eights.
__device__ __forceinline__ uint64_t descriptor(uint32_t low) {
  return (uint64_t)((1024u >> 4) | 1u << 14 | 2u << 29) << 32 | low;
}

__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// Bit e set when key jc + e is at or before position jc + eb.
__device__ __forceinline__ uint32_t upto_mask(int eb) {
  return eb < 0 ? 0u : eb >= 31 ? 0xffffffffu : (2u << eb) - 1u;
}

// Where the warp's 32 positions of a step lie: two tiles of 16, or nullptr.
template <int D, bool PREFIX>
struct Source {
  const uint8_t* head;           // tile 0 of page 0 of the KV head
  const uint8_t* any;            // of the cache
  const int32_t* table;
  int64_t page_bytes, pages;
  int shift, last, first;        // first: of the warp's positions, within a step
  __device__ Source(const ManyParams& p, const Item& it, int first)
      : table(PREFIX ? p.prefix : p.c.table + (int64_t)it.b * p.c.max_pages), pages(p.c.pages), shift(p.c.page_shift),
        last(it.last), first(first) {
    const int64_t tile = Layout<D>::kTileBytes;
    page_bytes = ((int64_t)p.c.H << (shift - 4)) * tile;
    any = p.c.data;
    head = p.c.data + ((int64_t)it.kvh << (shift - 4)) * tile;
  }
  // the table's entries of step s (-1: none needed)
  __device__ int2 entries(int s, int k0) const {
    const int at = BN * s + first;
    int2 e = make_int2(-1, -1);
    if (s >= k0 && at <= last) {
      e.x = table[at >> shift];
      if (at + kTile <= last) e.y = shift == 4 ? table[(at >> 4) + 1] : e.x;
    }
    return e;
  }
  // tile k of the two (an absent one: some tile, whose codes count for nothing)
  __device__ const uint8_t* tile(int s, int k, int32_t pg, bool& there) const {
    there = pg >= 0 && pg < pages;
    const int in_page = (BN * s + first + kTile * k) & ((1 << shift) - 1);
    return there ? head + pg * page_bytes + (in_page >> 4) * Layout<D>::kTileBytes : any;
  }
};

// N words from global memory.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* at, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 a = *reinterpret_cast<const uint4*>(at);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  } else {
    static_assert(N == 2, "a group of 32 or two");
    const uint2 a = *reinterpret_cast<const uint2*>(at);
    w[0] = a.x, w[1] = a.y;
  }
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

// Prefix: the last position that any sequence of the batch has come to, found by the
// warps that take codes apart while the list is made.  What lies behind it counts for
// nothing, be it not written, not there or no number.
template <int D>
__device__ __forceinline__ void find_tops(const ManyParams& p, Ctl<D>* ctl) {
  const int t = threadIdx.x - 32 * kKWarp;
  int top = -1;
#pragma unroll 4
  for (int b = t; b < p.c.B; b += 2 * kDeqThreads) {
    const int pos = p.pos[b];
    if (pos < p.limit) top = max(top, pos);
  }
  top = __reduce_max_sync(FULL, top);
  if ((t & 31) == 0) ctl->tops[t >> 5] = top;
  barrier_or(BAR_CODES, 2 * kDeqThreads, false);
}
template <int D, bool PREFIX>
__device__ __forceinline__ int last_seen(const Ctl<D>* ctl, int last) {
  if constexpr (PREFIX) {
    int top = -1;
#pragma unroll
    for (int w = 0; w < 2 * kDeqWarps; ++w) top = max(top, ctl->tops[w]);
    last = min(last, top);
  }
  return last;
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
  const uint64_t lim = p.wait_ns, item_lim = p.item_wait_ns;

  if (tid == 0) {
    for (int k = 0; k < 2; ++k) {
      mbar_init(bar(B_IFULL + k), 1);
      mbar_init(bar(B_IEMPTY + k), kSoftWarps + 2 * kDeqWarps + 1);
      mbar_init(bar(B_VREADY + k), kDeqWarps);
      mbar_init(bar(B_VEMPTY + k), 1);
      mbar_init(bar(B_KEMPTY + k), 1);
      mbar_init(bar(B_QFULL + k), kTileThreads);
      mbar_init(bar(B_SFULL + k), 1);
      mbar_init(bar(B_PFULL + k), kTileThreads);
      mbar_init(bar(B_ODONE + k), 1);
    }
    for (int k = 0; k < 4; ++k) {
      mbar_init(bar(B_KREADY + k), kDeqWarps);
      mbar_init(bar(B_INFO + k), 2 * kDeqWarps);
    }
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
  auto share = [&]() {
    const int64_t all = total * p.c.H, fair = (all + gridDim.x - 1) / gridDim.x;
    per = fair < kMinShare ? kMinShare : fair;
    begin = blockIdx.x * per;
    end = min(all, begin + per);
  };
  if constexpr (PREFIX) {
    // (all items are alike, nothing to sum: 64 sequences behind 8192 52.5 -> 51.1 us)
    const int cost = (p.keys + BN - 1) / BN + kItemCost;
    total = (int64_t)entries * cost;
    if (warp == kProdWarp) {
      share();
      const int e = (int)(begin % total / cost);
      ctl->found[0] = e;
      ctl->found[1] = (int64_t)e * cost;
    }
  } else {
    auto cost = [&](int e) -> int {
      int pos, rows, last;
      const int b = e / p.tiles, n = item_steps<false>(p, b, e - b * p.tiles, pos, rows, last);
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
    share();
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
    if (tid == 0) p.ends[blockIdx.x].x = -1;
    // rows without a position: idle sequences', and those past the limit
    for (int b = blockIdx.x; b < p.c.B; b += gridDim.x) {
      int pos;
      const int n = tokens_of(p, b, pos);
      const int rows = p.len == nullptr ? p.m : max(0, min(p.len[b], p.m));
      if (n == rows) continue;
      if (pos >= 0 && tid == 0) atomicOr(p.err, kErrCachePlace);
      const int64_t vecs = (int64_t)(rows - n) * (D / 8);     // of a head
      for (int64_t x = tid; x < vecs * p.Hq; x += kThreads) {
        const int64_t h = x / vecs, v = x - h * vecs;
        reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) +
                                 ((b * (int64_t)p.Hq + h) * p.m + n) * D)[v] = make_uint4(0, 0, 0, 0);
      }
    }
    __syncthreads();
  }

  if (warp >= kMmaWarp) {
    leave_registers<kRegsRest>();
  if (warp == kProdWarp) {
    // ----------------------------------------------------------------- items
    bool ok = true;
    int seq = 0, slot = 2 * blockIdx.x;
    auto publish = [&](const Item& it) {
      const int s = seq & 1;
      ok = __all_sync(FULL, mbar_wait(bar(B_IEMPTY + s), ((uint32_t)(seq >> 1) & 1u) ^ 1u, abort, item_lim));
      if (ok && lane == 0) {
        volatile int* v = reinterpret_cast<volatile int*>(&ctl->ring[s]);
        v[0] = it.valid; v[1] = it.b; v[2] = it.kvh; v[3] = it.row0; v[4] = it.row1;
        v[5] = it.k0; v[6] = it.k1; v[7] = it.pos; v[8] = it.last; v[9] = it.slot;
        mbar_arrive(bar(B_IFULL + s));
      }
      __syncwarp();
      ++seq;
    };
    if (begin < end && !p.stall) {
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
        const bool closes = till == base + cost, whole = t0 == 0 && closes;
        if (!PREFIX && closes && !whole && lane == 0) {
          const int i0 = (int)((base + kItemCost) / per);          // the CTA of its first step
          p.ends[blockIdx.x] = make_int4(kvh * entries + e, i0, base <= i0 * per ? 2 * i0 : 2 * i0 + 1, 0);
        }
        publish(Item{1, b, kvh, kItemRows * t, min(rows, kItemRows * (t + 1)), t0, t1, pos, last,
                     !whole ? slot : PREFIX ? (int)(2 * gridDim.x) + kvh * p.tiles + t : -1});
        slot = 2 * blockIdx.x + 1;
      }
    }
    if (ok && !p.stall) publish(Item{});
    if (!ok && lane == 0) {
      *abort = 1;
      atomicOr(p.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ the products
    // (The whole warp runs this, and one lane's predicate issues: so everything a
    // product takes stays in uniform registers.  With one lane in a branch of its own
    // they were moved there one by one, about 100 cycles a product of 64.  A
    // descriptor's upper word is a constant, its lower one an address / 16 and the
    // leading offset.)
    {
      const uint32_t lead = elect_one();
      const uint32_t tm = __shfl_sync(FULL, tmem, 0);
      constexpr uint32_t id_s = idesc_f16_f32(BM, BN, 0, 0), id_pv = idesc_f16_f32(BM, D, 0, 1);
      const uint32_t base = (__shfl_sync(FULL, sbase, 0) >> 4) & 0x3fffu;
      auto issue_s = [&](int tile, uint32_t kb) {
        const uint32_t q = (base + ((S::kQ + tile * S::kTileB) >> 4)) | (16u >> 4) << 16;
        const uint32_t k = (base + ((S::kK + kb * S::kTileB) >> 4)) | (16u >> 4) << 16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
          product_ss(lead, tm + tile * BN, descriptor(q + off), descriptor(k + off), id_s, kk > 0 ? 1u : 0u);
        }
        commit(lead, bar(B_SFULL + tile));
      };
      auto issue_pv = [&](int tile, uint32_t first, uint32_t vb) {
        const uint32_t v = (base + ((S::kV + vb * S::kTileB) >> 4)) | (kHalf >> 4) << 16;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          product_ts(lead, tm + kColO + tile * 128, tm + tile * BN + kColP + kk * 8,
                     descriptor(v + kk * (2048 >> 4)), id_pv, kk == 0 ? 1u - first : 1u);
      };
      auto wait = [&](int k, uint32_t parity) -> bool {
        return __all_sync(FULL, mbar_wait(bar(k), parity, abort, lim));
      };
      bool ok = true;
      // steps, steps with both tiles; items, items with both tiles (an item that leaves
      // the second tile out completes no phase of that tile's barriers)
      uint32_t g = 0, gb = 0, seq = 0, seqb = 0;
      int jj = 0, steps = 0;                     // step of the item, its steps (0: the end)
      bool two = false, ptwo = false, pfirst = false, plast = false;      // p: of the step before
      auto next_item = [&]() {
        ok = __all_sync(FULL, mbar_wait(bar(B_IFULL + (seq & 1)), (seq >> 1) & 1u, abort, item_lim));
        const volatile Item& it = ctl->ring[seq & 1];
        steps = __shfl_sync(FULL, ok && it.valid ? it.k1 - it.k0 : 0, 0);
        two = __shfl_sync(FULL, it.row1 - it.row0, 0) > BM;
        jj = 0;
      };
      // P V of the step before, tile A or B
      auto close_a = [&]() -> bool {
        const uint32_t vb = (g - 1) & 1;
        if (!wait(B_VREADY + vb, ((g - 1) >> 1) & 1u) || !wait(B_PFULL, (g - 1) & 1u)) return false;
        tc_fence_after();
        issue_pv(0, pfirst, vb);
        if (plast) commit(lead, bar(B_ODONE));
        if (!ptwo) commit(lead, bar(B_VEMPTY + vb));
        return true;
      };
      auto close_b = [&]() -> bool {
        const uint32_t vb = (g - 1) & 1;
        if (ptwo) {
          if (!wait(B_PFULL + 1, (gb - 1) & 1u)) return false;
          tc_fence_after();
          issue_pv(1, pfirst, vb);
          commit(lead, bar(B_VEMPTY + vb));
          if (plast) commit(lead, bar(B_ODONE + 1));
        }
        return true;
      };
      next_item();
      uint32_t done = 0;                         // items whose slot was released
      while (ok && steps > 0) {
        // (K first, which is ready long before: nothing stands between the two products)
        ok = wait(B_KREADY + (g & 3), (g >> 2) & 1u);
        if (!ok || (g > 0 && !(ok = close_a()))) break;
        if (jj == 0) ok = wait(B_QFULL, seq & 1u);
        if (!ok) break;
        tc_fence_after();
        issue_s(0, g & 1);
        if (!two) commit(lead, bar(B_KEMPTY + (g & 1)));
        if (g > 0) {
          if (!(ok = close_b())) break;
          if (plast && lead) mbar_arrive(bar(B_IEMPTY + (done & 1)));
          if (plast) ++done;
        }
        if (two) {
          if (jj == 0) ok = wait(B_QFULL + 1, seqb++ & 1u);
          if (!ok) break;
          tc_fence_after();
          issue_s(1, g & 1);
          commit(lead, bar(B_KEMPTY + (g & 1)));
          ++gb;
        }
        pfirst = jj == 0;
        ptwo = two;
        ++g;
        plast = ++jj == steps;
        if (plast) {
          ++seq;
          next_item();
        }
      }
      if (ok && g > 0) ok = close_a() && close_b();
      if (ok && g > 0 && lead) mbar_arrive(bar(B_IEMPTY + (done & 1)));
      if (!ok && lead) {
        *abort = 1;
        atomicOr(p.err, kErrTimeout);
      }
      // every product of this thread has completed once this arrives
      commit(lead, bar(B_DRAIN));
      mbar_drain(bar(B_DRAIN), 0);
    }
    __syncwarp();
  }
  } else if (warp >= kVWarp) {
    leave_registers<kRegsDeq>();
    // ------------------------------------------------- V's codes into f16 tiles
    const int dw = warp - kVWarp, t = 32 * dw + lane;            // t: a position of the step
    if constexpr (PREFIX) find_tops<D>(p, ctl);
    bool ok = true, range = false;
    int g = 0;
    float unit[Y];                       // 2^-R_y
#pragma unroll
    for (int y = 0; y < Y; ++y) unit[y] = 1.f;
    for (int seq = 0; ok; ++seq) {
      const int islot = seq & 1;
      ok = mbar_wait(bar(B_IFULL + islot), (uint32_t)(seq >> 1) & 1u, abort, item_lim);
      ok = barrier_and(BAR_V, kDeqThreads, ok);
      if (!ok) break;
      const Item it = read_item(ctl->ring, islot);
      if (!it.valid) break;
      const Source<D, PREFIX> src(p, it, 32 * dw);
      const int last = last_seen<D, PREFIX>(ctl, it.last);
      uint32_t pairs[Y], code[Y][4];       // of tile i / (Y / 2), groups 2 (i % (Y / 2)) and the next
      bool there;                          // whether this lane's position is
      const int pair_at = Layout<D>::kVPairs + Layout<D>::pair(lane & 15, 0);
      auto load = [&](int s, int2 e) {
        bool h0, h1;
        const uint8_t *t0 = src.tile(s, 0, e.x, h0), *t1 = src.tile(s, 1, e.y, h1);
        there = lane < 16 ? h0 : h1;
        load_words<Y>((lane < 16 ? t0 : t1) + pair_at, pairs);
        t0 += lane * 16;
        t1 += lane * 16;
#pragma unroll
        for (int i = 0; i < Y; ++i) load_words<4>((i < Y / 2 ? t0 : t1) + Layout<D>::kV + i % (Y / 2) * 512, code[i]);
      };
      load(it.k1 - 1, src.entries(it.k1 - 1, it.k0));
      int2 ahead = src.entries(it.k1 - 2, it.k0);
      for (int s = it.k1 - 1; s >= it.k0; --s, ++g) {
        const int st = g & 1;
        // -- this position's pairs
        const bool counts = BN * s + t <= last && there;
        uint32_t vw[Y];
#pragma unroll
        for (int y = 0; y < Y; ++y) vw[y] = pairs[y];
        int bad = 0;
        uint32_t seen = 0;                   // groups that are not 0, and of these the ones within reach of R_y
        float top[Y], most = 0.f;            // largest magnitudes: of the groups, of all in units of 2^R_y
#pragma unroll
        for (int y = 0; y < Y; ++y) {
          if (!counts) vw[y] = 0;
          // (at one of a group's ends; a NaN of either number is one of hi)
          const float hi = fmaf(15.f, pair_step(vw[y]), pair_lo(vw[y]));
          top[y] = fmaxf(fabsf(pair_lo(vw[y])), fabsf(hi));
          if (!(top[y] <= 3.402823466e38f) || hi != hi) {
            bad |= 1 << y;
            vw[y] = 0;
            top[y] = 0.f;
          }
          const float r = top[y] * unit[y];
          most = fmaxf(most, r);
          if (top[y] > 0.f) seen |= (r >= kVBelow ? 0x101u : 0x100u) << y;
        }
        // -- R_y: kept while every group of every 32 positions is near it, else moved
        // to the step's largest (an item's first step takes this way always)
        const bool first = s == it.k1 - 1;
        uint32_t all = 0;
        bool moved = false, near = false;
        if (!first) {
          all = __reduce_max_sync(FULL, __float_as_uint(most));
          seen = __reduce_or_sync(FULL, seen);
          near = (int)(all >> 23) - 127 < kVAbove && ((seen >> 8) & ~seen & 0xffu) == 0;
          near = barrier_and(BAR_V, kDeqThreads, ok && near);
        }
        if (!near) {
          // (lane y: group y)
          const int y0 = lane & (Y - 1);
          int own = kNoGroup, unit_of = 0;
#pragma unroll
          for (int y = 0; y < Y; ++y) {
            top[y] = fmaxf(fabsf(pair_lo(vw[y])), fabsf(fmaf(15.f, pair_step(vw[y]), pair_lo(vw[y]))));
            const uint32_t a = __reduce_max_sync(FULL, __float_as_uint(top[y]));
            if (y0 == y) {
              own = a == 0 ? kNoGroup : max((int)(a >> 23) - 127, -100);
              unit_of = __float_as_int(unit[y]);
            }
          }
          if (lane < Y) ctl->vmax[dw][lane] = own;
          const int high = first ? kNoGroup : ctl->vhigh[y0], now = 127 - (unit_of >> 23);
          int low = first ? -kNoGroup : ctl->vlow[y0];
          // (a wait that ran out is told to the other warps here, or behind the item)
          ok = barrier_and(BAR_V, kDeqThreads, ok);
          if (!ok) break;
          int e = kNoGroup;
#pragma unroll
          for (int w = 0; w < kDeqWarps; ++w) {
            const int v = ctl->vmax[w][y0];
            e = max(e, v);
            low = v == kNoGroup ? low : min(low, v);
          }
          const int base = __reduce_max_sync(FULL, e);
          const int none = !first ? now : base == kNoGroup ? 0 : min(base, 110);
          const int rise = max(0, min(e - low - kVRise, kVRiseMost));
          const int to = e == kNoGroup ? none : min(max(e - rise, high - kVSpan), 110);
          moved = __any_sync(FULL, !first && to != now);
          if (t < Y) {
            ctl->vr[islot][t] = to - 14;
            ctl->vhigh[t] = e == kNoGroup ? high : max(high, to);
            ctl->vlow[t] = low;
            ctl->vscale[g & 3][t] = pow2(now - to);
          }
          most = 0.f;
#pragma unroll
          for (int y = 0; y < Y; ++y) {
            unit[y] = pow2(-__shfl_sync(FULL, to, y));
            most = fmaxf(most, top[y] * unit[y]);
          }
          all = __reduce_max_sync(FULL, __float_as_uint(most));
          const int ev = all == 0 ? 0 : max(-48, min(48, (int)(all >> 23) - 127));
          range = range || __any_sync(FULL, own != kNoGroup && to + ev - own > kVLost);
        }
        const int ev = all == 0 ? 0 : max(-48, min(48, (int)(all >> 23) - 127));
        const bool any_bad = __any_sync(FULL, bad != 0);
        if (any_bad || moved) {
#pragma unroll
          for (int y = 0; y < Y; ++y) {
            const uint32_t w = __ballot_sync(FULL, (bad >> y) & 1);
            if (lane == 0) ctl->vnan[g & 3][y][dw] = w;
          }
          if (lane == 0) ctl->vmoved[g & 3][dw] = moved;
        }
        const float down = pow2(-ev), to = down * 0x1p14f;       // largest below 2^15
#pragma unroll
        for (int y = 0; y < Y; ++y) {
          const float up = unit[y] * to, vs = pair_step(vw[y]) * up, vl = pair_lo(vw[y]) * up;
          ctl->vq[y][t] = make_uint2(pack_f16(vs, vs), pack_f16(vl, vl));
        }
        if (lane == 0)
          ctl->vinfo[g & 3][dw] = make_uint2(__float_as_uint((float)ev), __float_as_uint(any_bad || moved ? -down : down));
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_INFO + (g & 3)));
        // -- a lane a quarter group of two neighbouring groups, four positions; the
        // codes are in registers before the tile is free
        ok = __all_sync(FULL, mbar_wait(bar(B_VEMPTY + st), ((uint32_t)(g >> 1) & 1u) ^ 1u, abort, lim));
        if (ok) {
          const int gq = lane >> 2, tq = lane & 3;
          const uint32_t row0 = sbase + S::kV + st * S::kTileB + (dw * 32 + 2 * tq) * 128;
          const uint32_t dst[2] = {row0 + ((gq ^ (2 * tq)) << 4), row0 + 128 + ((gq ^ (2 * tq + 1)) << 4)};
          const uint32_t scales = smem_u32(&ctl->vq[0][dw * 32 + 2 * tq]);
          // (step, lo of two positions and two groups, read one turn ahead: these
          // accesses stay in the order written)
          uint4 q0 = ld_shared_v4(scales), q1 = ld_shared_v4(scales + BN * 8);
#pragma unroll
          for (int n = 0; n < 2 * Y; ++n) {
            const int blk = n & 1, i = n >> 1, yy = i % (Y / 2), tile = i / (Y / 2);
            const uint32_t w0 = code[i][blk], w1 = code[i][2 + blk];
            const uint4 a = q0, b = q1;
            if (n + 1 < 2 * Y) {
              const int i1 = (n + 1) >> 1;
              const uint32_t at = scales + (2 * (i1 % (Y / 2)) * BN + i1 / (Y / 2) * 16 + ((n + 1) & 1) * 8) * 8;
              q0 = ld_shared_v4(at);
              q1 = ld_shared_v4(at + BN * 8);
            }
            uint32_t v[2][4];
#pragma unroll
            for (int par = 0; par < 2; ++par) {
              const uint32_t x0 = __byte_perm(w0, 0, par ? 0x4342 : 0x4140);
              const uint32_t x1 = __byte_perm(w1, 0, par ? 0x4342 : 0x4140);
              const uint32_t s0 = par ? a.z : a.x, l0 = par ? a.w : a.y;
              const uint32_t s1 = par ? b.z : b.x, l1 = par ? b.w : b.y;
              v[par][0] = hfma2(low_codes(x0), s0, l0);
              v[par][1] = hfma2(high_codes(x0), s0, l0);
              v[par][2] = hfma2(low_codes(x1), s1, l1);
              v[par][3] = hfma2(high_codes(x1), s1, l1);
            }
#pragma unroll
            for (int par = 0; par < 2; ++par)
              st_shared_v4(dst[par] + yy * kHalf + (tile * 16 + blk * 8) * 128, v[par][0], v[par][1], v[par][2], v[par][3]);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_VREADY + st));
        }
        if (s > it.k0) load(s - 1, ahead);
        ahead = src.entries(s - 2, it.k0);
      }
      if (!ok && lane == 0) *abort = 1;
      ok = barrier_and(BAR_V, kDeqThreads, ok);
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
  } else if (warp >= kKWarp) {
    leave_registers<kRegsDeq>();
    // ------------------------------------------------- K's codes into f16 tiles
    // (a warp takes its own 32 positions apart: nothing to tell the others)
    const int dw = warp - kKWarp, t = 32 * dw + lane;
    if constexpr (PREFIX) find_tops<D>(p, ctl);
    bool ok = true;
    int g = 0;
    for (int seq = 0; ok; ++seq) {
      const int islot = seq & 1;
      ok = __all_sync(FULL, mbar_wait(bar(B_IFULL + islot), (uint32_t)(seq >> 1) & 1u, abort, item_lim));
      if (!ok) break;
      const Item it = read_item(ctl->ring, islot);
      if (!it.valid) break;
      const Source<D, PREFIX> src(p, it, 32 * dw);
      const int last = last_seen<D, PREFIX>(ctl, it.last);
      // a lane a position and a quarter of each group; eight positions a turn, bit 2
      // of the position in bit 2 of the lane, so that eight lanes' stores lie in eight
      // different banks; two turns a tile
      const int u = lane & 3, r8 = (lane & 4) | ((lane >> 3) & 3);
      uint32_t kp[Y], code[4][Y];
      bool there;                          // whether this lane's position is
      const int pair_at = Layout<D>::kKPairs + Layout<D>::pair(lane & 15, 0);
      auto load = [&](int s, int2 e) {
        bool h0, h1;
        const uint8_t *t0 = src.tile(s, 0, e.x, h0), *t1 = src.tile(s, 1, e.y, h1);
        there = lane < 16 ? h0 : h1;
        // (pages that are needed and not there are told once, by K's warps)
        if (!there && BN * s + t <= last) atomicOr(p.err, kErrCachePlace);
        load_words<Y>((lane < 16 ? t0 : t1) + pair_at, kp);
        t0 += r8 * (D / 2) + u * (D / 8);
        t1 += r8 * (D / 2) + u * (D / 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) load_words<Y>((i < 2 ? t0 : t1) + (i & 1) * 4 * D, code[i]);
      };
      load(it.k1 - 1, src.entries(it.k1 - 1, it.k0));
      int2 ahead = src.entries(it.k1 - 2, it.k0);
      for (int s = it.k1 - 1; s >= it.k0; --s, ++g) {
        const int st = g & 1, ring = g & 3;
        const bool counts = BN * s + t <= last && there;
        uint32_t kw[Y];
#pragma unroll
        for (int y = 0; y < Y; ++y) kw[y] = kp[y];
        float top = 0.f;
#pragma unroll
        for (int y = 0; y < Y; ++y) {
          if (!counts) kw[y] = 0;
          const float k = fmaxf(fabsf(pair_lo(kw[y])), fabsf(fmaf(15.f, pair_step(kw[y]), pair_lo(kw[y]))));
          if (k <= 3.402823466e38f) top = fmaxf(top, k);
        }
        // the warp's largest below 2^15
        const int e = min(max((int)(__reduce_max_sync(FULL, __float_as_uint(top)) >> 23) - 127, -100), 126);
        const float up = pow2(14 - e);
#pragma unroll
        for (int y = 0; y < Y; ++y) {
          const float step = pair_step(kw[y]) * up, lo = pair_lo(kw[y]) * up;
          ctl->kq[t][y] = make_uint2(pack_f16(step, step), pack_f16(lo, lo));
        }
        const uint32_t positions = __ballot_sync(FULL, counts);
        ok = __all_sync(FULL, mbar_wait(bar(B_KEMPTY + st), ((uint32_t)(g >> 1) & 1u) ^ 1u, abort, lim));
        if (!ok) break;
        if (lane == 0) ctl->kinfo[ring][dw] = make_uint2(__float_as_uint(pow2(e - 14)), positions);
        __syncwarp();
        const uint32_t dst = sbase + S::kK + st * S::kTileB + (dw * 32 + r8) * 128 + ((u ^ r8) << 4);     // of even groups
        const uint32_t pairs = smem_u32(&ctl->kq[dw * 32 + r8][0]);
        // (step, lo of two groups, read one turn ahead)
        uint4 next = ld_shared_v4(pairs);
#pragma unroll
        for (int n = 0; n < 4 * (Y / 2); ++n) {
          const int i = n / (Y / 2), yy = n % (Y / 2);
          const uint4 k = next;
          if (n + 1 < 4 * (Y / 2)) next = ld_shared_v4(pairs + (n + 1) / (Y / 2) * 8 * Y * 8 + (n + 1) % (Y / 2) * 16);
          uint32_t v[2][4];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t w = code[i][2 * yy + y], hi = w >> 8, s = y ? k.z : k.x, l = y ? k.w : k.y;
            v[y][0] = hfma2(low_codes(w), s, l);
            v[y][1] = hfma2(high_codes(w), s, l);
            v[y][2] = hfma2(low_codes(hi), s, l);
            v[y][3] = hfma2(high_codes(hi), s, l);
          }
          st_shared_v4(dst + yy * kHalf + i * 1024, v[0][0], v[0][1], v[0][2], v[0][3]);
          st_shared_v4((dst ^ 64u) + yy * kHalf + i * 1024, v[1][0], v[1][1], v[1][2], v[1][3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(B_KREADY + ring));
          mbar_arrive(bar(B_INFO + ring));
        }
        if (s > it.k0) load(s - 1, ahead);
        ahead = src.entries(s - 2, it.k0);
      }
      if (!ok) break;
      if (lane == 0) mbar_arrive(bar(B_IEMPTY + islot));
    }
    if (!ok && lane == 0) {
      *abort = 1;
      atomicOr(p.err, kErrTimeout);
    }
    __syncwarp();
  } else {
    take_registers<kRegsSoftmax>();
    // ------------------------------------------------------ softmax, epilogue
    const int tile = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_col = tmem + lane_base + tile * BN + 64 * half, p_col = tmem + lane_base + tile * BN + kColP + 32 * half;
    const uint32_t o_col = tmem + lane_base + kColO + tile * 128;
    const int pair = BAR_PAIR + tile * 4 + quarter;
    const float norm = kLog2e * (D == 64 ? 0.125f : 0.08838834764831845f);
    bool ok = true;
    uint32_t g = 0, gt = 0, items = 0;   // steps, this tile's steps and items
    for (int seq = 0; ok; ++seq) {
      const int islot = seq & 1;
      // (whether a wait ran out is told to the two warps of a row, which alone share
      // barriers without a limit, before either leaves)
      ok = mbar_wait(bar(B_IFULL + islot), (uint32_t)(seq >> 1) & 1u, abort, item_lim);
      ok = barrier_and(pair, 64, ok);
      if (!ok) break;
      const Item it = read_item(ctl->ring, islot);
      if (!it.valid) break;
      const int row = it.row0 + tile * BM + r;
      if (tile == 1 && it.row1 - it.row0 <= BM) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_IEMPTY + islot));
        g += it.k1 - it.k0;
        continue;
      }
      // -- the row's query
      bool row_ok = row < it.row1, row_bad = false;
      int h = 0, pos = -1;
      int64_t at = 0;
      float slope = 0.f, qs;                 // qs: what q's power of two leaves of the scores' scale
      if (row_ok) {
        at = row_at<PREFIX, D>(p, it.b, it.kvh, it.pos, row, h, pos);
        slope = p.slope[h];
        row_ok = pos >= 0;
      }
      {
        // (half of the row)
        uint4 qv[D / 16];
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + at) + half * (D / 16);
        uint32_t mx = 0;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          qv[c] = row_ok ? src[c] : make_uint4(0, 0, 0, 0);
          mx = __vmaxu2(mx, qv[c].x & 0x7fff7fffu);
          mx = __vmaxu2(mx, qv[c].y & 0x7fff7fffu);
          mx = __vmaxu2(mx, qv[c].z & 0x7fff7fffu);
          mx = __vmaxu2(mx, qv[c].w & 0x7fff7fffu);
        }
        mx = max(mx & 0xffff0000u, mx << 16);
        // (each row's own: behind a prefix a tile's rows are several requests')
        ctl->pair[tile][half][r] = __uint_as_float(mx);
        ok = barrier_and(pair, 64, ok);
        mx = max(mx, __float_as_uint(ctl->pair[tile][half ^ 1][r]));
        row_bad = mx >= (110u + 127u) << 23;             // 2^110, infinities, NaN
        const int e = min(max((int)(mx >> 23) - 127, -100), 110);
        const float up = row_bad ? 0.f : pow2(14 - e);
        qs = pow2(e - 14) * norm;
        const uint32_t dst = sbase + S::kQ + tile * S::kTileB + r * 128;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int c = half * (D / 16) + i;
          const uint32_t w[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
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
      if (!row_ok) {                         // (a row of no one: it sees everything, and is not written)
        pos = 1 << 30;
        slope = 0.f;
      }
      const int pos_min = __reduce_min_sync(FULL, pos);
      const uint64_t rise2 = f2_pack(2.f * slope, 2.f * slope), rise4 = f2_pack(4.f * slope, 4.f * slope);      // of the bias
      float m_ref = -INFINITY, l = 0.f;
      int nan_groups = 0;
      for (int s = it.k1 - 1; s >= it.k0; --s, ++g, ++gt) {
        const int j0 = s * BN + 64 * half;               // this thread's keys: 64 from here
        const uint32_t kinfo = smem_u32(&ctl->kinfo[g & 3][2 * half]), vinfo = smem_u32(&ctl->vinfo[g & 3][2 * half]);
        // (The scores first: a tile that was left out of the item before runs ahead of
        // the others, and only behind its own scores is the step's phase of the scales'
        // barrier the next to complete.)
        ok = mbar_wait(bar(B_SFULL + tile), gt & 1u, abort, lim) &&
             mbar_wait(bar(B_INFO + (g & 3)), (g >> 2) & 1u, abort, lim);
        ok = __all_sync(FULL, ok);
        tc_fence_after();
        float mu = m_ref == -INFINITY ? 0.f : m_ref, sum;
        // The step's weights, kept in registers until it is known that the reference
        // they are taken against stands, for both threads of a row: they are below 2^15,
        // and the row has one.  Else the reference moves to the step's maximum, O and l
        // follow, and the weights are taken again (at the start of a piece, and where
        // scores jump).
        uint32_t pk[32], most;
        int rare = 0;
        // exponents of sixteen keys, x + ev - mu, -inf where masked (if any are)
        auto exponents = [&](auto masked, int c, const uint32_t (&rr)[16], uint2 kq, float ev, float (&x)[16]) {
          const int jc = j0 + 16 * c;
          const float cs = fminf(__uint_as_float(kq.x) * qs, 3.402823466e38f);
          const uint64_t cs2 = f2_pack(cs, cs);
          const float off = fmaf((float)(jc - pos), slope, ev - mu);
          uint64_t b[2];
          b[0] = f2_pack(off, off + slope);
          b[1] = f2_add(b[0], rise2);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f2_unpack(f2_fma(f2_pack(__uint_as_float(rr[2 * e]), __uint_as_float(rr[2 * e + 1])), cs2, b[e & 1]),
                      x[2 * e], x[2 * e + 1]);
            b[e & 1] = f2_add(b[e & 1], rise4);
          }
          if constexpr (decltype(masked)::value) {
            const uint32_t vm = upto_mask(pos - jc) & (kq.y >> (16 * (c & 1)));
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (!(vm & (1u << e))) x[e] = -INFINITY;
          }
        };
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          most = 0;
          sum = 0.f;
          const uint4 kk = ld_shared_v4(kinfo), vv = ld_shared_v4(vinfo);
          rare = (int)(vv.y | vv.w);
          auto take = [&](auto masked) {
            uint32_t ra[16], rb[16];
            tmem_ld16(s_col, ra);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t(&rr)[16] = c & 1 ? rb : ra;
              const uint2 kq = c < 2 ? make_uint2(kk.x, kk.y) : make_uint2(kk.z, kk.w);
              const uint2 vq = c < 2 ? make_uint2(vv.x, vv.y) : make_uint2(vv.z, vv.w);
              tmem_wait_ld();
              if (c < 3) tmem_ld16(s_col + 16 * (c + 1), c & 1 ? ra : rb);
              float x[16];
              exponents(masked, c, rr, kq, __uint_as_float(vq.x), x);
              uint64_t t[2];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float u = ex2(x[2 * e]), v = ex2(x[2 * e + 1]);
                t[e & 1] = e < 2 ? f2_pack(u, v) : f2_add(t[e & 1], f2_pack(u, v));
                pk[8 * c + e] = pack_f16(u, v);
                if (e & 1) most = __vimax3_u16x2(most, pk[8 * c + e - 1], pk[8 * c + e]);
              }
              float s0, s1;
              f2_unpack(f2_add(t[0], t[1]), s0, s1);
              sum = fmaf(s0 + s1, fabsf(__uint_as_float(vq.y)), sum);
            }
          };
          // (One decision a step: with one every sixteen keys nothing moved across it,
          // 2550 us against 2430 for 2048 tokens behind 63488.)
          if (pos_min < j0 + 63 || (kk.y & kk.w) != FULL)
            take(std::true_type());
          else
            take(std::false_type());
          const bool fresh = m_ref == -INFINITY;
          // does a weight reach 2^15 (or is it no number)?  or has the row no reference?
          const bool grow = fresh || ((most + 0x08000800u) & 0x80008000u) != 0;
          // (also: both have read the scores that the weights are written over)
          tc_fence_before();
          const bool again = barrier_or(pair, 64, grow || !ok);
          tc_fence_after();
          if (!again) break;
          float top = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t rr[16];
            float x[16];
            tmem_ld16(s_col + 16 * c, rr);
            const uint2 kc = ld_shared_v2(kinfo + 8 * (c >> 1)), vc = ld_shared_v2(vinfo + 8 * (c >> 1));
            tmem_wait_ld();
            exponents(std::true_type(), c, rr, kc, __uint_as_float(vc.x), x);
#pragma unroll
            for (int e = 0; e < 16; e += 2) top = max3(top, x[e], x[e + 1]);
          }
          ctl->pair[tile][half][r] = top;
          ok = barrier_and(pair, 64, ok);
          if (!ok) break;
          top = fmaxf(top, ctl->pair[tile][half ^ 1][r]);
          // (to no less than the maximum, whatever its own rounding: a second pass is
          // the last; the bound is for the third that no row needs)
          const bool move = pass < 2 && (top > kGrowLog2 || (fresh && top > -INFINITY));
          const float d = move ? fmaf(fabsf(mu + top), 0x1p-20f, top) : 0.f, f = fresh ? 0.f : ex2(-d);
          mu += d;
          if (move) m_ref = mu;
          l *= f;
          // (the commit behind these scores proves that P V of the step before is done)
#pragma unroll 1
          for (int k = s < it.k1 - 1 ? 0 : D / 32; k < D / 32; ++k) {
            uint32_t o[16];
            tmem_ld16(o_col + half * (D / 2) + k * 16, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(o_col + half * (D / 2) + k * 16, o);
          }
          if (!barrier_or(pair, 64, move)) break;          // (a row that sees nothing yet)
        }
        if (!ok) break;
        tmem_st32(p_col, pk);
        if (rare < 0) {
          // (before the arrival: behind it the products may hand the step's slot on)
          bool moved = false;
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            if ((int)ld_shared_u32(vinfo + 8 * q + 4) >= 0) continue;      // a group of V that is no number, or R_y moved
            moved = moved || ctl->vmoved[g & 3][2 * half + q] != 0;
            const uint32_t vm = upto_mask(pos - j0 - 32 * q) & ld_shared_u32(kinfo + 8 * q + 4);
            for (int y = 0; y < Y; ++y)
              if (ctl->vnan[g & 3][y][2 * half + q] & vm) nan_groups |= 1 << y;
          }
          if (moved && s < it.k1 - 1) {
            const int y = D == 64 ? 0 : 2 * half;          // (columns in turn, four of a group)
            const float f0 = ctl->vscale[g & 3][y], f1 = ctl->vscale[g & 3][y + 1];
#pragma unroll 1
            for (int k = 0; k < D / 32; ++k) {
              uint32_t o[16];
              tmem_ld16(o_col + half * (D / 2) + k * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * (e & 4 ? f1 : f0));
              tmem_st16(o_col + half * (D / 2) + k * 16, o);
            }
          }
        }
        l += sum;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(B_PFULL + tile));
      }
      if (!ok) break;
      // -- the row
      ok = mbar_wait(bar(B_ODONE + tile), items & 1u, abort, lim);
      // both threads' row sums and groups that are no numbers
      ctl->pair[tile][half][r] = l;
      ok = barrier_and(pair, 64, ok);
      if (!ok) break;
      ++items;
      tc_fence_after();
      l += ctl->pair[tile][half ^ 1][r];
      barrier_or(pair, 64, false);
      ctl->pair[tile][half][r] = __int_as_float(nan_groups);
      barrier_or(pair, 64, false);
      nan_groups |= __float_as_int(ctl->pair[tile][half ^ 1][r]);
      if (row_bad) l = NAN;
      const bool whole = it.slot < 0;
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      float* part = p.part + (int64_t)it.slot * part_floats<D>();
      const int pr = tile * BM + r;                        // row of the piece
      float up[Y];
#pragma unroll
      for (int y = 0; y < Y; ++y) up[y] = (nan_groups >> y) & 1 ? NAN : pow2(ctl->vr[islot][y]) * inv;
#pragma unroll 1
      for (int q = half * (D / 64); q < (half + 1) * (D / 64); ++q) {      // half of the columns
        uint32_t o[32];
        tmem_ld32(o_col + q * 32, o);
        tmem_wait_ld();
        // columns 8 c .. 8 c + 7 of O are values 4 g .. 4 g + 3 of groups y and y + 1,
        // c = 4 y + g, in the order 0, 2, 1, 3: here four quarters of each
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
        } else if (row_ok) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float u = c & 1 ? u1 : u0;
            reinterpret_cast<float4*>(part)[(8 * q + c) * kItemRows + pr] =
                make_float4(__uint_as_float(o[4 * c]) * u, __uint_as_float(o[4 * c + 1]) * u,
                            __uint_as_float(o[4 * c + 2]) * u, __uint_as_float(o[4 * c + 3]) * u);
          }
        }
      }
      if (!whole && half == 0) {
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
// A lane a row of 32 rows of an item.  Few pieces: a warp every eighth of the columns'
// quads (4 columns), all pieces.  kSplit pieces or more: a warp every eighth of the
// pieces of two quads, the warps' sums joined in their order; a CTA for each two quads.
// So an item that all CTAs work on (one sequence behind a long context) is read by many
// threads, with loads of several pieces in flight: one CTA for all columns and pieces
// took longer than the attention itself (131072 keys, one KV head: 100 of 121 us).
// (64 sequences behind a prefix of 8192, 16 pieces an item: 4 or 8 -> 55 us, 16 -> 59;
// 512 tokens behind 7680, 4 to 5: 4 -> 108, 8 -> 104.)
constexpr int kJoinThreads = 256, kSplit = 8;

template <int D>
__device__ __forceinline__ void store4(__nv_bfloat16* o, int quad, const float4& a) {
  // quad c: values 4 g .. 4 g + 3 of group y, in the order 0, 2, 1, 3
  const int c = quad >> 1, y = 2 * (c >> 3) + (quad & 1), g = c & 7;
  *reinterpret_cast<uint2*>(o + 32 * y + 4 * g) = make_uint2(pack_bf16(a.x, a.z), pack_bf16(a.y, a.w));
}

// A row's sum of pieces: maximum, sum of weights, columns of NQ quads.
template <int NQ>
struct RowSum {
  float m = kNothing, l = 0.f;
  float4 o[NQ];
  __device__ RowSum() {
#pragma unroll
    for (int c = 0; c < NQ; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ void scale(float f) {
    l *= f;
#pragma unroll
    for (int c = 0; c < NQ; ++c) o[c].x *= f, o[c].y *= f, o[c].z *= f, o[c].w *= f;
  }
  __device__ static void add(float4& a, float f, const float4& v) {
    a.x = fmaf(f, v.x, a.x);
    a.y = fmaf(f, v.y, a.y);
    a.z = fmaf(f, v.z, a.z);
    a.w = fmaf(f, v.w, a.w);
  }
};

// Pieces first, first + every, .. of n; quads q0, q0 + stride, ..
template <int D, int NQ, typename Piece>
__device__ __forceinline__ void add_pieces(RowSum<NQ>& a, Piece piece, int first, int every, int n, int pr, int q0,
                                           int stride) {
  float mm = kNothing;
#pragma unroll 8
  for (int k = first; k < n; k += every) mm = fmaxf(mm, piece(k)[kItemRows * D + pr]);
  a.m = mm;
#pragma unroll 4
  for (int k = first; k < n; k += every) {
    const float* pt = piece(k);
    const float l = pt[kItemRows * (D + 1) + pr], f = l == 0.f ? 0.f : ex2(pt[kItemRows * D + pr] - mm);
    a.l = fmaf(f, l, a.l);
#pragma unroll
    for (int c = 0; c < NQ; ++c) {
      float4 v = reinterpret_cast<const float4*>(pt)[(q0 + stride * c) * kItemRows + pr];
      if (l == 0.f) v = make_float4(0.f, 0.f, 0.f, 0.f);       // (not written, or of nothing)
      RowSum<NQ>::add(a.o[c], f, v);
    }
  }
}

// The warps' sums of a row (two quads), and the row.
template <int D>
__device__ __forceinline__ void join_warps(const RowSum<2>& a, __nv_bfloat16* o, int q0, bool there) {
  __shared__ float ms[8][32], ls[8][32];
  __shared__ float4 os[2][8][32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();                       // (another unit's were read)
  ms[w][lane] = a.m;
  ls[w][lane] = a.l;
  os[0][w][lane] = a.o[0];
  os[1][w][lane] = a.o[1];
  __syncthreads();
  if (w >= 2 || !there) return;
  float mm = kNothing, sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) mm = fmaxf(mm, ms[i][lane]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float l = ls[i][lane], f = l == 0.f ? 0.f : ex2(ms[i][lane] - mm);
    sum = fmaf(f, l, sum);
    RowSum<2>::add(acc, f, os[w][i][lane]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  store4<D>(o, q0 + w, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
}

template <int D, int NQ>
__device__ __forceinline__ void store_row(const RowSum<NQ>& a, __nv_bfloat16* o, int q0, int stride) {
  const float inv = a.l == 0.f ? 0.f : 1.f / a.l;
#pragma unroll
  for (int c = 0; c < NQ; ++c)
    store4<D>(o, q0 + stride * c, make_float4(a.o[c].x * inv, a.o[c].y * inv, a.o[c].z * inv, a.o[c].w * inv));
}

// Units (32 rows of an item, and two quads where its pieces are many) of all the items
// that end in a CTA, a CTA every gridDim.x-th.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) q4_many_join_kernel(const __grid_constant__ ManyParams p, int ctas) {
  grid_dep_wait();
  __shared__ int starts[kJoinThreads + 1], sums[kJoinThreads / 32];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, entries = p.c.B * p.tiles;
  auto rows_of = [&](const int4& end, int& e, int& kvh, int& b, int& pos) {      // rows of the item
    kvh = end.x / entries;
    e = end.x - kvh * entries;
    b = e / p.tiles;
    int rows, last;
    item_steps<false>(p, b, e - b * p.tiles, pos, rows, last);
    return min(rows - kItemRows * (e - b * p.tiles), kItemRows);
  };
  int units = 0;
  if (tid < ctas) {
    const int4 end = p.ends[tid];
    if (end.x >= 0) {
      int e, kvh, b, pos;
      units = ((rows_of(end, e, kvh, b, pos) + 31) / 32) * (tid - end.y + 1 >= kSplit ? D / 8 : 1);
    }
  }
  int upto = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(FULL, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) sums[w] = upto;
  __syncthreads();
  for (int i = 0; i < w; ++i) upto += sums[i];
  starts[tid + 1] = upto;
  if (tid == 0) starts[0] = 0;
  __syncthreads();
  const int total = starts[kJoinThreads];
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    int t = 0;                             // starts[t] <= u < starts[t + 1]
#pragma unroll
    for (int o = kJoinThreads / 2; o > 0; o >>= 1)
      if (starts[t + o] <= u) t += o;
    const int4 end = p.ends[t];
    const int n = t - end.y + 1;
    int e, kvh, b, pos0;
    const int rows = rows_of(end, e, kvh, b, pos0);
    const bool split = n >= kSplit;
    const int blk = split ? (u - starts[t]) / (D / 8) : u - starts[t], pr = 32 * blk + lane;
    const bool there = pr < rows;
    int h, pos;
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) +
                       row_at<false, D>(p, b, kvh, pos0, kItemRows * (e - b * p.tiles) + min(pr, rows - 1), h, pos);
    auto piece = [&](int k) { return p.part + (int64_t)(k == 0 ? end.z : 2 * (end.y + k)) * part_floats<D>(); };
    if (split) {
      const int q0 = 2 * (u - starts[t] - blk * (D / 8));
      RowSum<2> a;
      if (there) add_pieces<D>(a, piece, w, 8, n, pr, q0, 1);
      join_warps<D>(a, o, q0, there);
    } else if (there) {
      RowSum<D / 32> a;
      add_pieces<D>(a, piece, 0, 1, n, pr, w, 8);
      store_row<D>(a, o, w, 8);
    }
  }
}

// A decode step's rows: the prefix's pieces and those of the sequences' own keys.
struct PrefixJoin {
  int64_t total, per;                 // of the prefix's list: entries of a KV head, of a CTA
  const int4* rows;                   // own keys: per row {first piece, second, pieces, 0}
  const float* own;                   // their pieces: o [8][D], maximum [8], sum [8]
  int chunks, per_chunk, ctas;
};

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kJoinThreads)
q4_prefix_join_kernel(const __grid_constant__ ManyParams p, const __grid_constant__ PrefixJoin j) {
  grid_dep_wait();
  constexpr int kOwn = 8 * (D + 2), NQ = SPLIT ? 2 : D / 32;
  const int kvh = blockIdx.x / p.tiles, t = blockIdx.x - kvh * p.tiles, w = threadIdx.x >> 5;
  const int pr = blockIdx.y * 32 + (threadIdx.x & 31), rows = p.c.B * p.G, row = min(kItemRows * t + pr, rows - 1);
  const bool there = kItemRows * t + pr < rows;
  if (kItemRows * t + (int)blockIdx.y * 32 >= rows) return;
  int h, pos;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + row_at<true, D>(p, 0, kvh, 0, row, h, pos);
  // the item's entries [base, base + cost): its pieces' CTAs
  const int64_t cost = ((p.keys + BN - 1) / BN) + kItemCost, base = kvh * j.total + t * cost;
  const int i0 = (int)((base + kItemCost) / j.per), i1 = (int)((base + cost - 1) / j.per);
  const int n = i1 - i0 + 1, slot0 = n == 1 ? 2 * j.ctas + (int)blockIdx.x : base <= i0 * j.per ? 2 * i0 : 2 * i0 + 1;
  auto piece = [&](int k) { return p.part + (int64_t)(k == 0 ? slot0 : 2 * (i0 + k)) * part_floats<D>(); };
  const int q0 = SPLIT ? 2 * blockIdx.z : w, stride = SPLIT ? 1 : 8;
  RowSum<NQ> a;
  if (there) {
    add_pieces<D>(a, piece, SPLIT ? w : 0, SPLIT ? 8 : 1, n, pr, q0, stride);
    const int b = row / p.G, hh = row - b * p.G, ch = hh / j.per_chunk, hc = hh - ch * j.per_chunk;
    const int4 own = j.rows[((int64_t)b * p.c.H + kvh) * j.chunks + ch];
    for (int k = SPLIT ? w : 0; k < own.z; k += SPLIT ? 8 : 1) {
      const float* pt = j.own + (int64_t)(k == 0 ? own.x : own.y + 2 * (k - 1)) * kOwn;
      const float l = pt[8 * D + 8 + hc], m = pt[8 * D + hc], mm = fmaxf(a.m, m);
      if (l == 0.f) continue;
      a.scale(a.l == 0.f ? 0.f : ex2(a.m - mm));
      a.m = mm;
      const float f = ex2(m - mm);
      a.l = fmaf(f, l, a.l);
#pragma unroll
      for (int c = 0; c < NQ; ++c) {
        const int quad = q0 + stride * c, x = quad >> 1;
        const float4 v = *reinterpret_cast<const float4*>(pt + hc * D + 32 * (2 * (x >> 3) + (quad & 1)) + 4 * (x & 7));
        RowSum<NQ>::add(a.o[c], f, make_float4(v.x, v.z, v.y, v.w));
      }
    }
  }
  if constexpr (SPLIT)
    join_warps<D>(a, o, q0, there);
  else if (there)
    store_row<D>(a, o, q0, stride);
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
  p.item_wait_ns = std::min(a.wait_ns, UINT64_MAX / kItemWaits) * kItemWaits;
  p.stall = a.stall;
  for (int h = 0; h < a.Hq; ++h) p.slope[h] = a.slope_log2[h];
}

template <int D>
cudaError_t launch_chunk(const Q4DecodeArgs& a, cudaStream_t st) {
  ManyParams p;
  fill(p, a, a.work);
  p.tiles = (int)(((int64_t)p.m * p.G + kItemRows - 1) / kItemRows);
  auto kern = q4_many_kernel<D, false>;
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kern), (int)smem_bytes<D>());
  const int ctas = std::min(a.num_sms, kJoinThreads);
  if (e == cudaSuccess) e = launch_dependent(kern, dim3(ctas), kThreads, smem_bytes<D>(), st, p);
  if (e == cudaSuccess)
    e = launch_dependent(q4_many_join_kernel<D>, dim3(4 * a.num_sms), kJoinThreads, 0, st, p, ctas);
  return e;
}

template <int D>
cudaError_t launch_prefix(const Q4DecodeArgs& a, cudaStream_t st) {
  ManyParams p;
  const int64_t own = q4_own_work_bytes(D, a.num_sms, a.c.B, a.c.H, a.Hq / a.c.H);
  fill(p, a, static_cast<uint8_t*>(a.work) + own);
  p.tiles = (int)(((int64_t)a.c.B * p.G + kItemRows - 1) / kItemRows);
  PrefixJoin j;
  j.ctas = a.num_sms;
  j.chunks = (p.G + 7) / 8;
  j.per_chunk = (p.G + j.chunks - 1) / j.chunks;
  // (as the kernel finds them)
  j.total = (int64_t)p.tiles * ((p.keys + BN - 1) / BN + kItemCost);
  const int64_t all = j.total * a.c.H;
  j.per = std::max<int64_t>((all + a.num_sms - 1) / a.num_sms, kMinShare);
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
  // (pieces of an item: as many as its entries touch CTAs, or one less)
  const int64_t pieces = (j.total / p.tiles + j.per - 1) / j.per;
  if (e == cudaSuccess)
    e = pieces >= kSplit ? launch_dependent(q4_prefix_join_kernel<D, true>, dim3(a.c.H * p.tiles, kItemRows / 32, D / 8),
                                            kJoinThreads, 0, st, p, j)
                         : launch_dependent(q4_prefix_join_kernel<D, false>, dim3(a.c.H * p.tiles, kItemRows / 32),
                                            kJoinThreads, 0, st, p, j);
  return e;
}

}  // namespace

int64_t q4_many_work_bytes(int d, int num_sms, int64_t rows, int Hkv) {
  const int64_t items = (rows + kItemRows - 1) / kItemRows * Hkv;
  return num_sms * (int64_t)sizeof(int4) + (2 * num_sms + items) * (int64_t)sizeof(float) * kItemRows * (d + 2);
}

cudaError_t launch_q4_chunk(const Q4DecodeArgs& a, cudaStream_t st) {
  return a.c.d == 64 ? launch_chunk<64>(a, st) : launch_chunk<128>(a, st);
}
cudaError_t launch_q4_prefix(const Q4DecodeArgs& a, cudaStream_t st) {
  return a.c.d == 64 ? launch_prefix<64>(a, st) : launch_prefix<128>(a, st);
}

}  // namespace plsh
