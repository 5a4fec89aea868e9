// One decode step over the 4-bit paged cache, approximate and exact ALiBi.
//
// Per sequence b and query head h, with pos = pos[b] and the cached values
// k_j, v_j (value = lo + step c of each group of 32):
//   o = sum_j w_j e^{x_j} v_j / sum_j w_j e^{x_j},  x_j = q . k_j / sqrt(d),
//   approximate:  w_j = c_j = #{t : lo_t(pos) <= j},  j <= pos
//   exact:        w_j = e^{-(pos - j) / sigma_h},     j <= pos
// (Positional LSH, technical summary, Methodology 1 and 3, for one row.)
//
// What bounds it: the cache's bytes, 1.25 d a position and KV head, and next to
// them the instructions of taking it apart.  At HBM rate an SM has about 27
// issue slots for a position of d = 128 (K and V), which up to eight query
// heads share; products on the CUDA cores would take 2 d G / 32 of them alone,
// so they run as mma.sync m16n8k16 with the cached values as the A operand (16
// positions, or 16 values of a row) and the query heads as the eight columns
// of B.  (tcgen05 takes A from shared or tensor memory: the codes would be
// expanded to 16 bits, written there and read again, 512 bytes a position,
// which costs more than the products.)  The codes never become the values they
// stand for:
//   q . k_j = sum_y step_jy (sum_i q_yi c_jyi) + sum_y lo_jy (sum_i q_yi),
//   sum_j p_j v_jyi = sum_j (p_j step_jy) c_jyi + sum_j p_j lo_jy,
// so the products take the bare codes, step and lo act on sums of 32, in fp32.
// The cache holds the codes in the order of the operand registers, so that a
// word of eight codes gives four of them with four ANDs and a shift
// (two_codes), or, where the sums of c + 16 c' may stand for those of c', three
// ANDs and a byte permutation (V: 66.4 -> 65.0 us for 64 ragged sequences).
//   - q is scaled to f16 by a power of two per head (bf16: its largest
//     magnitude in [2^14, 2^15), exact down to 2^-24 of that; fp32: two terms
//     of integers whose sums are exact, 22 bits).
//   - p_j step_jy is scaled by a power of two per head (column) and group, which
//     follows the largest p_j step_jy met, and rounded to f16 (2^-11 relative, no
//     finer than 2^-33 of that largest; fp32: two terms, 2^-36).  A large step of
//     a key that weighs nothing, for this head or for all, takes no precision
//     from the others (one power for all heads, by the largest step, was half a
//     microsecond faster in the approximate step and 1.5 us in the exact one of 64
//     sequences, but a head's row could vanish under a key that it does not
//     see).  f16 because bf16's 2^-8 would show beside the output's own rounding.
// Each warp of a row's team takes every so-manieth block of 32 positions, with
// a maximum, row sums and accumulators of its own, from a ring of asynchronous
// copies that it alone fills and reads (no barrier in the loop); its maximum
// moves only when a score passes it by a factor 2^kLazy.  The team merges in
// shared memory, pieces of a row that went to several CTAs in a second kernel.
//
// Work split.  Exact: every CTA takes the same share of the flat list
// (sequence, KV head, block), found from the positions on the device, so that
// ragged sequences balance (counting 12 blocks for a row's beginning and end:
// 75.6 -> 66.0 us for 64 ragged sequences).  Approximate: a row's key envelope
// is short and known only after its bins are read; a team of 1 to 8 warps for
// it, by the reach that its scales let expect, or a cluster of 2 to 8 CTAs that
// joins its pieces in distributed shared memory (one sequence 9.2 -> 7.0 us).
//
// Measured on GB300 (CUDA graph, back to back; percentages of the measured copy
// rate of 6.80 TB/s): exact, 64 ragged sequences of up to 8192, 32/8 heads, 66
// us (346 MB, 77 %); 2 x 131072 positions, 40/8 heads, 64 us (336 MB, 77 %);
// one sequence of 8192 9.3 us.  Without the arithmetic the copies alone took
// 57 us for the long case when the whole took 66: it is bound by instructions
// (about 260 a tile of 16 positions, issued in 52 % of the cycles; the logic
// pipe, which takes the ANDs, is 53 % busy).  Approximate, s = 10: 64 ragged
// sequences 14.4 us (19.7 MB, means over draws), bound by instructions of
// beginning and ending rows (2600 a warp, half of them not in blocks, issued in
// 46 % of the cycles); one 7.6 us, bound by latency (position, bins, first
// block, 1.4 us a block in one warp, merge).  fp32 queries (twice the products,
// codes made normal numbers): the exact step of those 64 sequences 98 us, the
// approximate one 26 us, with one CTA an SM (launch_approx).
// Tried and dropped: one more warp per scheduler at 128 registers (spills, 73
// -> 79 us), products of the next block beside P V of this one (74 -> 81),
// K's codes as e4m3 operands of m16n8k32 (half the ANDs, but 65 -> 83), joining
// split rows in the CTA that arrives last (+3 us on the device), 16-warp teams
// (14.6 -> 17.1), dependents launched at a kernel's start (waiting CTAs take the
// slots unevenly: 14.2 -> 17.2).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "bins_dev.cuh"
#include "plsh_internal.h"
#include "q4.cuh"
#include "tc_ptx.cuh"

namespace plsh {
namespace {

using namespace q4;
using namespace ptx;

// Exact: three CTAs of four warps (168 registers a thread: 128 spill) and three
// blocks of 32 positions in a warp's ring.  Approximate: two CTAs of eight
// warps (one where the queries' operands or the bin starts take more than half of
// the shared memory: fp32 with d = 128; bf16 with d = 128 and 64 hashes), two
// blocks (an envelope is a few blocks long).
constexpr int kExactWarps = 4, kExactStages = 3, kExactCtas = 3;
constexpr int kApproxWarps = 8, kApproxStages = 2, kApproxCtas = 2;
constexpr int kHeads = 8;           // query heads of a CTA (columns of the products)
// exact: blocks of a CTA at least (one sequence of 8192: 4 -> 12.2 us, 8 -> 8.9, 12 -> 9.8)
constexpr int kMinBlocks = 8;
// exact: blocks that beginning and ending a row costs (64 ragged sequences: 0 ->
// 75.6 us, 6 -> 69.7, 12 -> 66.0, 20 -> 67.7)
constexpr int kRowCost = 12;
// approximate: blocks of a warp where not all warps fit at once, blocks of a CTA
// at most while there is room, beyond what a cluster takes (below that the
// cluster is faster: it needs no second kernel), CTAs of one row at most
constexpr double kTeamBlocks = 2.5, kShareBlocks = 40.0;
constexpr int kMaxShares = 64, kMaxCluster = 8;
constexpr int kMaxGroupOrder = 32;
constexpr unsigned FULL = 0xffffffffu;
constexpr float kNothing = -3.402823466e38f;   // a maximum over no score
constexpr float kLog2e = 1.4426950408889634f;

struct Slopes {
  float v[kMaxExactHeads];          // log2(e) / sigma_h
};

// What a launch of the exact step's kernel attends over:
//   kStep    one row a sequence, every key up to its position;
//   kRows    m rows a sequence (q, o [B, Hq, m, d]), row i at pos[b] + i, each a
//            row of the flat list by itself;
//   kPacked  the same where a KV head has at most four query heads: as many of a
//            sequence's rows as the eight columns hold (`tokens`) are one row of the
//            flat list, column i G + h for head h of the i-th of them, and the keys'
//            codes are taken apart once for all of them (64 sequences of 4096
//            positions, 32/8 heads, 4 tokens: 210 -> 137 us, 8 tokens 401 -> 252;
//            as a matter of kRows with one row of eight heads the columns'
//            positions cost 7 %);
//   kShared  as kStep, the first pages being a prefix's that all sequences share;
//   kOwn     as kStep, only the keys behind that prefix; rows are left as pieces,
//            which a kernel elsewhere joins with the prefix's part.
enum Form { kStep, kRows, kPacked, kShared, kOwn };
constexpr bool of_rows(int form) { return form == kRows || form == kPacked; }

struct DecodeParams {
  Q4Cache c;
  const void* q;
  void* o;
  const int32_t* pos;
  int Hq, G;                        // query heads, of a KV head
  int chunks, per_chunk;            // a KV head's query heads in shares of at most kHeads
  const BinRecord* rec;
  int s;
  int64_t W;
  int limit;                        // positions below this may be asked for
  int4* ends;                       // exact: per CTA {row, first CTA, first piece} of a row that ends in it
  float* part;                      // pieces: o [8][D], m [8], l [8]
  int* err;
  int m;                            // rows of a sequence
  int tokens, each;                 // of them that one row of the list holds, at most; rows of the list
  const int32_t* len;               // [B] rows that count, or null
  const int32_t* prefix;            // kShared: the prefix's pages
  int prefix_pages;
  int first;                        // kOwn: the prefix's positions
  int4* rows;                       // kOwn: per row {first piece, second, pieces, 0}
  int row_pieces;                   // kOwn: piece of row 0 where a CTA has all of it
};

template <int D>
__host__ __device__ constexpr int part_floats() { return kHeads * (D + 2); }

// 16 bytes from src + OFF to dst + OFF
template <int OFF>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;" ::"r"(dst), "l"(src), "n"(OFF)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// All threads of a cluster; what they wrote to shared memory is seen after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// address of `at` of this CTA's shared memory in that of CTA `rank` of the cluster
__device__ __forceinline__ uint32_t cluster_addr(uint32_t at, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t at) {
  float r;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t at) {
  float4 r;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
               : "r"(at)
               : "memory");
  return r;
}

// c += A (16 x 16, row) B (16 x 8): f16 operands (bf16 with BF), fp32 sums
template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
#define PLSH_MMA(TYPES)                                                                       \
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." TYPES ".f32 {%0, %1, %2, %3}, "       \
               "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"                                \
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])                               \
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if constexpr (BF)
    PLSH_MMA("bf16.bf16");
  else
    PLSH_MMA("f16.f16");
#undef PLSH_MMA
}
// c = A B
template <bool BF>
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
#define PLSH_MMA(TYPES)                                                                       \
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." TYPES ".f32 {%0, %1, %2, %3}, "       \
               "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"                            \
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])                               \
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f))
  if constexpr (BF)
    PLSH_MMA("bf16.bf16");
  else
    PLSH_MMA("f16.f16");
#undef PLSH_MMA
}
// transpose of an 8 x 8 matrix of 16-bit values, two per lane and row
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// Two codes of a word as f16 operands: in bits 0 - 3 of each half (HIGH: 4 - 7,
// as 16 c).  As they stand they are the subnormals c 2^-24; the matrix
// instruction multiplies those exactly but aligns its sums as if they were
// 2^-14, so that sums keep about 18 bits of their largest product: enough under
// bf16 queries.  Under fp32 ones (NORMAL) they become the number c itself, by
// way of 1024 + c.
template <bool NORMAL>
__device__ __forceinline__ uint32_t f16_codes(uint32_t c) {
  if constexpr (NORMAL) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(c | 0x64006400u), "r"(0x64006400u));
    return r;
  }
  return c;
}
template <bool NORMAL, bool HIGH>
__device__ __forceinline__ uint32_t two_codes(uint32_t w) {
  return f16_codes<NORMAL>(w & (HIGH ? 0x00f000f0u : 0x000f000fu));
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r, x, y;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  float2 o;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
  return o;
}
// 2^e for -126 <= e <= 127, 0 below
__device__ __forceinline__ float pow2(int e) {
  return e < -126 ? 0.f : __int_as_float((e + 127) << 23);
}
__device__ __forceinline__ float sum_rows(float v) {      // over the lanes of one column pair
  v += __shfl_xor_sync(FULL, v, 4);
  v += __shfl_xor_sync(FULL, v, 8);
  return v + __shfl_xor_sync(FULL, v, 16);
}
__device__ __forceinline__ float max_rows(float v) {
  v = fmaxf(v, __shfl_xor_sync(FULL, v, 4));
  v = fmaxf(v, __shfl_xor_sync(FULL, v, 8));
  return fmaxf(v, __shfl_xor_sync(FULL, v, 16));
}

// words of one lane: D / 32 consecutive 32-bit words of shared memory
template <int OFF, int N>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(addr), "n"(OFF)
                 : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];"
                 : "=r"(w[0]), "=r"(w[1])
                 : "r"(addr), "n"(OFF)
                 : "memory");
  else
    asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(w[0]) : "r"(addr), "n"(OFF) : "memory");
}

// the same with an offset that unrolling makes a constant
__device__ __forceinline__ void lds_at(uint32_t addr, int off, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(addr + off)
               : "memory");
}

__device__ __forceinline__ void store_row(float* p, const float (&o)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&o)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
}

// What a team of warps attends over: blocks [t0, t1) of 32 positions (two tiles) of
// sequence b, KV head kvh, for the query heads h0 .. h0 + heads - 1 (kPacked: `heads`
// columns, of several rows).
struct Piece {
  int b, kvh, h0, heads, pos, t0, t1;
  int first;         // first position any of the heads sees
  int i, tokens;     // first row of the sequence, and rows (the last at pos)
};

// Head of column c among the piece's, and how many rows before the last it is.
template <int FORM>
__device__ __forceinline__ int head_of(const DecodeParams& p, const Piece& pc, int c) {
  return FORM == kPacked ? c % p.G : c;
}
template <int FORM>
__device__ __forceinline__ int back_of(const DecodeParams& p, const Piece& pc, int c) {
  return FORM == kPacked ? pc.tokens - 1 - c / p.G : 0;
}
// Element of column c in q and o.
template <int FORM, int D>
__device__ __forceinline__ int64_t column_at(const DecodeParams& p, const Piece& pc, int c) {
  const int64_t bh = (int64_t)pc.b * p.Hq + pc.h0 + head_of<FORM>(p, pc, c);
  return (of_rows(FORM) ? bh * p.m + pc.i + (FORM == kPacked ? c / p.G : 0) : bh) * D;
}

// ROWS: rows that a CTA's warps may be attending at once (a team of warps each)
template <typename T, int D, int WARPS, int STAGES, int ROWS>
struct Smem {
  // the queries' B operands by lane (fp32: two terms), and zeros
  alignas(128) uint4 q[ROWS][sizeof(T) / 2][Layout<D>::kGroups][33];
  uint2 qlow[ROWS][32];
  float scale[ROWS][kHeads];
  alignas(128) uint8_t ring[WARPS][STAGES][2 * Layout<D>::kTileBytes];
  float m[WARPS][kHeads], l[WARPS][kHeads];
  float weight[2 * WARPS][kHeads + 1];   // of a warp's column in its head
  unsigned some[ROWS][kHeads];           // which of them saw anything (NaN too)
  int64_t sums[WARPS], found[2];         // exact: sequences' entries; the first sequence, its first entry
};

// Lane (g, t)'s values 8 t .. 8 t + 7 of every group of column g's query head.
template <typename T, int D, int PACK>
struct Query {
  uint4 w[Layout<D>::kGroups][sizeof(T) / 2];
  template <int FORM>
  __device__ void load(const DecodeParams& p, const Piece& pc, int rank) {
    if (rank >= Layout<D>::kGroups) return;        // (prepare_query)
    const int lane = threadIdx.x & 31, g = (lane >> 2) % (kHeads / PACK), t = lane & 3;
    const T* q = static_cast<const T*>(p.q) + column_at<FORM, D>(p, pc, g < pc.heads ? g : 0) + 8 * t;
#pragma unroll
    for (int y = 0; y < Layout<D>::kGroups; ++y)
#pragma unroll
      for (int k = 0; k < (int)sizeof(T) / 2; ++k)
        w[y][k] = g < pc.heads ? reinterpret_cast<const uint4*>(q + 32 * y)[k] : make_uint4(0, 0, 0, 0);
  }
  // bits of the largest magnitude of column g (a NaN's are larger than any)
  __device__ uint32_t largest() const {
    uint32_t m = 0;
#pragma unroll
    for (int y = 0; y < Layout<D>::kGroups; ++y)
#pragma unroll
      for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
        const uint32_t x[4] = {w[y][k].x, w[y][k].y, w[y][k].z, w[y][k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          m = sizeof(T) == 4 ? max(m, x[i] & 0x7fffffffu) : __vmaxu2(m, x[i] & 0x7fff7fffu);
      }
    if (sizeof(T) == 2) m = max(m & 0xffff0000u, m << 16);
    m = max(m, __shfl_xor_sync(FULL, m, 1));
    return max(m, __shfl_xor_sync(FULL, m, 2));
  }
  // the values of group y
  __device__ void get(int y, float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
      uint4 c = w[0][k];
#pragma unroll
      for (int z = 1; z < Layout<D>::kGroups; ++z)
        if (y == z) c = w[z][k];
      const uint32_t x[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          v[4 * k + i] = __uint_as_float(x[i]);
        } else {
          v[2 * i] = __uint_as_float(x[i] << 16);
          v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
        }
      }
    }
  }
};

// Copies N bytes, 16 a lane and turn; dst and src are the lane's own.
template <int N, int OFF = 0>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t* src, int lane) {
  if (OFF + 512 <= N || 16 * lane < N - OFF) cp_async16<OFF>(dst, src);
  if constexpr (OFF + 512 < N) copy_async<N, OFF + 512>(dst, src, lane);
}

// A warp's ring of blocks of one piece.  A block's two tiles lie one after the
// other in a page, except with pages of 16 positions.
template <typename T, int D, int FORM>
struct Ring {
  using L = Layout<D>;
  const uint8_t* head_data;
  const int32_t* table;
  const int32_t* prefix;
  int prefix_pages;
  int64_t page_bytes;
  uint32_t pages;
  uint32_t smem;
  int log_blocks, last, lane;
  uint32_t absent = 0;          // two bits a stage: tiles that have no page
  int* err;
  __device__ Ring(const DecodeParams& p, const Piece& pc, const void* ring)
      : table(p.c.table + (int64_t)pc.b * p.c.max_pages), prefix(p.prefix),
        prefix_pages(p.prefix_pages), pages((uint32_t)p.c.pages),
        smem(smem_u32(ring)), log_blocks(p.c.page_shift - 5), last(pc.pos >> 4),
        lane(threadIdx.x & 31), err(p.err) {
    page_bytes = ((int64_t)p.c.H << (p.c.page_shift - 4)) * L::kTileBytes;
    head_data = p.c.data + ((int64_t)pc.kvh << (p.c.page_shift - 4)) * L::kTileBytes + 16 * lane;
  }
  __device__ int32_t entry(int i) const {
    if constexpr (FORM == kShared) return i < prefix_pages ? prefix[i] : table[i];
    return table[i];
  }
  // the page of a block's first tile (and, in general, of its second)
  __device__ int32_t page_of(int block) const {
    return entry(log_blocks >= 0 ? block >> log_blocks : 2 * block);
  }
  // `first`: the first position that the row reaches back to
  __device__ void fetch(int block, int st, int32_t pg, int first) {
    const uint32_t dst = smem + st * (2 * L::kTileBytes) + 16 * lane;
    absent &= ~(3u << (2 * st));
    if (log_blocks >= 0) {
      if ((uint32_t)pg < pages)
        copy_async<2 * L::kTileBytes>(
            dst, head_data + pg * page_bytes + (block & ((1 << log_blocks) - 1)) * (2 * L::kTileBytes), lane);
      else
        absent |= 3u << (2 * st);
    } else {
      // the second tile's page is looked up only if the row reaches it; the first
      // one's counts only if the row reaches back to it
      const bool need0 = 32 * block + kTile > first, need1 = 2 * block + 1 <= last;
      const int32_t pg1 = need1 ? entry(2 * block + 1) : -1;
      if ((uint32_t)pg < pages)
        copy_async<L::kTileBytes>(dst, head_data + pg * page_bytes, lane);
      else
        absent |= 1u << (2 * st);
      if ((uint32_t)pg1 < pages)
        copy_async<L::kTileBytes>(dst + L::kTileBytes, head_data + pg1 * page_bytes, lane);
      else
        absent |= 2u << (2 * st);
      if ((!need0 || (uint32_t)pg < pages) && (!need1 || (uint32_t)pg1 < pages)) return;
    }
    if (((absent >> (2 * st)) & 3u) && lane == 0) atomicOr(err, kErrCachePlace);
  }
};

// The queries as B operands (lane (g, t) holds rows 2 t, 2 t + 1, ... of column
// g), a group of values a warp of the team and turn; qlow takes the products of
// q's sums over a group with K's lo, a bf16 number: k slots 2 t, 2 t + 1 and
// 2 t + 8 hold group t's sum as three bf16 terms (24 bits).  Visible to the
// team after a barrier.
template <typename T, int D, int PACK, typename S>
__device__ __forceinline__ void prepare_query(const Query<T, D, PACK>& query, int rank, int size, int row, S& sm) {
  constexpr int Y = Layout<D>::kGroups;
  constexpr bool kTwo = sizeof(T) == 4;         // two f16 terms
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (rank >= Y) return;
  const uint32_t mx = query.largest();
  const int e = min(max((int)(mx >> 23) - 127, -100), 110);
  // bf16: the largest in [2^14, 2^15); fp32: in [2^10, 2^11), as integers
  constexpr int kTop = kTwo ? 10 : 14;
  const float up = pow2(kTop - e);
  const float norm = kLog2e / sqrtf((float)D);
  if (rank == 0) {
    // what q's power of two and a code's (2^-24, or 1) leave
    const bool bad = mx >= (110u + 127u) << 23;           // 2^110, infinities, NaN
    if (t == 0) sm.scale[row][g] = bad ? NAN : pow2(e + (kTwo ? 0 : 24) - kTop) * norm;
    if (lane < (int)sizeof(T) / 2 * Y) sm.q[row][lane / Y][lane % Y][32] = make_uint4(0, 0, 0, 0);
    if (t >= Y) sm.qlow[row][lane] = make_uint2(0, 0);
  }
  // (not unrolled: most warps take one turn, all the same instructions)
#pragma unroll 1
  for (int y = rank; y < Y; y += size) {
    float v[8], sum = 0.f;
    query.get(y, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += v[i];
    sum += __shfl_xor_sync(FULL, sum, 1);
    sum += __shfl_xor_sync(FULL, sum, 2);
    uint32_t w[4], r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // odd codes are taken four bits up, as 16 c
      const float k = (i & 1) ? 0.0625f : 1.f;
      float a = v[i] * up, b = v[i + 4] * up;
      if constexpr (kTwo) {
        const float a0 = rintf(a), b0 = rintf(b);
        r[i] = pack_f16(rintf((a - a0) * 2048.f) * k, rintf((b - b0) * 2048.f) * k);
        a = a0;
        b = b0;
      }
      w[i] = pack_f16(a * k, b * k);
    }
    sm.q[row][0][y][lane] = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (kTwo) sm.q[row][1][y][lane] = make_uint4(r[0], r[1], r[2], r[3]);
    const float group = sum * norm;
    const float hi = __uint_as_float(__float_as_uint(group) & 0xffff0000u);
    const float mid = __uint_as_float(__float_as_uint(group - hi) & 0xffff0000u);
    if (t == y) sm.qlow[row][lane] = make_uint2(pack_bf16(hi, mid), pack_bf16(group - hi - mid, 0.f));
  }
}

// One piece; the result (all columns, the warps merged) goes to `o_row` (o of
// head h0; chunks: o itself; divided by the row sums) or, when that is null, to `part`.
// A step takes a block of two tiles.  PACK = 1: one after the other, the scores
// of eight heads in the eight columns of the product.  PACK = 2 (at most four
// heads): both at once, the first one's scores in columns 0 - 3 and the second
// one's in 4 - 7 (B is zero in the other tile's columns), so that what follows
// the products (a lane holds two positions and two columns either way) is done
// once for both.  Every column keeps a maximum, sums and accumulators of its
// own.  `ahead`: this warp's first block is in its ring already, not yet
// committed.
// The row's team: `size` warps from warp `first` on; all warps of the CTA call
// this together.  `starts`: its heads' bin starts, padded to whole int4 by numbers
// that no position reaches.
struct Team {
  int first, size, number;     // number: of the CTA's teams
};
template <typename T, int D, bool EXACT, int PACK, int FORM, int WARPS, int STAGES, int ROWS>
__device__ __forceinline__ void attend(const DecodeParams& p, const Piece& pc, const Team& team,
                                       const Query<T, D, PACK>& query, const float* slopes,
                                       const int4* starts, Smem<T, D, WARPS, STAGES, ROWS>& sm,
                                       Ring<T, D, FORM>& ring, bool ahead, T* o_row, float* part) {
  using L = Layout<D>;
  constexpr int Y = L::kGroups;
  constexpr bool kTwo = sizeof(T) == 4;         // two f16 terms
  constexpr float kLazy = EXACT ? 8.f : 4.f;    // weights up to 2^8, or 64 x 2^4
  constexpr int kCols = kHeads / PACK;          // columns of a tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = warp - team.first, kTeam = team.size;
  const int row = EXACT ? 0 : team.number;
  const int mine = PACK == 2 ? t >> 1 : 0;      // the tile whose scores this lane holds
  const int head = (2 * t) % kCols;             // and its heads: head, head + 1

  // ---- step i takes block newest - i kTeam, from the newest down (ALiBi's
  // weights fall with the distance: the running maximum is met early)
  const int newest = pc.t1 - 1 - rank;
  const int steps = newest >= pc.t0 ? (newest - pc.t0) / kTeam + 1 : 0;
  int32_t next_page;
  {
    int32_t pg[STAGES + 1];
#pragma unroll
    for (int i = 0; i <= STAGES; ++i) pg[i] = i < steps ? ring.page_of(newest - i * kTeam) : 0;
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
      if (i < steps && !(ahead && i == 0)) ring.fetch(newest - i * kTeam, i, pg[i], pc.first);
      cp_async_commit();
    }
    next_page = pg[STAGES];
  }

  if constexpr (EXACT) prepare_query<T, D, PACK>(query, rank, kTeam, row, sm);
  __syncthreads();
  const uint32_t qlow[2] = {sm.qlow[row][lane].x, sm.qlow[row][lane].y};
  const float qscale[2] = {sm.scale[row][2 * t], sm.scale[row][2 * t + 1]};
  // the lane's operands where column g belongs to tile u of the block, else zeros
  uint32_t q_at[PACK];
#pragma unroll
  for (int u = 0; u < PACK; ++u) q_at[u] = smem_u32(&sm.q[row][0][0][g / kCols == u ? lane : 32]);
  constexpr int kQ = 33 * 16;                   // bytes from a group's operands to the next's
  // all ones where column g belongs to tile u of the block
  uint32_t keep[PACK];
#pragma unroll
  for (int u = 0; u < PACK; ++u) keep[u] = g / kCols == u ? 0xffffffffu : 0u;
  float slope[2] = {0.f, 0.f}, back[2] = {0.f, 0.f};      // back: positions before the last row's
  int newest_start = 0;            // the largest bin start of the lane's heads
  const int quads = (p.s + 3) >> 2;
  if constexpr (EXACT) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (head + k < pc.heads) {
        slope[k] = slopes[pc.h0 + head_of<FORM>(p, pc, head + k)];
        back[k] = (float)back_of<FORM>(p, pc, head + k);
      }
  } else if (steps > 0) {
    for (int i = 0; i < 2 * quads; ++i) {
      const int4 v = starts[head * quads + i];
      const int a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) newest_start = a[k] <= pc.pos ? max(newest_start, a[k]) : newest_start;
    }
  }

  // ---- the loop
  float acc[Y][2][4];             // P V: values 32 y + 4 g + 2 tau + (r >> 1), columns 2 t + (r & 1)
  float low[Y][2];                // sum of p lo, this lane's positions
  float m[2] = {kNothing, kNothing}, l[2] = {0.f, 0.f};
  // Weights times step of a group and column are held times 2^-r.  r puts the
  // largest met into [2^kTop, 2^(kTop + 1)) and is raised when one reaches 2^15, so
  // that f16's smallest, 2^-24, lies far below the largest (bf16: with more room
  // above, so that it is raised less often: one sequence 9.7 -> 9.4 us).
  constexpr int kTop = kTwo ? 11 : 8;
  constexpr int kLeast = -100;    // r's smallest, where nothing was met
  float2 down[Y];                 // 2^-r, -100 <= r <= 124
#pragma unroll
  for (int y = 0; y < Y; ++y) {
    down[y] = make_float2(pow2(-kLeast), pow2(-kLeast));
    low[y][0] = low[y][1] = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[y][k >> 2][k & 3] = 0.f;
  }
  const uint32_t k_at = ring.smem + g * (D / 2) + t * (D / 8);
  const uint32_t pair_at = ring.smem + mine * L::kTileBytes + L::pair(g, 0);
  const uint32_t low_at = ring.smem + L::pair(g, t & (Y - 1));
  const uint32_t v_at = ring.smem + 16 * lane;
  for (int i = 0, st = 0; i < steps; ++i, st = st == STAGES - 1 ? 0 : st + 1) {
    const int block = newest - i * kTeam;
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    const uint32_t gone = (ring.absent >> (2 * st)) & 3u;
    const bool edge =
        32 * block < pc.first || 32 * block + 31 > pc.pos - (FORM == kPacked ? pc.tokens - 1 : 0) || gone;
#pragma unroll
    for (int sub = 2 / PACK - 1; sub >= 0; --sub) {
      // scores of positions j and j + 8 of the lane's tile, its two heads
      const uint32_t at = (uint32_t)((2 * st + sub) * L::kTileBytes);
      float x[4] = {0.f, 0.f, 0.f, 0.f}, z[4];
      {
        uint32_t k0[PACK][Y], k1[PACK][Y], w0[Y], w1[Y];
        lds<0>(k_at + at, k0[0]);
        lds<4 * D>(k_at + at, k1[0]);
        if constexpr (PACK == 2) {
          lds<L::kTileBytes>(k_at + at, k0[1]);
          lds<L::kTileBytes + 4 * D>(k_at + at, k1[1]);
        }
        lds<L::kKPairs>(pair_at + at, w0);
        lds<L::kKPairs + L::pair(8, 0)>(pair_at + at, w1);
        // q's sums times lo: every column for every tile, and the lane takes its
        // own tile's (a NaN of one tile must not reach the other's columns)
        auto low_products = [&](auto tile, float (&c)[4]) {
          constexpr int off = decltype(tile)::value * L::kTileBytes + L::kKPairs;
          uint32_t b0[1], b1[1];
          lds<off>(low_at + at, b0);
          lds<off + L::pair(8, 0)>(low_at + at, b1);
          b0[0] = __byte_perm(b0[0], 0, 0x1010);
          b1[0] = __byte_perm(b1[0], 0, 0x1010);
          mma16816_first<true>(c, b0[0], b1[0], b0[0], b1[0], qlow[0], qlow[1]);
        };
        low_products(std::integral_constant<int, 0>{}, z);
        if constexpr (PACK == 2) {
          float c[4];
          low_products(std::integral_constant<int, 1>{}, c);
#pragma unroll
          for (int k = 0; k < 4; ++k) z[k] = mine ? c[k] : z[k];
        }
#pragma unroll
        for (int y = 0; y < Y; ++y) {
          float c[4], c2[kTwo ? 4 : 1];
#pragma unroll
          for (int u = 0; u < PACK; ++u) {
            const uint32_t v0 = k0[u][y], v1 = k1[u][y], h0 = v0 >> 8, h1 = v1 >> 8;
            const uint32_t a[8] = {two_codes<kTwo, false>(v0), two_codes<kTwo, false>(v1),
                                   two_codes<kTwo, true>(v0),  two_codes<kTwo, true>(v1),
                                   two_codes<kTwo, false>(h0), two_codes<kTwo, false>(h1),
                                   two_codes<kTwo, true>(h0),  two_codes<kTwo, true>(h1)};
            uint32_t q[4];
            lds_at(q_at[u], y * kQ, q);
            if (u == 0)
              mma16816_first<false>(c, a[0], a[1], a[2], a[3], q[0], q[1]);
            else
              mma16816<false>(c, a[0], a[1], a[2], a[3], q[0], q[1]);
            mma16816<false>(c, a[4], a[5], a[6], a[7], q[2], q[3]);
            if constexpr (kTwo) {
              lds_at(q_at[u], (Y + y) * kQ, q);
              if (u == 0)
                mma16816_first<false>(c2, a[0], a[1], a[2], a[3], q[0], q[1]);
              else
                mma16816<false>(c2, a[0], a[1], a[2], a[3], q[0], q[1]);
              mma16816<false>(c2, a[4], a[5], a[6], a[7], q[2], q[3]);
            }
          }
          if constexpr (kTwo) {
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = fmaf(c2[k], 0x1p-11f, c[k]);
          }
          const float s0 = pair_step(w0[y]), s1 = pair_step(w1[y]);
          x[0] = fmaf(s0, c[0], x[0]);
          x[1] = fmaf(s0, c[1], x[1]);
          x[2] = fmaf(s1, c[2], x[2]);
          x[3] = fmaf(s1, c[3], x[3]);
        }
      }
      // the mask's weights; -inf where a head does not see a position
      const int j = 32 * block + (sub + mine) * kTile + g;
      float cnt[4];
      if constexpr (EXACT) {
        const float d0 = (float)(j - pc.pos), d1 = d0 + 8.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[k] = fmaf(x[k], qscale[k & 1],
                      fmaf((k < 2 ? d0 : d1) + (FORM == kPacked ? back[k & 1] : 0.f), slope[k & 1], z[k]));
      } else {
        // c_j: every start in the row's past, or those at or before j
        int n[4] = {p.s, p.s, p.s, p.s};
        if (!__all_sync(FULL, j - g >= newest_start)) {
          n[0] = n[1] = n[2] = n[3] = 0;
#pragma unroll 4
          for (int i = 0; i < quads; ++i) {
            const int4 u = starts[head * quads + i], v = starts[(head + 1) * quads + i];
            n[0] += (u.x <= j) + (u.y <= j) + (u.z <= j) + (u.w <= j);
            n[1] += (v.x <= j) + (v.y <= j) + (v.z <= j) + (v.w <= j);
            n[2] += (u.x <= j + 8) + (u.y <= j + 8) + (u.z <= j + 8) + (u.w <= j + 8);
            n[3] += (v.x <= j + 8) + (v.y <= j + 8) + (v.z <= j + 8) + (v.w <= j + 8);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          cnt[k] = (float)n[k];
          x[k] = n[k] == 0 ? -INFINITY : fmaf(x[k], qscale[k & 1], z[k]);
        }
      }
      uint32_t w0[Y], w1[Y];         // V's pairs of the lane's positions
      lds<L::kVPairs>(pair_at + at, w0);
      lds<L::kVPairs + L::pair(8, 0)>(pair_at + at, w1);
      if (edge) {
        __syncwarp();          // (a branch: selects would cost every step)
        // positions that no head sees may hold anything
        const bool none = (gone >> (sub + mine)) & 1;
        if (none || j < pc.first || j > pc.pos) {
          x[0] = x[1] = -INFINITY;
#pragma unroll
          for (int y = 0; y < Y; ++y) w0[y] = 0;
        }
        if (none || j + 8 < pc.first || j + 8 > pc.pos) {
          x[2] = x[3] = -INFINITY;
#pragma unroll
          for (int y = 0; y < Y; ++y) w1[y] = 0;
        }
        if constexpr (FORM == kPacked) {         // rows before the last
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (j + 8 * (k >> 1) > pc.pos - (int)back[k & 1]) x[k] = -INFINITY;
        }
      }
      // the weights, and P step of each group as f16 operands (times 2^-r):
      // positions j (e0) and j + 8 (e1) of two heads
      float pw[4];
      uint32_t e0[Y], e1[Y];
      auto weigh = [&](int y, float2& u0, float2& u1) {
        const float s0 = pair_step(w0[y]), s1 = pair_step(w1[y]);
        u0 = mul2(mul2(make_float2(pw[0], pw[1]), down[y]), make_float2(s0, s0));
        u1 = mul2(mul2(make_float2(pw[2], pw[3]), down[y]), make_float2(s1, s1));
      };
      auto weights = [&]() {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          pw[k] = ex2(x[k] - m[k & 1]);
          if constexpr (!EXACT) pw[k] *= cnt[k];
        }
      };
#pragma unroll 1
      for (bool again = false;; again = true) {
        weights();
        uint32_t top = 0;
#pragma unroll
        for (int y = 0; y < Y; ++y) {
          float2 u0, u1;
          weigh(y, u0, u1);
          e0[y] = pack_f16(u0.x, u0.y);
          e1[y] = pack_f16(u1.x, u1.y);
          top = __vimax3_u16x2(top, e0[y], e1[y]);
        }
        // does a score outgrow what it is measured against, or a product reach
        // 2^15 (or is it no number)?  (one vote for both, behind the exponentials:
        // with one each, 4 us in 66)
        const bool grow = fmaxf(x[0], x[2]) > m[0] + kLazy || fmaxf(x[1], x[3]) > m[1] + kLazy;
        if (again || !__any_sync(FULL, grow || ((top + 0x08000800u) & 0x80008000u))) break;
        const bool some = __any_sync(FULL, m[0] != kNothing || m[1] != kNothing);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // The maximum moves, and r by as many whole binary places, so that what
          // the accumulators hold keeps its place.  (The maximum itself, not the
          // next whole number: the key that it belongs to then weighs 1, and 1
          // times a step, eight bits, takes no rounding.)
          const float to = max_rows(fmaxf(m[k], fmaxf(x[k], x[k + 2])));
          const float by = m[k] - to;
          m[k] = to;
          if (!some) continue;               // a warp's first tile
          const int n = (int)fminf(rintf(-by), 400.f);
          const float f = ex2(by), rest = ex2(by + (float)n);
          l[k] *= f;
#pragma unroll
          for (int y = 0; y < Y; ++y) {
            low[y][k] *= f;
            float& dn = k == 0 ? down[y].x : down[y].y;
            const int r = 127 - (__float_as_int(dn) >> 23), least = max(r - n, kLeast);
            dn = pow2(-least);
            const float past = pow2(r - n - least) * rest;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[y][e >> 1][2 * (e & 1) + k] *= past;
          }
        }
        weights();
#pragma unroll
        for (int y = 0; y < Y; ++y) {
          // a step that is not a number: its group of the row of every head
          // that gives the position a weight is none either
          const bool nan0 = (w0[y] & 0x7f800000u) == 0x7f800000u, nan1 = (w1[y] & 0x7f800000u) == 0x7f800000u;
          if (nan0) w0[y] = 0;
          if (nan1) w1[y] = 0;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if ((nan0 && x[k] != -INFINITY) || (nan1 && x[k + 2] != -INFINITY)) low[y][k] = NAN;
          // the columns' largest, by the upper halves of their bits
          const float s0 = pair_step(w0[y]), s1 = pair_step(w1[y]);
          uint32_t most = __byte_perm(__float_as_uint(fmaxf(pw[0] * s0, pw[2] * s1)),
                                      __float_as_uint(fmaxf(pw[1] * s0, pw[3] * s1)), 0x7632);
          most = __vmaxu2(most, __shfl_xor_sync(FULL, most, 4));
          most = __vmaxu2(most, __shfl_xor_sync(FULL, most, 8));
          most = __vmaxu2(most, __shfl_xor_sync(FULL, most, 16));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int e = (int)((most >> (16 * k + 7)) & 255u) - 127;       // (128: infinite, or no number)
            float& dn = k == 0 ? down[y].x : down[y].y;
            const int r = 127 - (__float_as_int(dn) >> 23);
            const int to = e - r < 15 ? r : e == 128 ? 124 : e - kTop;
            dn = pow2(-to);
            const float f = pow2(r - to);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[y][i >> 1][2 * (i & 1) + k] *= f;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) l[k & 1] += pw[k];
      // P V, group by group
#pragma unroll
      for (int yy = 0; yy < Y; yy += 2) {
        uint32_t v4[PACK][4];
        if (yy == 0) {
          lds<L::kV>(v_at + at, v4[0]);
          if constexpr (PACK == 2) lds<L::kV + L::kTileBytes>(v_at + at, v4[PACK - 1]);
        } else {
          lds<L::kV + 512>(v_at + at, v4[0]);
          if constexpr (PACK == 2) lds<L::kV + 512 + L::kTileBytes>(v_at + at, v4[PACK - 1]);
        }
#pragma unroll
        for (int y = yy; y < yy + 2; ++y) {
          const float b0 = pair_lo(w0[y]), b1 = pair_lo(w1[y]);
          low[y][0] = fmaf(pw[0], b0, fmaf(pw[2], b1, low[y][0]));
          low[y][1] = fmaf(pw[1], b0, fmaf(pw[3], b1, low[y][1]));
          uint32_t f0 = 0, f1 = 0;
          if constexpr (kTwo) {
            float2 u0, u1;
            weigh(y, u0, u1);
            const float2 c0 = __half22float2(*reinterpret_cast<__half2*>(&e0[y]));
            const float2 c1 = __half22float2(*reinterpret_cast<__half2*>(&e1[y]));
            f0 = transpose8x8(pack_f16(u0.x - c0.x, u0.y - c0.y));
            f1 = transpose8x8(pack_f16(u1.x - c1.x, u1.y - c1.y));
          }
          const uint32_t g0 = transpose8x8(e0[y]), g1 = transpose8x8(e1[y]);
          // fp32: the tile's own sums first, then added: the products' fp32 sums
          // truncate, which over a long row would add up to one side
          float own[kTwo ? 2 : 1][4];
#pragma unroll
          for (int u = 0; u < PACK; ++u) {
            const uint32_t v0 = v4[u][2 * (y - yy)], v1 = v4[u][2 * (y - yy) + 1];
            // rows of c and of c + 16 c', whose c the merge takes off again: a
            // byte permutation gives the latter for the upper bytes at once
            const uint32_t n0 = v0 & 0x00ff00ffu, n1 = v1 & 0x00ff00ffu;
            const uint32_t h0 = __byte_perm(v0, 0, 0x4341), h1 = __byte_perm(v1, 0, 0x4341);
            const uint32_t a[8] = {two_codes<kTwo, false>(v0), f16_codes<kTwo>(n0),
                                   two_codes<kTwo, false>(v1), f16_codes<kTwo>(n1),
                                   two_codes<kTwo, false>(h0), f16_codes<kTwo>(h0),
                                   two_codes<kTwo, false>(h1), f16_codes<kTwo>(h1)};
            const uint32_t b[4] = {g0 & keep[u], g1 & keep[u], f0 & keep[u], f1 & keep[u]};
            if constexpr (kTwo) {
              if (u == 0) {
                mma16816_first<false>(own[0], a[0], a[1], a[2], a[3], b[2], b[3]);
                mma16816_first<false>(own[1], a[4], a[5], a[6], a[7], b[2], b[3]);
              } else {
                mma16816<false>(own[0], a[0], a[1], a[2], a[3], b[2], b[3]);
                mma16816<false>(own[1], a[4], a[5], a[6], a[7], b[2], b[3]);
              }
              mma16816<false>(own[0], a[0], a[1], a[2], a[3], b[0], b[1]);
              mma16816<false>(own[1], a[4], a[5], a[6], a[7], b[0], b[1]);
            } else {
              mma16816<false>(acc[y][0], a[0], a[1], a[2], a[3], b[0], b[1]);
              mma16816<false>(acc[y][1], a[4], a[5], a[6], a[7], b[0], b[1]);
            }
          }
          if constexpr (kTwo) {
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[y][k >> 2][k & 3] += own[k >> 2][k & 3];
          }
        }
      }
    }
    __syncwarp();            // the stage may be filled again
    if (i + STAGES < steps) {
      ring.fetch(block - STAGES * kTeam, st, next_page, pc.first);
      if (i + STAGES + 1 < steps) next_page = ring.page_of(block - (STAGES + 1) * kTeam);
    }
    cp_async_commit();
  }
  cp_async_wait<0>();

  // ---- merge the team's columns: head h has column h of every warp, and with
  // PACK = 2 column h + 4
  const int ways = kTeam * PACK, way0 = team.first * PACK;
  constexpr int kStride = STAGES * 2 * L::kTileBytes / 4;      // floats of a warp's ring
  static_assert(kStride >= kHeads * D, "a warp's columns fit its ring");
  __syncwarp();              // the warp's ring is done with
  float* all = reinterpret_cast<float*>(sm.ring);
  float* merge = all + warp * kStride;
  if (steps > 0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float sum = sum_rows(l[k]);
      if (g == 0) {
        sm.m[warp][2 * t + k] = m[k];
        sm.l[warp][2 * t + k] = sum;
      }
#pragma unroll
      for (int y = 0; y < Y; ++y) {
        const float b = sum_rows(low[y][k]);
        const float up = __uint_as_float((254u << 23) - __float_as_uint(k == 0 ? down[y].x : down[y].y));
        float4 v;
        constexpr float kLow = kTwo ? 1.f : 0x1p24f, kHigh = kTwo ? 0.0625f : 0x1p20f;
        v.x = fmaf(acc[y][0][k] * kLow, up, b);
        v.y = fmaf((acc[y][0][2 + k] - acc[y][0][k]) * kHigh, up, b);
        v.z = fmaf(acc[y][1][k] * kLow, up, b);
        v.w = fmaf((acc[y][1][2 + k] - acc[y][1][k]) * kHigh, up, b);
        *reinterpret_cast<float4*>(merge + (2 * t + k) * D + 32 * y + 4 * g) = v;
      }
    }
  } else if (lane < kHeads) {
    sm.m[warp][lane] = kNothing;
    sm.l[warp][lane] = 0.f;
  }
  __syncthreads();
  if (rank == 0) {
    // 32 / kCols lanes a head, two columns each at most; a row divides by its
    // sum, and one that sees nothing is 0
    constexpr int kPer = 32 / kCols;
    const int h = lane / kPer, w0 = lane % kPer;
    static_assert(2 * kPer >= WARPS * PACK, "two columns a lane");
    float mw[2], lw[2], mm = kNothing;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int w = w0 + k * kPer;
      mw[k] = kNothing;
      lw[k] = 0.f;
      if (w < ways) {
        mw[k] = sm.m[team.first + w / PACK][w % PACK * kCols + h];
        lw[k] = sm.l[team.first + w / PACK][w % PACK * kCols + h];
      }
      mm = fmaxf(mm, mw[k]);
    }
#pragma unroll
    for (int k = 1; k < kPer; k <<= 1) mm = fmaxf(mm, __shfl_xor_sync(FULL, mm, k));
    float ll = 0.f;
    unsigned some = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int w = w0 + k * kPer;
      const float f = ex2(mw[k] - mm);
      if (w < ways) sm.weight[way0 + w][h] = f;
      if (lw[k] != 0.f) {
        some |= 1u << w;
        ll = fmaf(f, lw[k], ll);
      }
    }
#pragma unroll
    for (int k = 1; k < kPer; k <<= 1) {
      ll += __shfl_xor_sync(FULL, ll, k);
      some |= __shfl_xor_sync(FULL, some, k);
    }
    if (w0 == 0) {
      sm.some[row][h] = some;
      sm.scale[row][h] = o_row == nullptr ? 1.f : 1.f / ll;      // (the query's scale is done with)
      if (o_row == nullptr && part != nullptr && h < pc.heads) {
        part[kHeads * D + h] = mm;
        part[kHeads * D + kHeads + h] = ll;
      }
    }
  }
  __syncthreads();
  if (o_row != nullptr || part != nullptr) {
    for (int e = 4 * (32 * rank + lane); e < pc.heads * D; e += 4 * 32 * kTeam) {
      const int h = e / D;
      float o[4] = {0.f, 0.f, 0.f, 0.f};
      const unsigned some = sm.some[row][h];
#pragma unroll 8
      for (int w = 0; w < ways; ++w) {
        const bool in = (some >> w) & 1;         // else the buffer holds anything
        const float f = sm.weight[way0 + w][h];
        const float4 v = *reinterpret_cast<const float4*>(
            all + (team.first + w / PACK) * kStride + w % PACK * kCols * D + e);
        o[0] = in ? fmaf(f, v.x, o[0]) : o[0];
        o[1] = in ? fmaf(f, v.y, o[1]) : o[1];
        o[2] = in ? fmaf(f, v.z, o[2]) : o[2];
        o[3] = in ? fmaf(f, v.w, o[3]) : o[3];
      }
      if (o_row == nullptr) {
        *reinterpret_cast<float4*>(part + e) = make_float4(o[0], o[1], o[2], o[3]);
      } else {
        const float inv = some ? sm.scale[row][h] : 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] *= inv;
        if constexpr (of_rows(FORM))
          store_row(o_row + column_at<FORM, D>(p, pc, h) + (e - h * D), o);
        else
          store_row(o_row + e, o);
      }
    }
  }
  __syncthreads();           // before the next piece fills the rings
}

// The row of entry b of the flat list (exact): its sequence (and rows), position
// and blocks, the first of them the one that position pc.first is in; none where
// the position is out of range.  Returns how many rows of the sequence the entry is
// for, pc.tokens of them with a position (chunks).
template <int FORM>
__device__ __forceinline__ int find_row(const DecodeParams& p, int b, Piece& pc, int& blocks) {
  int rows = 1;
  pc.b = b;
  pc.i = 0;
  pc.tokens = 1;
  pc.first = FORM == kOwn ? p.first : 0;
  if constexpr (of_rows(FORM)) {
    pc.b = b / p.each;
    pc.i = (b - pc.b * p.each) * p.tokens;
    const int count = p.len == nullptr ? p.m : min(p.len[pc.b], p.m);
    rows = max(0, min(p.tokens, count - pc.i));
    pc.pos = p.pos[pc.b];
    const int64_t room = pc.pos < 0 ? 0 : (int64_t)p.limit - pc.pos - pc.i;
    pc.tokens = (int)max((int64_t)0, min((int64_t)rows, room));
    if (pc.pos >= 0) pc.pos = (int)min((int64_t)pc.pos + pc.i + max(pc.tokens, 1) - 1, (int64_t)p.limit);
    blocks = pc.tokens == 0 ? 0 : (pc.pos >> 5) + 1;
  } else {
    pc.pos = p.pos[pc.b];
    blocks = pc.pos < pc.first || pc.pos >= p.limit ? 0 : (pc.pos >> 5) - (pc.first >> 5) + 1;
  }
  return rows;
}

// heads of chunk c of a KV head
__device__ __forceinline__ void unit_heads(const DecodeParams& p, int kvh, int c, Piece& pc) {
  pc.kvh = kvh;
  pc.h0 = pc.kvh * p.G + c * p.per_chunk;
  pc.heads = min(p.per_chunk, p.G - c * p.per_chunk);
}

// Exact ALiBi.  The flat list runs over sequences, the units of a sequence,
// and a row's blocks, each row preceded by kRowCost entries that stand for the
// time a row takes to begin and end; CTA i takes entries [i per, (i + 1) per).
// A row whose blocks lie within one CTA is finished there; of one that crosses
// CTAs, each leaves a piece (slot 2 i when it is the CTA's first, else
// 2 i + 1), and the CTA where it ends says in ends[i] which pieces to join.
template <typename T, int D, int PACK, int FORM>
__global__ void __launch_bounds__(32 * kExactWarps, kExactCtas)
q4_exact_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ Slopes slopes) {
  extern __shared__ __align__(128) uint8_t raw[];
  using S = Smem<T, D, kExactWarps, kExactStages, 1>;
  S& sm = *reinterpret_cast<S*>(raw);
  grid_dep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, units = p.c.H * p.chunks;
  const int list = of_rows(FORM) ? p.c.B * p.each : p.c.B;
  Piece pc;
  auto row_entries = [&](int b) -> int64_t {
    int n;
    find_row<FORM>(p, b, pc, n);
    return n == 0 ? 0 : n + kRowCost;
  };
  // all sequences' entries; idle sequences' rows are zeroed on the way, by a
  // thread each (made for a few of them: each is Hq D / 8 stores in a row)
  int64_t sum = 0;
#pragma unroll 4
  for (int b = tid; b < list; b += 32 * kExactWarps) {
    int n;
    const int rows = find_row<FORM>(p, b, pc, n);
    sum += n == 0 ? 0 : n + kRowCost;
    if constexpr (of_rows(FORM)) {
      if (pc.tokens < rows && b % gridDim.x == blockIdx.x) {
        if (p.pos[pc.b] >= 0) atomicOr(p.err, kErrCachePlace);
        for (int h = 0; h < p.Hq; ++h) {
          const int64_t at = ((int64_t)pc.b * p.Hq + h) * p.m + pc.i + pc.tokens;
          uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(p.o) + at * D);
          for (int e = 0; e < (rows - pc.tokens) * D * (int)sizeof(T) / 16; ++e) o[e] = make_uint4(0, 0, 0, 0);
        }
      }
    } else if (n == 0 && b % gridDim.x == blockIdx.x) {
      if (pc.pos >= p.limit) atomicOr(p.err, kErrCachePlace);
      if constexpr (FORM == kOwn) {
        for (int u = 0; u < units; ++u) p.rows[b * units + u] = make_int4(0, 0, 0, 0);
      } else {
        uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(p.o) + (int64_t)b * p.Hq * D);
        for (int e = 0; e < p.Hq * D * (int)sizeof(T) / 16; ++e) o[e] = make_uint4(0, 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
  if ((tid & 31) == 0) sm.sums[warp] = sum;
  if (tid == 0) p.ends[blockIdx.x].x = -1;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < kExactWarps; ++w) total += sm.sums[w];
  total *= units;
  const int64_t fair = (total + gridDim.x - 1) / gridDim.x, per = fair < kMinBlocks ? kMinBlocks : fair;
  const int64_t begin = blockIdx.x * per, end = min(total, begin + per);
  if (begin >= end) return;
  // the sequence that entry `begin` is of, a turn of one sequence a thread
  int64_t base = 0;                       // entries of one unit before the turn's sequences
  for (int b0 = 0;; b0 += 32 * kExactWarps) {
    const int64_t n = b0 + tid < list ? row_entries(b0 + tid) : 0;
    int64_t upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(FULL, upto, o);
      if ((tid & 31) >= o) upto += v;
    }
    __syncthreads();                      // the sums have been read
    if ((tid & 31) == 31) sm.sums[warp] = upto;
    __syncthreads();
    int64_t turn = 0;
#pragma unroll
    for (int w = 0; w < kExactWarps; ++w) {
      if (w < warp) upto += sm.sums[w];
      turn += sm.sums[w];
    }
    if (begin < (base + turn) * units) {
      if (begin >= (base + upto - n) * units && begin < (base + upto) * units) {
        sm.found[0] = b0 + tid;
        sm.found[1] = (base + upto - n) * units;
      }
      break;
    }
    base += turn;
  }
  __syncthreads();
  int at = (int)sm.found[0];
  base = sm.found[1];
  int slot = 2 * blockIdx.x;
  for (int64_t f = begin; f < end;) {
    const int64_t n = row_entries(at), rel = f - base;
    if (rel >= n * units) {
      base += n * units;
      ++at;
      continue;
    }
    const int u = (int)(rel / n);
    const int64_t row = base + u * n, till = min(end, row + n);     // [row, row + n): its entries
    pc.t0 = (int)max((int64_t)0, f - row - kRowCost);
    pc.t1 = (int)(till - row - kRowCost);
    f = till;
    if (pc.t1 <= pc.t0) continue;                 // the row's cost alone
    unit_heads(p, u / p.chunks, u % p.chunks, pc);
    if (FORM == kPacked) pc.heads *= pc.tokens;
    const bool first = pc.t0 == 0, last = till == row + n;
    if (tid == 0 && last && (FORM == kOwn || !first)) {
      const int i0 = (int)((row + kRowCost) / per);    // the CTA of its first block
      const int slot0 = row <= i0 * per ? 2 * i0 : 2 * i0 + 1;
      if constexpr (FORM == kOwn) {
        const int r = at * units + u;
        p.rows[r] = first ? make_int4(p.row_pieces + r, 0, 1, 0)
                          : make_int4(slot0, 2 * (i0 + 1), (int)blockIdx.x - i0 + 1, 0);
      } else {
        p.ends[blockIdx.x] = make_int4(at * units + u, i0, slot0, 0);
      }
    }
    int64_t piece = slot;
    if constexpr (FORM == kOwn) {
      pc.t0 += pc.first >> 5;
      pc.t1 += pc.first >> 5;
      if (first && last) piece = p.row_pieces + at * units + u;
    }
    Query<T, D, PACK> query;
    query.template load<FORM>(p, pc, tid >> 5);
    Ring<T, D, FORM> ring(p, pc, sm.ring[tid >> 5]);
    attend<T, D, true, PACK, FORM>(
        p, pc, Team{0, kExactWarps, 0}, query, slopes.v, nullptr, sm, ring, false,
        FORM != kOwn && first && last
            ? static_cast<T*>(p.o) + (of_rows(FORM) ? 0 : ((int64_t)pc.b * p.Hq + pc.h0) * D)
            : nullptr,
        p.part + piece * part_floats<D>());
    slot = 2 * blockIdx.x + 1;
  }
}

// One head of a row from its pieces: slot `first`, then first2 + step k, n
// pieces in all.  A warp takes every kJoinWarps-th piece, kJoinAhead of them
// in flight (the kernel is one round of loads long where that covers them), a
// lane D / 32 values; the warps join in shared memory.
constexpr int kJoinWarps = 8, kJoinAhead = 4;
template <typename T, int D>
__device__ void join_pieces(const DecodeParams& p, int first, int first2, int step, int n, int h,
                            T* o) {
  constexpr int V = D / 32;
  __shared__ float acc_s[kJoinWarps][D];
  __shared__ float m_s[kJoinWarps], l_s[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float mm = kNothing, ll = 0.f, acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  for (int k0 = warp; k0 < n; k0 += kJoinWarps * kJoinAhead) {
    float mk[kJoinAhead], lk[kJoinAhead], v[kJoinAhead][V];
#pragma unroll
    for (int a = 0; a < kJoinAhead; ++a) {
      const int k = k0 + a * kJoinWarps;
      mk[a] = kNothing;
      lk[a] = 0.f;
      if (k >= n) continue;
      const float* pt = p.part + (int64_t)(k == 0 ? first : first2 + step * (k - 1)) * part_floats<D>();
      mk[a] = pt[kHeads * D + h];
      lk[a] = pt[kHeads * D + kHeads + h];
      if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4*>(pt + h * D + 4 * lane);
        v[a][0] = x.x, v[a][1] = x.y, v[a][2] = x.z, v[a][3] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(pt + h * D + 2 * lane);
        v[a][0] = x.x, v[a][1] = x.y;
      }
    }
    float to = mm;
#pragma unroll
    for (int a = 0; a < kJoinAhead; ++a) to = fmaxf(to, mk[a]);
    const float f0 = ex2(mm - to);
    mm = to;
    ll *= f0;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= f0;
#pragma unroll
    for (int a = 0; a < kJoinAhead; ++a) {
      if (lk[a] == 0.f) continue;          // nothing of the piece was seen, or written
      const float f = ex2(mk[a] - mm);
      ll = fmaf(f, lk[a], ll);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = fmaf(f, v[a][e], acc[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) acc_s[warp][V * lane + e] = acc[e];
  if (lane == 0) {
    m_s[warp] = mm;
    l_s[warp] = ll;
  }
  __syncthreads();
  if (threadIdx.x < D) {
    float to = m_s[0], sum = 0.f, a = 0.f;
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) to = fmaxf(to, m_s[w]);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = ex2(m_s[w] - to);
      sum = fmaf(f, l_s[w], sum);
      a = fmaf(f, acc_s[w][threadIdx.x], a);
    }
    o[threadIdx.x] = Elem<T>::put(sum == 0.f ? 0.f : a / sum);
  }
}

template <typename T, int D, int FORM>
__global__ void __launch_bounds__(32 * kJoinWarps) q4_exact_join_kernel(const __grid_constant__ DecodeParams p) {
  grid_dep_wait();
  const int4 end = p.ends[blockIdx.x];
  if (end.x < 0) return;
  const int units = p.c.H * p.chunks, h = blockIdx.y;
  Piece pc;
  int blocks;
  find_row<FORM>(p, end.x / units, pc, blocks);
  unit_heads(p, end.x % units / p.chunks, end.x % p.chunks, pc);
  if (FORM == kPacked) pc.heads *= pc.tokens;
  if (h >= pc.heads) return;
  join_pieces<T, D>(p, end.z, 2 * (end.y + 1), 2, (int)blockIdx.x - end.y + 1, h,
                    static_cast<T*>(p.o) + column_at<FORM, D>(p, pc, h));
}

// Approximate.  KV heads by the largest scale of their query heads, widest
// first (the longest envelopes start first), all rows (sequences and chunks) of
// a KV head together.  A row is attended by a team of 1, 2, 4 or 8 warps, so
// that a warp has a few blocks however wide the head's envelopes; a CTA has
// 8 / team rows.  Rows wider than eight warps' worth go to several CTAs, where
// the grid has room: to a cluster, which joins them in its shared memory, or,
// where 8 CTAs leave too much for one, to more that a second kernel joins.
struct Groups {
  int first[kMaxGroupOrder + 1];          // first CTA of each KV head, in order
  uint8_t order[kMaxGroupOrder];
  uint8_t shares[kMaxGroupOrder];         // CTAs of a row, in order
  uint8_t team[kMaxGroupOrder];           // log2 of the warps of a row, in order
  int ordered;                            // 0: index order, shares[0] and team[0] for all
  int cluster;                            // > 1: a row's shares, and the CTAs of a cluster
};

// CTAs of a KV head: `rows` rows by teams of `team` warps, or by `shares` CTAs each
__host__ __device__ __forceinline__ int group_ctas(int rows, int team, int shares) {
  const int held = kApproxWarps / team;
  return shares > 1 ? rows * shares : (rows + held - 1) / held;
}

// The pieces of one row that the CTAs of a cluster hold at `part` of their
// shared memory, joined and stored by the first; all threads call it.
template <typename T, int D>
__device__ __forceinline__ void join_cluster(const float* part, int rank, int n, int heads, T* o) {
  static_assert(kHeads * D <= 4 * 32 * kApproxWarps, "four values a thread");
  cluster_sync();
  const int e = 4 * threadIdx.x, h = e / D;
  if (rank == 0 && h < heads) {
    const uint32_t at = smem_u32(part);
    float m[kMaxCluster], l[kMaxCluster];
    float4 v[kMaxCluster];
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) {
      m[k] = kNothing;
      l[k] = 0.f;
      if (k < n) {
        const uint32_t there = cluster_addr(at, k);
        m[k] = ld_cluster(there + 4 * (kHeads * D + h));
        l[k] = ld_cluster(there + 4 * (kHeads * D + kHeads + h));
        v[k] = ld_cluster4(there + 4 * e);
      }
    }
    float mm = m[0], sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 1; k < kMaxCluster; ++k) mm = fmaxf(mm, m[k]);
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) {
      if (l[k] == 0.f) continue;           // nothing of the piece was seen
      const float f = ex2(m[k] - mm);
      sum = fmaf(f, l[k], sum);
      acc[0] = fmaf(f, v[k].x, acc[0]);
      acc[1] = fmaf(f, v[k].y, acc[1]);
      acc[2] = fmaf(f, v[k].z, acc[2]);
      acc[3] = fmaf(f, v[k].w, acc[3]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] *= inv;
    store_row(o + e, acc);
  }
  __syncwarp();
  cluster_sync();                          // the others' shared memory has been read
}

template <typename T, int D, int PACK>
__global__ void __launch_bounds__(32 * kApproxWarps, kApproxCtas)
q4_approx_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ Groups gr) {
  extern __shared__ __align__(128) uint8_t raw[];
  using S = Smem<T, D, kApproxWarps, kApproxStages, kApproxWarps>;
  S& sm = *reinterpret_cast<S*>(raw);
  grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, rows = p.c.B * p.chunks;
  int cta = blockIdx.x, k = 0;
  if (gr.ordered) {
    while (k + 1 < p.c.H && cta >= gr.first[k + 1]) ++k;
    cta -= gr.first[k];
  }
  const int log_size = gr.team[k], size = 1 << log_size, shares = gr.shares[k];
  int kvh = gr.ordered ? gr.order[k] : 0;
  if (!gr.ordered) {
    const int each = group_ctas(rows, size, shares);
    kvh = cta / each;
    cta -= kvh * each;
  }
  Team team;
  team.size = size;
  team.first = warp & -size;
  team.number = warp >> log_size;
  const int rank = warp - team.first, number = team.number;
  const int share = shares > 1 ? cta % shares : 0;
  const int row = shares > 1 ? cta / shares : cta * (kApproxWarps >> log_size) + number;
  const bool valid = row < rows;
  Piece pc;
  const int b = p.chunks == 1 ? row : row / p.chunks;
  pc.b = valid ? b : 0;
  unit_heads(p, kvh, row - b * p.chunks, pc);
  pc.pos = valid ? p.pos[pc.b] : -1;
  const bool none = pc.pos < 0 || pc.pos >= p.limit;
  if (valid && none && rank == 0 && lane == 0 && pc.pos >= 0) atomicOr(p.err, kErrCachePlace);
  Query<T, D, PACK> query;
  query.template load<kStep>(p, pc, rank);
  Ring<T, D, kStep> ring(p, pc, sm.ring[warp]);
  // A warp's first block is copied before the bins are known: the newest of the
  // row, always needed, or the next ones, which the team's size makes likely
  // (a page of its own only if its index is good: whether it is needed, and to
  // be reported, is not known yet).
  const int next = (pc.pos >> 5) - rank;
  bool ahead = share == 0 && !none && p.c.page_shift > 4 && next >= 0;
  int32_t next_page = ahead ? ring.page_of(next) : -1;
  // the heads' bin starts: a head a warp and turn, a hash a lane; the first 32
  // hashes' are on their way while the query is prepared
  const int quads = (p.s + 3) >> 2, width = 4 * quads;
  int4* starts = reinterpret_cast<int4*>(raw + sizeof(S)) + number * kHeads * quads;
  auto start_of = [&](int h, int x) {
    return bin_lo(load_record(p.rec, ((int64_t)(pc.h0 + h) * p.s + x) * p.W + (pc.pos >> 5)), pc.pos);
  };
  int v[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = rank + (i << log_size);
    v[i] = INT_MAX;
    if (h < pc.heads && !none && lane < p.s) v[i] = start_of(h, lane);
  }
  ahead = ahead && (uint32_t)next_page < (uint32_t)p.c.pages;
  if (ahead) ring.fetch(next, 0, next_page, 0);       // (a page holds both tiles)
  prepare_query<T, D, PACK>(query, rank, size, number, sm);
  int oldest = INT_MAX;
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = rank + (i << log_size);
    if (h >= kHeads) break;
    oldest = min(oldest, v[i]);
    if (lane < width) reinterpret_cast<int*>(starts)[h * width + lane] = v[i];
    if (lane + 32 < width) {
      const int w = h < pc.heads && lane + 32 < p.s && !none ? start_of(h, lane + 32) : INT_MAX;
      oldest = min(oldest, w);
      reinterpret_cast<int*>(starts)[h * width + lane + 32] = w;
    }
  }
  oldest = __reduce_min_sync(FULL, oldest);
  if (lane == 0) sm.some[0][warp] = (unsigned)oldest;       // (a row of kHeads, before its use)
  __syncthreads();
  pc.first = pc.pos;
  pc.t0 = pc.t1 = 0;
  if (!none) {
    for (int w = 0; w < size; ++w) pc.first = min(pc.first, (int)sm.some[0][team.first + w]);
    const int t_first = pc.first >> 5, n = (pc.pos >> 5) + 1 - t_first;
    const int len = (n + shares - 1) / shares;
    pc.t1 = t_first + n - share * len;            // share 0 the newest
    pc.t0 = max(t_first, pc.t1 - len);
  }
  T* o = static_cast<T*>(p.o) + ((int64_t)pc.b * p.Hq + pc.h0) * D;
  // (the queries' operands are done with when a piece is written)
  static_assert(sizeof(sm.q) >= sizeof(float) * part_floats<D>(), "a piece fits");
  float* part = gr.cluster > 1 ? reinterpret_cast<float*>(sm.q)
                               : p.part + (int64_t)blockIdx.x * part_floats<D>();
  attend<T, D, false, PACK, kStep>(p, pc, team, query, nullptr, starts, sm, ring, ahead,
                            valid && shares == 1 ? o : nullptr, valid && shares > 1 ? part : nullptr);
  if (gr.cluster > 1 && shares > 1 && valid) join_cluster<T, D>(part, share, shares, pc.heads, o);
}

template <typename T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
q4_approx_join_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ Groups gr) {
  grid_dep_wait();
  const int rows = p.c.B * p.chunks, k = blockIdx.x / rows, row = blockIdx.x - k * rows, h = blockIdx.y;
  const int shares = gr.shares[gr.ordered ? k : 0];
  Piece pc;
  unit_heads(p, gr.ordered ? gr.order[k] : k, row % p.chunks, pc);
  if (h >= pc.heads || shares == 1) return;
  const int first = (gr.ordered ? gr.first[k] : k * rows * shares) + row * shares;
  join_pieces<T, D>(p, first, first + 1, 1, shares, h,
                    static_cast<T*>(p.o) + ((int64_t)(row / p.chunks) * p.Hq + pc.h0 + h) * D);
}

int max_ctas(int num_sms) { return num_sms * kExactCtas; }

template <typename T, int D, int FORM>
cudaError_t launch_exact(DecodeParams& p, const Q4DecodeArgs& a, cudaStream_t st) {
  using S = Smem<T, D, kExactWarps, kExactStages, 1>;
  Slopes s;
  for (int h = 0; h < a.Hq; ++h) s.v[h] = a.slope_log2[h];
  // (a limit up to 2^31 - 16)
  const int64_t list = (int64_t)p.c.B * (of_rows(FORM) ? p.each : 1);
  const int columns = p.per_chunk * (FORM == kPacked ? p.tokens : 1);
  const int64_t entries = list * p.c.H * p.chunks * (((int64_t)p.limit + 31) / 32 + kRowCost);
  const int64_t want = (entries + kMinBlocks - 1) / kMinBlocks;
  const unsigned grid = (unsigned)std::min<int64_t>(max_ctas(a.num_sms), want);
  auto kern = columns <= 4 ? q4_exact_kernel<T, D, 2, FORM> : q4_exact_kernel<T, D, 1, FORM>;
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kern), (int)sizeof(S));
  if (e == cudaSuccess) e = launch_dependent(kern, dim3(grid), 32 * kExactWarps, sizeof(S), st, p, s);
  if (e == cudaSuccess && FORM != kOwn)
    e = launch_dependent(q4_exact_join_kernel<T, D, FORM>, dim3(grid, columns), 32 * kJoinWarps, 0, st, p);
  return e;
}

template <typename T, int D>
cudaError_t launch_approx(DecodeParams& p, const Q4DecodeArgs& a, cudaStream_t st) {
  const int H = p.c.H, rows = p.c.B * p.chunks;
  // The distance back to the start of a position's bin exceeds a with probability
  // e^{-a/sigma}, so that the furthest of the s n bin starts of a KV head's n query
  // heads lies about sigma (0.58 + ln(s n)) back; 1 for a little more than the mean.
  const double reach = 1.0 + log((double)p.s * std::min(p.G, kHeads));
  Groups gr;
  // (more KV heads are not ordered, and all get the team of the widest: 8 sequences
  // of 64 heads with ALiBi's scales 19.5 us, of 32 heads 10.2)
  gr.ordered = H <= kMaxGroupOrder && a.sigma != nullptr;
  const int groups = gr.ordered ? H : 1;
  double blocks[kMaxGroupOrder] = {};             // a row's, expected, by KV head; [0] the widest if not ordered
  for (int h = 0; h < a.Hq; ++h) {
    const double sigma = a.sigma ? a.sigma[h] : 1e30;
    double& x = blocks[gr.ordered ? h / p.G : 0];
    x = std::max(x, std::min(reach * sigma, (double)p.limit) / 32.0 + 1.0);
  }
  for (int k = 0; k < groups; ++k) gr.order[k] = (uint8_t)k;
  std::stable_sort(gr.order, gr.order + groups, [&](int x, int y) { return blocks[x] > blocks[y]; });
  // the fewest blocks a warp for which all warps fit `room` (found in steps of a
  // fifth; in halves: 64 sequences 14.3 us against 13.8, 16 of 20 hashes 12.5
  // against 10.1, means over ten draws), a KV head that
  // wants more than a CTA's taking a cluster (of eight CTAs, no more than 288 of
  // 304 find room); else kTeamBlocks, in turns
  // (two CTAs an SM are counted on; where one fits, such a grid runs in two turns:
  // 16 sequences of 32/8 heads of 128, s = 10, 17.8 us in fp32, 10.5 in bf16)
  const int64_t room = (int64_t)a.num_sms * kApproxCtas;
  int64_t grid = 0;
  for (double each = 1.0;; each *= 1.19) {
    const bool last = each > 8.0;
    if (last) each = kTeamBlocks;
    gr.cluster = 1;
    while (!last && gr.cluster < kMaxCluster && gr.cluster * kApproxWarps * each < blocks[gr.order[0]]) gr.cluster *= 2;
    grid = 0;
    for (int k = 0; k < groups; ++k) {
      const double wide = blocks[gr.order[k]];
      int team = 0;
      while ((1 << team) < kApproxWarps && (1 << team) * each < wide) ++team;
      gr.team[k] = (uint8_t)team;
      gr.shares[k] = (uint8_t)(kApproxWarps * each < wide ? gr.cluster : 1);
      grid += group_ctas(rows, 1 << team, gr.shares[k]);
    }
    if (!gr.ordered) grid *= H;
    if (last || grid <= (gr.cluster > 2 ? room - room / 16 : room)) break;
  }
  // and rows of more than kShareBlocks a CTA to more of them, evenly, while they fit
  bool split = false;
  for (double each = kShareBlocks; each * gr.cluster < blocks[gr.order[0]]; each *= 2.0) {
    int64_t g = 0;
    uint8_t shares[kMaxGroupOrder];
    for (int k = 0; k < groups; ++k) {
      shares[k] = (uint8_t)std::min((double)kMaxShares, std::max(1.0, ceil(blocks[gr.order[k]] / each)));
      if ((1 << gr.team[k]) < kApproxWarps) shares[k] = 1;
      g += (int64_t)(gr.ordered ? 1 : H) * group_ctas(rows, 1 << gr.team[k], shares[k]);
    }
    if (g > room) continue;
    std::copy(shares, shares + groups, gr.shares);
    gr.cluster = 1;
    split = gr.shares[0] > 1;
    grid = g;
    break;
  }
  grid = (grid + gr.cluster - 1) / gr.cluster * gr.cluster;     // (rows past the last group's are none)
  int64_t at = 0;
  for (int k = 0; k < groups; ++k) {
    gr.first[k] = (int)at;
    at += group_ctas(rows, 1 << gr.team[k], gr.shares[k]);
  }
  gr.first[groups] = (int)at;
  using S = Smem<T, D, kApproxWarps, kApproxStages, kApproxWarps>;
  const size_t smem = sizeof(S) + sizeof(int4) * kApproxWarps * kHeads * ((p.s + 3) / 4);
  auto kern = p.per_chunk <= 4 ? q4_approx_kernel<T, D, 2> : q4_approx_kernel<T, D, 1>;
  cudaError_t e = set_smem_limit(reinterpret_cast<const void*>(kern),
                                 (int)(sizeof(S) + sizeof(int) * kApproxWarps * kHeads * kMaxS));
  if (e == cudaSuccess)
    e = launch_clusters((unsigned)gr.cluster, kern, dim3((unsigned)grid), 32 * kApproxWarps, smem, st, p, gr);
  if (e == cudaSuccess && split)
    e = launch_dependent(q4_approx_join_kernel<T, D>, dim3((unsigned)(rows * H), p.per_chunk),
                         32 * kJoinWarps, 0, st, p, gr);
  return e;
}

template <typename T, int D>
cudaError_t launch_typed(DecodeParams& p, const Q4DecodeArgs& a, cudaStream_t st) {
  if (a.rec) return launch_approx<T, D>(p, a, st);
  if (a.m > 0) return p.tokens > 1 ? launch_exact<T, D, kPacked>(p, a, st) : launch_exact<T, D, kRows>(p, a, st);
  if constexpr (sizeof(T) == 2)
    if (a.rows != nullptr) return launch_exact<T, D, kOwn>(p, a, st);
  if (a.prefix != nullptr) return launch_exact<T, D, kShared>(p, a, st);
  return launch_exact<T, D, kStep>(p, a, st);
}

}  // namespace

// ends [CTAs] int4, then two pieces of a CTA (exact), or one of a share
int64_t q4_decode_work_bytes(int d, int num_sms) {
  return (int64_t)max_ctas(num_sms) * (sizeof(int4) + 2 * sizeof(float) * kHeads * (d + 2));
}

// behind these, a piece and an int4 of every row
int q4_own_rows(int B, int Hkv, int G) { return B * Hkv * ((G + kHeads - 1) / kHeads); }
int64_t q4_own_work_bytes(int d, int num_sms, int B, int Hkv, int G) {
  return q4_decode_work_bytes(d, num_sms) +
         (int64_t)q4_own_rows(B, Hkv, G) * (sizeof(int4) + sizeof(float) * kHeads * (d + 2));
}

const float* q4_own_pieces(const void* work, int num_sms) {
  return reinterpret_cast<const float*>(static_cast<const int4*>(work) + max_ctas(num_sms));
}

cudaError_t launch_q4_decode(const Q4DecodeArgs& a, cudaStream_t st) {
  DecodeParams p;
  p.c = a.c;
  p.q = a.q;
  p.o = a.o;
  p.pos = a.pos;
  p.Hq = a.Hq;
  p.G = a.Hq / a.c.H;
  p.chunks = (p.G + kHeads - 1) / kHeads;
  p.per_chunk = (p.G + p.chunks - 1) / p.chunks;
  p.rec = a.rec;
  p.s = a.s;
  p.W = a.W;
  const int64_t held = a.c.max_pages << a.c.page_shift;
  p.limit = (int)(a.rec ? std::min(held, a.bins_n) : held);
  p.ends = static_cast<int4*>(a.work);
  p.part = reinterpret_cast<float*>(p.ends + max_ctas(a.num_sms));
  p.err = a.err;
  p.m = a.m;
  // (evenly: nine rows of one head are five and four)
  const int most = p.G <= 4 ? kHeads / p.G : 1;
  p.each = std::max(1, (a.m + most - 1) / most);
  p.tokens = std::max(1, (a.m + p.each - 1) / p.each);
  p.len = a.len;
  p.prefix = a.prefix;
  p.prefix_pages = a.prefix_pages;
  p.first = a.prefix_pages << a.c.page_shift;
  p.rows = a.rows;
  p.row_pieces = 2 * max_ctas(a.num_sms);
  if (a.dtype == PLSH_BF16)
    return a.c.d == 64 ? launch_typed<__nv_bfloat16, 64>(p, a, st)
                       : launch_typed<__nv_bfloat16, 128>(p, a, st);
  return a.c.d == 64 ? launch_typed<float, 64>(p, a, st) : launch_typed<float, 128>(p, a, st);
}

}  // namespace plsh
