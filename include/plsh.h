/*
 * plsh.h -- C ABI of the Positional LSH approximate-ALiBi attention library
 * for GB300 (sm_103a).
 *
 * The method ("Positional LSH: Binary Block Matrix Approximation for
 * Attention with Linear Biases", Wolfson & Wagner; technical summary):
 *   Methodology 1   L*_ij = exp(-|i-j|/sigma) is a Laplacian kernel on token
 *                   positions.  A random-binning hash of the integer positions
 *                   splits 0..n-1 into contiguous bins; M(h) is 1 where i and
 *                   j share a bin, and L* = E_h[M(h)].
 *   Methodology 2   (Theorem 2.1) the mean M~ of s i.i.d. masks approximates
 *                   L*; bin widths follow a Gamma law.
 *   Methodology 3   (Theorem 2.2) ALiBi attention becomes s sets of short
 *                   block attentions with no positional bias:
 *                     T~ = D~^-1 (M~ o exp(QK^T/sqrt(d))) V,
 *                   numerator and row sums both averaged over the s masks.
 *
 * Conventions shared by every call:
 *   - Tensors are [B, H, n, d] contiguous row-major, on the CUDA device
 *     that is current when the call is made, 16-byte aligned.  Query head h
 *     reads KV head h / (Hq / Hkv) (contiguous GQA groups).
 *   - The caller owns Q, K, V and O.  The library owns plsh_bins handles and
 *     its per-device work-queue state.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Every call
 *     is asynchronous on it except where a comment says it synchronises.
 *   - Arguments are validated before anything is launched; on a validation
 *     error nothing is written and the status says why (plsh_last_error()
 *     holds a message for the calling thread).  No call aborts or prints.
 */
#ifndef PLSH_H_
#define PLSH_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PLSH_OK = 0,
  PLSH_ERR_INVALID = 1,      /* bad argument: shape, dtype, range, pointer  */
  PLSH_ERR_CUDA = 2,         /* a CUDA runtime/driver call failed           */
  PLSH_ERR_NOMEM = 3,        /* device or host allocation failed            */
  PLSH_ERR_TIMEOUT = 4,      /* a device-side bounded wait ran out          */
  PLSH_ERR_UNSUPPORTED = 5,  /* valid request the library does not serve    */
  PLSH_ERR_RANGE = 6         /* input values beyond the range the kernel
                                computes in (V beyond +-65504 on the
                                tensor-core path; over a 4-bit cache V's
                                groups too far apart), found on the device  */
} plsh_status;

/* Which kernel serves an attention call (plsh_attn_path). */
typedef enum { PLSH_PATH_CUDA_CORES = 0, PLSH_PATH_TENSOR_CORES = 1 } plsh_path;

typedef enum { PLSH_F32 = 0, PLSH_BF16 = 1 } plsh_dtype;

/* A device tensor [B, H, n, d], contiguous, element type `dtype`.
 * `data` is a device pointer the caller owns. */
typedef struct {
  void* data;
  int32_t dtype;   /* plsh_dtype */
  int64_t B, H, n, d;
} plsh_tensor;

/* Opaque set of s bin partitions per head (one per hash), resident on one
 * device.  Owns its device memory; reusable by any number of attention
 * calls (the same draws serve every batch element and layer). */
typedef struct plsh_bins plsh_bins;

/*
 * plsh_sample_bins -- draw s random-binning hashes per head and build their
 * bins on the device (Methodology 1-2).
 *
 * For head h and sample t the counter-based generator Philox4x32-10 (key =
 * seed, counter = (t, h, 0, 0)) gives U0, U1, U2 = (x + 0.5) 2^-32; the width
 * is w = sigma_h (-ln U0 - ln U1) ~ Gamma(shape 2, scale sigma_h) and the
 * offset u = w U2 ~ U(0, w).  Bin starts are 0 and ceil(u + k w) for
 * k = 0, 1, ... below n, u + k w one fused multiply-add (every position its
 * own bin when w < 1).  The arithmetic is fp64, each operation (a fused
 * multiply-add counts as one) rounded once, so the starts agree bit for bit
 * with any other implementation of the same recipe.
 *
 *   n        sequence length, 1 <= n < 2^31
 *   sigma_h  host array [H], each finite and > 0 (sigma = 1 / ALiBi slope)
 *   H        number of query heads, >= 1
 *   s        hashes per head, 1 <= s <= 64
 *   seed     64-bit generator key
 *   out      receives a new handle (free with plsh_bins_free)
 * Allocates device memory (synchronous allocation), then launches the
 * sampler on `stream`.  On error *out is left unchanged.
 */
plsh_status plsh_sample_bins(int64_t n, const double* sigma_h, int32_t H,
                             int32_t s, uint64_t seed, void* stream,
                             plsh_bins** out);

/*
 * plsh_bins_resample -- redraw an existing handle in place with new sigma_h
 * and seed (same n, H, s).  Allocates nothing; fully asynchronous.  The
 * previous contents must no longer be in use by work queued on other
 * streams.
 */
plsh_status plsh_bins_resample(plsh_bins* bins, const double* sigma_h,
                               uint64_t seed, void* stream);

/*
 * plsh_bins_from_host -- build a handle from explicit bin boundaries (for
 * deterministic variants such as fixed blocks, or draws made elsewhere).
 *   offsets  host int64 [H*s + 1]; hash (h, t) owns
 *            starts[offsets[h*s+t] .. offsets[h*s+t+1])
 *   starts   host int32; each hash's list begins with 0, strictly increases
 *            and ends with the terminal n
 * Validated on the host; synchronous upload.
 */
plsh_status plsh_bins_from_host(int64_t n, int32_t H, int32_t s,
                                const int64_t* offsets, const int32_t* starts,
                                void* stream, plsh_bins** out);

/*
 * plsh_bins_fixed -- deterministic fixed blocks in place of random hashes (the
 * "fixed blocks" baseline of the summary's Mistral fine-tuning experiment,
 * Experimental validation): hash t of head h cuts 0..n-1 into contiguous
 * blocks of width_h[h] positions, shifted by o = floor(t * width_h[h] / s),
 * i.e. bin starts {0} u {o + k * width_h[h] : k >= 0} inside [1, n).  With
 * s = 1 these are plain blocks [0, w), [w, 2w), ...; larger s averages s
 * evenly shifted grids, the deterministic counterpart of the random offsets.
 *   width_h: host array [H], every entry >= 1.  1 <= s <= 64, 1 <= n < 2^31.
 * The records are built on the device in closed form; the call waits for it
 * (the host arrays it uploads are its own).  The handle is used exactly like
 * one from plsh_sample_bins (plsh_bins_draws reports w = width, u = o);
 * plsh_bins_resample on it draws random bins.
 */
plsh_status plsh_bins_fixed(int64_t n, const int32_t* width_h, int32_t H, int32_t s,
                            void* stream, plsh_bins** out);

/*
 * plsh_alibi_attn_backward -- gradients of sum(T~ * dO) with respect to Q, K
 * and V (the backward pass of plsh_alibi_attn, Methodology 3's estimator with
 * the multiplicities c_ij held fixed):
 *   P_ij = c_ij e^{S_ij} / sum_j c_ij e^{S_ij},  dP_ij = dO_i . v_j,
 *   dS_ij = P_ij (dP_ij - sum_l P_il dP_il),
 *   dQ_i = sum_j dS_ij k_j / sqrt(d),  dK_j = sum_i dS_ij q_i / sqrt(d),
 *   dV_j = sum_i P_ij dO_i,
 * a KV head collecting the sums of every query head that reads it.
 *   Q, dO, dQ [B,Hq,n,d]; K, V, dK, dV [B,Hkv,n,d]; one dtype (PLSH_BF16 or
 *   PLSH_F32), d in {64, 128}; bins and causal as for plsh_alibi_attn.
 * Tensor cores (bf16, d = 128, s <= 16, Hq / Hkv <= 64; plsh_attn_path names
 * the path): the forward kernel in a row statistics mode writes each row's
 * max, sum and Delta_i = dO_i . O_i, then a kernel per (batch, KV head, key
 * tile) forms S^T, dP^T, dV, dK and dS K with tcgen05 products (P and dS
 * rounded to bf16, fp32 accumulation), the dS K rows added to an fp32 dQ
 * accumulator by TMA reductions and converted to bf16 at the end.
 * CUDA cores (every other case), fp32 accumulation, no atomics: a warp per
 * row computes the row's max, sum and sum_j P_ij dP_ij and dQ_i; a warp per
 * key then sums dK_j and dV_j over the rows whose bins contain it.
 * Scratch (2 or 3 B Hq n floats of row statistics, plus B Hq n d floats of
 * dQ accumulator on the tensor cores) lives in a device buffer the library
 * keeps per device between calls, grown on demand in stream order on
 * `stream` (from the device's stream-ordered memory pool); calls on
 * different streams are ordered on it by an event.
 * Asynchronous on `stream`.
 */
plsh_status plsh_alibi_attn_backward(const plsh_tensor* Q, const plsh_tensor* K,
                                     const plsh_tensor* V, const plsh_tensor* dO,
                                     const plsh_bins* bins, int32_t causal, plsh_tensor* dQ,
                                     plsh_tensor* dK, plsh_tensor* dV, void* stream);

/*
 * plsh_alibi_attn_backward_lse -- the same gradients from the forward pass's
 * output O and log-sum-exp lse (written by plsh_alibi_attn_lse for the same
 * Q, K, V, bins and causal), as a training step has them: the rows'
 * Delta_i = dO_i . O_i comes from O (bf16, as stored) in a pass over the rows
 * instead of a recomputation of the forward pass.
 *   O [B,Hq,n,d] with Q's shape and dtype; lse [B*Hq*n] fp32 device memory.
 * Tensor cores only (bf16, d = 128, s <= 16, Hq / Hkv <= 64): other inputs
 * return PLSH_ERR_UNSUPPORTED.  Scratch, ordering and errors as for
 * plsh_alibi_attn_backward.  Asynchronous on `stream`.
 */
plsh_status plsh_alibi_attn_backward_lse(const plsh_tensor* Q, const plsh_tensor* K,
                                         const plsh_tensor* V, const plsh_tensor* O,
                                         const float* lse, const plsh_tensor* dO,
                                         const plsh_bins* bins, int32_t causal, plsh_tensor* dQ,
                                         plsh_tensor* dK, plsh_tensor* dV, void* stream);

/*
 * plsh_bias_error -- the bias of the averaged mask for head h of `bins`:
 * ||L* - M~||_max and ||L* - M~||_2 with L*_ij = e^{-|i-j|/sigma} (Problem
 * statement) and M~ = (1/s) sum_t M(h_t) (Methodology 1-2), the two norms the
 * summary's convergence experiment follows against s (Results).  Neither
 * n x n matrix is formed: the max norm is exact (per row over its key
 * envelope); the spectral norm, the largest eigenvalue magnitude of the
 * symmetric difference, is estimated by `lanczos_iters` Lanczos steps from a
 * start vector drawn from `seed`, with O(n s) products (the Laplace kernel as
 * two linear recurrences, the mask through prefix sums).  fp64 throughout.
 *   sigma > 0 (the scale L* is taken at), 0 <= h < H,
 *   2 <= lanczos_iters <= 1000 when spectral is requested.
 *   max_abs, spectral: host outputs; either may be NULL to skip it.
 * Blocks until done (device scratch of 6 n doubles, allocated per call).
 */
plsh_status plsh_bias_error(const plsh_bins* bins, double sigma, int32_t h,
                            int32_t lanczos_iters, uint64_t seed, double* max_abs,
                            double* spectral, void* stream);

/*
 * plsh_bins_share_groups -- hashes shared across a GQA group: bins for Hq
 * query heads in which head h uses every hash (records, draws and scale) of
 * head floor(h / (Hq / G)) of `src`, G = src's number of heads, Hq % G == 0.
 * Drawn with one scale per KV group (plsh_sample_bins with G heads), the heads
 * of a group then cut the positions identically, so the key envelopes of two
 * heads of one group coincide.  A variant outside the summary's method (each
 * of its heads draws its own hashes).  Device-to-device copies; the call
 * waits for them.  plsh_bins_resample on the result draws per-head hashes.
 */
plsh_status plsh_bins_share_groups(const plsh_bins* src, int32_t Hq, void* stream,
                                   plsh_bins** out);

/* Shape of a handle.  n_entries (bins + terminals over all hashes) needs the
 * device contents: this call synchronises `stream` when n_entries != NULL. */
plsh_status plsh_bins_info(const plsh_bins* bins, int64_t* n, int32_t* H,
                           int32_t* s, int64_t* n_entries, void* stream);

/*
 * plsh_bins_to_host -- copy the bin boundaries back in the plsh_bins_from_host
 * layout.  offsets [H*s+1]; starts must hold `cap` entries (query the size
 * with plsh_bins_info).  Synchronises `stream`.
 */
plsh_status plsh_bins_to_host(const plsh_bins* bins, int64_t* offsets,
                              int32_t* starts, int64_t cap, void* stream);

/* Draws (w, u) of every (h, t), host arrays [H*s] (either may be NULL).
 * Synchronises `stream`. */
plsh_status plsh_bins_draws(const plsh_bins* bins, double* w, double* u,
                            void* stream);

/* Frees the handle's device memory (synchronises the device first). */
void plsh_bins_free(plsh_bins* bins);

/*
 * plsh_alibi_attn -- approximate ALiBi attention T~ (Methodology 3).
 *
 * For each batch b, query head h and row i, with J_t(i) the bin of i under
 * hash t of head h (clipped to j <= i when causal):
 *   O_i = sum_t sum_{j in J_t(i)} e^{S_ij} v_j / sum_t sum_{j in J_t(i)} e^{S_ij},
 *   S_ij = q_i . k_j / sqrt(d).
 * Computed as sum_j c_ij e^{S_ij} v_j / sum_j c_ij e^{S_ij}, with c_ij the
 * number of hashes that put i and j in one bin.
 *
 *   Q [B,Hq,n,d]; K, V [B,Hkv,n,d]; O [B,Hq,n,d], all the same dtype,
 *   Hq % Hkv == 0, bins->n == n, bins->H == Hq, d in {64, 128}.
 *   causal   non-zero: keys j <= i only.
 * Kernels (plsh_attn_path tells which one a call takes, without launching):
 *   tensor cores  bf16 with d in {64, 128} and s within the kernel's shared
 *                 memory (s <= 52 causal, s <= 29 without the mask; d = 64
 *                 runs zero-padded to 128 columns in shared memory, at the
 *                 cost of d = 128): QK^T in
 *                 bf16, the weights P and V in f16 for P V (every bf16
 *                 value of V up to 65504 is an f16 value; P keeps 11
 *                 significant bits), fp32 accumulation and softmax.  A value of V beyond +-65504 is reported by
 *                 plsh_stream_status() as PLSH_ERR_RANGE (O is then not
 *                 valid); T~ is linear in V, so V scaled down by a power of
 *                 two gives O scaled down by the same power.
 *   CUDA cores    everything else (fp32, larger s): fp32 throughout.
 * Asynchronous on `stream`.  A device-side wait that runs out (a bug, never
 * expected) is reported by the next plsh_stream_status().  The tensor-core
 * path keeps a work-item table per shape and head order on the device
 * (allocated and uploaded on `stream` at the first call of a shape, in stream
 * order; up to 16 are cached, and the least recently used one that no call
 * holds is freed, in stream order behind the work of the calls that used
 * it, when a seventeenth shape arrives).
 */
plsh_status plsh_alibi_attn(const plsh_tensor* Q, const plsh_tensor* K,
                            const plsh_tensor* V, const plsh_bins* bins,
                            int32_t causal, plsh_tensor* O, void* stream);

/*
 * plsh_alibi_attn_lse -- plsh_alibi_attn that also writes every row's
 * base-2 log-sum-exp of its scaled scores with their multiplicities,
 *   lse_i = log2 sum_j c_ij 2^{x_ij},  x_ij = q_i . k_j log2(e) / sqrt(d)
 * (so that T~_i = sum_j c_ij 2^{x_ij - lse_i} v_j), the statistic the backward
 * pass needs (plsh_alibi_attn_backward_lse).
 *   lse [B*Hq*n] fp32 device memory, row (b, h, i) at (b*Hq + h)*n + i.
 * Tensor-core path only (bf16, d in {64, 128}, s within its budget;
 * plsh_attn_path):
 * other inputs return PLSH_ERR_UNSUPPORTED.  O as for plsh_alibi_attn.
 * Asynchronous on `stream`.
 */
plsh_status plsh_alibi_attn_lse(const plsh_tensor* Q, const plsh_tensor* K,
                                const plsh_tensor* V, const plsh_bins* bins, int32_t causal,
                                plsh_tensor* O, float* lse, void* stream);

/*
 * plsh_alibi_attn_noalloc -- plsh_alibi_attn for callers that may not
 * allocate device memory.  The paper has no counterpart: this is a
 * deployment variant, not part of the method.
 *
 * Some callers cannot let a library call cudaMalloc: a serving process that
 * has reserved all of HBM for its own pools (a late allocation would fail or
 * fragment it), or a latency-bound loop where an allocation's implicit
 * device synchronisation is not acceptable.  This entry point computes the
 * same result as plsh_alibi_attn with the same arguments and rules, but keeps
 * its working memory (the work-item table and the work-queue counters) in a
 * fixed array compiled into the library, about 1 MiB per device, held by
 * every device that loads the library until the process exits.  It calls no
 * allocation routine.
 *
 * Limits: bf16, d = 128, s within the tensor-core kernel's shared-memory
 * budget (s <= 52 causal, s <= 29 without the mask), at most 1023 query
 * heads and 65536 work items (one item per two 128-row query tiles:
 * B * Hq * ceil(n/128) / 2, e.g.
 * n = 131072 with 40 heads uses 20480); larger requests return
 * PLSH_ERR_UNSUPPORTED and launch nothing.
 * The first call on each device resolves the array's device address
 * (cudaGetSymbolAddress) and keeps it for the life of the device's primary
 * context (a process that resets the device must not call this entry point
 * again).
 * Every call on a device shares the one array and each call resets its work
 * counters before use, so calls whose kernels overlap on the GPU (different
 * streams without ordering) race and must not be issued.  A device-side wait
 * that runs out (limit: plsh_set_wait_limit_ns) and a value of V beyond
 * +-65504 are recorded in the array's error word, which persists across calls
 * until plsh_noalloc_status() reads and clears it; plsh_stream_status() does
 * not see them.
 */
plsh_status plsh_alibi_attn_noalloc(const plsh_tensor* Q, const plsh_tensor* K,
                                    const plsh_tensor* V, const plsh_bins* bins,
                                    int32_t causal, plsh_tensor* O, void* stream);

/*
 * plsh_noalloc_status -- the error word of plsh_alibi_attn_noalloc on the
 * current device.  Synchronises `stream`, reads the word from the fixed
 * array (no allocation), clears it, and returns PLSH_ERR_TIMEOUT if a wait
 * ran out, else PLSH_ERR_RANGE if a value of V was beyond +-65504, else
 * PLSH_OK, covering every allocation-free call since the last report.  Call
 * it once the calls it should cover are queued on `stream` (or on streams
 * `stream` waits for).
 */
plsh_status plsh_noalloc_status(void* stream);

/*
 * plsh_alibi_attn_host -- plsh_alibi_attn on tensors in host memory.  The
 * paper has no counterpart: this is a deployment variant, not part of the
 * method.
 *
 * Q, K, V and O follow the plsh_alibi_attn rules except that their `data`
 * are host pointers (page-locked memory lets the copies run asynchronously
 * and overlap; pageable memory works but each copy then blocks the calling
 * thread).  The library stages the tensors through device buffers it keeps
 * per device (grown on demand in stream order, behind the previous call of
 * this entry point; held until the process exits) and splits the query rows
 * into up to four chunks on the tensor-core path: chunk c + 1 is copied in
 * and chunk c - 1 copied out, on two copy streams of its own, while the
 * fused kernel runs on chunk c (with
 * the causal mask only the keys up to a chunk's last row are needed before
 * it starts).  The call returns once everything is queued; O is complete on
 * the host when `stream` reaches the point of the call (synchronise it before
 * reading O).  Calls on one device share the staging buffers: issue them on
 * one stream, or order their streams.
 */
plsh_status plsh_alibi_attn_host(const plsh_tensor* Q, const plsh_tensor* K,
                                 const plsh_tensor* V, const plsh_bins* bins, int32_t causal,
                                 plsh_tensor* O, void* stream);

/*
 * plsh_alibi_exact -- exact ALiBi attention T* (the dense comparator, Problem
 * statement: O(n^2) in the bias matrix):
 *   O_i = sum_j e^{S_ij - |i-j|/sigma_h} v_j / sum_j e^{S_ij - |i-j|/sigma_h}
 * over all j (j <= i when causal).  sigma_h: host array [Hq], finite, > 0.
 * Same tensor rules as plsh_alibi_attn.
 */
plsh_status plsh_alibi_exact(const plsh_tensor* Q, const plsh_tensor* K,
                             const plsh_tensor* V, const double* sigma_h,
                             int32_t causal, plsh_tensor* O, void* stream);

/*
 * plsh_alibi_decode -- one decode step of the approximation: row `pos` of T~
 * (Methodology 3) with the causal mask, for a query given on its own against
 * cached keys and values.  With J_t(pos) = [lo_t(pos), pos], lo_t(pos) the
 * start of the bin of pos under hash t of head h,
 *   o = sum_j c_j e^{S_j} v_j / sum_j c_j e^{S_j},  S_j = q . k_j / sqrt(d),
 *   c_j = #{t : lo_t(pos) <= j},  j in [min_t lo_t(pos), pos]:
 * the work is the row's key envelope, O(s b) keys, not pos.
 *
 *   q [B,Hq,1,d]: the query of position pos; o [B,Hq,1,d]: its output.
 *   K, V [B,Hkv,n,d]: the cache; rows above pos are not read.
 *   All the same dtype (PLSH_BF16 or PLSH_F32), d in {64, 128}, Hq % Hkv == 0,
 *   B * Hq <= 65535, bins->n == n, bins->H == Hq, 0 <= pos < n.
 * A CTA serves the query heads of one KV group (up to 8) over one share of
 * the union of their envelopes; the shares' partial results (max, row sum,
 * unnormalised P V) are merged into o.  The partials live in a device buffer
 * the library keeps per device (B * Hq * S * (d + 2) floats, S <= 64 shares
 * chosen so that about 12 CTAs per SM run, at most the 64-key shares of the
 * envelope the widest bins are expected to reach; grown on demand in stream
 * order on `stream`; calls on different streams are ordered on it by an
 * event).  Up to 32 KV groups are listed widest scale first, and on large
 * grids each group takes the shares its own expected envelope wants.  Both
 * kernels of a call start as programmatic dependents of the kernel before
 * them on `stream` (neither touches global memory before it completes).
 * Asynchronous on `stream`; errors in the arguments return before any launch.
 */
plsh_status plsh_alibi_decode(const plsh_tensor* q, const plsh_tensor* K,
                              const plsh_tensor* V, const plsh_bins* bins, int64_t pos,
                              plsh_tensor* o, void* stream);

/* ------------------------------------------------------------------------
 * 4-bit paged K/V cache.  The paper has no counterpart: this is a deployment
 * variant of the decode step, not part of the method.
 *
 * A cache held in 4-bit codes takes 5 bits a value (codes and the scales of
 * their groups) instead of bf16's 16, and a decode step, which reads its keys
 * and values once, is bound by those bytes.  It is paged, so that sequences of
 * different lengths share one pool, and every sequence of a batch has its own
 * position, read on the device (a captured graph of a decode loop replays
 * while the positions and the page table change).
 *
 * Format.  A row of d values is cut into groups of 32; a group is held as 32
 * codes c in 0..15 and two bf16 numbers lo and step, and its values read back
 * as lo + step c.  Writing x (each operation in fp32, rounded once; bit for
 * bit the same from any implementation):
 *   lo = min x rounded down to bf16,  step = (max x - lo) / 15 rounded up to
 *   bf16,  c = (x - lo) / step rounded to the nearest integer, ties to even,
 *   within 0..15 (0 where step is 0): a value is off by at most about step / 2.
 * -0 counts as less than +0: a group whose least value is 0 has lo = -0 if one
 * of its zeros is -0.
 * A group that holds a NaN or an infinity, or spans more than fp32 does, is
 * stored as lo = 0, step = NaN: it reads back as NaN, and so does every
 * attention row that gives one of its keys a weight.
 * Positions are held in tiles of 16, 20 d bytes each, a page's tiles one after
 * the other.  Within a tile, position r = 0..15 (= 8 blk + 2 t + par) and
 * value e = 32 y + i of its row:
 *   K codes  byte r d/2 + (i / 8) d/8 + 4 y + (i % 8) / 2
 *   V codes  byte 8 d + (y / 2) 512 + (4 (i / 4) + t) 16 + (y % 2) 8 + 4 blk
 *            + 2 par + (i % 4) / 2
 *   (even values in the low nibble), then at 16 d + 4 (r d/32 + y) K's pairs
 *   (lo, step) and from 18 d V's.
 * These are the orders in which the decode step's matrix instructions take
 * the codes, so that a lane loads its operands with 16-byte loads.
 */
typedef struct {
  void* data;            /* device uint8 [pages, H, page / 16, 20 d], 16-byte
                            aligned; the caller owns it */
  const int32_t* table;  /* device int32 [B, max_pages]: sequence b holds its
                            positions [i page, (i + 1) page) in page
                            table[b, i] of data; entries past the pages a call
                            needs are not read */
  int64_t B;             /* sequences, >= 1 */
  int64_t H;             /* KV heads, >= 1 */
  int64_t pages;         /* pages of data, 1 .. 2^31 - 1 */
  int64_t max_pages;     /* pages of a sequence, >= 1, max_pages page < 2^31 */
  int32_t page;          /* positions of a page: 16, 32, 64, 128 or 256 */
  int32_t d;             /* 64 or 128 */
} plsh_q4_cache;

/* Bytes of plsh_q4_cache.data: pages * H * (page / 16) * 20 d. */
plsh_status plsh_q4_cache_bytes(int64_t pages, int64_t H, int32_t page, int32_t d,
                                int64_t* bytes);

/*
 * plsh_q4_cache_write -- quantise rows of K and V into the cache: row i <
 * len[b] of sequence b becomes its position pos[b] + i, for every head; the
 * rest of the cache is left as it was.
 *   K, V [B, H, m, d] (PLSH_BF16 or PLSH_F32) of the cache's B, H and d.
 *   pos  device int32 [B].
 *   len  device int32 [B], taken within 0..m, or NULL for m rows of each.
 * A row whose position is negative or not below max_pages * page, or whose
 * page index is not in [0, pages), is not written; plsh_stream_status then
 * reports PLSH_ERR_INVALID.  Two sequences that write the same position of
 * the same page leave one or a mixture of the two rows there: give each
 * sequence pages of its own where it writes (shared pages may be read).
 * Asynchronous on `stream`; allocates nothing.
 */
plsh_status plsh_q4_cache_write(const plsh_tensor* K, const plsh_tensor* V,
                                const plsh_q4_cache* cache, const int32_t* pos,
                                const int32_t* len, void* stream);

/*
 * plsh_q4_cache_read -- the values that positions pos[b] + i, i < len[b], of
 * the cache stand for, as rows of K and V [B, H, m, d] (PLSH_BF16, rounded
 * once, or PLSH_F32, exact up to one fp32 rounding).  Rows from len[b] on, and
 * rows whose position or page index is out of range (reported as for
 * plsh_q4_cache_write), are left as they were.  K and V must not overlap.
 * Asynchronous on `stream`; allocates nothing.
 */
plsh_status plsh_q4_cache_read(const plsh_q4_cache* cache, const int32_t* pos,
                               const int32_t* len, plsh_tensor* K, plsh_tensor* V,
                               void* stream);

/*
 * plsh_q4_cache_reserve -- the cache's page table kept on the device from the
 * positions that its sequences ask for.
 *   table  (of the cache; it is written, and must be writable) row b holds
 *          sequence b's pages in its first held[b] entries, -1 behind them.
 *   need   device int32 [B]: positions sequence b is to hold; <= 0: none.
 *   held   device int32 [B]: pages that it holds, updated.
 *   pool   device int32 [1 + pool_pages]: the number of free pages, then their
 *          stack from the bottom, updated.
 *   prefix device int32 [prefix_pages], 0 <= prefix_pages <= max_pages: pages of
 *          a prompt that all sequences share; the first prefix_pages entries of
 *          every row that holds anything are these.  They never come from or go
 *          to the stack.  NULL with prefix_pages = 0.
 * A sequence wants w = max(ceil(need[b] / page), prefix_pages) pages (0 for
 * need[b] <= 0).  First the pages held beyond w are pushed, from the last
 * sequence's last page to the first one's first, and their entries become -1;
 * then, from the first sequence on, the missing pages are popped, first entry
 * first, as long as a sequence's fit: the first one whose do not and all after
 * it that want more than they hold are left as they were (held[b] * page <
 * need[b] says which).  Growing and then releasing leaves the stack as it was.
 * A sequence with held[b] outside 0..max_pages, or that wants more than
 * max_pages, is left as it was; a free count outside 0..pool_pages counts as the
 * nearest, and pages pushed beyond pool_pages are dropped: each is reported as
 * PLSH_ERR_INVALID by plsh_stream_status.  The table, held and pool must overlap
 * neither one another nor need and prefix (a prefix is a copy of a row's entries).
 * Asynchronous on `stream`; allocates nothing; may be captured.
 */
plsh_status plsh_q4_cache_reserve(const plsh_q4_cache* cache, const int32_t* need, int32_t* held,
                                  int32_t* pool, int64_t pool_pages, const int32_t* prefix,
                                  int64_t prefix_pages, void* stream);

/*
 * plsh_q4_cache_slots -- the slot of every new row: row i < len[b] of sequence b
 * is position p = pos[b] + i and has slot table[b, p / page] * page + p % page
 * (whatever else is kept by slot: a position of every head of the cache, its
 * token, its owner); -1 for rows from len[b] on, rows whose position is negative,
 * and rows whose page index is not in [0, pages).  A row whose position is not
 * below max_pages * page is -1 too and reported as PLSH_ERR_INVALID by
 * plsh_stream_status.  Rows count by their own positions, as plsh_q4_cache_write and
 * plsh_q4_cache_read take them: a negative pos[b] with several rows is no idle
 * sequence here (its rows from position 0 on have slots); give that len 0.
 *   pos    device int32 [B];  len  device int32 [B] or NULL for m rows of each
 *   slots  device int64 [B, m], 16-byte aligned; B * m < 2^31 - 512
 * Asynchronous on `stream`; allocates nothing; may be captured.
 */
plsh_status plsh_q4_cache_slots(const plsh_q4_cache* cache, const int32_t* pos, const int32_t* len,
                                int64_t m, int64_t* slots, void* stream);

/* Bytes of workspace of a plsh_alibi_decode_q4 or plsh_alibi_exact_decode_q4
 * call with these q and cache on the current device. */
plsh_status plsh_q4_decode_work_bytes(const plsh_tensor* q, const plsh_q4_cache* cache,
                                      int64_t* bytes);

/*
 * plsh_alibi_decode_q4 -- plsh_alibi_decode over the 4-bit cache: for every
 * sequence b the row of T~ at its own position pos[b],
 *   o_b = sum_j c_j e^{S_j} v_j / sum_j c_j e^{S_j},  S_j = q_b . k_j / sqrt(d),
 *   c_j = #{t : lo_t(pos[b]) <= j},  j in [min_t lo_t(pos[b]), pos[b]],
 * with k_j, v_j the cached values.
 *   q, o [B, Hq, 1, d], PLSH_BF16 or PLSH_F32, which must not overlap; Hq a
 *        multiple of the cache's H;
 *   bins->H == Hq, bins of any length: pos[b] must lie below bins->n.
 *   pos  device int32 [B]; a negative one is an idle slot: o_b = 0.
 *   work device memory of plsh_q4_decode_work_bytes, 16-byte aligned, used by
 *        this call alone until it completes (calls that may overlap, and
 *        graphs that may replay at once, take one each).
 * A pos[b] not below max_pages * page or bins->n gives o_b = 0, and a key
 * whose page index is not in [0, pages) counts as absent; either is reported
 * as PLSH_ERR_INVALID by plsh_stream_status.  A key or value of c_j = 0, a
 * position past pos[b] and whatever else a page holds have no effect, be it
 * NaN.  A head whose q holds a NaN or an infinity, or reaches 2^110, gives a
 * row of NaN.  bf16: products of codes with q run as f16 ones of q scaled by a
 * power of two, so a value below 2^-24 of its head's largest counts as 0, and
 * P step is rounded to f16: 2^-11 of itself, no finer than 2^-33 of the largest
 * P step of the head's row and group of 32 values; sums of such products over
 * 16 values or 16 positions keep about 18 bits of their largest one.  fp32: two
 * such terms each, 2^-22 of a head's largest q and of P step itself (no finer
 * than 2^-36 of the largest), in fp32 sums.  What a key does to a row is bound
 * by its weight there: a value of a key that weighs nothing, however large,
 * takes no precision from the others.  All other sums are fp32's.  Asynchronous
 * on `stream`; allocates nothing; may be captured.
 */
plsh_status plsh_alibi_decode_q4(const plsh_tensor* q, const plsh_q4_cache* cache,
                                 const plsh_bins* bins, const int32_t* pos, plsh_tensor* o,
                                 void* work, int64_t work_bytes, void* stream);

/*
 * plsh_alibi_exact_decode_q4 -- one decode step of exact ALiBi attention (the
 * dense comparator, plsh_alibi_exact) over the 4-bit cache:
 *   o_b = sum_j e^{S_j - (pos[b] - j) / sigma_h} v_j / sum_j (the weights),
 *   0 <= j <= pos[b].
 * sigma_h: host array [Hq], finite, > 0; at most 512 heads.  Everything else
 * as for plsh_alibi_decode_q4.
 */
plsh_status plsh_alibi_exact_decode_q4(const plsh_tensor* q, const plsh_q4_cache* cache,
                                       const double* sigma_h, const int32_t* pos,
                                       plsh_tensor* o, void* work, int64_t work_bytes,
                                       void* stream);

/* Bytes of workspace of a plsh_alibi_exact_chunk_q4 call with these q and cache
 * on the current device. */
plsh_status plsh_q4_chunk_work_bytes(const plsh_tensor* q, const plsh_q4_cache* cache,
                                     int64_t* bytes);

/*
 * plsh_alibi_exact_chunk_q4 -- exact ALiBi attention of several new tokens of
 * every sequence over the 4-bit cache (a prompt's next piece, drafted tokens to
 * verify): row i < len[b] of sequence b is at position p = pos[b] + i,
 *   o_bi = sum_j e^{S_j - (p - j) / sigma_h} v_j / sum_j (the weights),
 *   S_j = q_bi . k_j / sqrt(d),  0 <= j <= p,
 * with k_j, v_j the cached values, the new tokens' own among them: they are
 * written (plsh_q4_cache_write) before the call.
 *   q, o [B, Hq, m, d], which must not overlap; B * Hq * m < 2^30.
 *   pos  device int32 [B]; a negative one is an idle slot: o_bi = 0, i < len[b].
 *   len  device int32 [B], or NULL for m rows of each; rows from len[b] on are
 *        left as they were.
 *   work device memory of plsh_q4_chunk_work_bytes, as for plsh_alibi_decode_q4.
 * A row whose position is not below max_pages * page gives 0, and a key whose
 * page index is not in [0, pages) counts as absent; either is reported as
 * PLSH_ERR_INVALID by plsh_stream_status.  What lies behind a row's position has
 * no effect on it (what another row of the call sees there may take part in the
 * powers of two below).  Everything else as for plsh_alibi_exact_decode_q4.
 *
 * bf16 calls of many rows (decided by sizes alone: tokens and query heads of a KV
 * head, and the table's length, also where the sequences are far shorter than that;
 * and no sigma_h below 1.4e-6) run on the tensor cores with the cached values
 * themselves in f16: q, k and v are rounded to 2^-11 of themselves, but
 *   q  no finer than 2^-39 of the largest of its row;
 *   k  no finer than 2^-39 of the largest of its 32 positions (from a multiple of 32);
 *   v  no finer than 2^-24 of the largest of its group of 32 values in its 32
 *      positions;
 *   weights  no finer than 2^-14 of the row's largest, and 2^-22 where a group of the
 *      position's value is 2^15 times others of the group and more (2^-25 and 2^-33
 *      unless such a position has the row's largest; 2^k times less fine in 32
 *      positions that are 2^k times smaller than others in all their groups).
 * So a key 2^31 times the others, or a group of V 2^16 times the others, leaves the 31
 * positions beside it (of V: the same group of theirs) precise to 2^-8 of themselves,
 * and less where it is larger still; no value takes that from other groups or positions.
 * Where a group of V of 32 positions would keep no 2^-14 of itself, which is when a
 * step's groups of 32 positions, each divided by the largest of its group in the step,
 * differ by more than 2^31 within 32 positions (a position that is large in all its
 * groups alike does not count: up to 2^79 between positions, 2^151 between steps), the
 * call is reported as PLSH_ERR_RANGE by plsh_stream_status, and o is then not to be
 * used.
 */
plsh_status plsh_alibi_exact_chunk_q4(const plsh_tensor* q, const plsh_q4_cache* cache,
                                      const double* sigma_h, const int32_t* pos, const int32_t* len,
                                      plsh_tensor* o, void* work, int64_t work_bytes, void* stream);

/* Bytes of workspace of a plsh_alibi_exact_prefix_decode_q4 call with these q and
 * cache on the current device. */
plsh_status plsh_q4_prefix_work_bytes(const plsh_tensor* q, const plsh_q4_cache* cache,
                                      int64_t* bytes);

/*
 * plsh_alibi_exact_prefix_decode_q4 -- plsh_alibi_exact_decode_q4 for sequences
 * that share their first positions: positions below prefix_pages * page are read
 * from the pages prefix[0 .. prefix_pages), the others from the cache's table at
 * the same index as ever (its first prefix_pages entries are not read).
 *   prefix device int32 [prefix_pages], 1 <= prefix_pages <= max_pages.
 *   work   device memory of plsh_q4_prefix_work_bytes, as for
 *          plsh_alibi_decode_q4.
 * A sequence may be anywhere, within the prefix too (pos[b] negative: idle).
 * Everything else as for plsh_alibi_exact_decode_q4; bf16 calls of many sequences
 * behind a long prefix take the prefix's part on the tensor cores, once for all of
 * them, as described at plsh_alibi_exact_chunk_q4; other calls read it once a
 * sequence.  Positions of the prefix that no sequence has come to have no effect.
 */
plsh_status plsh_alibi_exact_prefix_decode_q4(const plsh_tensor* q, const plsh_q4_cache* cache,
                                              const double* sigma_h, const int32_t* pos,
                                              const int32_t* prefix, int64_t prefix_pages,
                                              plsh_tensor* o, void* work, int64_t work_bytes,
                                              void* stream);

/* Synchronises `stream`, then reports CUDA errors and the library's device
 * error flag, clearing the flag: PLSH_ERR_TIMEOUT when a bounded device wait
 * ran out, else PLSH_ERR_RANGE when a tensor-core attention call met a value
 * of V beyond +-65504 (over a 4-bit cache: values as far apart as
 * plsh_alibi_exact_chunk_q4 says), else PLSH_ERR_INVALID when a call on a 4-bit cache met
 * a position or a page index out of range. */
plsh_status plsh_stream_status(void* stream);

/*
 * plsh_attn_path -- the kernel plsh_alibi_attn (bins != NULL) or
 * plsh_alibi_exact (bins == NULL) takes for a query tensor of Q's shape and
 * dtype, written to *path (a plsh_path).  Launches nothing, allocates
 * nothing; PLSH_ERR_INVALID for a NULL Q or path.
 */
plsh_status plsh_attn_path(const plsh_tensor* Q, const plsh_bins* bins, int32_t causal,
                           int32_t* path);

/* Debug knob: limit in nanoseconds of every device-side wait launched after
 * this call on the current device (0 restores the default of 2 s), but for a thread
 * block's wait for its own copies and products before it ends, which is 2 s always. */
plsh_status plsh_set_wait_limit_ns(uint64_t ns);

/*
 * plsh_set_split_parts -- how the tensor-core attention calls on the current
 * device cut long work items over their key range (the varlen scheduling
 * step: items are pairs of 128-row query tiles, each item's key envelope is
 * found on the device from its rows' bins).
 *   0   automatic (the default): an item whose expected key tiles exceed
 *       half the call's per-SM share (at least 2) is cut into parts of at
 *       most that size, so that no single item outlasts the others;
 *   1   never cut;
 *   2..16  cut every item into that many parts (a tuning and testing knob).
 * Each part covers a consecutive range of its item's key tiles (a part past
 * the envelope does nothing); parts write their unnormalised P V, running max
 * and row sum to a library-owned workspace and a second kernel combines them
 * into O.  Calls made afterwards use the setting; the workspace is allocated
 * with the item table of a shape.
 */
plsh_status plsh_set_split_parts(int32_t parts);

const char* plsh_status_string(plsh_status status);

/* Message of the last error raised on the calling thread ("" if none). */
const char* plsh_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* PLSH_H_ */
