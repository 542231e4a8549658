/*
 * attnres.h -- C ABI of libattnres: Block Attention Residuals (Block AttnRes)
 * depth aggregation on NVIDIA GB300 (sm_103a).
 *
 * What the operations compute (sources cited by page title and section):
 *
 *  - [Deep-dive 2] "Kimi K3 deep-dive series (2): AttnRes and Stable
 *    LatentMoE", §2: for one token and layer l with sources H (S rows of d)
 *    and a learned pseudo-query w_l,
 *        a_l = softmax_s( w_l . RMSNorm(H_s) ),     r_l = sum_s a_l[s] H_s,
 *    RMSNorm without a gain, no temperature, values are the raw sources.
 *    [Atlas] "LLM Atlas · Kimi K3", §07 Attention Residuals, states the same
 *    weights alpha_{i->l} and h_l = sum_i alpha_{i->l} v_i.
 *  - [Parts 6] "Kimi K3 model structure (6): inputs and parts", odd facts:
 *    RMSNorm eps = 1e-5 model-wide.  Here rms(h) = sqrt(mean_c h_c^2 + eps).
 *  - [Tutorial] Kimi K3 chaptered tutorial (kimi.papertok.ai), ch. 4.3,
 *    Eq. 10: layers are split into blocks of B layers; a completed block is
 *    kept as the SUM of its layers' outputs b_n; layer i of block n reads
 *    [b_0 .. b_{n-1}] if i = 1 and [b_0 .. b_{n-1}, partial] if i >= 2,
 *    where b_0 is the embedding h_0 and the partial sum holds the outputs of
 *    layers 1..i-1 of block n.  The final output layer aggregates all block
 *    representations.  Ch. 4.5: K3 uses B = 12 over 93 layers (the 8th block
 *    has 9 layers), so at most 9 sources.  Ch. 4.6: block representations
 *    are produced once at the block boundary and then stay resident.
 *
 * Conventions for every call:
 *  - Tensors are row-major [T, d] (token-major, channel contiguous) in device
 *    memory of the CURRENT device (cudaGetDevice), on which every call
 *    launches; `sources` / `block_reps` are HOST arrays of DEVICE pointers.
 *  - The caller owns and allocates every buffer.  The library makes no
 *    device allocation and keeps no device-side global state, with one
 *    exception: the fixed scratch array built into it for
 *    attnres_aggregate_backward_noalloc (see there).
 *  - Calls are asynchronous on `stream` (a cudaStream_t passed as void*;
 *    NULL = the legacy default stream) and never synchronise the device.
 *  - Argument errors are detected on the host before any launch and return
 *    a negative attnres_status; nothing is written then.  A failed launch
 *    returns ATTNRES_ECUDA; attnres_last_error() gives the CUDA message
 *    (per host thread).
 *  - dev_err (nullable): a device int32 the kernels OR error bits into
 *    (ATTNRES_DEVERR_*); they never clear it.  Every spin-wait inside the
 *    kernels has a time limit; when one runs out the kernel sets the bit,
 *    writes NaN to the affected outputs, drains its own copies and returns.
 *  - Any pointer alignment and any d >= 1 is accepted; rows that start on a
 *    16-byte boundary with 16-byte-multiple row length take the bulk-copy
 *    (TMA) path, others a plain-load kernel (still on the GPU).
 *  - Environment, read once per process: ATTNRES_NO_PDL=1 launches without
 *    programmatic dependent launch; ATTNRES_SPLIT=1 lets a launch of at most
 *    9 sources over few tokens (T times the cluster size within the SM
 *    count) share each token across a thread-block cluster of 2, 4 or 8
 *    CTAs.  Results agree with the default path to the order of fp32 sums.
 */
#ifndef ATTNRES_H
#define ATTNRES_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTNRES_OK = 0,
  ATTNRES_EINVAL = -1, /* null pointer, non-positive size, bad eps */
  ATTNRES_EDTYPE = -2, /* dtype code not one of attnres_dtype */
  ATTNRES_ERANGE = -4, /* S > ATTNRES_MAX_SOURCES, too many blocks, T*d overflow */
  ATTNRES_ECUDA = -5,  /* a CUDA runtime call or launch failed */
  ATTNRES_ESTATE = -6  /* stack call out of order (see attnres_state) */
} attnres_status;

typedef enum { ATTNRES_F32 = 0, ATTNRES_BF16 = 1 } attnres_dtype;

/* bits ORed into *dev_err by the kernels */
#define ATTNRES_DEVERR_WAIT_TIMEOUT 0x1 /* a bounded wait on a copy gave up */

#define ATTNRES_MAX_SOURCES 128
#define ATTNRES_MAX_BLOCKS (ATTNRES_MAX_SOURCES - 1)
#define ATTNRES_DEFAULT_EPS 1e-5f

/* ------------------------------------------------------------------------
 * attnres_aggregate -- one layer of depth-wise attention ([Deep-dive 2] §2).
 *
 *   for every token t in [0, T):
 *     z[s]  = (sum_c w_l[c] * src_s[t,c]) / sqrt(mean_c src_s[t,c]^2 + eps)
 *     a[t,:] = softmax_s(z)                         (fp32)
 *     r[t,c] = sum_s a[t,s] * src_s[t,c]            (fp32 accumulate)
 *
 * sources     host array of S device pointers, each [T, d] of src_dtype
 *             (a [S, T, d] slab: sources[s] = base + s*T*d elements)
 * S           1 .. ATTNRES_MAX_SOURCES
 * T, d        T >= 0 (T = 0 launches nothing and accepts NULL buffers), d >= 1
 * src_dtype   ATTNRES_F32 or ATTNRES_BF16
 * w_l         device [d] fp32 pseudo-query
 * eps         > 0 or 0 (1e-5 in K3)
 * out_r       device [T, d] of out_dtype; bf16 is rounded to nearest even
 * out_weights device [T, S] fp32, or NULL to skip
 * Each source row is read from device memory once.  out_r and out_weights
 * may not share a byte with a source or with each other (ATTNRES_EINVAL);
 * sources may repeat.  Returns ATTNRES_OK or a negative attnres_status.
 * ---------------------------------------------------------------------- */
int attnres_aggregate(const void* const* sources, int S, int64_t T, int d, int src_dtype,
                      const float* w_l, float eps, void* out_r, int out_dtype,
                      float* out_weights, int* dev_err, void* stream);

/* ------------------------------------------------------------------------
 * attnres_aggregate_fold -- one layer whose last source is a partial sum
 * formed in the same launch ([Tutorial] ch. 4.3: the partial sum of a block
 * is the sum of its layer outputs so far), i.e. attnres_layer_step without
 * a state:
 *
 *   p[t,c] = round(prev[t,c] + F[t,c])   (or round(F[t,c]) when prev is
 *            NULL; fp32 add, rounded to dtype), stored to dst;
 *   then attnres_aggregate over [sources[0..n_stored-1], p] (p as read back
 *   from dst's rounding, so the weights see exactly the stored bits).
 *
 * sources     host array of n_stored (0..127) device pointers [T, d] of
 *             dtype (NULL when n_stored = 0)
 * prev        device [T, d] or NULL; F: device [T, d]; dst: device [T, d]
 *             (may be prev itself, updated in place, but no other row)
 * dtype       of every row and of out_r
 * w_l, eps, out_r, out_weights ([T, n_stored + 1] fp32 or NULL), dev_err,
 *             stream: as attnres_aggregate.
 * flags       0, or ATTNRES_STATE_EARLY_LOADS: the stored rows and prev of
 *             the first token are loaded before the kernel launched just
 *             before this call has finished, only F after it -- under the
 *             conditions given at that flag (here: that kernel writes
 *             nothing this call reads except F).
 * Results equal attnres_fold followed by attnres_aggregate bit for bit,
 * with one launch and one row fewer per token.  Outputs may not share
 * memory with any row (ATTNRES_EINVAL).
 * ---------------------------------------------------------------------- */
int attnres_aggregate_fold(const void* const* sources, int n_stored, const void* prev, const void* F, void* dst,
                           int64_t T, int d, int dtype, const float* w_l, float eps, void* out_r,
                           float* out_weights, int flags, int* dev_err, void* stream);

/* ------------------------------------------------------------------------
 * attnres_aggregate_host -- attnres_aggregate on sources, query and outputs
 * that live in HOST memory.  The pages have no counterpart: this is the
 * library's way in for data that starts on the CPU.
 *
 * The tokens are cut into chunks of chunk_tokens (the last may be shorter).
 * Chunk c goes to staging slot c mod nslots of `workspace`: its S source
 * rows are copied in, aggregated as soon as they have arrived, and its r
 * (and weights) copied out while later chunks are still coming in, so the
 * host link carries both directions at once.  Results are those of
 * attnres_aggregate on the same data (each token is computed alone).
 *
 * sources_host host array of S HOST pointers, each [T, d] of src_dtype.
 *             Page-locked memory (cudaHostAlloc, cudaHostRegister) lets the
 *             copies run at the link's rate, asynchronously; pageable memory
 *             works, but the driver then stages each copy and the call
 *             returns only once the sources have been read.
 * w_host      host [d] fp32 pseudo-query
 * r_host      host [T, d] of out_dtype; weights_host host [T, S] fp32 or NULL
 * chunk_tokens >= 1 (values above T act as T)
 * workspace   device buffer owned by the caller, 256-byte aligned, of
 *             workspace_bytes >= attnres_aggregate_host_workspace_size(...,
 *             1); the call uses as many slots as fit, at most 8 and at most
 *             the number of chunks (2 to 3 slots let copies and compute
 *             overlap).  Its contents on entry do not matter.
 * stream      work already on `stream` comes first; work issued on `stream`
 *             after the call waits until r_host / weights_host hold the
 *             results, so synchronise `stream` before reading them or
 *             writing the inputs again.  The copies run on two streams that
 *             the call creates and destroys (CUDA defers their release until
 *             their work is done).  A stream being captured into a graph
 *             is refused (ATTNRES_EINVAL).  If a CUDA call fails part way
 *             (ATTNRES_ECUDA), the copies already queued are still joined
 *             into `stream` before the call returns.
 * Other arguments, bounds and errors as attnres_aggregate; nothing is
 * copied or launched when an argument is rejected.
 * ---------------------------------------------------------------------- */
int attnres_aggregate_host(const void* const* sources_host, int S, int64_t T, int d,
                           int src_dtype, const float* w_host, float eps, void* r_host,
                           int out_dtype, float* weights_host, int64_t chunk_tokens,
                           void* workspace, int64_t workspace_bytes, int* dev_err,
                           void* stream);

/* Bytes of workspace attnres_aggregate_host needs for `slots` staging slots
 * of chunk_tokens tokens (the query, then per slot the [S, chunk_tokens, d]
 * sources, r and, if with_weights, the weights, each part 256-byte
 * aligned); slots 1..8.  Host only.  Negative attnres_status on bad
 * arguments. */
int64_t attnres_aggregate_host_workspace_size(int S, int64_t chunk_tokens, int d, int src_dtype,
                                              int out_dtype, int with_weights, int slots);

/* ------------------------------------------------------------------------
 * attnres_aggregate_backward -- gradients of attnres_aggregate.  In training
 * AttnRes runs under activation checkpointing ([Tutorial] ch. 4.6): nothing
 * is kept from the forward; the logits and weights are recomputed here from
 * the sources.  Per token, with rho_s = rms(h_s), z_s = w.h_s / rho_s,
 * a = softmax(z) and dr the gradient of the loss with respect to r:
 *   g_s = dr.h_s,  gbar = sum_s a_s g_s,  dz_s = a_s (g_s - gbar),
 *   alpha_s = dz_s / rho_s,  beta_s = alpha_s z_s / (d rho_s)
 *   grad_sources[s][t,:]  =  (or +=)  a_s dr + alpha_s w - beta_s h_s
 *   grad_w[c]             =  sum_t sum_s alpha_s h_s[t,c]
 *
 * sources, S, T, d, w_l, eps  as in attnres_aggregate; dtype is that of the
 *             sources, of grad_r and of grad_sources
 * grad_r      device [T, d] of dtype
 * grad_sources host array of S device pointers [T, d] of dtype, none of them
 *             sharing memory with a source, with grad_r or with each other
 *             (ATTNRES_EINVAL); overwritten (accumulate = 0)
 *             or added to (accumulate = 1: a source read by several layers
 *             collects the gradient of each)
 * grad_w      device [d] fp32, overwritten (fp32 sums in a fixed order:
 *             bit-reproducible)
 * workspace   device scratch, 4-byte aligned, at least
 *             attnres_aggregate_backward_workspace_size(T, d) bytes, owned
 *             by the caller; its contents on entry do not matter
 * Reads (S + 1) rows and writes S rows per token (S more read with
 * accumulate).  T = 0 only zeroes grad_w.
 * ---------------------------------------------------------------------- */
int attnres_aggregate_backward(const void* const* sources, int S, int64_t T, int d, int dtype,
                               const float* w_l, float eps, const void* grad_r,
                               void* const* grad_sources, int accumulate, float* grad_w,
                               void* workspace, int64_t workspace_bytes, int* dev_err,
                               void* stream);

/* Bytes of workspace attnres_aggregate_backward needs for T tokens of d
 * channels on the current device (one fp32 row of d per CTA it runs, at most
 * one CTA per SM).  Negative attnres_status on error. */
int64_t attnres_aggregate_backward_workspace_size(int64_t T, int d);

/* ------------------------------------------------------------------------
 * attnres_aggregate_backward_noalloc -- attnres_aggregate_backward without
 * a caller workspace, for callers that cannot allocate device memory (code
 * that runs under a fixed device-memory budget or must not call cudaMalloc
 * once it is running, e.g. inside a serving or replay loop).  The pages
 * have no counterpart: this is a library convenience.
 *
 * The workspace is a scratch array built into the library (1,310,720 fp32
 * values, 5 MiB, held by every GPU that loads the library until the process
 * exits).  Calls needing more (CTAs x d fp32 values, CTAs = min(T, SMs); on
 * a 152-SM GB300 any T with d <= 8192 fits) return ATTNRES_ERANGE with a
 * message naming the sizes; use attnres_aggregate_backward then.  Nothing
 * is allocated and no allocating library routine is called.
 *
 * The first call on a device looks up the array's device address (one
 * cudaGetSymbolAddress, with that device current) and caches it, keyed by
 * the device and its current context: make that first call before any
 * stream capture, and again after the device's context was torn down and
 * recreated (cudaDeviceReset), when the address is looked up anew.  All calls share the array and it
 * keeps the previous call's contents (every value a call reads it has
 * written first, so nothing needs clearing); calls whose kernels overlap on
 * a GPU (other streams or host threads) race on it and must be serialised.
 * Arguments, results and errors otherwise as attnres_aggregate_backward.
 * ---------------------------------------------------------------------- */
int attnres_aggregate_backward_noalloc(const void* const* sources, int S, int64_t T, int d,
                                       int dtype, const float* w_l, float eps,
                                       const void* grad_r, void* const* grad_sources,
                                       int accumulate, float* grad_w, int* dev_err,
                                       void* stream);

/* ------------------------------------------------------------------------
 * Stack state: the resident depth sources of one batch of T tokens.
 * ([Tutorial] ch. 4.3-4.6: b_0 = embedding, b_1 .. b_N completed block sums
 * kept resident, one running partial sum of the current block.)
 *
 * The caller allocates the buffers (each [T, d] of `dtype`) and fills the
 * struct with attnres_state_init; the library only updates `folded`.
 * `folded` = number of layer outputs v_1 .. v_folded already folded into the
 * partial sum / block representations.  Layer outputs must be folded in
 * order: attnres_block_step(p) needs folded == p-1; attnres_layer_step(l)
 * needs folded == l-2 when it is given v_{l-1} to fold, folded == l-1
 * when not; attnres_layer_sources(l) needs folded == l-1.  Anything else
 * returns ATTNRES_ESTATE.
 * ---------------------------------------------------------------------- */
typedef struct attnres_state {
  const void* h0;                          /* device [T, d]: b_0, the embedding */
  void* block_reps[ATTNRES_MAX_BLOCKS];    /* block_reps[k-1] = b_k, k = 1..N */
  void* partial;                           /* device [T, d]: running partial sum */
  int64_t T;
  int d;
  int dtype;                               /* attnres_dtype of every buffer */
  int num_layers;                          /* L */
  int block_size;                          /* B */
  float eps;
  int folded;                              /* progress, maintained by the library */
  int flags;                               /* ATTNRES_STATE_*, set by the caller after init */
} attnres_state;

/* attnres_state.flags bit: a layer step that folds F_prev (the fused step)
 * may load the first token's stored rows -- h0, the block sums, the
 * partial sum -- before the kernel launched just before it on the stream
 * has finished (programmatic dependent launch), so that their DRAM latency
 * overlaps that kernel; only F_prev waits for it.  attnres_intrablock_step
 * with F_prev does the same with the partial sum and r_inter.  Set it only
 * when, before every such step, (a) the kernel launched just before it on
 * the stream writes none of the rows the step reads other than F_prev (in
 * a stack that kernel is the layer body; a step issued directly after
 * another step of the same state breaks this), and (b) that kernel is
 * launched without programmatic dependent launch, or signals its
 * dependents only after it has waited for its own prerequisites, as every
 * kernel of this library does: then everything launched before it has
 * completed when the step starts.  The stack drivers of the Python package
 * set it; results are the same bits either way. */
#define ATTNRES_STATE_EARLY_LOADS 0x1

/* Fill *st.  n_block_reps must be >= ceil(L/B) (ATTNRES_ERANGE if
 * ceil(L/B) > ATTNRES_MAX_BLOCKS).  The buffers may not share memory with
 * each other (ATTNRES_EINVAL; *st is not written then).
 * Host only; sets folded = 0 and flags = 0. */
int attnres_state_init(attnres_state* st, const void* h0, void* const* block_reps,
                       int n_block_reps, void* partial, int64_t T, int d, int dtype,
                       int num_layers, int block_size, float eps);

/* Rewind to layer 1 (folded = 0).  Host only; buffers are left as they are. */
int attnres_state_reset(attnres_state* st);

/* attnres_state_resume -- take up a stack after layer `folded` (0..L), for
 * a pipeline stage that starts at layer folded + 1 ([Tutorial] ch. 4.6:
 * cache-based pipeline communication sends a later stage only the blocks
 * completed since it last received, plus the open partial sum).  Host only:
 * sets st->folded and touches no buffer.  The caller has already placed in
 * the state's buffers what layer folded + 1 reads: h0, b_1 .. b_c
 * (c = completed blocks after layer `folded`) and, when layer `folded`
 * does not end its block, the partial sum of v_{first..folded} of the open
 * block; the sender forms them with attnres_block_step(folded) after its
 * last layer.  The next call is attnres_layer_step(folded + 1) with
 * F_prev = NULL (or attnres_layer_sources(folded + 1)).  ATTNRES_EINVAL for
 * folded outside 0..L; other errors as attnres_state_reset. */
int attnres_state_resume(attnres_state* st, int folded);

/* Number of sources layer `layer_idx` (1..L, or L+1 for the final output
 * aggregation) reads: n + [i >= 2] for layer i of block n, ceil(L/B) + 1 for
 * L+1 ([Tutorial] ch. 4.3 Eq. 10; [Atlas] §28 workbench: ceil(L/S) +
 * embedding).  Host only, pure.  Negative status on bad arguments. */
int attnres_num_sources(int layer_idx, int block_size, int num_layers);

/* Host only: the device pointers of layer `layer_idx`'s sources in order
 * [h_0, b_1 .. b_{n-1}, partial (if non-empty)] into out_ptrs (capacity
 * ATTNRES_MAX_SOURCES), their count into *out_S.  Needs folded ==
 * layer_idx - 1.  With attnres_block_step this gives the unfused path:
 * block_step(p) then aggregate(layer_sources(p+1)). */
int attnres_layer_sources(const attnres_state* st, int layer_idx, const void** out_ptrs,
                          int* out_S);

/* ------------------------------------------------------------------------
 * attnres_block_step -- fold layer `layer_idx`'s output v = F_out into the
 * block bookkeeping ([Tutorial] ch. 4.3, 4.6):
 *   new = (partial non-empty) ? partial + v : v      (fp32 add, one rounding)
 *   if layer_idx ends its block (layer_idx % B == 0 or layer_idx == L):
 *        b_n = new, partial becomes empty
 *   else partial = new
 * F_out: device [T, d] of st->dtype, sharing no memory with the state's
 * rows (ATTNRES_EINVAL).  Needs folded == layer_idx - 1; advances folded.
 * One elementwise launch.
 * ---------------------------------------------------------------------- */
int attnres_block_step(attnres_state* st, const void* F_out, int layer_idx, int* dev_err,
                       void* stream);

/* ------------------------------------------------------------------------
 * attnres_layer_step -- the fused hot path of one layer: fold F_prev =
 * v_{l-1} (exactly as attnres_block_step(l-1) would, same rounding, written
 * to the partial sum or to b_n) and aggregate layer l over its sources,
 * using the freshly formed partial / b_n as the last source without reading
 * it back.  One launch.
 *   layer_idx  1..L+1 (L+1 = the final output aggregation over [h_0, b_1..b_N])
 *   F_prev     device [T, d] of st->dtype; NULL when v_{l-1} is already
 *              folded (layer 1, or a state resumed with attnres_state_resume
 *              at folded == l-1): then layer l is aggregated over the
 *              state's sources as they are
 *   w_l        device [d] fp32 pseudo-query of this layer
 *   out_r      device [T, d] of st->dtype; it and out_weights may not share
 *              memory with the state's rows or F_prev (ATTNRES_EINVAL)
 *   out_weights device [T, S_l] fp32 or NULL
 * Needs folded == layer_idx - 2 with F_prev, layer_idx - 1 without;
 * leaves folded at layer_idx - 1.  Bit-identical to block_step(l-1) +
 * aggregate(layer_sources(l)).
 * ---------------------------------------------------------------------- */
int attnres_layer_step(attnres_state* st, const void* F_prev, const float* w_l, int layer_idx,
                       void* out_r, float* out_weights, int* dev_err, void* stream);

/* ------------------------------------------------------------------------
 * Two-phase schedule of inference ([Tutorial] ch. 4.4 and 4.6): the cached
 * sources [h_0, b_1 .. b_{n-1}] do not change inside block n, so one
 * batched inter-block pass reads each of them once and aggregates them for
 * every layer query of the block; each layer then folds in its own partial
 * sum with an online-softmax merge.  Same results as attnres_layer_step up
 * to fp32 rounding.  Both calls need rows of a 16-byte multiple with at
 * most 2 x 448 16-byte vectors (d <= 7168 bf16 / 3584 fp32) and 16-byte
 * aligned buffers (ATTNRES_ERANGE / ATTNRES_EINVAL otherwise).
 *
 * attnres_interblock -- phase 1 for one block.
 *   sources    host array of n (1..9) device pointers [T, d] of dtype
 *   w_queries  host array of Q (1..16) device pointers [d] fp32 (the
 *              block's layer queries in order), each 16-byte aligned
 *   out_r      device [Q, T, d] fp32: per query, the softmax-weighted sum
 *              over the n sources (normalised)
 *   out_lse    device [Q, T] fp32: log sum_s exp(z_qs) of those logits
 *   out_weights device [Q, T, n] fp32 (softmax over the n sources) or NULL
 *   out_r0     device [T, d] of dtype, 16-byte aligned, or NULL: query 0's
 *              row rounded to dtype -- the output of the block's first
 *              layer, the same bits attnres_intrablock_step writes for it
 *              (which the caller may then skip: it folds nothing there)
 *   out_weights0 device [T, n] fp32 or NULL: query 0's weights, the first
 *              layer's (the same bits attnres_intrablock_step writes)
 *   workspace  NULL, or device scratch of at least
 *              attnres_interblock_workspace_size(n, T, d, dtype, Q) bytes,
 *              256-byte aligned, owned by the caller, sharing no memory
 *              with an input or output (its contents on entry do not
 *              matter).  With it (bf16 sources, d a multiple of 64) the
 *              Q x n logits of all tokens are taken on the tensor cores
 *              (tcgen05.mma): the queries split into three bf16 terms
 *              (hi + mid + lo, fp32 accumulation), tiles of tokens x
 *              sources loaded by TMA, the channels split across CTAs; the
 *              softmax and the weighted sums then read the sources again.
 *              Without it (or when the size is 0) every step runs on the
 *              CUDA cores in one pass.  Results agree to fp32 rounding.
 *   workspace_bytes  its size
 *   Every source row is read once for all Q queries (twice with the
 *   workspace: once for the logits, once for the weighted sums).  No output
 *   may share memory with a source or with another output (ATTNRES_EINVAL).
 * ---------------------------------------------------------------------- */
int attnres_interblock(const void* const* sources, int n, int64_t T, int d, int dtype,
                       const float* const* w_queries, int Q, float eps, float* out_r,
                       float* out_lse, float* out_weights, void* out_r0, float* out_weights0,
                       void* workspace, int64_t workspace_bytes, int* dev_err, void* stream);

/* Bytes of workspace attnres_interblock's tensor-core logits need for n
 * sources of T tokens and d channels and Q queries on the current device
 * (the partial dot products of every channel split); 0 when that path does
 * not apply (fp32 sources, d not a multiple of 64).  Negative
 * attnres_status on bad arguments. */
int64_t attnres_interblock_workspace_size(int n, int64_t T, int d, int dtype, int Q);

/* attnres_intrablock_step -- phase 2 for layer l (1..L) of block n:
 *   first layer of its block (i = 1): F_prev NULL and the previous block
 *     already closed (attnres_block_step); r = r_inter.
 *   later layers (i >= 2): F_prev = v_{l-1} is folded into the partial sum
 *     exactly as attnres_layer_step folds it, p = the new partial sum,
 *     z_p = w_l . RMSNorm(p), m = max(lse, z_p) and
 *       r = (e^{lse-m} r_inter + e^{z_p-m} p) / (e^{lse-m} + e^{z_p-m}).
 *   r_inter, lse_inter, a_inter: this layer's rows of attnres_interblock's
 *     outputs ([T, d], [T], [T, n] or NULL).
 *   out_r: device [T, d] of st->dtype; out_weights: [T, S_l] fp32 or NULL
 *     (the cached sources' weights scaled into the merged softmax, then the
 *     partial sum's).
 * Needs folded == l-1 (i = 1) or l-2 (i >= 2); advances folded like
 * attnres_layer_step.  The final aggregation (L+1) uses attnres_layer_step.
 * Later layers with bf16 rows of d = 7168 stream their rows (previous
 * partial, F_prev, r_inter) through the persistent TMA ring; its waits are
 * bounded, and one that runs out sets ATTNRES_DEVERR_WAIT_TIMEOUT in
 * dev_err and leaves NaN in that token's outputs. */
int attnres_intrablock_step(attnres_state* st, const void* F_prev, const float* w_l,
                            int layer_idx, const float* r_inter, const float* lse_inter,
                            const float* a_inter, void* out_r, float* out_weights,
                            int* dev_err, void* stream);

/* ------------------------------------------------------------------------
 * attnres_synthetic_layer -- the stand-in layer body used to drive a stack
 * forward without trained weights (not part of the method):
 *   out[t,c] = tanh(x[t,c] * g[c]) * s[c], fp32 math, rounded to `dtype`.
 * x, out: device [T, d] of dtype (may alias); g, s: device [d] fp32.
 * ---------------------------------------------------------------------- */
int attnres_synthetic_layer(const void* x, const float* g, const float* s, void* out, int64_t T,
                            int d, int dtype, void* stream);

/* ------------------------------------------------------------------------
 * attnres_synthetic_layer_backward -- gradient of attnres_synthetic_layer
 * (the stand-in body, not part of the method), for a stack backward:
 *   grad_x[t,c] = (grad_out_a + grad_out_b)[t,c] * (1 - tanh(x g)^2) * g[c] * s[c]
 * x: the layer's input [T, d] of dtype; grad_out_a: [T, d] of dtype, the
 * gradient of the loss with respect to the layer's output; grad_out_b: a
 * second such term added to it, or NULL; grad_x: [T, d] of dtype (may alias
 * either gradient input); g, s: [d] fp32.  fp32 math, rounded to dtype.
 * T = 0 launches nothing and accepts NULL buffers.
 * ---------------------------------------------------------------------- */
int attnres_synthetic_layer_backward(const void* x, const float* g, const float* s, const void* grad_out_a,
                                     const void* grad_out_b, void* grad_x, int64_t T, int d, int dtype,
                                     void* stream);

/* ------------------------------------------------------------------------
 * attnres_fold -- the block bookkeeping of [Tutorial] ch. 4.3 (Eq. 10) on
 * plain buffers, without a state: dst = prev + F (fp32 sum, one rounding to
 * dtype), or dst = F when prev is NULL (a block's first layer output opens
 * its partial sum).  prev, F, dst: device [T, d] of dtype; elementwise, so
 * dst may alias prev or F.  Used where the partial sums of a block are kept
 * per layer (the recomputed forward of a stack backward).
 * ---------------------------------------------------------------------- */
int attnres_fold(const void* prev, const void* F, void* dst, int64_t T, int d, int dtype, void* stream);

/* ------------------------------------------------------------------------
 * Operators of a layer body.  Between two aggregations a layer maps r_l to
 * its output v_l; the calls below are what such a body is made of: the
 * projections around it (attnres_linear), the norm and rotation of its heads
 * (attnres_qk_norm_rope) and a token mixer with a state of fixed size
 * (attnres_linear_attention).  It is a simpler mixer than the pages' own (a
 * delta rule with forgetting per channel, gated latent attention, experts),
 * which are not here; the formulas here define the operations.
 *
 * Row strides (ld*, *_stride) are in elements between consecutive rows
 * (tokens) of a tensor whose rows are otherwise contiguous: slices of one
 * wider buffer can be passed as they are.  A row stride is at least the
 * row's length.
 * ---------------------------------------------------------------------- */

/* activations of attnres_linear */
typedef enum {
  ATTNRES_ACT_NONE = 0,
  ATTNRES_ACT_GELU = 1,      /* z Phi(z), Phi the normal distribution function */
  ATTNRES_ACT_GELU_TANH = 2, /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) */
  ATTNRES_ACT_SILU = 3       /* z / (1 + exp(-z)) */
} attnres_activation;

/* ------------------------------------------------------------------------
 * attnres_linear -- matrix product with bias, activation and residual in
 * its epilogue:
 *   z[m,n] = sum_k x[m,k] w[n,k] + bias[n]     (fp32 accumulate)
 *   out[m,n] = round(act(z[m,n]) + residual[m,n])
 * x         device [M, K] of dtype, row stride ldx
 * w         device [N, K] of dtype, contiguous
 * bias      device [N] fp32 or NULL
 * residual  device [M, N] of dtype, row stride ldr, or NULL; it may be out
 *           itself (with ldr = ldo)
 * out       device [M, N] of dtype, row stride ldo
 * M 0..2^31 - 65 (0 launches nothing and accepts NULL buffers), N, K 1..2^30
 *           (ATTNRES_ERANGE above)
 * act       one of attnres_activation
 * workspace NULL, or device scratch of workspace_bytes, 256-byte aligned,
 *           sharing no memory with an operand (its contents on entry do not
 *           matter).  bf16 operands whose rows start on 16-byte boundaries go
 *           to the tensor cores (tcgen05) without one.  Others are first
 *           copied into it: bf16 to aligned rows, fp32 as three bf16 terms
 *           each, whose six leading products keep fp32 precision (there an
 *           infinite operand gives NaN).  Where it is too small for that, and
 *           for small fp32 products, the CUDA cores take the call.
 * No output may share memory with an input (but residual, as above).
 * Calls that overlap in time need a workspace each.
 * ---------------------------------------------------------------------- */
int attnres_linear(const void* x, int64_t ldx, const void* w, const float* bias, const void* residual, int64_t ldr,
                   void* out, int64_t ldo, int64_t M, int N, int K, int dtype, int act, void* workspace,
                   int64_t workspace_bytes, int* dev_err, void* stream);

/* Bytes of workspace with which attnres_linear takes its fastest path for
 * contiguous operands of these sizes (0: it needs none).  Negative
 * attnres_status on bad arguments. */
int64_t attnres_linear_workspace_size(int64_t M, int N, int K, int dtype);

/* The same for these operands, wherever they lie (x, w: pointers or NULL for
 * aligned ones, not dereferenced): bf16 rows off the 16-byte boundaries have
 * room for their copies, without which the CUDA cores take the call. */
int64_t attnres_linear_operands_workspace_size(const void* x, int64_t ldx, const void* w, int64_t M, int N, int K,
                                               int dtype);

/* ------------------------------------------------------------------------
 * attnres_linear_backward -- gradients of attnres_linear, nothing kept from
 * the forward (z is recomputed where the activation needs it):
 *   dz = grad_out * act'(z)      (grad_out itself without an activation)
 *   grad_x[m,k] = sum_n dz[m,n] w[n,k]
 *   grad_w[n,k] = sum_m dz[m,n] x[m,k]
 *   grad_bias[n] = sum_m dz[m,n]
 * The residual's gradient is grad_out.
 * x, w, bias, act, sizes  as in attnres_linear (bias is only read with an
 *             activation)
 * grad_out    device [M, N] of dtype, row stride ldg
 * grad_x      device [M, K] of dtype, contiguous, or NULL to skip
 * grad_w      device [N, K] of dtype, contiguous, or NULL
 * grad_bias   device [N] fp32, or NULL
 * workspace   device scratch of at least
 *             attnres_linear_backward_workspace_size(...) bytes, 256-byte
 *             aligned (required)
 * All outputs are overwritten, with sums in a fixed order (bit-reproducible);
 * with bf16 tensors the products grad_x and grad_w take dz rounded to bf16
 * (grad_bias sums it in fp32).  M = 0 zeroes grad_w and grad_bias.
 * ---------------------------------------------------------------------- */
int attnres_linear_backward(const void* x, int64_t ldx, const void* w, const float* bias, const void* grad_out,
                            int64_t ldg, void* grad_x, void* grad_w, float* grad_bias, int64_t M, int N, int K,
                            int dtype, int act, void* workspace, int64_t workspace_bytes, int* dev_err,
                            void* stream);

/* Bytes of workspace attnres_linear_backward needs.  Negative
 * attnres_status on bad arguments. */
int64_t attnres_linear_backward_workspace_size(int64_t M, int N, int K, int dtype, int act);

/* The same with room for the copies of these operands (as
 * attnres_linear_operands_workspace_size); never less than by sizes alone. */
int64_t attnres_linear_backward_operands_workspace_size(const void* x, int64_t ldx, const void* w, const void* grad_out,
                                                        int64_t ldg, int64_t M, int N, int K, int dtype, int act);

/* ------------------------------------------------------------------------
 * attnres_qk_norm_rope -- RMSNorm of every head of q and k and rotation by
 * position, in one launch.  Per token t and head row x of D channels:
 *   y = gain * x / sqrt(mean_c x_c^2 + eps)
 *   pair i of the first `rot` channels, (a, b) = (y_i, y_{i + rot/2}), or
 *   (y_{2i}, y_{2i+1}) when interleaved, turns by p = positions[t] inv_freq[i]:
 *   out_a = a cos p - b sin p,  out_b = b cos p + a sin p;
 *   channels rot .. D-1 stay.
 * q           device [T, Hq, D] of dtype, token stride q_stride; NULL if Hq = 0
 * k           device [T, Hk, D] of dtype, token stride k_stride; NULL if Hk = 0
 * q_gain, k_gain  device [D] fp32 or NULL (no gain)
 * positions   device [T] int64 (NULL allowed when rot = 0).  The angle is
 *             reduced before it is rounded to fp32: far positions keep the
 *             precision of near ones.
 * inv_freq    device [rot / 2] fp32 (NULL allowed when rot = 0)
 * rot         even, 0 .. D
 * q_out, k_out  device [T, H, D] of dtype with their own token strides; each
 *             may be its input itself (same stride), and may share no other
 *             memory with an input or output
 * T >= 0 (0 launches nothing), D 1..1024, Hq + Hk >= 1.
 * ---------------------------------------------------------------------- */
int attnres_qk_norm_rope(const void* q, int64_t q_stride, int Hq, const void* k, int64_t k_stride, int Hk, int64_t T,
                         int D, int dtype, const float* q_gain, const float* k_gain, float eps,
                         const int64_t* positions, const float* inv_freq, int rot, int interleaved, void* q_out,
                         int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* stream);

/* ------------------------------------------------------------------------
 * attnres_qk_norm_rope_backward -- its gradients, from the forward's inputs.
 * With dy the incoming gradient turned back, h = x / rho and n = gain * dy:
 *   grad_x = (n - h mean_c(n_c h_c)) / rho,   grad_gain[c] = sum_{t,heads} dy_c h_c
 * grad_q_out, grad_k_out  device [T, H, D] of dtype, token strides given
 * grad_q, grad_k          device [T, H, D] of dtype, token strides given
 *             (each may be the incoming gradient itself, same stride)
 * grad_q_gain, grad_k_gain  device [D] fp32, overwritten, or NULL to skip;
 *             summed in a fixed order (bit-reproducible)
 * workspace   device scratch, 4-byte aligned, of at least
 *             attnres_qk_norm_rope_backward_workspace_size(T, Hq, Hk, D)
 *             bytes; may be NULL when neither gain gradient is wanted
 * T = 0 only zeroes the gain gradients.
 * ---------------------------------------------------------------------- */
int attnres_qk_norm_rope_backward(const void* q, int64_t q_stride, int Hq, const void* k, int64_t k_stride, int Hk,
                                  int64_t T, int D, int dtype, const float* q_gain, const float* k_gain, float eps,
                                  const int64_t* positions, const float* inv_freq, int rot, int interleaved,
                                  const void* grad_q_out, int64_t gqo_stride, const void* grad_k_out,
                                  int64_t gko_stride, void* grad_q, int64_t gq_stride, void* grad_k,
                                  int64_t gk_stride, float* grad_q_gain, float* grad_k_gain, void* workspace,
                                  int64_t workspace_bytes, void* stream);

/* Bytes of workspace the gain gradients need on the current device. */
int64_t attnres_qk_norm_rope_backward_workspace_size(int64_t T, int Hq, int Hk, int D);

/* ------------------------------------------------------------------------
 * attnres_linear_attention -- causal linear attention with one decay per
 * head, over prompts.  Each of num_seqs sequences and H heads keeps a state
 * S [Dk, Dv], decayed by exp(log_decay[h]) before every token:
 *   S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T,    out_t = scale q_t S_t
 * q, k        device [T, H, Dk] of dtype, token strides given
 * v           device [T, H, Dv] of dtype, token stride given
 * log_decay   device [H] fp32, <= 0 (-inf: each token alone; a constant of
 *             the head: it gets no gradient)
 * cu_seqlens  device [num_seqs + 1] int32, non-decreasing, 0 <= .. <= T:
 *             sequence n is rows cu_seqlens[n] .. cu_seqlens[n+1] - 1 (it may
 *             be empty).  Rows outside every sequence are left as they are.
 *             Values outside 0..T are clamped.  NULL: one sequence of T rows
 *             (num_seqs = 1).
 * initial_state device [num_seqs, H, Dk, Dv] fp32 or NULL (zero)
 * final_state device [num_seqs, H, Dk, Dv] fp32 or NULL; it may be
 *             initial_state itself
 * scale       finite; 1/sqrt(Dk) is usual
 * out         device [T, H, Dv] of dtype, token stride given
 * workspace   device scratch of at least
 *             attnres_linear_attention_workspace_size(...) bytes, 256-byte
 *             aligned (NULL when that is 0).  Calls that overlap in time need
 *             one each.
 * T >= 0, H 1..65535, Dk, Dv 1..256, num_seqs 1..65535 (ATTNRES_ERANGE
 * above).  The state is held in fp32.  bf16 tensors with Dk and Dv up to 128
 * and multiples of 16, 16-byte aligned rows, run in chunks of 128 tokens on
 * the tensor cores (tcgen05): the state and the chunk's scores enter an
 * output's products with 16 bits, the state's own sums keep fp32 precision.
 * Others run on the CUDA cores in fp32.  Where the sequences do not fill the
 * GPU evenly they are cut into pieces (whose states lie in the workspace).
 * Infinities and NaN reach the tokens behind them and no others; a token's
 * infinity becomes NaN in the state (one of the initial state stays what it
 * is).
 * ---------------------------------------------------------------------- */
int attnres_linear_attention(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                             int64_t v_stride, int64_t T, int H, int Dk, int Dv, int dtype, const float* log_decay,
                             const int32_t* cu_seqlens, int num_seqs, const float* initial_state, float* final_state,
                             float scale, void* out, int64_t out_stride, void* workspace, int64_t workspace_bytes,
                             int* dev_err, void* stream);

/* Bytes of workspace that every call of up to T tokens in up to num_seqs
 * sequences needs (0: none; other arguments as in the calls). */
int64_t attnres_linear_attention_workspace_size(int64_t T, int H, int Dk, int Dv, int dtype, int num_seqs);

/* ------------------------------------------------------------------------
 * attnres_linear_attention_backward -- its gradients, from the forward's
 * inputs (nothing is kept).  With R_t the gradient at S_t,
 *   R_t = scale q_t do_t^T + exp(log_decay) R_{t+1}
 *   (R of the last token: scale q do^T + grad_final_state)
 *   grad_q_t = scale S_t do_t,  grad_k_t = R_t v_t,  grad_v_t = R_t^T k_t,
 *   grad_initial_state = exp(log_decay) R_{first}
 *   (grad_final_state itself for an empty sequence).
 * grad_out    device [T, H, Dv] of dtype, token stride given
 * grad_q, grad_k, grad_v  device, contiguous [T, H, D] of dtype, or NULL to
 *             skip (its scan does not run); rows outside every sequence are
 *             left as they are
 * grad_final_state    device [num_seqs, H, Dk, Dv] fp32 or NULL (zero)
 * grad_initial_state  the same shape or NULL; it may be grad_final_state.  It
 *             comes with grad_v (ATTNRES_EINVAL without, but for T = 0)
 * Other arguments as in attnres_linear_attention; workspace of at least
 * attnres_linear_attention_backward_workspace_size(...) bytes.  Infinities
 * and NaN reach grad_q of the tokens behind them, grad_k and grad_v of those
 * before them.
 * ---------------------------------------------------------------------- */
int attnres_linear_attention_backward(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                      int64_t v_stride, int64_t T, int H, int Dk, int Dv, int dtype,
                                      const float* log_decay, const int32_t* cu_seqlens, int num_seqs,
                                      const float* initial_state, float scale, const void* grad_out,
                                      int64_t grad_out_stride, const float* grad_final_state, void* grad_q,
                                      void* grad_k, void* grad_v, float* grad_initial_state, void* workspace,
                                      int64_t workspace_bytes, int* dev_err, void* stream);

/* The same for attnres_linear_attention_backward. */
int64_t attnres_linear_attention_backward_workspace_size(int64_t T, int H, int Dk, int Dv, int dtype, int num_seqs);

/* ------------------------------------------------------------------------
 * attnres_linear_attention_step -- the recurrent form for decoding: row b of
 * the batch is one token of the sequence whose state lies in slot slots[b].
 * q, k        device [B, H, Dk] of dtype, row strides given
 * v, out      device [B, H, Dv] of dtype, row strides given
 * state       device [num_slots, H, Dk, Dv] fp32, updated in place
 * slots       device [B] int32, or NULL (row b in slot b, B <= num_slots).
 *             A row whose slot is outside 0..num_slots-1 is padding: its out
 *             row is left as it is.  Rows that name the same slot are
 *             consecutive tokens of that sequence, in the order of the rows.
 * B 0..65535 (0 launches nothing); Dk, Dv, H, log_decay, scale as above.
 * ---------------------------------------------------------------------- */
int attnres_linear_attention_step(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                  int64_t v_stride, int B, int H, int Dk, int Dv, int dtype, const float* log_decay,
                                  float* state, int num_slots, const int32_t* slots, float scale, void* out,
                                  int64_t out_stride, void* stream);

/* ------------------------------------------------------------------------
 * attnres_layer_norm -- layer norm of whole rows:
 *   h = (x - mean_c x) / sqrt(mean_c (x - mean)^2 + eps),  out = gain h + bias
 * x, out      device [T, d] of dtype, row strides given; out may be x itself
 *             (same stride) and may share no other memory with an input
 * gain, bias  device [d] fp32 or NULL (1 and 0)
 * eps         finite, >= 0
 * T >= 0 (0 launches nothing and accepts NULL buffers), d 1..2^24
 * (ATTNRES_ERANGE above).  Sums are fp32; the mean is held as two numbers, so
 * rows whose mean is far from zero keep their digits.  Their squares have to
 * lie within fp32: x - mean up to 1.8e19 / sqrt(d) (beyond it a row comes out as
 * its bias, or NaN).  Infinities and NaN of a row reach no other row's result.
 * ---------------------------------------------------------------------- */
int attnres_layer_norm(const void* x, int64_t x_stride, int64_t T, int d, int dtype, const float* gain, const float* bias,
                       float eps, void* out, int64_t out_stride, void* stream);

/* ------------------------------------------------------------------------
 * attnres_layer_norm_backward -- its gradients, from the forward's input
 * (nothing is kept).  With n = gain * grad_out and sigma the row's divisor:
 *   grad_x = (n - mean_c n - h mean_c(n h)) / sigma
 *   grad_gain[c] = sum_t grad_out h,   grad_bias[c] = sum_t grad_out
 * grad_out    device [T, d] of dtype, row stride given
 * grad_x      the same, or NULL to skip; it may be grad_out itself (same
 *             stride).  Infinities and NaN of a row of x or grad_out reach no
 *             other row of it.
 * grad_gain, grad_bias  device [d] fp32, overwritten, or NULL to skip; summed
 *             in fp32 in a fixed order (bit-reproducible)
 * workspace   device scratch, 256-byte aligned, of at least
 *             attnres_layer_norm_backward_workspace_size(T, d) bytes; may be
 *             NULL when neither grad_gain nor grad_bias is wanted.  Calls that
 *             overlap in time need one each.
 * T = 0 only zeroes grad_gain and grad_bias.
 * ---------------------------------------------------------------------- */
int attnres_layer_norm_backward(const void* x, int64_t x_stride, int64_t T, int d, int dtype, const float* gain, float eps,
                                const void* grad_out, int64_t grad_out_stride, void* grad_x, int64_t grad_x_stride,
                                float* grad_gain, float* grad_bias, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace the gain and bias gradients of up to T rows need on the
 * current device. */
int64_t attnres_layer_norm_backward_workspace_size(int64_t T, int d);

/* ------------------------------------------------------------------------
 * attnres_gated_recurrence -- gated linear recurrence over prompts: a state
 * of C channels per sequence, forgetting by a gate per token and channel:
 *   a_t = 1 / (1 + exp(-forget_t)),   h_t = a_t h_{t-1} + (1 - a_t) x_t
 *   out_t = h_t gate_t / (1 + exp(-gate_t))   (h_t where gate is NULL)
 * x, forget   device [T, C] of dtype, row strides given (slices of one
 *             projection's rows, say)
 * gate        the same or NULL
 * cu_seqlens  device [num_seqs + 1] int32, non-decreasing, 0 <= .. <= T:
 *             sequence n is rows cu_seqlens[n] .. cu_seqlens[n+1] - 1 (it may
 *             be empty).  Rows outside every sequence are left as they are.
 *             Values outside 0..T are clamped; offsets that decrease give
 *             unspecified results.  NULL: one sequence of T rows (num_seqs =
 *             1).
 * initial_state device [num_seqs, C] fp32 or NULL (zero)
 * final_state device [num_seqs, C] fp32 or NULL; it may be initial_state
 *             itself
 * out         device [T, C] of dtype, row stride given; it shares no memory
 *             with an input
 * chunk_states device [ceil(T / ATTNRES_RECURRENCE_CHUNK), C] fp32 or NULL:
 *             the states ahead of every 64th row, which the backward goes on
 *             from (rows of it that lie in no sequence are unspecified)
 * T 0..2^31 - 65537, C 1..2^24, num_seqs 1..65535 (ATTNRES_ERANGE above).
 * dev_err     device int or NULL.  CTAs that share channels wait for one
 *             another's spans; a wait that runs out (a bound of seconds) ORs
 *             ATTNRES_DEVERR_WAIT_TIMEOUT into *dev_err, and what depends on it
 *             is NaN
 * The state is held in fp32, and so is a_t (off by some 2^-22 of itself, which a
 * memory of n tokens sees n times).  Either gate below -83 (minus infinity too)
 * counts as -83: a_t of 1e-36.  Infinities and NaN reach the tokens of their
 * channel and sequence behind them and no others (an infinite state may become
 * NaN).  The last bits of a result do not depend on how the rows lie in memory.
 * ---------------------------------------------------------------------- */
#define ATTNRES_RECURRENCE_CHUNK 64
int attnres_gated_recurrence(const void* x, int64_t x_stride, const void* forget, int64_t forget_stride, const void* gate,
                             int64_t gate_stride, int64_t T, int C, int dtype, const int32_t* cu_seqlens, int num_seqs,
                             const float* initial_state, float* final_state, void* out, int64_t out_stride,
                             float* chunk_states, int* dev_err, void* stream);

/* ------------------------------------------------------------------------
 * attnres_gated_recurrence_backward -- its gradients, from the forward's
 * inputs and its chunk_states.  With s = gate / (1 + exp(-gate)) (1 without a
 * gate) and dh_t the gradient at h_t:
 *   dh_t = grad_out_t s_t + a_{t+1} dh_{t+1}
 *   (of a sequence's last token: grad_out s + grad_final_state)
 *   grad_x = (1 - a) dh,   grad_forget = dh (h_{t-1} - x) a (1 - a),
 *   grad_gate = grad_out h ds/dgate,
 *   grad_initial_state = a dh of the first token (grad_final_state itself for
 *   an empty sequence).
 * chunk_states  as the forward wrote them for the same arguments
 * grad_out      device [T, C] of dtype, row stride given
 * grad_x, grad_forget, grad_gate  device [T, C] of dtype, row strides given,
 *             or NULL to skip; rows outside every sequence are left as they
 *             are.  grad_gate needs gate.
 * grad_final_state    device [num_seqs, C] fp32 or NULL (zero)
 * grad_initial_state  the same shape or NULL; it may be grad_final_state
 * Other arguments as in attnres_gated_recurrence.
 * ---------------------------------------------------------------------- */
int attnres_gated_recurrence_backward(const void* x, int64_t x_stride, const void* forget, int64_t forget_stride,
                                      const void* gate, int64_t gate_stride, int64_t T, int C, int dtype,
                                      const int32_t* cu_seqlens, int num_seqs, const float* initial_state,
                                      const float* chunk_states, const void* grad_out, int64_t grad_out_stride,
                                      const float* grad_final_state, void* grad_x, int64_t grad_x_stride, void* grad_forget,
                                      int64_t grad_forget_stride, void* grad_gate, int64_t grad_gate_stride,
                                      float* grad_initial_state, int* dev_err, void* stream);

/* ------------------------------------------------------------------------
 * attnres_gated_recurrence_step -- the form for decoding: row b of the batch
 * is one token of the sequence whose state lies in slot slots[b].
 * x, forget, gate, out  device [B, C] of dtype, row strides given (gate: or
 *             NULL)
 * state       device [num_slots, C] fp32, updated in place
 * slots       device [B] int32, or NULL (row b in slot b, B <= num_slots).
 *             A row whose slot is outside 0..num_slots-1 is padding: its out
 *             row is left as it is.  Rows that name the same slot are
 *             consecutive tokens of that sequence, in the order of the rows.
 * B 0..65535 (0 launches nothing); C as above.
 * ---------------------------------------------------------------------- */
int attnres_gated_recurrence_step(const void* x, int64_t x_stride, const void* forget, int64_t forget_stride, const void* gate,
                                  int64_t gate_stride, int B, int C, int dtype, float* state, int num_slots,
                                  const int32_t* slots, void* out, int64_t out_stride, void* stream);

/* ------------------------------------------------------------------------
 * attnres_grad_clip -- the norm of a list of gradients taken as one vector,
 * and their clipping:
 *   norm = sqrt(sum over all tensors of g^2)
 *   out = g * (max_norm / norm) where norm > max_norm, else g
 * A norm that is not finite (a gradient is an infinity or NaN) scales nothing:
 * out = g, and out_norm says so.  A finite norm above fp32's numbers clips like
 * any other; out_norm is then the largest of them (3.4e38).
 * grads       host array of n device pointers, contiguous tensors
 * outs        host array of n device pointers, or NULL (only the norm).
 *             outs[i] may be grads[i] itself (in place: nothing is written
 *             where nothing is clipped); it shares no other memory with a
 *             tensor of the call
 * numels      host array of n element counts (0: the pointers may be NULL)
 * dtypes      host array of n attnres_dtype (outs[i] has that of grads[i])
 * n 0..65535 (ATTNRES_ERANGE above)
 * max_norm    >= 0 (infinity: nothing is clipped); not read without outs
 * out_norm    device fp32 [1]
 * workspace   device scratch, 256-byte aligned, of at least
 *             attnres_grad_clip_workspace_size() bytes.  Calls that overlap in
 *             time need one each.
 * The host arrays are read during the call only.  The squares are summed in
 * fp32 over chunks, those in fp64 (in fp64 throughout where fp32 does not
 * hold the squares), in a fixed order (bit-reproducible).
 * ---------------------------------------------------------------------- */
int attnres_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes, int n,
                      float max_norm, float* out_norm, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace attnres_grad_clip needs on the current device. */
int64_t attnres_grad_clip_workspace_size(void);

/* ------------------------------------------------------------------------
 * attnres_debug_wait_test -- a diagnostic with no counterpart in the pages:
 * makes the bounded waits of the ring kernels launched afterwards from this
 * process run out on a healthy GPU, so that their timeout path can be tested
 * without a fault.
 *   wait_limit_ns  limit of every main-loop wait (a ring slot's landing or
 *                  release); 0 = the default, 2 s.  The drain at a kernel's
 *                  exit always waits up to 2 s for the copies it issued.
 *   withhold_row   0..7: every CTA's producer arms that row of its first
 *                  token but issues no copy for it, so the consumers' wait
 *                  on it runs out after wait_limit_ns; -1 = none.
 * Expected effect: ATTNRES_DEVERR_WAIT_TIMEOUT in dev_err, NaN outputs for
 * the abandoned token, the kernel returns (no slot is refilled under a copy
 * in flight; its copies are drained), the context stays usable.  Outputs of
 * kernels launched in this mode are not meaningful.  (0, -1) restores
 * normal operation.  Process-wide; not for use while other threads launch.
 * Returns ATTNRES_OK, or ATTNRES_EINVAL for withhold_row outside -1..7.
 * ---------------------------------------------------------------------- */
int attnres_debug_wait_test(uint64_t wait_limit_ns, int withhold_row);

/* Human-readable name of a status code (static string). */
const char* attnres_status_string(int status);

/* Detail of the last error returned on this host thread ("" if none). */
const char* attnres_last_error(void);

/* ABI version: (major << 16) | minor. */
int attnres_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTNRES_H */
