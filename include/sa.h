/*
 * sa.h -- C ABI of the Sketch Attention (SA) compression library (libsa.so).
 *
 * What it computes.  One SA layer of SequenceO1, as section 2.1 ("Sketch
 * Attention") of the reading notes "SequenceO1：用可缓存的低秩草图实现端到端十万级用户历史建模"
 * defines it.  For each user b with history X_b (n_b x d, one row per
 * behaviour), shared prototypes P (k x d) and projections W_Q, W_K (d x d):
 *
 *     S   = (P W_Q)(X_b W_K)^T * scale                 k x n_b affinities
 *     A   = softmax of S over the PROTOTYPE axis j      every column sums to 1
 *     X~_b = A X_b                                      k x d sketch, no value projection
 *     m_b  = A 1                                        k per-prototype masses
 *
 * (sum_j m_bj = n_b; X~_bj / m_bj is the mass-normalised sketch.)  The
 * library evaluates S through Q' = P W_Q W_K^T * scale, the rearrangement
 * section 1 of the same notes describes for single-query cross-attention,
 * so the key projection X W_K is never formed; and it fuses affinity,
 * stable softmax and aggregation in one pass over X without writing the
 * k x n matrices to memory, as section 2.4 describes for FlashSA, over
 * ragged batches.
 *
 * Conventions.
 *  - Device pointers are CUDA device memory of the current device (the one
 *    current when the query was prepared).  Host pointers are host memory.
 *  - All arrays are dense and row-major.  bf16 data is IEEE bfloat16 bit
 *    patterns (uint16); fp32 data is IEEE binary32.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    Device-side work is enqueued on it and runs asynchronously unless an
 *    entry point says otherwise.
 *  - The caller owns every buffer it passes; the library owns only what is
 *    inside an sa_query (freed by sa_sketch_free).
 *  - Host-side argument errors are reported immediately and nothing is
 *    enqueued.  Offsets live on the device, so their validity is checked on
 *    the device: a bad offsets array never causes an out-of-bounds access,
 *    but it makes the outputs unspecified and raises a device flag that
 *    sa_read_device_status reports.
 */
#ifndef SA_H_
#define SA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum sa_status {
  SA_OK = 0,
  SA_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misaligned buffer, wrong device */
  SA_ERR_UNSUPPORTED = 2,  /* shape/dtype/GPU without a kernel in this build */
  SA_ERR_WORKSPACE = 3,    /* workspace smaller than sa_workspace_bytes() */
  SA_ERR_CUDA = 4,         /* a CUDA runtime call or kernel launch failed */
  SA_ERR_DEVICE_FLAG = 5   /* a kernel flagged bad offsets or a timed-out wait */
} sa_status;

typedef enum sa_dtype {
  SA_BF16 = 0, /* bf16 inputs, tensor-core pass, fp32 accumulation */
  SA_FP32 = 1  /* fp32 inputs, CUDA-core pass, fp64 accumulation */
} sa_dtype;

/* Device flag bits reported through sa_read_device_status. */
#define SA_DEVFLAG_OFFSET0_NONZERO 1u  /* offsets[0] != 0 */
#define SA_DEVFLAG_OFFSETS_DECREASE 2u /* offsets[b] > offsets[b+1] for some b */
#define SA_DEVFLAG_OFFSET_LAST 4u      /* offsets[batch] != total_rows */
#define SA_DEVFLAG_TIMEOUT 8u          /* a kernel's bounded wait gave up */
#define SA_DEVFLAG_SMEM_ALIGN 16u      /* a kernel found its shared memory misaligned (no work done) */
#define SA_DEVFLAG_ACTION_TYPE 32u     /* an action type id >= the producer's n_types */
#define SA_DEVFLAG_DECAY 64u           /* a head's log decay is positive or NaN */
#define SA_DEVFLAG_SLOT 128u           /* a state slot past the pool, or taken twice in one step */

/* Opaque handle: the precomputed query Q' for one weight set. */
typedef struct sa_query_s* sa_query;

/*
 * sa_prepare_query -- precompute Q' = P W_Q W_K^T * scale (times log2 e) for
 * one set of SA parameters (section 2.1: P^(0) in R^{k x d}, W_Q, W_K in
 * R^{d x d}; section 1: the query/key rearrangement).
 *
 *   P     device, k x d, dtype          shared prototypes P^(0)
 *   W_Q   device, d x d, dtype          query projection
 *   W_K   device, d x d, dtype          key projection
 *   k     1 <= k <= 1024                number of prototypes
 *   d     64, 128 or 256                embedding width
 *   scale finite                        affinity scale (1/sqrt(d) in the paper's setting)
 *   dtype SA_BF16 or SA_FP32            element type of P, W_Q, W_K and of X later
 *   stream                              the precompute kernel runs on it
 *   out   host; receives the handle
 *
 * Allocates device memory (cudaMalloc) for Q' and for W_Q W_K^T * scale
 * (d x d fp32, used by sa_sketch_forward_user_queries).  P, W_Q and W_K are read by
 * a kernel enqueued on `stream`; they must stay alive until it completes.
 * Returns SA_ERR_UNSUPPORTED for shapes without a kernel, or for a GPU
 * other than sm_100.  bf16: d = 64 and 128 take any k <= 1024 (k > 128 runs
 * on clusters of ceil(k / 128) CTAs, each holding 128 prototypes; section
 * 2.2 of the notes puts the final layers at about a thousand prototypes),
 * d = 256 takes k <= 256 (k > 64 on pairs of CTAs).  fp32: k <= 256.
 */
sa_status sa_prepare_query(const void* P, const void* W_Q, const void* W_K, int k, int d,
                           float scale, sa_dtype dtype, void* stream, sa_query* out);

/* Releases a query and its device memory (synchronises with the device).
 * NULL is a no-op. */
void sa_sketch_free(sa_query q);

/* Bytes of device workspace sa_sketch_forward needs for a batch of `batch`
 * users and `total_rows` rows.  Independent of the batch size beyond a fixed
 * bound (it scales with the number of SMs, not with the number of users).
 * Per-user queries need more: sa_workspace_bytes_user_queries. */
size_t sa_workspace_bytes(sa_query q, int64_t batch, int64_t total_rows);

/*
 * sa_sketch_forward -- one SA layer over a ragged batch (section 2.1; ragged
 * batches and fused tiling: section 2.4).
 *
 *   q           prepared query
 *   X           device, total_rows x d, q's dtype; user b owns rows
 *               [offsets[b], offsets[b+1]).  16-byte aligned.
 *   offsets     device, int64, batch + 1 entries: offsets[0] == 0,
 *               non-decreasing, offsets[batch] == total_rows.  No padding:
 *               rows outside a user's range never contribute to it
 *               (section 3.1: padding must not receive mass).
 *   batch       number of users B >= 0
 *   total_rows  N >= 0, < 2^31 - 256
 *   X_tilde     device out, B x k x d fp32 (16-byte aligned): the sketches
 *   mass        device out, B x k fp32: m_bj = sum_i A_ji
 *   workspace   device, >= sa_workspace_bytes(q, B, N) bytes, 256-byte
 *               aligned; no initial contents needed; one call at a time
 *   stream      work is enqueued here; outputs are ready when it is done
 *
 * A user with no rows gets X~ = 0 and m = 0.  Results are bitwise
 * reproducible for the same inputs on the same GPU model.
 */
sa_status sa_sketch_forward(sa_query q, const void* X, const int64_t* offsets, int64_t batch,
                            int64_t total_rows, float* X_tilde, float* mass, void* workspace,
                            size_t workspace_bytes, void* stream);

/*
 * sa_sketch_forward_user_queries -- the SA step of a refinement layer: user
 * b's rows are queried by its own k x d matrix Q_b in place of P (section
 * 2.2 "Stacked Refinement" of the same notes: layer l starts from the shared
 * prototypes and queries the original X with the previous layer's sketch).
 * For each user b:
 *
 *     S_b = (Q_b W_Q)(X_b W_K)^T * scale,  A_b = softmax over prototypes,
 *     X~_b = A_b X_b,  m_b = A_b 1
 *
 * with W_Q, W_K and scale those of `q` (its P is not used).  The library
 * forms Q'_b = Q_b (W_Q W_K^T * scale) in fp32 for every user (a kernel on
 * `stream`, into the workspace) and runs the same fused pass, which loads
 * each user's Q'_b where that user's rows begin.
 *
 *   q           prepared query (supplies d, k, dtype, W_Q, W_K, scale)
 *   queries     device, B x k x d fp32 (4-byte aligned): Q_b for every user
 *               (for example the previous layer's X~, or a function of it);
 *               not modified
 *   X, offsets, batch, total_rows, X_tilde, mass, stream
 *               as for sa_sketch_forward
 *   workspace   device, >= sa_workspace_bytes_user_queries(q, B, N) bytes,
 *               256-byte aligned; one call at a time
 *
 * Every query shape that sa_sketch_forward runs takes per-user queries.
 * Returns SA_ERR_INVALID_ARG if queries is NULL with B > 0 or if B * k_pad
 * reaches 2^31 (k_pad as sa_query_info reports), otherwise as
 * sa_sketch_forward.  An empty user gets X~ = 0 and m = 0 whatever its Q_b.
 */
size_t sa_workspace_bytes_user_queries(sa_query q, int64_t batch, int64_t total_rows);
/* The first two of the three kernels (Q'_b for every user, then the fused
 * pass); sa_sketch_finalize with the same arguments (minus `queries`)
 * completes the layer, as for sa_sketch_partials. */
sa_status sa_sketch_partials_user_queries(sa_query q, const float* queries, const void* X,
                                          const int64_t* offsets, int64_t batch,
                                          int64_t total_rows, float* X_tilde, float* mass,
                                          void* workspace, size_t workspace_bytes, void* stream);
sa_status sa_sketch_forward_user_queries(sa_query q, const float* queries, const void* X,
                                         const int64_t* offsets, int64_t batch,
                                         int64_t total_rows, float* X_tilde, float* mass,
                                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * The two kernels sa_sketch_forward enqueues, for callers that schedule (or
 * time) them separately.  sa_sketch_partials runs the fused pass over X,
 * writing users that lie inside one CTA's row range to the outputs and the
 * others to partial slots in the workspace; sa_sketch_finalize then sums the
 * partial slots in a fixed order, zero-fills empty users and validates the
 * offsets.  Calling both, in this order, on one stream with the same
 * arguments equals sa_sketch_forward.
 */
sa_status sa_sketch_partials(sa_query q, const void* X, const int64_t* offsets, int64_t batch,
                             int64_t total_rows, float* X_tilde, float* mass, void* workspace,
                             size_t workspace_bytes, void* stream);
sa_status sa_sketch_finalize(sa_query q, const void* X, const int64_t* offsets, int64_t batch,
                             int64_t total_rows, float* X_tilde, float* mass, void* workspace,
                             size_t workspace_bytes, void* stream);

/*
 * sa_sketch_forward_host -- the same layer on HOST buffers (end-to-end use).
 *
 *   X_host        host, total_rows x d, q's dtype (pinned memory copies fastest)
 *   offsets_host  host, batch + 1 int64 (validated on the host before any copy)
 *   X_tilde_host  host out, B x k x d fp32
 *   mass_host     host out, B x k fp32
 *   device_buffer device, >= sa_host_path_device_bytes(q, B, N), 256-byte aligned
 *
 * Copies X and the offsets to device_buffer, runs sa_sketch_forward there,
 * copies the results back and synchronises `stream` before returning.
 */
size_t sa_host_path_device_bytes(sa_query q, int64_t batch, int64_t total_rows);
sa_status sa_sketch_forward_host(sa_query q, const void* X_host, const int64_t* offsets_host,
                                 int64_t batch, int64_t total_rows, float* X_tilde_host,
                                 float* mass_host, void* device_buffer,
                                 size_t device_buffer_bytes, void* stream);

/*
 * sa_read_device_status -- synchronises `stream`, reads the device flags of
 * the last call that used `workspace` and clears them.  Returns SA_OK if no
 * flag was set, SA_ERR_DEVICE_FLAG otherwise (with the SA_DEVFLAG_* bits in
 * *flags_out if it is not NULL), SA_ERR_CUDA if the copy failed.
 */
sa_status sa_read_device_status(void* workspace, size_t workspace_bytes, void* stream,
                                uint32_t* flags_out);

/*
 * sa_sketch_forward_noalloc -- sa_sketch_forward for callers that cannot
 * allocate device memory.  (The SequenceO1 paper has no counterpart to this
 * entry point; it exists for callers of this library.)
 *
 * Some callers cannot call cudaMalloc or any other allocator where they run
 * the SA layer: code inside an allocator's own hooks, code under a memory
 * pool that must not grow, or hosts that hand the library only fixed,
 * pre-registered buffers.  This call takes the same inputs and outputs as
 * sa_sketch_forward, but in place of a caller-provided workspace it uses a
 * fixed 32 MiB scratch array inside the library's device image.  Every GPU
 * that loads the library's module holds that array until the process exits.
 * Under CUDA's default lazy module loading the module, and with it the
 * array, is loaded on a device by the first call there; a call with
 * batch = 0 does only that set-up, so a caller can make it while allocating
 * is still allowed.  Later calls allocate nothing.
 *
 *   q, X, offsets, batch, total_rows, X_tilde, mass, stream
 *                     as for sa_sketch_forward
 *   device_flags_out  device, 2 uint32 words (4-byte aligned), or NULL:
 *                     receives, in stream order, this call's device flags
 *                     (word 0: the SA_DEVFLAG_OFFSET* bits, word 1:
 *                     SA_DEVFLAG_TIMEOUT and SA_DEVFLAG_SMEM_ALIGN), which sa_read_device_status
 *                     reports for the workspace path
 *
 * Returns SA_ERR_WORKSPACE when the call needs more scratch than the array
 * holds (sa_workspace_bytes(q, batch, total_rows) > 32 MiB; this covers
 * every query with k * d <= 128 * 128 on a 148-SM GPU), SA_ERR_CUDA if the
 * array's address cannot be looked up, and otherwise what sa_sketch_forward
 * returns.
 *
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current) and caches it with the
 * ID of the device's context; make that first call before any stream
 * capture on the device.  After a device reset the next call runs in a new
 * context and looks the address up again (the module is reloaded then).
 * All calls share the one array, so calls whose work overlaps on the GPU
 * (other streams, other host threads) race on it and give wrong results:
 * serialise them.
 */
sa_status sa_sketch_forward_noalloc(sa_query q, const void* X, const int64_t* offsets,
                                    int64_t batch, int64_t total_rows, float* X_tilde,
                                    float* mass, uint32_t* device_flags_out, void* stream);

/*
 * sa_mass_normalise -- the mass-normalised sketch X~_bj / m_bj (0 where
 * m_bj == 0), the weighted mean of user b's rows under prototype j (section
 * 2.1: the sketch is a weighted aggregation; its masses make it a mean),
 * e.g. as the query of the next refinement layer (section 2.2).
 *
 *   X_tilde  device, batch x k x d fp32 (16-byte aligned), as written by
 *            sa_sketch_forward
 *   mass     device, batch x k fp32
 *   batch    B >= 0;  k >= 1;  d >= 4, a multiple of 4
 *   out      device, batch x k x d fp32 (16-byte aligned); may be X_tilde
 *   stream   the kernel is enqueued here
 *
 * Returns SA_ERR_INVALID_ARG for bad sizes, null pointers or misalignment.
 */
sa_status sa_mass_normalise(const float* X_tilde, const float* mass, int64_t batch, int k, int d,
                            float* out, void* stream);

/*
 * sa_sketch_backward -- gradients of one SA layer (section 2.2 of the notes:
 * the compression module is trained end to end by the ranking loss; the
 * page prints no backward, so these follow from section 2.1's forward by
 * the chain rule).  For upstream gradients G_b = dL/dX~_b and g_b = dL/dm_b:
 *
 *     dA  = G X^T + g 1^T,   dS = A * (dA - 1 c^T),  c_i = sum_j A_ji dA_ji
 *     dX  = A^T G + dS^T Q'              (Q' = P W_Q W_K^T * scale)
 *     R   = dS X,   dP = scale R W_K W_Q^T,
 *     dW_Q = scale P^T R W_K,   dW_K = scale R^T P W_Q
 *
 * One tcgen05 pass over X recomputes the softmax per 128-row tile (no saved
 * activations), writes dX and accumulates R per user; small GEMMs turn R
 * into the parameter gradients.
 *
 *   q           prepared bf16 query with d in {64, 128} and k <= 128
 *               (others: SA_ERR_UNSUPPORTED)
 *   queries     device B x k x d fp32 (per-user queries, as for
 *               sa_sketch_forward_user_queries) or NULL (the shared P)
 *   P_f32       device k x d fp32: the prototypes q was prepared with (read
 *               only when queries is NULL)
 *   W_Q_f32, W_K_f32   device d x d fp32: the projections q was prepared with
 *   X, offsets, batch, total_rows   as for sa_sketch_forward
 *   G           device B x k x d fp32: dL/dX~
 *   g           device B x k fp32: dL/dm, or NULL (zero)
 *   dX          device out, total_rows x d bf16 (16-byte aligned)
 *   dP          device out, k x d fp32 summed over users (shared P), or
 *               B x k x d fp32 per user (with queries: dL/dQ_b)
 *   dW_Q, dW_K  device out, d x d fp32, summed over users
 *   workspace   device, >= sa_workspace_bytes_backward(q, B, N) bytes,
 *               256-byte aligned; one call at a time
 *
 * Device flags (bad offsets, timeouts) are read with sa_read_device_status
 * on the workspace.  Rows of empty users contribute nothing.
 */
size_t sa_workspace_bytes_backward(sa_query q, int64_t batch, int64_t total_rows);
sa_status sa_sketch_backward(sa_query q, const float* queries, const float* P_f32,
                             const float* W_Q_f32, const float* W_K_f32, const void* X,
                             const int64_t* offsets, int64_t batch, int64_t total_rows,
                             const float* G, const float* g, void* dX, float* dP, float* dW_Q,
                             float* dW_K, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Stacked refinement layers (section 2.2 "Stacked Refinement" of the same
 * notes).  Layer l queries the ORIGINAL history X with the previous layer's
 * sketches (layer 1 with the shared prototypes: X~^(0) = P^(0)) and then
 * updates every (user, prototype) row of width d:
 *
 *     z   = LN1(prev_bj + X~_bj / m_bj)          (X~/m is 0 where m_bj = 0)
 *     out = LN2(z + (SiLU(z W1) * (z W3)) W2)
 *
 * where X~, m are that layer's SA outputs, LN normalises over the d features
 * (biased variance, eps 1e-5) with gain gamma and shift beta, and the FFN is
 * SwiGLU-gated with hidden width h and no biases.  The page lost the layer's
 * formulas; this is the reading its text supports (the aggregation added to
 * the previous state and normalised, then a residual feed-forward network):
 * the aggregation enters mass-normalised, a weighted mean of the user's
 * rows, whose scale does not grow with the history length.  Every layer has
 * its own sa_query (W_Q, W_K, scale) and sa_refine (LN and FFN parameters).
 */
typedef struct sa_refine_s* sa_refine;

/*
 * sa_prepare_refine -- the LN and FFN parameters of one refinement layer.
 *
 *   W1, W3   device, d x h fp32, row-major (z W1, z W3)
 *   W2       device, h x d fp32, row-major
 *   gamma1, beta1, gamma2, beta2   device, d fp32 each (LN1, LN2)
 *   d        64 or 128 (256: SA_ERR_UNSUPPORTED)
 *   h        hidden width, a multiple of 128, 128 <= h <= 4096
 *   stream   the copies (bf16, transposed) are made by kernels on it
 *   out      host; receives the handle
 *
 * Allocates device memory for the parameters; the inputs may be freed once
 * `stream` has passed this call.  Errors: SA_ERR_INVALID_ARG (null,
 * misaligned, bad d or h), SA_ERR_UNSUPPORTED (d = 256, or not sm_100),
 * SA_ERR_CUDA.
 */
sa_status sa_prepare_refine(const float* W1, const float* W3, const float* W2,
                            const float* gamma1, const float* beta1, const float* gamma2,
                            const float* beta2, int d, int h, void* stream, sa_refine* out);

/* Releases a refinement handle and its device memory.  NULL is a no-op. */
void sa_refine_free(sa_refine r);

/*
 * sa_refine_update -- the update after a layer's SA step, for batch * k rows
 * (one tcgen05 kernel: LN1, the FFN on the tensor cores in bf16 with fp32
 * accumulation, LN2; the norms in fp32).
 *
 *   prev         device fp32, 16-byte aligned: batch x k x d, or k x d
 *                shared by every user when prev_shared != 0 (layer 1: P)
 *   X_tilde      device, batch x k x d fp32 (16-byte aligned): the layer's
 *                SA sketches
 *   mass         device, batch x k fp32: the layer's masses
 *   batch, k     batch >= 0, k >= 1
 *   out          device, batch x k x d fp32 (16-byte aligned); must not
 *                overlap the inputs
 *   device_flags device uint32 (or NULL): SA_DEVFLAG_TIMEOUT is OR-ed in if
 *                a bounded wait in the kernel gave up
 *   stream       the kernel is enqueued here
 */
sa_status sa_refine_update(sa_refine r, const float* prev, int prev_shared, const float* X_tilde,
                           const float* mass, int64_t batch, int k, float* out,
                           uint32_t* device_flags, void* stream);

/*
 * sa_refine_layer_forward -- one refinement layer over a ragged batch: the
 * SA step (section 2.1 with the layer's query; per-user queries for l >= 2)
 * followed by sa_refine_update.
 *
 *   q          the layer's SA query (its W_Q, W_K, scale; its P for layer 1)
 *   r          the layer's LN and FFN parameters (same d as q; q bf16)
 *   prev       device fp32: NULL for layer 1 (the query and the residual are
 *              the shared prototypes, given as P_f32), else the previous
 *              layer's sketches, batch x k x d
 *   P_f32      device, k x d fp32: the prototypes q was prepared with, as
 *              fp32 (read only when prev is NULL)
 *   X, offsets, batch, total_rows   as for sa_sketch_forward
 *   out        device, batch x k x d fp32: X~^(l); must not overlap prev
 *   workspace  device, >= sa_workspace_bytes_refine_layer(q, batch,
 *              total_rows), 256-byte aligned; one call at a time
 *
 * Device flags (bad offsets, timeouts) are read with sa_read_device_status
 * on the workspace, as for sa_sketch_forward.
 */
size_t sa_workspace_bytes_refine_layer(sa_query q, int64_t batch, int64_t total_rows);
sa_status sa_refine_layer_forward(sa_query q, sa_refine r, const float* prev, const float* P_f32,
                                  const void* X, const int64_t* offsets, int64_t batch,
                                  int64_t total_rows, float* out, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * sa_refine_stack_forward -- `layers` refinement layers in sequence (the
 * final configuration of section 2.2 has two): layer 1 from P_f32, each
 * later layer queried by the previous layer's output; every layer reads the
 * original X.  qs[l], rs[l] are layer l's handles (all with the same k, d).
 *
 *   out        device, batch x k x d fp32: X~^(layers)
 *   workspace  device, >= sa_workspace_bytes_refine_stack(qs[0], batch,
 *              total_rows) (which also holds the layers' intermediate
 *              sketches), 256-byte aligned
 */
size_t sa_workspace_bytes_refine_stack(sa_query q, int64_t batch, int64_t total_rows);
sa_status sa_refine_stack_forward(int layers, const sa_query* qs, const sa_refine* rs,
                                  const float* P_f32, const void* X, const int64_t* offsets,
                                  int64_t batch, int64_t total_rows, float* out, void* workspace,
                                  size_t workspace_bytes, void* stream);

/*
 * Sketch cache (section 2.4 "Local KVCache" of the same notes; section 2.3,
 * Figure 2: hit -> the stored sketch, miss -> one compression).  Only the
 * user-side sketch (X~_b and m_b, k x d and k fp32) is stored, keyed by the
 * user, the model version, the history timestamp and the sketch
 * configuration, for a time-to-live, in a device pool of `capacity` slots.
 * Times are seconds on any clock the caller chooses (passed as `now`).
 *
 * Decisions (the page names the key, the TTL and capacity eviction and no
 * more; this is the reading built):
 *  - an entry is fresh while now - t_insert < ttl; a lookup that finds an
 *    expired entry counts a miss and drops it;
 *  - a hit refreshes the entry's last-use time;
 *  - an insert of a new key takes the free slot with the smallest index,
 *    else evicts the expired entry inserted earliest, else the least
 *    recently used entry (ties: the smaller slot);
 *  - inserting a key that is present replaces its sketch in place and
 *    restarts its TTL; within one call, of two equal keys the later wins.
 * The index is host memory guarded by a mutex; the sketches move only on
 * the device.  Calls on one cache that move data (lookup, insert, forward)
 * must be ordered with one another by the caller: the library reuses one
 * device slot list, so use one stream per cache.  Every call must be made
 * with the cache's device current (SA_ERR_INVALID_ARG otherwise), and `now`
 * must be finite (SA_ERR_INVALID_ARG otherwise).  SA_ERR_CUDA from a call
 * also covers a failed host allocation in the index; the cache's index may
 * then be partly updated, so free the cache.
 */
typedef struct sa_cache_key {
  int64_t user;
  int64_t model_version;
  int64_t history_ts;
  int64_t config;
} sa_cache_key;

typedef struct sa_cache_s* sa_cache;

/* A cache of `capacity` sketches of k x d (k >= 1, d >= 4 and a multiple of
 * 4, capacity >= 1) with a time-to-live of ttl_seconds (> 0).  Allocates
 * capacity * k * (d + 1) * 4 bytes on the current device (SA_ERR_INVALID_ARG
 * if that count does not fit in size_t).  Errors: SA_ERR_INVALID_ARG,
 * SA_ERR_CUDA. */
sa_status sa_cache_create(int k, int d, int64_t capacity, double ttl_seconds, sa_cache* out);

/* Waits for the cache's device, then releases the cache and its device
 * memory (any device may be current; it is current again on return).  NULL
 * is a no-op. */
void sa_cache_free(sa_cache c);

/*
 * sa_cache_lookup -- for each of `batch` keys (host array): hit[b] (host
 * out) = 1 if a fresh entry exists, else 0; for each hit a kernel on
 * `stream` copies the entry into X_tilde[b] (device, batch x k x d fp32,
 * 16-byte aligned) and mass[b] (device, batch x k fp32).  Rows of misses
 * are left as they were.  The decisions are taken on the host before the
 * call returns; the copies complete with the stream.
 */
sa_status sa_cache_lookup(sa_cache c, const sa_cache_key* keys, int64_t batch, double now,
                          uint8_t* hit, float* X_tilde, float* mass, void* stream);

/*
 * sa_cache_insert -- stores X_tilde[b], mass[b] (device, layout as for
 * lookup) under keys[b] (host) at time `now`, evicting as described above.
 * The copies are kernels on `stream`; the sources must stay unchanged until
 * they complete.
 */
sa_status sa_cache_insert(sa_cache c, const sa_cache_key* keys, int64_t batch, double now,
                          const float* X_tilde, const float* mass, void* stream);

/* Host-side counters: entries held, hits, misses (expired ones included),
 * evictions.  Any pointer may be NULL. */
sa_status sa_cache_stats(sa_cache c, int64_t* entries, int64_t* hits, int64_t* misses,
                         int64_t* evictions);

/*
 * sa_cache_forward -- one SA layer served through the cache: look the keys
 * up and copy the hits to the outputs; each run of consecutive missed users
 * (whose rows and outputs are contiguous) is compressed in place by one
 * sa_sketch_forward over its range of X, and its sketches are inserted.
 *
 *   c, q           a cache and a prepared query of the same k and d
 *   keys           host, batch keys
 *   offsets_host   host, batch + 1 int64 (validated on the host): the same
 *                  ragged layout as sa_sketch_forward's device offsets
 *   X              device, total_rows x d, q's dtype, 16-byte aligned
 *   X_tilde, mass  device outputs as for sa_sketch_forward
 *   hit            host out, batch bytes: 1 where the cache served the user
 *   workspace      device, >= sa_cache_forward_workspace_bytes(q, batch,
 *                  total_rows), 256-byte aligned; the SA pass's device
 *                  flags are read with sa_read_device_status on it, as for
 *                  sa_sketch_forward
 *
 * Returns once the host work is done and everything is enqueued on `stream`.
 */
size_t sa_cache_forward_workspace_bytes(sa_query q, int64_t batch, int64_t total_rows);
sa_status sa_cache_forward(sa_cache c, sa_query q, const sa_cache_key* keys, double now,
                           const void* X, const int64_t* offsets_host, int64_t batch,
                           int64_t total_rows, float* X_tilde, float* mass, uint8_t* hit,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * Width adapter (section 2.3): Y = X~ W_A with W_A in R^{d x D} and no bias,
 * mapping every sketch row to the ranking model's width (D = 1024 in the
 * final configuration).  The adapted sketch is shared by a request's targets
 * but not cached (section 2.4).  One tcgen05 kernel: X~ rounded to bf16,
 * W_A held as bf16, fp32 accumulation, Y written as bf16.
 */
typedef struct sa_adapter_s* sa_adapter;

/* W_A: device, d x D fp32 (4-byte aligned); d 64 or 128; D a positive
 * multiple of 256.  A kernel on `stream` makes the bf16 copy; W_A may be
 * freed once the stream has passed this call.  Errors: SA_ERR_INVALID_ARG,
 * SA_ERR_UNSUPPORTED (not sm_100), SA_ERR_CUDA. */
sa_status sa_prepare_adapter(const float* W_A, int d, int D, void* stream, sa_adapter* out);

/* Releases an adapter.  NULL is a no-op. */
void sa_adapter_free(sa_adapter a);

/*
 * sa_adapter_forward -- Y (device out, rows x D bf16, 16-byte aligned) =
 * X_tilde (device, rows x d fp32, 16-byte aligned) W_A, for rows = batch * k
 * sketch rows.  device_flags (device uint32, or NULL): SA_DEVFLAG_TIMEOUT or
 * SA_DEVFLAG_SMEM_ALIGN is OR-ed in if the kernel gave up.
 */
sa_status sa_adapter_forward(sa_adapter a, const float* X_tilde, int64_t rows, void* out,
                             uint32_t* device_flags, void* stream);

/*
 * Action-side fusion (section 2.2 "Stacked Refinement 与动作侧融合" of the
 * same notes): the producer of the history matrix X.  For behaviour i with
 * item embedding e_i (d wide) and action type id t_i:
 *
 *     x_i = e_i + (SiLU(z_i W1) * (z_i W3)) W2,   z_i = [e_i ; table[t_i]],
 *
 * W1, W3 (d + d_a) x h with the e-rows first, W2 h x d, no biases, the
 * action table n_types x d_a.  The page gives the abstract form (a SwiGLU
 * network over the concatenation, residual on e_i) and no more; this is
 * the reading built.  The library folds table W1[d:] and table W3[d:] into
 * per-type rows at prepare time, so the producer's products have K = d.
 */
typedef struct sa_action_s* sa_action;

/*
 * sa_prepare_action -- the producer's parameters.
 *
 *   W1, W3        device, (d + d_a) x h fp32, row-major, 4-byte aligned
 *   W2            device, h x d fp32
 *   action_table  device, n_types x d_a fp32
 *   d             64 or 128
 *   d_a           1 <= d_a <= 4096
 *   h             a multiple of 64, 64 <= h <= 4096
 *   n_types       1 <= n_types <= 16
 *   stream        the bf16 copies and the per-type rows are made by a kernel
 *                 on it; the inputs may be freed once the stream has passed
 *                 this call
 *
 * Errors: SA_ERR_INVALID_ARG, SA_ERR_UNSUPPORTED (not sm_100), SA_ERR_CUDA.
 */
sa_status sa_prepare_action(const float* W1, const float* W3, const float* W2,
                            const float* action_table, int d, int d_a, int h, int n_types,
                            void* stream, sa_action* out);

/* Waits for the producer's device, then releases the producer (any device
 * may be current; it is current again on return).  NULL is a no-op. */
void sa_action_free(sa_action act);

/*
 * sa_action_fuse -- X = the fused rows for `rows` behaviours (one tcgen05
 * kernel; bf16 products with fp32 accumulation, the gate in fp32, X rounded
 * to bf16).
 *
 *   E             device, rows x d bf16, 16-byte aligned: item embeddings
 *   types         device, rows uint8: action type ids; an id >= n_types
 *                 contributes no action term and raises SA_DEVFLAG_ACTION_TYPE
 *   rows          0 <= rows < 2^31 - 256
 *   X             device out, rows x d bf16, 16-byte aligned; must not
 *                 overlap E
 *   device_flags  device uint32 (or NULL): SA_DEVFLAG_* bits OR-ed in
 */
sa_status sa_action_fuse(sa_action act, const void* E, const uint8_t* types, int64_t rows, void* X,
                         uint32_t* device_flags, void* stream);

/*
 * sa_action_sketch_forward -- the producer followed by one SA layer over its
 * output: X is written to the workspace and compressed by sa_sketch_forward
 * (q bf16, the same d as act).  offsets, batch, total_rows, X_tilde, mass
 * as for sa_sketch_forward; workspace >=
 * sa_workspace_bytes_action_sketch(q, batch, total_rows), 256-byte aligned.
 * Device flags of both kernels are read with sa_read_device_status on the
 * workspace.
 */
size_t sa_workspace_bytes_action_sketch(sa_query q, int64_t batch, int64_t total_rows);
sa_status sa_action_sketch_forward(sa_action act, sa_query q, const void* E, const uint8_t* types,
                                   const int64_t* offsets, int64_t batch, int64_t total_rows,
                                   float* X_tilde, float* mass, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * Linear attention with a decay per head, over a ragged batch of histories:
 * the causal companion of the sketch.  Per user and head, with rows in
 * order and S_0 the initial state (zeros when none is given):
 *
 *     S_t = exp(log_decay_h) S_{t-1} + k_t v_t^T      d_k x d_v state
 *     o_t = scale S_t^T q_t                           row t counts itself
 *
 * so a history of any length is read once and leaves a state of fixed size,
 * which sa_linear_attention_step advances by one behaviour.
 *
 * Element type of q, k, v, out and their gradients: dtype.  SA_BF16: bf16
 * products with fp32 accumulation on the tensor cores; the weights of a
 * tile (q . k times the decay) and the copy of the state that outputs are
 * taken from are rounded to bf16, and the state itself is kept in fp32, its
 * sums formed from operands split into two bf16 parts (three where a final
 * state or a d_initial_state is asked for).  SA_FP32: fp32 arithmetic on the
 * CUDA cores.  A value that is not finite reaches only the rows that the
 * formula lets see it (and the state).
 *
 * Common arguments
 *   q, k, v     device; row t, head h of q starts at q + t * q_row + h *
 *               q_head elements (d_k of them, adjacent), likewise k, and v
 *               (d_v of them): slices of a fused projection need no copy.
 *               Any alignment of the element type; addresses and strides
 *               that are multiples of 16 bytes take the tensor-core path
 *   log_decay   device, heads fp32, each <= 0 (0: no decay; -inf: a row
 *               sees itself only).  A positive or NaN entry raises
 *               SA_DEVFLAG_DECAY and counts as 0 or as -inf
 *   offsets     device, int64, batch + 1 entries: offsets[0] == 0,
 *               non-decreasing, offsets[batch] <= total_rows.  Rows behind
 *               offsets[batch] belong to nobody: what they hold does not
 *               matter, and their output rows are left as they were
 *   batch       0 <= batch < 2^21; with 0 nothing is launched, and the
 *               workspace's flags stay as they were
 *   total_rows  0 <= total_rows < 2^31 - 256
 *   max_rows    the longest history, if known, else 0: batches with few and
 *               long histories are split along the rows, and a bound saves
 *               splitting.  A history longer than the bound is still exact
 *   heads       1 <= heads <= 1024
 *   d_k, d_v    64 or 128 each
 *   scale       finite, 1e-20 <= |scale| <= 1e20
 *   workspace   device, 256-byte aligned, at least
 *               sa_workspace_bytes_linear_attention(...) bytes of the same
 *               sizes; one call at a time.  Device flags are read with
 *               sa_read_device_status on it
 *
 * Results are bitwise reproducible for the same inputs on the same GPU
 * model.  Errors: SA_ERR_INVALID_ARG, SA_ERR_UNSUPPORTED (not sm_100),
 * SA_ERR_WORKSPACE, SA_ERR_CUDA.
 */
size_t sa_workspace_bytes_linear_attention(int heads, int d_k, int d_v, int64_t batch,
                                           int64_t total_rows, int64_t max_rows);

/*
 * sa_linear_attention_forward
 *   initial_state  device, batch x heads x d_k x d_v fp32, or NULL: zeros
 *   out            device out, total_rows x heads x d_v, dense; must not
 *                  overlap the inputs
 *   final_state    device out, batch x heads x d_k x d_v fp32, or NULL;
 *                  may be initial_state.  A user without rows keeps its
 *                  initial state
 * States and out are 16-byte aligned.
 */
sa_status sa_linear_attention_forward(const void* q, int64_t q_row, int64_t q_head, const void* k,
                                      int64_t k_row, int64_t k_head, const void* v, int64_t v_row,
                                      int64_t v_head, const float* log_decay,
                                      const int64_t* offsets, int64_t batch, int64_t total_rows,
                                      int64_t max_rows, int heads, int d_k, int d_v,
                                      sa_dtype dtype, float scale, const float* initial_state,
                                      void* out, float* final_state, void* workspace,
                                      size_t workspace_bytes, void* stream);

/*
 * sa_linear_attention_backward -- the gradients of q, k, v and the initial
 * state for d_out = dL/d out and d_final_state = dL/d final_state.  The
 * decay is a constant of the model and gets none.
 *   d_out            device, strided as q with d_v elements per head
 *   d_final_state    device, batch x heads x d_k x d_v fp32, or NULL: zeros
 *   dq, dk, dv       device out, dense, total_rows x heads x d_k (d_k, d_v)
 *   d_initial_state  device out, batch x heads x d_k x d_v fp32, or NULL
 * The outputs must not overlap the inputs or one another.
 */
sa_status sa_linear_attention_backward(const void* q, int64_t q_row, int64_t q_head, const void* k,
                                       int64_t k_row, int64_t k_head, const void* v, int64_t v_row,
                                       int64_t v_head, const float* log_decay,
                                       const int64_t* offsets, int64_t batch, int64_t total_rows,
                                       int64_t max_rows, int heads, int d_k, int d_v,
                                       sa_dtype dtype, float scale, const float* initial_state,
                                       const void* d_out, int64_t d_out_row, int64_t d_out_head,
                                       const float* d_final_state, void* dq, void* dk, void* dv,
                                       float* d_initial_state, void* workspace,
                                       size_t workspace_bytes, void* stream);

/*
 * sa_linear_attention_step -- one row for each of `batch` stored states,
 * which are updated in place (fp32 arithmetic):
 *   S <- exp(log_decay_h) S + k v^T;  out = scale S^T q
 *   q, k, v       device, strided as above with the batch entry as the row
 *   slots         device, batch int64, or NULL (entry b uses state b).  A
 *                 negative slot marks a padded entry: no state is touched
 *                 and its output is zero.  A slot >= states, and a slot that
 *                 an earlier entry of the call has, raise SA_DEVFLAG_SLOT
 *                 and are treated the same way.  Slots are compared in pairs:
 *                 time that grows with the square of the batch, a tenth of
 *                 the call at 10000 entries of 8 heads of 64 x 64
 *   states        states in the pool; >= batch without slots
 *   d_k           1 to 256;  d_v a multiple of 4, 4 to 256
 *   state         device, states x heads x d_k x d_v fp32, 16-byte aligned
 *   out           device out, batch x heads x d_v, dense
 *   device_flags  device uint32 (or NULL): SA_DEVFLAG_DECAY and
 *                 SA_DEVFLAG_SLOT are OR-ed in
 */
sa_status sa_linear_attention_step(const void* q, int64_t q_row, int64_t q_head, const void* k,
                                   int64_t k_row, int64_t k_head, const void* v, int64_t v_row,
                                   int64_t v_head, const float* log_decay, const int64_t* slots,
                                   int64_t batch, int64_t states, int heads, int d_k, int d_v,
                                   sa_dtype dtype, float scale, float* state, void* out,
                                   uint32_t* device_flags, void* stream);

/*
 * The norms before and after a block, fused with its gate and residual
 * scale.  Per row of `d` columns:
 *
 *     n = norm(block; post_gain, post_bias)     n = block without post_gain
 *     r = residual + res_scale * act(gate) * n  residual_out
 *     u = norm(r; pre_gain, pre_bias)           normed: the next block's input
 *
 * norm(x; g, b) = g (x - mean) / sqrt(var + eps) + b in the layer form
 * (biased variance, as sa_refine_update), g x / sqrt(mean(x^2) + eps) + b in
 * the root-mean-square form.  Arithmetic is fp32; each output is rounded
 * once, and u is taken from the unrounded r.
 */
typedef enum sa_norm_kind { SA_NORM_LAYER = 0, SA_NORM_RMS = 1 } sa_norm_kind;
typedef enum sa_gate_kind {
  SA_GATE_IDENTITY = 0, /* act(z) = z */
  SA_GATE_SIGMOID = 1,  /* act(z) = 1 / (1 + exp(-z)) */
  SA_GATE_SILU = 2      /* act(z) = z / (1 + exp(-z)) */
} sa_gate_kind;

/*
 * sa_block_norm_forward
 *   residual      device, rows of residual_dtype, ld_residual elements apart
 *   block         device, rows of dtype, ld_block apart, or NULL: r =
 *                 residual, only u is computed (the first block's norm)
 *   gate          device, rows of dtype, ld_gate apart, or NULL: act = 1
 *   post_gain, post_bias, res_scale, pre_gain, pre_bias
 *                 device, d fp32 each, or NULL: no norm after the block, no
 *                 bias, scale 1, no norm before the next block (then normed
 *                 is NULL), no bias.  A bias needs its gain; gate, post_gain
 *                 and res_scale need a block
 *   rows          0 <= rows < 2^40;  d  1 to 8192;  every ld >= d
 *   residual_dtype, dtype   SA_BF16 or SA_FP32; bf16 residuals need dtype
 *                 SA_BF16
 *   eps           positive
 *   residual_out  device out, rows x d of residual_dtype, dense; NULL if and
 *                 only if block is; may be residual where that is dense
 *   normed        device out, rows x d of dtype, dense, NULL if and only if
 *                 pre_gain is
 * Rows whose addresses and widths are multiples of 16 bytes run fastest; any
 * others are taken element by element.
 */
sa_status sa_block_norm_forward(const void* residual, int64_t ld_residual, const void* block,
                                int64_t ld_block, const void* gate, int64_t ld_gate,
                                const float* post_gain, const float* post_bias,
                                const float* res_scale, const float* pre_gain,
                                const float* pre_bias, int64_t rows, int d,
                                sa_dtype residual_dtype, sa_dtype dtype, sa_norm_kind kind,
                                sa_gate_kind gate_kind, float eps, void* residual_out,
                                void* normed, void* stream);

/*
 * sa_block_norm_backward -- the gradients, at the forward's residual_out.
 * Nothing is saved by the forward: the statistics are taken again.
 *   residual_out        the forward's output r (read only with d_normed)
 *   block, gate, gains, scale, kinds, eps   as in the forward
 *   d_residual_out      device, rows of residual_dtype, ld_d_residual apart:
 *                       dL/dr from what else reads r, or NULL: zeros
 *   d_normed            device, rows of dtype, ld_d_normed apart: dL/du;
 *                       NULL if and only if pre_gain is
 *   d_residual          device out, rows x d of residual_dtype, dense; may
 *                       be d_residual_out where that is dense
 *   d_block, d_gate     device out, rows x d of dtype, dense; NULL if and
 *                       only if block (gate) is
 *   d_post_gain, d_post_bias, d_res_scale, d_pre_gain, d_pre_bias
 *                       device out, d fp32, the sums over the rows, each or
 *                       NULL; zeros for rows == 0
 *   workspace           device, 16-byte aligned, at least
 *                       sa_workspace_bytes_block_norm(rows, d) bytes; may be
 *                       NULL when none of those sums is asked for
 * The sums are added in a fixed order: bitwise reproducible.
 */
size_t sa_workspace_bytes_block_norm(int64_t rows, int d);
sa_status sa_block_norm_backward(const void* residual_out, int64_t ld_residual, const void* block,
                                 int64_t ld_block, const void* gate, int64_t ld_gate,
                                 const float* post_gain, const float* post_bias,
                                 const float* res_scale, const float* pre_gain, int64_t rows,
                                 int d, sa_dtype residual_dtype, sa_dtype dtype,
                                 sa_norm_kind kind, sa_gate_kind gate_kind, float eps,
                                 const void* d_residual_out, int64_t ld_d_residual,
                                 const void* d_normed, int64_t ld_d_normed, void* d_residual,
                                 void* d_block, void* d_gate, float* d_post_gain,
                                 float* d_post_bias, float* d_res_scale, float* d_pre_gain,
                                 float* d_pre_bias, void* workspace, size_t workspace_bytes,
                                 void* stream);

/*
 * The global gradient norm over many tensors, and clipping by it:
 *
 *     norm = sqrt(sum of g^2 over all elements of all tensors)
 *     out  = g * min(1, max_norm / (norm + 1e-6))
 *
 *   grads       host array of `tensors` device addresses; tensor i holds
 *               numel[i] (host) adjacent elements of dtypes[i] (host).  The
 *               arrays are read before the call returns and nothing is kept;
 *               a captured call keeps the addresses it was captured with
 *   tensors     0 <= tensors <= 2^20; empty tensors are allowed
 *   norm        device out, one fp32
 *   workspace   device, 8-byte aligned, at least
 *               sa_workspace_bytes_grad_norm(tensors) bytes
 *   out         host array of device addresses (sizes and types of grads),
 *               or NULL: in place.  No written tensor may overlap another
 *               tensor of the call, so a tensor listed twice is refused;
 *               out[i] may be grads[i]
 *   max_norm    finite, >= 0
 *
 * Squares are summed in fp64 over the whole range of fp32, in a fixed order
 * (bitwise reproducible).  If *norm is not finite, also because finite values
 * have a norm beyond fp32, the values are left (copied) as they are.
 */
size_t sa_workspace_bytes_grad_norm(int64_t tensors);
sa_status sa_grad_norm(const void* const* grads, const int64_t* numel, const sa_dtype* dtypes,
                       int64_t tensors, float* norm, void* workspace, size_t workspace_bytes,
                       void* stream);
sa_status sa_clip_grad_norm(void* const* grads, void* const* out, const int64_t* numel,
                            const sa_dtype* dtypes, int64_t tensors, float max_norm, float* norm,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Static description of a status code. */
const char* sa_status_string(sa_status s);

/* Shape of a prepared query: k, d, dtype, and the padded prototype count
 * the tensor-core pass uses (0 for fp32). */
sa_status sa_query_info(sa_query q, int* k, int* d, int* dtype, int* k_pad);

#ifdef __cplusplus
}
#endif

#endif /* SA_H_ */
