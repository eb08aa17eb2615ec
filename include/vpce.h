/*
 * vpce.h -- vocab-parallel cross-entropy on one GB300 (sm_103a).
 *
 * The operation ("Distributed Training III: Model Parallelism", CMU 11-868
 * Lecture 16 notes, §5.5 "Embedding and output layer"; "LLM Internals" §7.3
 * "Model and tensor parallelism", §7.3.4): the LM-head logits z[s, V] are split
 * along the vocabulary into t shards.  Each shard reduces, per row, its
 * maximum, its sum of exponentials and -- if the row's target column falls in
 * the shard's [vocab_start, vocab_end) -- the target logit.  The partials
 * combine into logsumexp(z_r) and the loss CE_r = logsumexp(z_r) - z_r[y_r]
 * without ever gathering the full rows.  Here all t shards live on one GPU and
 * the combine runs on the device, in a fixed order.
 *
 * The backward (not given by the pages; the standard derivative of the reduced
 * loss) overwrites the shards in place with
 *     dlogits_rk = g * (softmax(z_r)_k - [k == y_r]) / n_valid    (mean)
 *     dlogits_rk = g * (softmax(z_r)_k - [k == y_r])              (sum)
 *     dlogits_rk = g_r * (softmax(z_r)_k - [k == y_r])            (none)
 * and with zeros on rows whose target is ignore_index.  'none' is the
 * per-row mode of torch.nn.functional.cross_entropy, the routine the CMU notes
 * check the sharded loss against: one loss per row, and one upstream gradient
 * g_r per row (the *_rows entry points take them as a device vector).
 *
 * Conventions for every entry point
 * ---------------------------------
 * - All calls are asynchronous and ordered on `stream` (a cudaStream_t; NULL
 *   is the legacy default stream), except vpce_read_error_flag, which
 *   synchronises the stream.  The current CUDA device must be the one that
 *   owns every device pointer, and it must be a compute-capability 10.3 GPU.
 * - The caller owns every buffer.  The library allocates nothing and keeps no
 *   per-call state; the only thing carried from forward to backward is the
 *   caller's workspace.
 * - Host-detectable argument errors return a non-OK status and launch
 *   nothing.  A launch failure returns VPCE_ERR_CUDA.
 * - Logits layout: shard i is a row-major [s, w_i] array of `dtype` elements
 *   at device address shards[i], w_i = vocab_start[i+1] - vocab_start[i], with
 *   a row stride of `ld` elements (ld = 0: each shard is dense, stride w_i).
 *   A shard may be a column block of one big [s, V] tensor (shards[i] =
 *   base + vocab_start[i], ld = V).  Shard pointers need only element
 *   alignment; rows that are not 16-byte aligned take a scalar path for their
 *   ragged head and tail elements.
 * - Targets: int64[s] on the device, replicated view of the whole batch.  A
 *   target equal to ignore_index drops its row; any other target outside
 *   [0, V) is not trapped: the row's loss, lse and gradient become NaN and the
 *   workspace error flag gets bit 0 (read it with vpce_read_error_flag).
 */
#ifndef VPCE_H
#define VPCE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t (the runtime's opaque stream handle). */
typedef struct CUstream_st* vpce_stream_t;

typedef enum {
  VPCE_OK = 0,
  VPCE_ERR_INVALID_ARG = 1,       /* null pointer, bad t/s/ld/vocab_start/reduction */
  VPCE_ERR_ALIGNMENT = 2,         /* a pointer not aligned to its element / 256 B workspace */
  VPCE_ERR_DTYPE = 3,             /* dtype is not VPCE_FP32 or VPCE_BF16 */
  VPCE_ERR_WORKSPACE = 4,         /* workspace_bytes < vpce_workspace_bytes(t, s) */
  VPCE_ERR_CUDA = 5,              /* a CUDA runtime call or a launch failed */
  VPCE_ERR_UNSUPPORTED_DEVICE = 6 /* current device is not compute capability 10.3 */
} vpce_status;

typedef enum { VPCE_FP32 = 0, VPCE_BF16 = 1 } vpce_dtype;

/* Reduction of the per-row losses, as torch.nn.functional.cross_entropy. */
typedef enum { VPCE_MEAN = 0, VPCE_SUM = 1, VPCE_NONE = 2 } vpce_reduction;

#define VPCE_MAX_SHARDS 64

/* Error-flag bits written to the workspace by the device. */
#define VPCE_FLAG_BAD_TARGET 1    /* some target is neither ignore_index nor in [0, V) */
#define VPCE_FLAG_WAIT_TIMEOUT 2  /* a pipeline wait gave up (never expected) */

/*
 * Bytes of device workspace vpce_forward / vpce_backward need for t shards
 * and s rows (t in [1, VPCE_MAX_SHARDS], s >= 0).  Returns 0 for arguments out
 * of range.  The workspace holds the per-(shard, row) partials (8 B each), the
 * per-row target logit and logsumexp (4 B each), the batch count n_valid, the
 * error flag and the combine's per-block sums.  Caller allocated, 256-byte
 * aligned, no initialisation needed.
 */
size_t vpce_workspace_bytes(int t, int64_t s);

/*
 * Forward: loss of the vocab-sharded logits.  Implements the pages' sharded
 * cross-entropy ("Distributed Training III: Model Parallelism", CMU 11-868
 * Lecture 16 notes, §5.5 "Embedding and output layer": each card reduces its
 * block to a maximum, a sum of exponentials and, where it holds the target,
 * the target logit; the blocks combine to logsumexp minus the target logit;
 * "LLM Internals" §7.3.4: the same three quantities for the [8192, 128256]
 * head split 16032 columns per card), with the t shards on one GPU and the
 * combine on the device.  A wait that gave up (VPCE_FLAG_WAIT_TIMEOUT) makes
 * every valid row's loss and the reduced loss NaN.
 *   shards       host array of t device pointers (read only here).
 *   dtype        element type of every shard.
 *   t            number of shards, 1..VPCE_MAX_SHARDS.
 *   s            rows (tokens), >= 0.  s = 0 gives loss NaN (mean) or 0 (sum).
 *   vocab_start  host array of t+1 offsets: vocab_start[0] = 0, strictly
 *                increasing, V = vocab_start[t] < 2^31.  Shard i holds global
 *                columns [vocab_start[i], vocab_start[i+1]); widths may differ
 *                (a V not divisible by t needs no padding).
 *   ld           row stride in elements shared by all shards, >= every
 *                width; 0 means each shard is dense.
 *   targets      device int64[s].
 *   ignore_index target value that drops a row (torch default -100).
 *   reduction    VPCE_MEAN: sum of valid-row losses / n_valid (NaN when
 *                n_valid = 0); VPCE_SUM: the plain sum; VPCE_NONE: the
 *                per-row losses are the result (row_loss_out required).
 *   loss_out     device float, receives the reduced loss.  With VPCE_NONE
 *                it may be NULL; when given it receives the plain sum.
 *   row_loss_out device float[s] or NULL (required for VPCE_NONE when s > 0); receives
 *                CE_r for valid rows, 0 for ignored rows, NaN for
 *                out-of-range targets.
 *   workspace    device buffer of workspace_bytes >= vpce_workspace_bytes.
 * Results are bitwise reproducible for fixed inputs and t: the shards fold
 * in ascending index order and the batch sum runs in a fixed order (a
 * compensated fp32 pair per lane, about 48 bits, added across warps in
 * fp64).
 */
vpce_status vpce_forward(const void* const* shards, vpce_dtype dtype, int t, int64_t s,
                         const int64_t* vocab_start, int64_t ld,
                         const int64_t* targets, int64_t ignore_index,
                         vpce_reduction reduction, float* loss_out, float* row_loss_out,
                         void* workspace, size_t workspace_bytes, vpce_stream_t stream);

/*
 * Backward: overwrite the shards in place with dlogits (same dtype; bf16 is
 * rounded to nearest-even from the fp32 value).  Not on the pages, which
 * give no backward: the standard derivative of the reduced cross-entropy,
 * g * (softmax - onehot) / n_valid for 'mean', computed shard by shard from
 * the forward's logsumexp (the combine of the CMU notes' §5.5 and "LLM
 * Internals" §7.3.4 is what makes softmax available per shard).  Every argument describing the
 * logits and targets must equal the preceding vpce_forward's, the shards must
 * still hold that call's logits, and `workspace` must be that call's,
 * unmodified (it carries logsumexp, n_valid and the reduction).
 * grad_output is the upstream gradient g of the reduced loss (1.0 normally);
 * after a VPCE_NONE forward it is applied to every row, as VPCE_SUM.
 * vocab_start[0] may be > 0 when the shards are one process's part of the
 * vocabulary and the workspace comes from vpce_combine_partials.
 * Padding columns (ld > w_i) are neither read nor written.
 */
vpce_status vpce_backward(void* const* shards, vpce_dtype dtype, int t, int64_t s,
                          const int64_t* vocab_start, int64_t ld,
                          const int64_t* targets, int64_t ignore_index,
                          float grad_output, const void* workspace, size_t workspace_bytes,
                          vpce_stream_t stream);

/*
 * Backward of the per-row losses (reduction 'none'): as vpce_backward, but
 * with one upstream gradient per row, dlogits_rk = grad_rows[r] *
 * (softmax(z_r)_k - [k == y_r]), whatever reduction the forward used.
 *   grad_rows  device float[s] (4-byte aligned), read only; entry r is
 *              d(outer loss)/d(CE_r).  Ignored rows get zeros whatever their
 *              entry; any other entry is used as given (0 gives zeros, a
 *              negative value flips the sign, NaN gives NaN).
 */
vpce_status vpce_backward_rows(void* const* shards, vpce_dtype dtype, int t, int64_t s,
                               const int64_t* vocab_start, int64_t ld,
                               const int64_t* targets, int64_t ignore_index,
                               const float* grad_rows, const void* workspace, size_t workspace_bytes,
                               vpce_stream_t stream);

/*
 * The two halves of vpce_forward, for shards spread over several processes
 * (one GPU each), with the exchange in between done by the caller -- the
 * pages' multi-card method ("Distributed Training III: Model Parallelism",
 * CMU 11-868 Lecture 16 notes, §5.5; "LLM Internals" §7.3.4): each card
 * reduces its columns to per-row partials, the cards exchange them, and every
 * card combines them.
 *
 * vpce_partials: this process's shards (vocab_start: t+1 global column
 * offsets, vocab_start[0] >= 0, the shards' part of the vocabulary) reduced
 * per (shard, row) to part_out[i * s + r] = (max, sum exp(z - max)) (device
 * float2 [t][s]) and tgt_out[r] = the target logit when this process holds
 * the target's column, else 0 (device float [s], cleared here).  workspace
 * as vpce_forward's (vpce_workspace_bytes(t, s)); other arguments as
 * vpce_forward.
 *
 * vpce_combine_partials: n_part partials [n_part][s] (all processes' part_out
 * gathered, in a fixed order) and tgt [s] (the sum over processes of tgt_out,
 * exact since one term per row is non-zero) combined into logsumexp, the row
 * losses and the reduced loss with vpce_forward's per-row arithmetic (folded
 * in index order; the batch sum in fp64 over fixed blocks).  V is the whole vocabulary (the bad-target
 * check).  The workspace is laid out for t_local shards so that
 * vpce_backward on this process's t_local shards (with their global
 * vocab_start) reads its logsumexp and n_valid; its header is cleared here.
 */
vpce_status vpce_partials(const void* const* shards, vpce_dtype dtype, int t, int64_t s,
                          const int64_t* vocab_start, int64_t ld, const int64_t* targets,
                          int64_t ignore_index, float* part_out, float* tgt_out,
                          void* workspace, size_t workspace_bytes, vpce_stream_t stream);
vpce_status vpce_combine_partials(const float* part, int n_part, const float* tgt, int64_t s, int64_t V,
                                  const int64_t* targets, int64_t ignore_index, vpce_reduction reduction,
                                  float* loss_out, float* row_loss_out, int t_local,
                                  void* workspace, size_t workspace_bytes, vpce_stream_t stream);

/*
 * One process's partials folded to one (max, sum exp) pair per row before
 * the exchange, so that each process sends the pages' three scalars per
 * token -- maximum, sum of exponentials and (through the target all-reduce)
 * the target logit -- whatever number of shards it holds ("Distributed
 * Training III: Model Parallelism", CMU 11-868 Lecture 16 notes, §5.5: 12
 * bytes per token instead of the logits).  part: device float2 [t][s] as
 * vpce_partials writes it; out: device float2 [s] (8-byte aligned, may not
 * overlap part), out[r] = (M, S) with M = max_i part[i][r].max and
 * S = sum over i ascending of part[i][r].sum * exp(part[i][r].max - M), the
 * combine's arithmetic.  Folded pairs of all processes, gathered in process
 * order, go to vpce_combine_partials as n_part = (number of processes)
 * partials.  Errors: t outside 1..VPCE_MAX_SHARDS or s < 0
 * (VPCE_ERR_INVALID_ARG), misaligned pointers (VPCE_ERR_ALIGNMENT).
 */
vpce_status vpce_fold_partials(const float* part, int t, int64_t s, float* out, vpce_stream_t stream);

/*
 * Forward and backward in one call: the loss (as vpce_forward) and the shards
 * overwritten in place with dlogits for upstream gradient grad_output (as
 * vpce_backward), for the common case where the loss is the last op and g is
 * known before the forward runs (1.0, or a loss scale).  Each row's backward
 * follows its forward while the row is still in L2 (a CTA's stats warps
 * stream a row in, its grad warps re-read it from L2 about a row later), so
 * the logits cross HBM about once in each direction instead of three passes.  Arguments
 * as vpce_forward plus grad_output; the workspace afterwards holds logsumexp
 * and n_valid like a forward's.  Rows that are not 16-byte aligned (shard
 * pointer, row stride or width in bytes) run the two-call path instead, with
 * the same results.  The batch loss is summed in a fixed order (compensated
 * fp32 pairs, fp64 across warps), so results are bitwise reproducible; they
 * agree with the two-call path within rounding.
 */
vpce_status vpce_forward_backward(void* const* shards, vpce_dtype dtype, int t, int64_t s,
                                  const int64_t* vocab_start, int64_t ld,
                                  const int64_t* targets, int64_t ignore_index,
                                  vpce_reduction reduction, float grad_output,
                                  float* loss_out, float* row_loss_out,
                                  void* workspace, size_t workspace_bytes, vpce_stream_t stream);

/*
 * vpce_forward_backward with one upstream gradient per row (known before the
 * call, e.g. per-token loss weights): the loss as vpce_forward with
 * `reduction`, and dlogits as vpce_backward_rows with grad_rows (device
 * float[s], 4-byte aligned).  Same single pass over HBM and same fallback.
 */
vpce_status vpce_forward_backward_rows(void* const* shards, vpce_dtype dtype, int t, int64_t s,
                                       const int64_t* vocab_start, int64_t ld,
                                       const int64_t* targets, int64_t ignore_index,
                                       vpce_reduction reduction, const float* grad_rows,
                                       float* loss_out, float* row_loss_out,
                                       void* workspace, size_t workspace_bytes, vpce_stream_t stream);

/*
 * How vpce_forward_backward would run the given problem on the current
 * device (no launch): *kernel = 0 two-call path (a shard's width in bytes is
 * not a multiple of 16; misaligned pointers or strides also take it),
 * 1 fused streaming kernel on a persistent grid of *grid CTAs, one per SM.
 * *cluster is 1, or 2 when rows are longer than 224 KB: a pair of CTAs then
 * shares each row, so that the rows kept live between the two passes still
 * fit in L2 with room for the statistics pass to run ahead.
 */
vpce_status vpce_fused_plan(vpce_dtype dtype, int t, const int64_t* vocab_start, int64_t s,
                            int* kernel, int* cluster, int* grid);

/*
 * Forward without a workspace argument, for callers that cannot allocate
 * device memory where they need the loss: a plugin inside a framework whose
 * pooling allocator already owns the GPU's memory (a raw cudaMalloc would fail
 * or fragment that pool), a path that cannot afford cudaMalloc's implicit
 * device synchronisation, or a deployment that forbids device allocation
 * after start-up.  The pages have no counterpart: this is a packaging
 * variant of vpce_forward, with identical arguments and results except that
 * the scratch is a file-scope device array of VPCE_STATIC_SCRATCH_BYTES held
 * by every GPU that loads this library until the process exits.  The caller
 * still passes the logits, targets and outputs.
 *   - Calls the library makes: no cudaMalloc, cudaFree or other allocating
 *     routine; the first call on each device looks the array's address up
 *     (cudaGetSymbolAddress, with that device current), so make that first
 *     call before any stream capture.
 *   - Limit: returns VPCE_ERR_WORKSPACE, launching nothing, when
 *     vpce_workspace_bytes(t, s) > VPCE_STATIC_SCRATCH_BYTES (8 MiB covers,
 *     e.g., t = 16 at s = 32768, t = 8 at s = 65536 and t = 64 at s = 8192;
 *     roughly 8 * t * s + 12 * s bytes are needed).
 *   - Every call on a device shares the one array and the next call overwrites
 *     it (each call clears what must start at zero), so calls that may
 *     overlap on the GPU -- on different streams, or from different threads --
 *     race: serialise them on one stream.  The workspace stays inside the
 *     library, so no vpce_backward can follow this forward, and its error
 *     flag cannot be read: a bad target gives that row, and a wait that gave
 *     up gives every row, a NaN loss, so a NaN loss_out is the signal.
 *   - The array's address is cached per device after the first call, so a
 *     device reset (cudaDeviceReset) after that call is not supported.
 */
#define VPCE_STATIC_SCRATCH_BYTES (8u * 1024u * 1024u)
vpce_status vpce_forward_static(const void* const* shards, vpce_dtype dtype, int t, int64_t s,
                                const int64_t* vocab_start, int64_t ld,
                                const int64_t* targets, int64_t ignore_index,
                                vpce_reduction reduction, float* loss_out, float* row_loss_out,
                                vpce_stream_t stream);

/*
 * LM-head GEMM fused with the forward loss: the logits of shard i are
 * z_i = X W_i^T, computed tile by tile on the tensor cores (bf16 in, fp32
 * accumulate) and reduced in the tile's epilogue to the per-row maximum, sum
 * of exponentials and target logit, so the [s, V] logits are never written
 * ("Distributed Training III: Model Parallelism", CMU 11-868 Lecture 16
 * notes, §5.5: do not assemble the big tensor, move the later computation to
 * the data; "LLM Internals" §7.3.4: the LM head [128256, 8192] split by
 * vocabulary, 16032 rows per card at t = 8).  The combine and the batch sum
 * are vpce_forward's, so loss_out, row_loss_out, the reduction and the
 * workspace's logsumexp / n_valid / error flag mean the same.
 *   hidden         device bf16 [s, h], row stride ld_hidden elements (0 = h);
 *                  16-byte aligned base, ld_hidden * 2 a multiple of 16.
 *   weight_shards  host array of t device pointers; shard i is bf16
 *                  [w_i, h] (one row per vocabulary entry, K contiguous),
 *                  row stride ld_weight elements (0 = h); 16-byte aligned,
 *                  ld_weight * 2 a multiple of 16.
 *   t              1..32 shards; vocab_start as vpce_forward (t+1 offsets).
 *   h              hidden size, a positive multiple of 64.
 *   workspace      vpce_lmhead_workspace_bytes(s) bytes, 256-byte aligned.
 * Other arguments and errors as vpce_forward.  The backward is
 * vpce_lmhead_backward.
 */
#define VPCE_LMHEAD_MAX_GROUPS 256
size_t vpce_lmhead_workspace_bytes(int64_t s);
vpce_status vpce_lmhead_forward(const void* hidden, int64_t ld_hidden,
                                const void* const* weight_shards, int64_t ld_weight,
                                int t, int64_t s, int64_t h, const int64_t* vocab_start,
                                const int64_t* targets, int64_t ignore_index,
                                vpce_reduction reduction, float* loss_out, float* row_loss_out,
                                void* workspace, size_t workspace_bytes, vpce_stream_t stream);

/*
 * Backward of vpce_lmhead_forward (the pages give none; the standard
 * derivative): with dZ = (softmax(z) - onehot) * g / n_valid ('mean'; g for
 * 'sum'; g_r = grad_rows[r] when grad_rows is given),
 *     grad_hidden         = dZ W              bf16 [s, h], overwritten
 *     grad_weight_shards[i] += dZ_i^T X       fp32 [w_i, h], accumulated
 * The logits are formed again tile by tile on the tensor cores (the forward
 * kept none) and written as bf16 dZ for one chunk of rows at a time into
 * `workspace`; two more tensor-core kernels then form the products (bf16 in,
 * fp32 accumulate): dX with the contraction over all t shards in one
 * accumulator, rounded once to bf16; dW_i added into grad_weight_shards[i]
 * by tile reductions, one add per element per chunk, so the result is the
 * same on every run.  Every argument describing X, the head, the targets and
 * fwd_workspace must be the preceding vpce_lmhead_forward's, unmodified
 * (it carries logsumexp, n_valid and the reduction).
 *   grad_output / grad_rows  as vpce_backward / vpce_backward_rows (grad_rows
 *                   device float[s] or NULL).
 *   grad_hidden     device bf16 [s, h], row stride ld_grad_hidden (0 = h).
 *   grad_weight_shards  host array of t device float pointers, [w_i, h],
 *                   row stride ld_grad_weight (0 = h), 16-byte aligned,
 *                   ld_grad_weight a multiple of 4.
 *   workspace       256-byte aligned; vpce_lmhead_backward_workspace_bytes(V, h)
 *                   bytes give 8192-row chunks (the chunk's bf16 dZ, each
 *                   shard's columns padded to a multiple of 8).  A smaller
 *                   workspace gives smaller chunks, in steps of 128 rows;
 *                   less than 128 rows' worth returns VPCE_ERR_WORKSPACE.
 * Calls launch kernels only (no allocation, no host synchronisation).
 */
size_t vpce_lmhead_backward_workspace_bytes(int64_t V, int64_t h);
vpce_status vpce_lmhead_backward(const void* hidden, int64_t ld_hidden,
                                 const void* const* weight_shards, int64_t ld_weight,
                                 int t, int64_t s, int64_t h, const int64_t* vocab_start,
                                 const int64_t* targets, int64_t ignore_index,
                                 float grad_output, const float* grad_rows,
                                 const void* fwd_workspace, size_t fwd_workspace_bytes,
                                 void* grad_hidden, int64_t ld_grad_hidden,
                                 float* const* grad_weight_shards, int64_t ld_grad_weight,
                                 void* workspace, size_t workspace_bytes, vpce_stream_t stream);

/*
 * vpce_lmhead_forward followed by vpce_lmhead_backward in one call, for a
 * training step whose upstream gradient is known up front (grad_output, or
 * grad_rows per row): loss, dX and dW without forming any logits twice.
 * Per row chunk, the tensor-core kernel writes the loss statistics and keeps
 * the chunk's fp32 logits in the workspace (a chunk is the unit the CMU notes
 * (§5.5) keep resident instead of the whole [s, V] tensor).  A row kernel
 * then forms each row's logsumexp, loss and bf16 dZ from them, and the
 * tensor-core kernels of vpce_lmhead_backward compute dX = dZ W and
 * dW += dZ^T X.
 *   loss_out, row_loss_out, reduction   as vpce_lmhead_forward (the mean
 *                  divides by the batch's n_valid; the loss sum runs over
 *                  fixed 256-row blocks in compensated fp32 pairs, fp64
 *                  across warps).
 *   grad_output, grad_rows, grad_hidden, grad_weight_shards, their strides
 *                  as vpce_lmhead_backward.  VPCE_NONE requires grad_rows.
 *   workspace      256-byte aligned.  With
 *                  vpce_lmhead_forward_backward_workspace_bytes(s, V, h)
 *                  bytes, chunks are min(8192, s rounded up to 128) rows.
 *                  Each chunk holds [R, V] fp32 logits and [R, V] bf16 dZ,
 *                  4.2 GB and 2.1 GB at R = 8192, V = 128256 (rows padded
 *                  per shard).  A smaller workspace gives chunks smaller
 *                  by steps of 128 rows; less than 128 rows' worth returns
 *                  VPCE_ERR_WORKSPACE.  The workspace starts with the loss
 *                  header: vpce_read_error_flag works on it.
 * Other arguments and errors as vpce_lmhead_forward and vpce_lmhead_backward.
 * The results equal those two calls' up to the column grouping of the
 * logsumexp (the same arithmetic on a different split of the columns).
 */
size_t vpce_lmhead_forward_backward_workspace_bytes(int64_t s, int64_t V, int64_t h);
vpce_status vpce_lmhead_forward_backward(const void* hidden, int64_t ld_hidden,
                                         const void* const* weight_shards, int64_t ld_weight,
                                         int t, int64_t s, int64_t h, const int64_t* vocab_start,
                                         const int64_t* targets, int64_t ignore_index,
                                         vpce_reduction reduction, float grad_output,
                                         const float* grad_rows, float* loss_out, float* row_loss_out,
                                         void* grad_hidden, int64_t ld_grad_hidden,
                                         float* const* grad_weight_shards, int64_t ld_grad_weight,
                                         void* workspace, size_t workspace_bytes, vpce_stream_t stream);

/*
 * Vocabulary-parallel input embedding ("Distributed Training III: Model
 * Parallelism", CMU 11-868 Lecture 16 notes, §5.5; "LLM Internals" §7.3.4):
 * the table [V, h] is split by vocabulary into t shards; card i looks up only
 * the ids in its range and writes zeros elsewhere, and an all-reduce sums the
 * cards.  On one GPU the sum has one non-zero term per row, so
 *     out[r] = table_shard_i[ids[r] - vocab_start[i]]  for the shard i holding ids[r],
 *     out[r] = 0                                          for an id outside [0, V).
 *   table_shards  host array of t device pointers, shard i [w_i, h] of dtype,
 *                 row stride ld_table elements (0 = h); element-aligned.
 *   ids           device int64[s].
 *   out           device [s, h] of dtype, row stride ld_out (0 = h).
 *   flag_out      device int or NULL: set to 0, then bit 0
 *                 (VPCE_FLAG_BAD_TARGET) if some id is outside [0, V).
 * Rows whose source and destination are 16-byte aligned (and h * element
 * size a multiple of 16) are copied in 16-byte vectors; others by element.
 */
vpce_status vpce_embedding_forward(const void* const* table_shards, vpce_dtype dtype, int t,
                                   const int64_t* vocab_start, int64_t h, int64_t ld_table,
                                   const int64_t* ids, int64_t s, void* out, int64_t ld_out,
                                   int* flag_out, vpce_stream_t stream);

/*
 * Backward of vpce_embedding_forward (not on the pages; the adjoint of the
 * lookup): adds each output-gradient row into the fp32 gradient-table row of
 * its id, accumulating into what grad_shards already hold:
 *     grad_shard_i[j] += sum over r with ids[r] = vocab_start[i] + j of grad_out[r].
 * Ids outside [0, V) contribute nothing.  Deterministic: the rows of an id
 * with at most 64 rows in a chunk are summed in ascending row order (fp32);
 * an id with more is summed as eight contiguous slices of its rows, each in
 * ascending order, then the slices in order; the sum is then added once.
 * Batches longer than 16384 rows run in 16384-row chunks in order.
 *   grad_out      device [s, h] of grad_dtype, row stride ld_grad (0 = h);
 *                 16-byte aligned, ld_grad * element size a multiple of 16.
 *   grad_shards   host array of t device float pointers, shard i [w_i, h],
 *                 row stride ld_grad_table (0 = h); 16-byte aligned,
 *                 ld_grad_table a multiple of 4.
 *   h             a positive multiple of 4.
 *   workspace     vpce_embedding_backward_workspace_bytes() bytes, 256-byte
 *                 aligned, caller owned.  It starts with the same header as
 *                 the loss workspace: vpce_read_error_flag on it returns
 *                 VPCE_FLAG_WAIT_TIMEOUT if a bounded wait of the kernels gave
 *                 up (the gradient is then incomplete), else 0.
 */
size_t vpce_embedding_backward_workspace_bytes(void);
vpce_status vpce_embedding_backward(const void* grad_out, vpce_dtype grad_dtype, int64_t ld_grad,
                                    const int64_t* ids, int64_t s, float* const* grad_shards, int t,
                                    const int64_t* vocab_start, int64_t h, int64_t ld_grad_table,
                                    void* workspace, size_t workspace_bytes, vpce_stream_t stream);

/*
 * Log probabilities of given tokens, with the entropy and the most likely
 * alternatives of each row, from vocabulary-sharded logits: what a sampler, an
 * evaluation or a policy-gradient step reads off the LM head.  The pages'
 * combine ("Distributed Training III: Model Parallelism", CMU 11-868 Lecture
 * 16 notes, §5.5) carries over: each shard's part of a row reduces to its
 * maximum and its sums, and no full row is gathered.  With x = z / temperature
 * and p = softmax(x) over all V columns,
 *     logp[r]    = ln p_r[y_r]
 *     entropy[r] = -sum_k p_rk ln p_rk
 *     top_ids[r] = the `top` columns of largest logit, largest first; equal
 *                  logits rank by column, lowest first
 *     top_logp[r][j] = ln p_r[top_ids[r][j]].
 * The logits are read once, and the stretches that may hold alternatives
 * again (3 to 5% more bytes at V = 128256); nothing but the outputs is written.
 * Two kinds of rows are read a second time by a single warp, right but slower
 * (s = 8192, V = 128256 bf16, every row such a one, against 0.38 ms):
 *   - rows whose largest logit is 726817 temperature (2^20 ln 2) or more from 0,
 *     as ordinary logits are from temperatures of about 1e-5 down: 6.5 ms;
 *   - with alternatives, rows in which over 128 columns come into question for
 *     them (many equal logits, fewer unmasked ones than `top`): 1.0 ms.
 *   shards .. ld     as vpce_forward (read only).
 *   targets          device int64[s], or NULL when logp_out is NULL.  A target
 *                    equal to ignore_index skips its row: its logits are not
 *                    read, its top ids are -1 and its other outputs 0.  A
 *                    target outside [0, V) gives logp NaN; the row's other
 *                    outputs do not depend on the target.  Without targets
 *                    every row is scored.
 *   temperature      1e-30 .. 1e30.
 *   top              0..VPCE_MAX_TOP alternatives, at most V.
 *   logp_out, entropy_out   device float[s], or NULL.
 *   top_ids_out      device int64[s][top]; required when top > 0, else NULL.
 *   top_logp_out     device float[s][top], or NULL.
 *   stats_out        device float[s][4], 16-byte aligned, or NULL: the row's
 *                    largest logit, ln sum_k exp((z_k - largest) /
 *                    temperature), its entropy and 0, for
 *                    vpce_logprob_backward.
 *   flag_out         device int or NULL: set to 0, then bit 0
 *                    (VPCE_FLAG_BAD_TARGET) if some target is outside [0, V),
 *                    bit 1 (VPCE_FLAG_WAIT_TIMEOUT) if a wait gave up.
 * At least one output is required.  Logits of -inf (masked columns) have
 * probability 0 and add nothing to the entropy; as alternatives they come
 * last, with top_logp -inf.  A row with no finite largest logit (every column
 * -inf, or some +inf or NaN) has no distribution: logp, entropy, top_logp and
 * the statistics past the first are NaN, and the alternatives are ordered by
 * value, NaN first.  Results are bitwise reproducible.
 */
#define VPCE_MAX_TOP 32
vpce_status vpce_logprob_forward(const void* const* shards, vpce_dtype dtype, int t, int64_t s,
                                 const int64_t* vocab_start, int64_t ld, const int64_t* targets,
                                 int64_t ignore_index, float temperature, int top, float* logp_out,
                                 float* entropy_out, int64_t* top_ids_out, float* top_logp_out, float* stats_out,
                                 int* flag_out, vpce_stream_t stream);

/*
 * Gradient of vpce_logprob_forward's outputs with respect to the logits.  With
 * upstream gradients g_l of logp, g_H of entropy and g_j of top_logp,
 *     dz_k = (g_l [k = y] + sum_j g_j [k = top_ids_j]
 *             - p_k (g_l + sum_j g_j + g_H (ln p_k + entropy))) / temperature
 * in the shards' dtype (one rounding from fp32).
 *   shards .. temperature   the forward's (unchanged logits).
 *   stats            the forward's stats_out.
 *   grad_logp        device float[s] or NULL (no such gradient); needs targets.
 *   grad_entropy     device float[s] or NULL.
 *   top, top_ids, grad_top_logp   device int64[s][top] and float[s][top], or
 *                    top = 0.  Entries outside [0, V) are skipped; an id that
 *                    occurs twice counts twice.
 *   grad_shards      host array of t device pointers of the shards' dtype, row
 *                    stride ld_grad elements (0: dense), written in full: rows
 *                    of ignored targets get zeros.  grad_shards[i] may be
 *                    shards[i] (in place, same stride); other overlaps are not
 *                    allowed.  Padding columns are not written.
 * At least one upstream gradient is required.  Columns at -inf have p = 0 and
 * get 0 plus their onehot terms.  A row
 * without a distribution gets NaN, and so does, when grad_logp is given, a row
 * whose target is outside [0, V).
 */
vpce_status vpce_logprob_backward(const void* const* shards, vpce_dtype dtype, int t, int64_t s,
                                  const int64_t* vocab_start, int64_t ld, const int64_t* targets,
                                  int64_t ignore_index, float temperature, const float* stats,
                                  const float* grad_logp, const float* grad_entropy, int top,
                                  const int64_t* top_ids, const float* grad_top_logp, void* const* grad_shards,
                                  int64_t ld_grad, vpce_stream_t stream);

/*
 * Scaled embedding lookup with dropout over a table split by vocabulary
 * (vpce_embedding_forward's table and method):
 *     out[r, c] = scale / (1 - D / 65536) * m(r, c) * table[ids[r], c],
 *     m(r, c)   = 0 where the 16 random bits of (r, c) are < D, else 1,
 *     D         = drop_p * 65536 rounded to the nearest integer, at most 65535,
 * so the expectation is scale * table[ids[r], c] exactly.  The bits come from
 * Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
 * as 1, 2, 3", SC 2011): key = the seed's two 32-bit words, low first; counter
 * = (c / 8, r, offset's low word, offset's high word); the 16 bits of column c
 * are half c % 8 of the block's four words, low halves first.  The mask is
 * never stored: vpce_embedding_dropout_backward forms it again.
 *   table_shards, dtype, t, vocab_start, h, ld_table   as
 *                 vpce_embedding_forward (V, h < 2^31).
 *   s             rows, 0 .. 2^31, and s ceil(h / 1024) < 2^34.
 *   ids           device int64[s].  padding_id gives a zero row, whether it
 *                 lies in [0, V) or not (INT64_MIN: no padding); any other id
 *                 outside [0, V) gives a zero row and the flag.
 *   scale         finite.
 *   drop_p        0 <= drop_p < 1; D = 0 drops nothing and reads no rng.
 *   rng           device int64[2]: seed and offset, any bits; read by the
 *                 kernel, so that a captured graph draws new masks after the
 *                 two words change.  May be NULL when D = 0.
 *   out           device [s, h] of out_dtype, row stride ld_out (0 = h); the
 *                 product is formed in fp32 and rounded once.
 *   flag_out      device int or NULL, as vpce_embedding_forward.
 * A dropped element is 0 whatever the table holds.
 */
vpce_status vpce_embedding_dropout_forward(const void* const* table_shards, vpce_dtype dtype, int t,
                                           const int64_t* vocab_start, int64_t h, int64_t ld_table,
                                           const int64_t* ids, int64_t s, int64_t padding_id, float scale,
                                           float drop_p, const int64_t* rng, void* out, vpce_dtype out_dtype,
                                           int64_t ld_out, int* flag_out, vpce_stream_t stream);

/*
 * Gradient of vpce_embedding_dropout_forward with respect to the table:
 *     grad_table[v, c] (=, or += when accumulate) scale / (1 - D / 65536) *
 *         sum over r with ids[r] = v of m(r, c) * grad_out[r, c],
 * v != padding_id; ids equal to padding_id or outside [0, V) contribute
 * nothing.  Sums are fp32 in an order fixed by the ids, so results are bitwise
 * reproducible.
 *   grad_out      device [s, h] of grad_dtype, row stride ld_grad (0 = h),
 *                 element aligned.
 *   s             rows, 0 .. 2^31 - 4096.
 *   ids, padding_id, scale, drop_p, rng   the forward's (rng's words as the
 *                 forward read them).
 *   grad_shards   host array of t device float pointers, shard i [w_i, h], row
 *                 stride ld_grad_table (0 = h), element aligned.
 *   accumulate    0: every element of the shards is written (zeros for ids
 *                 that do not occur); 1: the sums are added to what they hold,
 *                 and rows of ids that do not occur are left alone.
 *   workspace     vpce_embedding_dropout_backward_workspace_bytes(s, V, h)
 *                 bytes (0 for sizes out of range), 256-byte aligned, caller
 *                 owned, no initialisation needed.
 */
size_t vpce_embedding_dropout_backward_workspace_bytes(int64_t s, int64_t V, int64_t h);
vpce_status vpce_embedding_dropout_backward(const void* grad_out, vpce_dtype grad_dtype, int64_t ld_grad,
                                            const int64_t* ids, int64_t s, int64_t padding_id, float scale,
                                            float drop_p, const int64_t* rng, float* const* grad_shards, int t,
                                            const int64_t* vocab_start, int64_t h, int64_t ld_grad_table,
                                            int accumulate, void* workspace, size_t workspace_bytes,
                                            vpce_stream_t stream);

/*
 * Root-mean-square norm with the residual's addition: what stands in front of
 * the LM head (its `hidden`) and of every product of a transformer.  Per row
 *     r = x + residual            (x alone without a residual),
 *     rstd = 1 / sqrt(mean_c r_c^2 + eps),
 *     out_c = r_c rstd weight_c,
 * all in fp32 from the inputs as they are; r is rounded once where it is
 * stored, and so is out (the norm is the unrounded r's).
 *   x              device [s, h] of dtype, row stride ld_x elements (0 = h).
 *   residual       device [s, h] of residual_dtype, stride ld_residual, or
 *                  NULL.  residual_dtype: dtype, or VPCE_FP32 beside bf16 x.
 *   weight         device [h] of weight_dtype.
 *   eps            finite, >= 0.
 *   s, h           rows 0 .. 2^31, columns 1 .. VPCE_MAX_NORM_COLUMNS.
 *   residual_out   device [s, h] of residual_dtype, stride ld_residual_out: r.
 *                  Required with a residual, NULL without one.
 *   out            device [s, h] of dtype, stride ld_out.
 *   rstd_out       device float[s], or NULL; for vpce_rmsnorm_backward.
 * Every pointer needs only element alignment; rows of whole 16-byte vectors
 * (h a multiple of 8, all addresses and strides multiples of 16 bytes) are
 * read in vectors.  In place: residual_out may be residual, and residual_out
 * or out may be x, where type and stride are the same; no other overlap of an
 * output with another operand is allowed.  Columns past h are not written.
 * The squares' sum is fp32 in a fixed order: rows whose mean square
 * passes fp32's range (|r| about 2^64) give rstd 0, and out 0 (NaN at an
 * infinite r); a NaN makes its row NaN, and so does a row of zeros at eps 0.
 * Squares below fp32's smallest number (|r| under 2^-75) count as 0: a row of
 * them alone has an infinite rstd at eps 0.
 * Results are bitwise reproducible.
 */
#define VPCE_MAX_NORM_COLUMNS 32768
vpce_status vpce_rmsnorm_forward(const void* x, vpce_dtype dtype, int64_t ld_x, const void* residual,
                                 vpce_dtype residual_dtype, int64_t ld_residual, const void* weight,
                                 vpce_dtype weight_dtype, float eps, int64_t s, int64_t h, void* residual_out,
                                 int64_t ld_residual_out, void* out, int64_t ld_out, float* rstd_out,
                                 vpce_stream_t stream);

/*
 * The same norm with its output in 8 bits, for products in 8 bits: per row and
 * group of `group` consecutive columns (the last may be shorter),
 *     scale = max_c |out_c| / 448, at least 2^-126,
 *     q_c = out_c / scale, in fp32, rounded to the nearest e4m3 value,
 * from the unrounded out, so q_c scale is within 2^-4 of out_c (or half of
 * e4m3's smallest step, 2^-10 scale).  A NaN or infinite out makes its group's scale
 * so; its own codes are NaN.
 *   group          0 (one scale per row) or a multiple of 16.
 *   q_out          device bytes [s, h], stride ld_q (0 = h): e4m3 codes.
 *   scale_out      device float [s][ceil(h / group)] ([s] for group 0): a row's
 *                  scales are consecutive, rows follow one another without a gap.
 * Other arguments as vpce_rmsnorm_forward; vector rows also need q_out and
 * ld_q to be multiples of 8.
 */
vpce_status vpce_rmsnorm_quantized_forward(const void* x, vpce_dtype dtype, int64_t ld_x, const void* residual,
                                           vpce_dtype residual_dtype, int64_t ld_residual, const void* weight,
                                           vpce_dtype weight_dtype, float eps, int64_t s, int64_t h, int64_t group,
                                           void* residual_out, int64_t ld_residual_out, void* q_out, int64_t ld_q,
                                           float* scale_out, float* rstd_out, vpce_stream_t stream);

/*
 * Gradient of vpce_rmsnorm_forward with respect to r (so to x and to residual
 * alike) and to the weight.  With n = r rstd and dy = grad_out,
 *     grad_in_c = grad_residual_c + rstd (weight_c dy_c - n_c mean_k(weight_k dy_k n_k)),
 *     grad_weight_c (=, or += when accumulate) sum over rows dy_c n_c,
 * in fp32, rounded once.  r is read as the forward stored it.
 *   grad_out       device [s, h] of grad_dtype, stride ld_grad (0 = h).
 *   x              device [s, h] of x_dtype, stride ld_x: the forward's
 *                  residual_out, or its x where it had no residual.  x_dtype:
 *                  grad_dtype, or VPCE_FP32 beside bf16 grad_out.
 *   rstd           the forward's rstd_out.
 *   grad_residual  device [s, h] of x_dtype, stride ld_grad_residual, or NULL:
 *                  the gradient that reaches r through residual_out.
 *   grad_in        device [s, h] of x_dtype, stride ld_grad_in.  May be
 *                  grad_residual, x or grad_out where type and stride are the
 *                  same (in place); other overlaps are not allowed.
 *   grad_weight    device float[h].
 *   workspace      vpce_rmsnorm_backward_workspace_bytes(s, h) bytes, 256-byte
 *                  aligned, no initialisation needed.
 * The rows' terms of grad_weight are summed in fp32 in an order that s, h, the
 * types, alignments and the GPU's SM count fix: bitwise reproducible.  s = 0
 * writes zeros to grad_weight (or leaves it alone when accumulate).
 */
size_t vpce_rmsnorm_backward_workspace_bytes(int64_t s, int64_t h);
vpce_status vpce_rmsnorm_backward(const void* grad_out, vpce_dtype grad_dtype, int64_t ld_grad, const void* x,
                                  vpce_dtype x_dtype, int64_t ld_x, const void* weight, vpce_dtype weight_dtype,
                                  const float* rstd, const void* grad_residual, int64_t ld_grad_residual,
                                  int64_t s, int64_t h, void* grad_in, int64_t ld_grad_in, float* grad_weight,
                                  int accumulate, void* workspace, size_t workspace_bytes, vpce_stream_t stream);

/*
 * One tensor of an optimizer step: n consecutive elements of each array.
 * Arrays need only element alignment; a tensor is moved in vectors where all of
 * them are on 16 bytes (8-bit states on 8).
 *   param         fp32 or bf16, read and written.
 *   grad          fp32 or bf16, read.
 *   copy          bf16[n], written with the new param rounded, or NULL: the
 *                 weights that the LM head reads beside fp32 masters.
 *   exp_avg, exp_avg_sq   float[n] each; or e4m3 codes, a byte each, with
 *   exp_avg_scale, exp_avg_sq_scale   float[ceil(n / 256)] (NULL in 32 bits).
 *   weight_decay  of this tensor, finite.
 * n = 0 is skipped.
 */
typedef struct {
  void* param;
  const void* grad;
  void* copy;
  void* exp_avg;
  void* exp_avg_sq;
  float* exp_avg_scale;
  float* exp_avg_sq_scale;
  int64_t n;
  float weight_decay;
} vpce_adamw_tensor;

/*
 * Norm of all gradients and the factor that clips it, left on the device:
 *     norm = sqrt(sum of g^2 over every element of every tensor),
 *     scale = min(1, max_norm / norm), and 0 where norm is not finite,
 * so that vpce_adamw_step with grad_scale = scale_out clips, and skips the
 * step of a batch with an infinity or NaN in its gradients.
 *   tensors       host array; only grad and n are looked at.  n < 2^40.
 *   grad_dtype    of every grad.
 *   max_norm      > 0; infinity never clips.
 *   norm_out, scale_out   device float, or NULL (not both).
 *   workspace     vpce_grad_norm_workspace_bytes(n_tensors) bytes, 256-byte
 *                 aligned, no initialisation needed.
 * Squares are summed in fp32 (elements of about 2^64 overflow to an infinite
 * norm, ones below 2^-63 lose their squares' last bits, below 2^-75 all) and
 * joined in fp64, in a fixed order: bitwise reproducible.
 */
size_t vpce_grad_norm_workspace_bytes(int64_t n_tensors);
vpce_status vpce_grad_norm(const vpce_adamw_tensor* tensors, int64_t n_tensors, vpce_dtype grad_dtype,
                           float max_norm, float* norm_out, float* scale_out, void* workspace,
                           size_t workspace_bytes, vpce_stream_t stream);

/*
 * One AdamW step (Loshchilov and Hutter, "Decoupled weight decay
 * regularization", ICLR 2019) of many tensors, in as few launches as the
 * kernels' parameters hold (440 tensors each).  Per element, with g = grad *
 * grad_scale and t = *step, in fp32:
 *     m = beta1 m + (1 - beta1) g,    v = beta2 v + (1 - beta2) g^2,
 *     p = p (1 - lr weight_decay)
 *         - lr / (1 - beta1^t) * m / (sqrt(v / (1 - beta2^t)) + eps).
 * param is rounded to nearest in its own type: a bf16 param without an fp32
 * master loses updates below 2^-9 of it.
 *   param_dtype, grad_dtype   of every param and grad.  copy needs fp32 params.
 *   state_bits    32: exp_avg and exp_avg_sq hold m and v.  8: they hold e4m3
 *                 codes of m and of sqrt(v) in blocks of 256 consecutive
 *                 elements of a tensor, value = code * scale, scale = the
 *                 block's largest magnitude / 448, at least 2^-126; all-zero
 *                 codes and scales are states of 0.  Codes are rounded
 *                 stochastically, since v moves by 1 - beta2 a step and e4m3's
 *                 steps are 6 to 12%: rounding to nearest would never move
 *                 an element's v against its block's.  With u the element's 16
 *                 random bits, a value x between neighbouring codes' values
 *                 lo, hi takes hi where (u + 1/2) / 2^16 < (x - lo) / (hi -
 *                 lo); for sqrt(v) the three are squared, which leaves v's
 *                 expectation as it was.  A v above 0 takes at least the
 *                 smallest code above 0, so that m never meets a v of 0.  m
 *                 and v are formed with every fp32 operation rounded by itself,
 *                 so that the codes are those of a plain evaluation (scale =
 *                 largest magnitude times fl(1 / 448)).  The update itself
 *                 uses the unrounded m and v.  u is half k % 8 (low
 *                 halves first) of the Philox4x32-10 block of
 *                 vpce_embedding_dropout_forward with counter = (k / 8, the
 *                 tensor's position in `tensors`, offset's two words), k the
 *                 element's index.  A NaN or infinity in a block's m or v
 *                 spreads over all of the block's codes of it.
 *   step          device int64[1]: t, from 1 (smaller is taken as 1); read by
 *                 the kernel, so that a captured graph advances with it.
 *   lr, lr_dev    the rate; lr_dev, a device float, replaces lr where not NULL.
 *                 lr finite, >= 0 (lr_dev's value is not checked).
 *   beta1, beta2  0 <= beta < 1.
 *   eps           0, or 2^-126 or more, finite.
 *   grad_scale    device float, or NULL (1).  A value of 0 skips the step:
 *                 nothing is written.  A caller that counts steps should not
 *                 count it (beta^t belongs to the updates that m and v have
 *                 had): on the device, t += grad_scale != 0 before the call.
 *   rng           device int64[2]: seed and offset, for state_bits 8 (else
 *                 NULL is taken too); pass another offset every step, and
 *                 another seed than a dropout's.
 * No two arrays of the list may overlap (two tensors may share a grad).
 * Results are bitwise reproducible.
 */
vpce_status vpce_adamw_step(const vpce_adamw_tensor* tensors, int64_t n_tensors, vpce_dtype param_dtype,
                            vpce_dtype grad_dtype, int state_bits, const int64_t* step, float lr,
                            const float* lr_dev, double beta1, double beta2, float eps, const float* grad_scale,
                            const int64_t* rng, vpce_stream_t stream);

/*
 * Synchronise `stream`, then copy the workspace error flag to *flag (bit 0:
 * bad target seen by the last forward; bit 1: a device wait timed out, in
 * which case the forward's loss is NaN).
 */
vpce_status vpce_read_error_flag(const void* workspace, int* flag, vpce_stream_t stream);

/* Static, human-readable name of a status code. */
const char* vpce_status_string(vpce_status status);

#ifdef __cplusplus
}
#endif

#endif /* VPCE_H */
