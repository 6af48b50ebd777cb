/*
 * embbwd — backward pass of pooled (EmbeddingBag) and unpooled embedding
 * lookups over many tables, with SGD or row-wise Adagrad applied in place to
 * every unique touched row. GB300 (sm_103a) CUDA kernels behind a plain C ABI.
 *
 * The operation (the problem statement of "fbgemm_gpu/codegen/
 * embedding_backward_split_template.cu", host function
 * split_embedding_backward_codegen_{optimizer}_{weighted}_exact_cuda):
 *
 *   For table t and bag b with lookups i in [offsets[t*B+b], offsets[t*B+b+1]):
 *     G_t[indices[i]] += s_i * grad_output[b, D_offsets[t] : D_offsets[t+1]]
 *   with s_i = per_sample_weights[i] (if given) * (1/L under mean pooling),
 *   L the bag's length. Unpooled ("nobag"): G_t[indices[l]] += grad_output[l, :].
 *   Then, once for every unique touched row (t, idx):
 *     SGD:               w <- w - lr * G
 *     row-wise Adagrad:  m <- m + sum_d(G_d^2)/D_t ;  w <- w - lr * G / (sqrt(m) + eps)
 *   ("tt_embeddings_cuda.cu": update_tt_cores_sgd_kernel and
 *    cache_backward_rowwise_adagrad_approx_kernel give the two update rules;
 *    here they act on the de-duplicated row gradient.)
 *   The update is computed in fp32 and rounded once (round-to-nearest-even,
 *   or stochastically with EMB_FLAG_STOCHASTIC_ROUNDING) to the weight's
 *   storage type. Rows that no lookup touches are not written.
 *
 * Also declared here: elementwise Adagrad (emb_bag_bwd_adagrad), the
 * dense-gradient mode (emb_bag_bwd_dense_grad, emb_nobag_bwd_dense_grad), the
 * forward pooled lookup (emb_bag_fwd), an allocation-free unpooled update
 * (emb_nobag_bwd_sgd_atomic_noalloc), and the exchange step of row-sharded
 * tables over several ranks (emb_shard_*), and the vocabulary operators of a
 * language model (emb_logits_process, emb_distill_*, emb_micro_*, emb_rms_norm_*,
 * emb_dropout, emb_cross_entropy_*). emb_shard_bucketize is the one call
 * that synchronises (it returns the exchange's split sizes).
 *
 * Layouts (all element offsets, not bytes):
 *   weights        flat; row idx of table t starts at weights_offsets[t] + idx*D_t
 *   momentum       fp32; row idx of table t at momentum_offsets[t] + idx
 *                  (momentum_offsets NULL => hash_size_cumsum[t] + idx)
 *   indices        int64[N], row ids local to their table
 *   offsets        int64[B*T+1], CSR over bags in table-major order (bag t*B+b)
 *   grad_output    pooled: [B, D_offsets[T]] row-major; unpooled: [N, D]
 *   per_sample_weights  fp32[N] or NULL
 *
 * Ownership: every tensor pointer passed to a call is caller-owned device
 * memory. Host arrays given to emb_bwd_plan are copied. The plan owns all of
 * its scratch (device memory sized from max_N at plan time); calls allocate
 * nothing.
 *
 * Execution: calls enqueue work on `stream` (a cudaStream_t; NULL = legacy
 * default stream) and return without synchronising. Argument errors are
 * returned synchronously. Errors found on the device (an index outside its
 * table, malformed offsets, a bounded wait that ran out) are latched in the
 * plan, leave weights and momentum unmodified, and are returned by the next
 * emb_plan_status(). One plan serves one call at a time: calls on one plan
 * must be ordered (same stream, or synchronised), because they share scratch.
 * A call contains no host synchronisation and no allocation, so it can be
 * captured in a CUDA graph.
 */
#ifndef EMBBWD_H
#define EMBBWD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  EMB_OK = 0,
  EMB_ERR_INVALID_ARG = 1,         /* bad argument, or malformed offsets found on the device */
  EMB_ERR_UNSUPPORTED = 2,         /* valid but not supported by this library (see each call) */
  EMB_ERR_INDEX_OUT_OF_RANGE = 3,  /* an index outside [0, rows of its table) */
  EMB_ERR_OOM = 4,                 /* plan scratch could not be allocated */
  EMB_ERR_CUDA = 5,                /* a CUDA runtime call failed */
  EMB_ERR_TIMEOUT = 6              /* a bounded inter-block wait ran out; nothing was updated */
} emb_status;

typedef enum { EMB_F32 = 0, EMB_F16 = 1, EMB_BF16 = 2 } emb_dtype;
typedef enum { EMB_POOL_SUM = 0, EMB_POOL_MEAN = 1 } emb_pooling;
typedef enum { EMB_NOBAG_AUTO = 0, EMB_NOBAG_SORTED = 1, EMB_NOBAG_ATOMIC = 2 } emb_nobag_path;

/* emb_bwd_plan flags. Index range checking is always on. */
#define EMB_FLAG_CHECK_INDICES 0x1u
/* Launch the kernels of a call as plain stream-ordered launches instead of
 * programmatic dependent launches (for A/B timing; results are identical). */
#define EMB_FLAG_NO_PDL 0x2u
/* Stochastic rounding of fp16 / bf16 weight stores ("embedding_backward_split_
 * template.cu", the stochastic_rounding argument of the per-row kernels and
 * their Philox-seeded 16-bit stores): an update is rounded to one of its two
 * representable neighbours, away from zero with probability equal to the
 * fraction of an ulp it lies past the one toward zero (unbiased in expectation). Applies to the SGD and Adagrad updates of plans
 * with 16-bit weights (fp32 weights and the dense-gradient mode store as usual).
 * Element d of the row with linear index K, in the update call numbered c, draws
 * word d mod 4 of Philox4x32-10 (Salmon et al., SC 2011) at counter
 * (K, d / 4, c mod 2^32, c / 2^32) under the key (seed mod 2^32, seed / 2^32).
 * bf16: the 16 low bits of the word are added to the fp32 pattern, then it is
 * truncated; fp16: the neighbour away from zero is taken iff (word >> 8) <
 * floor(fraction * 2^24). The call number starts at 0; each SGD or Adagrad
 * call with N > 0 on a plan with 16-bit weights takes the next one;
 * emb_plan_set_rounding sets seed and number.
 * A call captured in a CUDA graph keeps the number it was captured with. */
#define EMB_FLAG_STOCHASTIC_ROUNDING 0x4u
/* Sort with the multi-block front (histogram kernel, radix passes, run-length
 * kernel) even where the small-batch front applies. That front takes calls of
 * at most 2^16 lookups whose tables fit one cluster of CTAs each, all resident
 * at once; a cluster sorts and run-length encodes one table's lookups in
 * shared memory in a single launch. For A/B timing and tests: both fronts
 * give identical results. */
#define EMB_FLAG_NO_CLUSTER_FRONT 0x8u
/* Test only: every block that would wait on another one gives up at once and
 * reports EMB_ERR_TIMEOUT, exercising the error path without a real stall. */
#define EMB_FLAG_DEBUG_FORCE_TIMEOUT 0x100u

typedef struct emb_plan emb_plan;

/* Creates a plan for a fixed set of tables.
 *   device            CUDA device ordinal the plan and all its calls use.
 *   T                 number of tables, 1..4096.
 *   hash_size_cumsum  host int64[T+1]: hash_size_cumsum[t] = rows of tables < t;
 *                     strictly increasing, hash_size_cumsum[0] = 0, total rows < 2^32.
 *                     Row idx of table t has linear index hash_size_cumsum[t] + idx
 *                     ("embedding_backward_split_template.cu", the per-row kernels).
 *   D_offsets         host int32[T+1]: D_t = D_offsets[t+1] - D_offsets[t], each a
 *                     positive multiple of 4 (the pages' vector width) and <= 4096.
 *   weights_offsets   host int64[T], each a multiple of 4.
 *   momentum_offsets  host int64[T] or NULL.
 *   weight_dtype      storage type of weights (fp32, fp16, bf16).
 *   grad_dtype        type of grad_output (fp32, fp16, bf16).
 *   max_N             largest lookup count any call will pass (< 2^30, and
 *                     max_N * ceil(max D_t / 256) < 2^31).
 *   max_B             largest batch any call will pass (max_B * T < 2^31).
 *   max_segment_length_per_warp  runs at least this long take the block-level
 *                     path ("embedding_backward_split_template.cu",
 *                     *_find_long_segments); <= 0 selects 32.
 *   flags             EMB_FLAG_* bits.
 * Returns EMB_ERR_INVALID_ARG for malformed arguments, EMB_ERR_OOM if scratch
 * cannot be allocated, EMB_ERR_CUDA on other runtime failures. *out is NULL on error. */
emb_status emb_bwd_plan(emb_plan** out, int device, int32_t T, const int64_t* hash_size_cumsum,
                        const int32_t* D_offsets, const int64_t* weights_offsets,
                        const int64_t* momentum_offsets, emb_dtype weight_dtype,
                        emb_dtype grad_dtype, int64_t max_N, int32_t max_B,
                        int32_t max_segment_length_per_warp, uint32_t flags);

/* Stochastic rounding state of the plan: `seed` keys the random words and
 * `next_call` is the call number the next update call uses (see
 * EMB_FLAG_STOCHASTIC_ROUNDING). Host-side only; no synchronisation.
 * emb_plan_get_rounding reads both back (either pointer may be NULL). */
emb_status emb_plan_set_rounding(emb_plan* plan, uint64_t seed, uint64_t next_call);
emb_status emb_plan_get_rounding(const emb_plan* plan, uint64_t* seed, uint64_t* next_call);

/* Frees the plan and its scratch (synchronises the device). NULL is accepted. */
emb_status emb_plan_destroy(emb_plan* plan);

/* Pooled backward + SGD, in place on `weights` (plan's weight_dtype).
 * offsets has B*T+1 entries with offsets[0] = 0 and offsets[B*T] = N; B <= max_B,
 * N <= max_N. per_sample_weights may be NULL. N = 0 returns EMB_OK and does nothing
 * ("embedding_backward_split_template.cu": the exact_cuda host function's
 * empty-indices short-circuit and its T > 0, B > 0 checks). */
emb_status emb_bag_bwd_sgd(emb_plan* plan, void* weights, const int64_t* indices,
                           const int64_t* offsets, int64_t N, int32_t B,
                           const float* per_sample_weights, const void* grad_output,
                           emb_pooling mode, float lr, void* stream);

/* Pooled backward + row-wise Adagrad, in place on `weights` and fp32 `momentum`.
 * Same arguments as emb_bag_bwd_sgd plus momentum and eps. Rows of every supported
 * width (D_t <= 4096): when some D_t > 1024 the reduce runs twice on the stream,
 * first finding each row's new state from the sums of squares of its 1024-wide
 * chunks (added in chunk order), then updating the weights. */
emb_status emb_bag_bwd_rowwise_adagrad(emb_plan* plan, void* weights, float* momentum,
                                       const int64_t* indices, const int64_t* offsets,
                                       int64_t N, int32_t B, const float* per_sample_weights,
                                       const void* grad_output, emb_pooling mode, float lr,
                                       float eps, void* stream);

/* Pooled backward + elementwise Adagrad, in place on `weights` and fp32 `momentum`,
 * whose layout is that of the weights (momentum[weights_offsets[t] + idx*D_t + d],
 * 16-byte aligned): for every unique row, with G its de-duplicated gradient,
 *   m_d <- m_d + G_d^2 ;  w_d <- w_d - lr * G_d / (sqrt(m_d) + eps)
 * ("tt_embeddings_cuda.cu", update_tt_cores_adagrad_kernel). Other arguments as
 * for emb_bag_bwd_sgd; rows of any supported width. */
emb_status emb_bag_bwd_adagrad(emb_plan* plan, void* weights, float* momentum,
                               const int64_t* indices, const int64_t* offsets, int64_t N,
                               int32_t B, const float* per_sample_weights,
                               const void* grad_output, emb_pooling mode, float lr, float eps,
                               void* stream);

/* Dense-gradient mode: instead of updating, writes the de-duplicated gradient G of
 * every touched row into `grad_weights`, a buffer of the plan's weight_dtype with
 * the layout of the weights (row idx of table t at grad_weights[weights_offsets[t] +
 * idx*D_t]), after zeroing it over the plan's whole weights extent (the largest
 * weights_offsets[t] + rows_t*D_t), so untouched rows read zero ("embedding_backward_
 * split_template.cu", the dense variant: grad_dev_weights = zeros_like(dev_weights),
 * then grad_sum stored per touched row). G is rounded once to the storage type.
 * Pooled: arguments as for emb_bag_bwd_sgd without lr. Unpooled: as for
 * emb_nobag_bwd_sgd without lr and path (the sorted, deterministic path). */
emb_status emb_bag_bwd_dense_grad(emb_plan* plan, void* grad_weights, const int64_t* indices,
                                  const int64_t* offsets, int64_t N, int32_t B,
                                  const float* per_sample_weights, const void* grad_output,
                                  emb_pooling mode, void* stream);
emb_status emb_nobag_bwd_dense_grad(emb_plan* plan, void* grad_weights, const int64_t* indices,
                                    const int64_t* offsets, int64_t N, int32_t B,
                                    const void* grad_output, void* stream);

/* Unpooled backward + SGD: lookup l adds grad_output[l, :] (shape [N, D], every
 * table has the same D) to row indices[l] of its table, the table given by the
 * CSR offsets (B*T+1 entries; only table membership matters). There is no
 * weighted variant ("embedding_backward_split_template.cu" generates no
 * weighted nobag kernel).
 *   path EMB_NOBAG_SORTED: sort + de-duplicated, deterministic update.
 *   path EMB_NOBAG_ATOMIC: one float atomic add of -lr*g per element, no sort
 *        ("tinygrad/nn/__init__.py", _embedding_bwd_kernel; "tt_embeddings_cuda.cu",
 *        cache_backward_sgd_kernel); fp32 weights only, else EMB_ERR_UNSUPPORTED.
 *   path EMB_NOBAG_AUTO: the faster of the two for the plan's types. */
emb_status emb_nobag_bwd_sgd(emb_plan* plan, void* weights, const int64_t* indices,
                             const int64_t* offsets, int64_t N, int32_t B,
                             const void* grad_output, float lr, emb_nobag_path path,
                             void* stream);

/* Forward pooled lookup (EmbeddingBag forward) over the plan's tables:
 *   output[b, D_offsets[t] + d] = sum over lookups i of bag (t, b) of
 *                                 s_i * weights[weights_offsets[t] + indices[i]*D_t + d],
 *   s_i = per_sample_weights[i] (if not NULL) times 1/L (EMB_POOL_MEAN, L = bag length),
 * the scale the backward applies to the same lookup (the forward is the adjoint
 * of the backward's scatter). "tt_embeddings_cuda.cu", cache_forward_kernel and
 * reduce_output_kernel: a bag's output row is the sum of the rows it indexes.
 *   weights     the plan's weight_dtype, layout as for the backward (read only).
 *   indices, offsets, N, B, per_sample_weights  as for emb_bag_bwd_sgd.
 *   output      [B, D_offsets[T]] of output_dtype (fp32, fp16 or bf16), overwritten
 *               entirely: an empty bag gives zeros; rounded once from fp32 sums.
 * Asynchronous on `stream`; uses no plan scratch, so it may run while no
 * backward call of the plan is in flight on another stream. An index outside its
 * table or malformed offsets latch EMB_ERR_INDEX_OUT_OF_RANGE / EMB_ERR_INVALID_ARG
 * (read with emb_plan_status); the offending lookup or bag is left out. */
emb_status emb_bag_fwd(emb_plan* plan, const void* weights, const int64_t* indices,
                       const int64_t* offsets, int64_t N, int32_t B,
                       const float* per_sample_weights, emb_pooling mode, void* output,
                       emb_dtype output_dtype, void* stream);

/* Allocation-free unpooled atomic SGD (the same update as emb_nobag_bwd_sgd with
 * EMB_NOBAG_ATOMIC), for callers that cannot allocate device memory when they run
 * it: inside a CUDA graph capture, under a runtime that owns all device memory,
 * or where the library must not call the device allocator. The pages have no
 * counterpart of this entry point; it exists for those callers.
 *   No plan is used and nothing is allocated (no cudaMalloc, cudaFree or
 *   allocating library call). Scratch is one fixed static device array in the
 * library image, about 21 KB, present on every GPU that loads the library
 *   until the process exits. Limits: N <= 4194304 lookups, T <= 4096 tables,
 *   B*T < 2^31, D a multiple of 4 and <= 4096; beyond them EMB_ERR_INVALID_ARG.
 *   hash_size_cumsum (int64[T+1]) and weights_offsets (int64[T]) are caller-owned
 *   DEVICE arrays here, checked on the device before any update: hash_size_cumsum
 *   starts at 0, strictly increases and stays below 2^32; every weights_offsets[t]
 *   is >= 0 and a multiple of 4. weights are fp32; grad_output is [N, D] of
 *   grad_dtype. device_status (device uint32, may be NULL) receives this call's
 *   device error bits: 1 = an index outside its table, 2 = malformed offsets,
 *   hash_size_cumsum or weights_offsets; 0 = none. Nothing is updated when a bit
 *   is set.
 *   The first call on a device looks up the scratch array's device address
 *   (cudaGetSymbolAddress); make that first call before any stream capture.
 *   All calls share the scratch array: calls that overlap on the GPU race, so
 *   order them (one stream, or events). Asynchronous on `stream`. */
emb_status emb_nobag_bwd_sgd_atomic_noalloc(int device, int32_t T,
                                            const int64_t* hash_size_cumsum,
                                            const int64_t* weights_offsets, int32_t D,
                                            float* weights, const int64_t* indices,
                                            const int64_t* offsets, int64_t N, int32_t B,
                                            const void* grad_output, emb_dtype grad_dtype,
                                            float lr, uint32_t* device_status, void* stream);

/* Waits for the plan's last call, then returns and clears the latched device
 * error (EMB_OK if none). */
emb_status emb_plan_status(emb_plan* plan);

/* Host copies of the last sorted call's integer outputs, for parity checks:
 * run_keys (ascending unique linear indices), run_len, cum (exclusive scan of
 * run_len, num_runs+1 entries), num_runs, long_ids (runs with run_len >=
 * max_segment_length_per_warp; the order is unspecified, compare as a set) and
 * num_long. Arrays need `capacity` entries (cum: capacity+1); any pointer may be
 * NULL. Synchronises. EMB_ERR_INVALID_ARG if the last call was not a sorted one or
 * a count exceeds capacity. */
emb_status emb_plan_debug_runs(emb_plan* plan, int64_t capacity, int64_t* run_keys,
                               int32_t* run_len, int32_t* cum, int32_t* num_runs,
                               int32_t* long_ids, int32_t* num_long);

/* Profiling: when enabled, calls record CUDA events between their stages. */
emb_status emb_plan_set_profiling(emb_plan* plan, int enable);

/* Stage durations (ms) of the last profiled call; synchronises. Sorted path:
 * [0] linearise + histogram, [1] radix sort passes, [2] run-length encode and
 * long-run partition (one kernel), [3] 0, [4] reduce + optimizer. Atomic path:
 * [0] index check, [4] atomic scatter, others 0. Writes min(n, 5) values. */
emb_status emb_plan_stage_ms(emb_plan* plan, float* ms, int32_t n);

/* ---- Row-wise sharding over W ranks (the exchange step before the backward).
 * Every rank trains on its own batch and owns a contiguous row range of every
 * table: rank r holds rows [row_bounds[t*(W+1)+r], row_bounds[t*(W+1)+r+1]) of
 * table t, the vocabulary sharding of "Function _embedding_bwd_kernel" (tinygrad:
 * a device owns one slice of the rows; lookups outside it add nothing there).
 * A step on rank r:
 *   1. emb_shard_bucketize its batch: per owner, the lookups of its rows;
 *   2. all-to-all the parts (offsets: W*(T*B+1) each way; indices and scales
 *      with the per-owner counts as split sizes) and all-gather grad_output into
 *      [W*B, sum D] in rank order (e.g. NCCL through torch.distributed);
 *   3. emb_shard_merge the received parts into one batch of W*B bags per table;
 *   4. the ordinary backward on the rank's own plan (its local tables: row range
 *      sizes as hash_size_cumsum, rows relative to the range) with B' = W*B, the
 *      merged offsets and indices, the merged scales as per_sample_weights (or
 *      NULL when the batch is unweighted and sum-pooled) and EMB_POOL_SUM.
 * The forward runs 1-3 the same way, then emb_bag_fwd with B' = W*B gives the
 * rank's partial sums of every rank's bags, and a reduce-scatter over ranks
 * gives each rank its own bags' output. */
typedef struct emb_shard emb_shard;

/* Creates the shard map of one rank: T tables (1..4096), W ranks (1..256),
 * row_bounds host int64[T*(W+1)] (row_bounds[t*(W+1)] = 0, non-decreasing, last
 * = rows of table t > 0; empty ranges are allowed here, but a rank whose plan
 * has an empty table cannot create that plan), max_B the largest per-rank batch
 * (W * T * max_B < 2^31). Allocates its scratch on `device` (about
 * 12 * W * T * max_B bytes). */
emb_status emb_shard_create(emb_shard** out, int device, int32_t T, int32_t W,
                            const int64_t* row_bounds, int32_t max_B);

/* The cyclic map: rank r owns rows r, r + W, r + 2W, ... of every table (its
 * local row k is row k*W + r), so a skewed id distribution spreads over all
 * ranks. rows: host int64[T], each > 0. Rows are then relative as row / W in
 * send_indices; a rank's plan has ceil((rows_t - r) / W) rows of table t. */
emb_status emb_shard_create_cyclic(emb_shard** out, int device, int32_t T, int32_t W,
                                   const int64_t* rows, int32_t max_B);
emb_status emb_shard_destroy(emb_shard* shard);

/* Step 1 on `stream`; synchronises it (the exchange needs the sizes on the
 * host). Inputs as for emb_bag_bwd_sgd (device indices [N], offsets [T*B+1],
 * optional per_sample_weights [N], mode). Outputs (device, caller-owned):
 *   send_offsets int64[W][T*B+1]: owner r's bag offsets counted from its first lookup;
 *   send_indices int64[N]: owner 0's lookups first, then owner 1's, ..., each row
 *     relative to the owner's range (cyclic map: row / W), in bag order and
 *     lookup order within a bag;
 *   send_scales float[N] or NULL: per-sample weight (1 if none), divided in fp32
 *     by the length of its whole bag under mean pooling;
 *   send_counts host int64[W]: lookups per owner (the all-to-all split sizes).
 * EMB_ERR_INDEX_OUT_OF_RANGE for an index outside its table, EMB_ERR_INVALID_ARG
 * for malformed offsets; nothing usable is written then. */
emb_status emb_shard_bucketize(emb_shard* shard, const int64_t* indices, const int64_t* offsets,
                               int64_t N, int32_t B, const float* per_sample_weights,
                               emb_pooling mode, int64_t* send_offsets, int64_t* send_indices,
                               float* send_scales, int64_t* send_counts, void* stream);

/* Step 3 on `stream`, asynchronous. recv_offsets device int64[W][T*B+1] (source
 * s's send_offsets for this rank, in source order), recv_indices / recv_scales
 * the n_recv received lookups concatenated in source order (recv_scales may be
 * NULL, then merged_scales must be NULL too). Writes merged_offsets int64[T*W*B+1]
 * and merged_indices / merged_scales [n_recv]: bag s*B + b of table t holds
 * source s's bag (t, b). Received offsets inconsistent with n_recv are skipped
 * and reported by emb_shard_status as EMB_ERR_INVALID_ARG. */
emb_status emb_shard_merge(emb_shard* shard, const int64_t* recv_offsets, const int64_t* recv_indices,
                           const float* recv_scales, int64_t n_recv, int32_t B,
                           int64_t* merged_offsets, int64_t* merged_indices, float* merged_scales,
                           void* stream);

/* Waits for the shard's last call and returns (and clears) its latched errors. */
emb_status emb_shard_status(emb_shard* shard);

/* ---- Vocabulary operators of a language model: its token table is also the matrix
 * of its output logits. They need no plan and no workspace, allocate nothing and
 * never synchronise, so they can be captured in a CUDA graph. `device` is the CUDA
 * device of the pointers and of `stream`. Row strides are in elements and matter
 * where there is more than one row. Argument errors are returned synchronously.
 * device_status (device uint32, may be NULL) collects device error bits: they are
 * added to it (the caller clears it) - 1 = an id outside its range (the entry is
 * left out), 2 = malformed CSR offsets (the list is taken as empty), 4 = a bounded
 * wait ran out (what was not finished of the output is NaN). */

/* Logits before a token is chosen. B requests (<= 65535), V tokens (<= 2^20). For
 * token v of request b, with z its logit and c the times v occurs in the request's
 * output ids:
 *   v in the prompt or output ids:  z <- z > 0 ? z / repetition[b] : z * repetition[b]
 *   v in the output ids:            z <- z - frequency[b] * c - presence[b]
 *   z <- z + the biases of v, in the order of the list
 *   bit v % 32 of mask[b, v / 32] clear:  z <- -infinity
 * in fp32 (the division as a product with the reciprocal), rounded once to out_dtype.
 * prompt/output/bias lists are CSR: ids int64[n], n < 2^31, offsets int64[B+1] with values in
 * 0..n (both NULL and n = 0: no list; a bias list has fp32 bias_values). A request has fewer
 * than 2^30 output ids (a longer list counts as malformed offsets).
 * repetition, frequency, presence: fp32[B], NULL = 1, 0, 0.
 * mask: uint32 [B, mask_stride >= ceil(V / 32)] or NULL. `out` may be `logits` itself
 * (same type and stride), and must not overlap it otherwise. */
emb_status emb_logits_process(int device, const void* logits, emb_dtype logits_dtype,
                              int64_t logits_stride, int32_t B, int32_t V,
                              const int64_t* prompt_ids, const int64_t* prompt_offsets,
                              int64_t prompt_n, const int64_t* output_ids,
                              const int64_t* output_offsets, int64_t output_n,
                              const float* repetition, const float* frequency,
                              const float* presence, const int64_t* bias_ids,
                              const int64_t* bias_offsets, const float* bias_values,
                              int64_t bias_n, const uint32_t* mask, int64_t mask_stride, void* out,
                              emb_dtype out_dtype, int64_t out_stride, uint32_t* device_status,
                              void* stream);

/* Distillation from a teacher's top logits. Row n of the student's logits z [N, V]
 * (N <= 2^23, V <= 2^20), tau = temperature > 0, p = softmax(z / tau), and the teacher's list of
 * K <= 1024 entries (teacher_ids int64, teacher_logits; row stride teacher_stride for
 * both), q_k = exp(t_k / tau - L):
 *   teacher_lse given (fp32[N], L = log of the teacher's whole sum of exp(t / tau)):
 *     r = max(0, 1 - sum q), u = mass of p off the list,
 *     loss = tau^2 * (sum_k q_k (log q_k - log p_{id_k}) + r (log r - log u))
 *   teacher_lse NULL: L = log sum_k exp(t_k / tau) and r = 0.
 *   d loss / d z_v = tau * (p_v - q of the entries with id v)   on the list,
 *                    tau * p_v * (1 - r / u)                    off it.
 * Entries with id -1 are padding. Rows without entries, and rows with L = -infinity (a
 * teacher without mass), have loss 0 and gradient 0. Entries that repeat an id add. Where no
 * logit off the list is finite (u = 0), an r within rounding of 0 counts as 0; a larger one
 * makes the loss infinite, and the gradient off the list is 0.
 *   emb_distill_forward   loss fp32[N]; stats fp32[N, 4], 16-byte aligned: {largest z,
 *                         sum of exp((z - largest) / tau), 1 - r / u, L}; for r / u above
 *                         2^64 its binary logarithm stands in place of 1 - r / u
 *   emb_distill_backward  dlogits (logits_dtype) = row_weight[n] * dloss/dz from the
 *                         forward's stats; row_weight fp32[N] or NULL = 1
 *   emb_distill_step      loss and dlogits in one call, for a row_weight known
 *                         beforehand; z is read twice, the second time from L2 while
 *                         the rows under way fit it (16-bit rows of 128256 do)
 * dlogits may be logits itself (same stride) and must not overlap it otherwise. */
emb_status emb_distill_forward(int device, const void* logits, emb_dtype logits_dtype,
                               int64_t logits_stride, int32_t N, int32_t V,
                               const int64_t* teacher_ids, const void* teacher_logits,
                               emb_dtype teacher_dtype, int64_t teacher_stride, int32_t K,
                               const float* teacher_lse, float temperature, float* loss,
                               float* stats, uint32_t* device_status, void* stream);
emb_status emb_distill_backward(int device, const void* logits, emb_dtype logits_dtype,
                                int64_t logits_stride, int32_t N, int32_t V,
                                const int64_t* teacher_ids, const void* teacher_logits,
                                emb_dtype teacher_dtype, int64_t teacher_stride, int32_t K,
                                const float* stats, const float* row_weight, float temperature,
                                void* dlogits, int64_t dlogits_stride, uint32_t* device_status,
                                void* stream);
emb_status emb_distill_step(int device, const void* logits, emb_dtype logits_dtype,
                            int64_t logits_stride, int32_t N, int32_t V,
                            const int64_t* teacher_ids, const void* teacher_logits,
                            emb_dtype teacher_dtype, int64_t teacher_stride, int32_t K,
                            const float* teacher_lse, const float* row_weight, float temperature,
                            float* loss, void* dlogits, int64_t dlogits_stride,
                            uint32_t* device_status, void* stream);

/* Microscaled floating point: 4-bit E2M1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
 * negatives) or 8-bit E4M3 elements (up to 448) with a scale for every block.
 *   EMB_MICRO_MX: blocks of 32 share 2^(byte - 127), exponent floor(log2(amax)) - 2 (at
 *     least -127); byte 255 = NaN. No tensor scale (pass 1).
 *   EMB_MICRO_NV: blocks of 16 share an E4M3 scale times the tensor's fp32 scale g
 *     (1e-15..1e15): E4M3(amax / (6 g)), saturating.
 *   EMB_MICRO_MX8: E4M3 elements, blocks of 32 share 2^(byte - 127), the smallest (at least
 *     2^-127) that brings amax to 448 or less; byte 255 = NaN. No tensor scale (pass 1).
 * An element is multiplied by the scale's reciprocal (rounded to fp32; exact for MX and MX8), rounded
 * to the nearest code (ties to even) and saturates at the largest. A block that holds an
 * infinity or a NaN gets a NaN scale: all its elements read back as NaN.
 * codes: [rows, 16 * ceil(K / 32)] bytes; element k in bits 0-3 (k even) or 4-7 (k odd)
 *   of byte k / 2; padded with zeros. MX8: [rows, 32 * ceil(K / 32)], element k in byte k.
 * scales: tiles of 512 bytes for 128 rows x 4 blocks, tile (i, j) at (i * ceil(blocks / 4)
 *   + j) * 512 with blocks = ceil(K / 32) * (MX, MX8: 1, NV: 2); block j of row r at byte
 *   (r % 32) * 16 + (r % 128 / 32) * 4 + j % 4 of tile (r / 128, j / 4); padded with zeros.
 * Both 16-byte aligned, and written entirely by emb_micro_quantize. K <= 2^20. */
typedef enum { EMB_MICRO_MX = 0, EMB_MICRO_NV = 1, EMB_MICRO_MX8 = 8 } emb_micro_format;

/* x [R, K] -> codes, scales. */
emb_status emb_micro_quantize(int device, const void* x, emb_dtype x_dtype, int64_t x_stride,
                              int64_t R, int32_t K, emb_micro_format format, float tensor_scale,
                              uint8_t* codes, uint8_t* scales, void* stream);

/* Rows ids[0..n) of a microscaled table of R rows as values, out [n, K]: code * block
 * scale * tensor scale, rounded once to out_dtype. ids NULL: rows 0..n-1 (n <= R). An id
 * outside the table gives a row of zeros and error bit 1. */
emb_status emb_micro_lookup(int device, const uint8_t* codes, const uint8_t* scales, int64_t R,
                            int32_t K, emb_micro_format format, float tensor_scale,
                            const int64_t* ids, int64_t n, void* out, emb_dtype out_dtype,
                            int64_t out_stride, uint32_t* device_status, void* stream);

/* out[m, n] = sum_k X[m, k] * W[n, k] for microscaled X [M, K] and W [N, K] of one format
 * (M, N <= 2^21), summed in fp32 and rounded once: the logits of M hidden states against
 * a table of N tokens. */
emb_status emb_micro_matmul(int device, const uint8_t* x_codes, const uint8_t* x_scales,
                            float x_tensor_scale, int32_t M, const uint8_t* w_codes,
                            const uint8_t* w_scales, float w_tensor_scale, int32_t N, int32_t K,
                            emb_micro_format format, void* out, emb_dtype out_dtype,
                            int64_t out_stride, uint32_t* device_status, void* stream);

/* Root-mean-square norm of N rows of D <= 16384 elements, with the residual's addition before it.
 *   s = x + residual (NULL: x),  rstd = 1 / sqrt(mean(s^2) + eps),  y = s * rstd * weight
 * in fp32 (y is computed from the sum before it is rounded), weight [D] of a type of its own, NULL =
 * 1. Outputs: sum (s; may be NULL), rstd fp32[N] (may be NULL), and either out (y), all of x's type, or
 * codes and scales: y as an EMB_MICRO_MX8 matrix of N rows, written entirely. out or sum
 * may be x or residual themselves (same stride), and must not overlap them or each other
 * otherwise.
 * The gradient, with h = sum * rstd and g = grad * weight, grad the gradient of y:
 *   out = rstd * (g - h * mean(g * h)) + grad_sum   (of x, and of residual)
 *   grad_weight[d] = sum_n grad[n, d] * h[n, d]     (of weight_dtype; NULL: not computed)
 * grad_sum: the gradient that arrives at s by other ways, NULL = 0. out may be grad, sum or
 * grad_sum themselves (same stride). With grad_weight it needs a workspace (16-byte aligned, not
 * shared by calls that may run at once) of emb_rms_norm_workspace bytes (-1: sizes
 * out of range). The same call gives the same bits: the order of sums depends on the sizes, on
 * where in 16 bytes rows lie and on the number of SMs, never on timing. */
emb_status emb_rms_norm_forward(int device, const void* x, emb_dtype dtype, int64_t x_stride, int64_t N,
                                int32_t D, const void* residual, int64_t residual_stride,
                                const void* weight, emb_dtype weight_dtype, float eps, void* out,
                                int64_t out_stride, uint8_t* codes, uint8_t* scales, void* sum,
                                int64_t sum_stride, float* rstd, void* stream);
int64_t emb_rms_norm_workspace(int device, int64_t N, int32_t D);
emb_status emb_rms_norm_backward(int device, const void* grad, emb_dtype dtype, int64_t grad_stride,
                                 int64_t N, int32_t D, const void* sum, int64_t sum_stride,
                                 const void* weight, emb_dtype weight_dtype, const float* rstd,
                                 const void* grad_sum, int64_t grad_sum_stride, void* out,
                                 int64_t out_stride, void* grad_weight, void* workspace,
                                 int64_t workspace_bytes, void* stream);

/* Dropout of N < 2^31 rows of D <= 2^20 elements, with the residual's addition after it:
 *   out = (kept ? x / (1 - p) : 0) + residual (NULL: 0),  0 <= p < 1
 * Element d of row r is kept iff word d mod 4 of Philox4x32-10 (Salmon et al., SC 2011) at
 * counter (r, d / 4, c mod 2^32, c / 2^32) under the key (seed mod 2^32, seed / 2^32) is at
 * least p * 2^32, with c = call + *device_call (device int64, NULL: 0; read when the call
 * runs, so that a captured graph draws new words when the caller has advanced it). The
 * gradient of x is the same call on the gradient, without residual. Products with
 * 1 / (1 - p) in fp32; a dropped element is 0 whatever it held. out may be x or
 * residual themselves (same stride), and must not overlap them otherwise. */
emb_status emb_dropout(int device, const void* x, emb_dtype dtype, int64_t x_stride, int64_t N,
                       int32_t D, const void* residual, int64_t residual_stride, double p,
                       uint64_t seed, uint64_t call, const int64_t* device_call, void* out,
                       int64_t out_stride, void* stream);

/* Softmax cross entropy of N hidden states against a table of V tokens (N, V <= 2^20, width
 * D <= 2^15; hidden [N, D] and table [V, D] both fp16 or both bf16), without the N x V
 * logits in memory. With z = hidden table^T, summed in fp32:
 *   lse[n] = log sum_v exp(z[n, v]),  loss[n] = lse[n] - z[n, targets[n]]
 *   G[n, v] = row_weight[n] * (exp(z[n, v] - lse[n]) - [v = targets[n]])
 *   grad_hidden = G table,  grad_table = G^T hidden   (of hidden's type)
 * targets int64[N]. A row with a negative target takes no part: its loss, lse and grad_hidden
 * are 0, and nothing that it holds reaches another output. So does a target >= V, with error
 * bit 1. row_weight fp32[N] or NULL = 1; lse fp32[N] (may be NULL in the forward call). G is
 * rounded to hidden's type before it is multiplied, up to 64 tokens to a sum of two such numbers.
 * (fp16: scaled by a power of two that brings the largest weight of a row that takes part to
 * 2^14..2^15, so that probabilities down to 2^-28 keep all bits in a row of that weight, and
 * down to 2^(k - 28) in one whose weight is 2^-k of it.) Sums are fp32, in a fixed order: the
 * same call (sizes, places in 16 bytes, targets that take part, number of SMs) gives the same
 * bits, and a row's loss and lse do not depend on the other rows' targets. An accumulator of a
 * gradient sums 2^13 (fp16) or 2^16 (bf16) elements at most. Probabilities and products below
 * 2^-126 may count as 0.
 *   emb_cross_entropy_forward    loss, lse
 *   emb_cross_entropy_backward   gradients from the forward's lse; the logits are computed
 *                                again. A NULL grad_hidden or grad_table is not computed
 *   emb_cross_entropy_step       loss and gradients in one call
 * With N = 0 grad_table is set to zero. The outputs must not overlap the inputs nor each
 * other. These calls
 * need a workspace (256-byte aligned, not shared by calls that may run at once) of
 * emb_cross_entropy_workspace bytes, for the same sizes, table pointer and stride, either type;
 * gradients != 0 for the backward and the step. With N rounded up to 256 and D to 64 it takes up
 * to N (V / 16 + 2 D + 16 SMs + 64) bytes; with gradients also 2 N V or 512 MB for G, whichever is
 * less (512 N at least), and for the parts of grad_hidden up to the largest of 8 N D, 256 MB,
 * 24 KB for each column, and 256 KB for each SM + 1 KB for each column; a table that bulk copies
 * cannot read (off 16-byte boundaries, or D not a multiple of 8) 2 V D more.
 * It returns -1 for sizes out of range. */
int64_t emb_cross_entropy_workspace(int device, int64_t N, int32_t V, int32_t D, const void* table,
                                    int64_t table_stride, int gradients);
emb_status emb_cross_entropy_forward(int device, const void* hidden, emb_dtype dtype,
                                     int64_t hidden_stride, int64_t N, const void* table,
                                     int64_t table_stride, int32_t V, int32_t D,
                                     const int64_t* targets, float* loss, float* lse, void* workspace,
                                     int64_t workspace_bytes, uint32_t* device_status, void* stream);
emb_status emb_cross_entropy_backward(int device, const void* hidden, emb_dtype dtype,
                                      int64_t hidden_stride, int64_t N, const void* table,
                                      int64_t table_stride, int32_t V, int32_t D,
                                      const int64_t* targets, const float* lse,
                                      const float* row_weight, void* grad_hidden,
                                      int64_t grad_hidden_stride, void* grad_table,
                                      int64_t grad_table_stride, void* workspace,
                                      int64_t workspace_bytes, uint32_t* device_status,
                                      void* stream);
emb_status emb_cross_entropy_step(int device, const void* hidden, emb_dtype dtype,
                                  int64_t hidden_stride, int64_t N, const void* table,
                                  int64_t table_stride, int32_t V, int32_t D,
                                  const int64_t* targets, const float* row_weight, float* loss,
                                  void* grad_hidden, int64_t grad_hidden_stride, void* grad_table,
                                  int64_t grad_table_stride, void* workspace,
                                  int64_t workspace_bytes, uint32_t* device_status, void* stream);

/* Static description of a status code. */
const char* emb_status_string(emb_status status);

#ifdef __cplusplus
}
#endif

#endif /* EMBBWD_H */
