/*
 * rar.h -- C ABI of librar.so: ring all-reduce-mean and the synchronous SGD
 * update of data-parallel training, for N logical ranks whose gradient
 * buffers all sit in the HBM of one MI355X (gfx950).
 *
 * Sources (short names):
 *   [Gibiansky]  "Bringing HPC Techniques to Deep Learning", A. Gibiansky,
 *                Baidu SVAIL (Korean translation at wonjae.kim).
 *   [TrainMGPU]  "[AI System] Training With Multiple GPUs".
 *   [DDPpage]    "[PyTorch] GPU 분산 학습 1 - DP / DDP / FSDP 개념".
 *
 * The problem ([Gibiansky] §Scatter-reduce, opening paragraph): N ranks each
 * hold an array of the same length P; afterwards every rank holds the same
 * array.  Here that array is the element-wise MEAN of the N inputs, because
 * data-parallel SGD averages the per-rank gradients and applies the average
 * to the weights ([Gibiansky] §The communication problem; [TrainMGPU]
 * §Training Process, steps 2-3; [DDPpage] §DDP: every rank ends with the
 * identical gradient and updates on its own).
 *
 * Numerics contract (binary32):
 *   - Chunk c of the plan's chunk table is summed in ring order, starting at
 *     rank c: ((g_c + g_{c+1}) + g_{c+2}) + ... + g_{c+N-1} (ranks mod N).
 *     That is the order the scatter-reduce of [Gibiansky] §Scatter-reduce
 *     produces (rank n starts by sending chunk n).
 *   - mean = S / N, one correctly rounded IEEE division.
 *   - SGD: w = w - (lr * mean), the product and the difference each rounded
 *     once (no fused multiply-add).
 *   - No flush of subnormals; NaN and infinity propagate.
 *   With these, every algorithm below gives bit-identical results.
 * bf16: values are widened exactly to binary32, summed and divided as above,
 * and each bf16 buffer receives the mean rounded to nearest-even; the SGD
 * update uses the binary32 mean.
 *
 * Memory and streams: every device pointer is owned by the caller and must
 * stay valid until the work enqueued on `stream` (a hipStream_t passed as
 * void*, NULL = the default stream) has finished.  Calls return after
 * enqueueing; they never synchronise, except rar_rank_stride_tune, which
 * times work on its stream and waits for it.  Rank buffers, weights and bucket
 * buffers must be 16-byte aligned; bucket tensors need only element
 * alignment.  The only device allocations are binary32 workspaces of bf16
 * rings: a bf16 plan set to RAR_ALGO_RING (rar_plan_set_algo, or a bucket call
 * that builds such a plan for itself), which lives until the plan is
 * destroyed, and a bf16 RAR_ALGO_RING bucket call over per-rank arenas (one
 * float per element of the plan, kept with the bucket handle until it is
 * destroyed).
 *
 * Graph capture: the execute and bucket calls only enqueue kernels and
 * stream waits (no allocation, synchronisation or memset), so they can be
 * captured into a HIP graph and replayed, once the plans they use exist and
 * any bf16 ring workspace has been allocated by rar_plan_set_algo.  Bucket
 * calls make their per-size plans on first use (a bf16 RAR_ALGO_RING bucket
 * call allocates the workspaces then): make one call before capturing.  The
 * ready events of a captured rar_bucket_allreduce_arena must be recorded
 * inside the same capture (on a stream forked from the capturing one).
 *
 * Errors: every argument is checked before any device work is enqueued; on
 * an argument error nothing is enqueued and a negative rar_status is
 * returned.  RAR_EHIP means a HIP launch or runtime call failed, RAR_ENOMEM
 * that a device allocation did; a call of several launches that fails that
 * way part-way may leave its earlier launches enqueued, and the buffers'
 * contents are then unspecified.  The library clears HIP's last-error state
 * when it returns either, so the caller's next HIP call does not report it
 * again.
 * Thread safety: a plan is immutable after rar_plan_set_algo; a plan without
 * a workspace may be used from several host threads and streams at once.  A
 * bf16 ring plan owns one workspace and must be used by one stream at a time.
 * A bucket handle may be used from several threads and streams at once (its
 * plan cache is locked), except with dtype bf16 and RAR_ALGO_RING, whose
 * binary32 workspaces (one per bucket size for bucket buffers, one per handle
 * for arenas) are shared by every call: one stream at a time.
 */
#ifndef RAR_H
#define RAR_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RAR_MAX_RANKS 64
#define RAR_MAX_STRIDE_CANDIDATES 64
/* binary32 elements of the library's static device workspace (64 MiB on each
 * device it runs on), used by rar_allreduce_ring_noalloc */
#define RAR_STATIC_WS_ELEMS (1 << 24)

typedef struct rar_plan_s *rar_plan_t;
typedef struct rar_buckets_s *rar_buckets_t;

typedef enum { RAR_F32 = 0, RAR_BF16 = 1 } rar_dtype;

/* How P elements are cut into N chunks ([Gibiansky] §Scatter-reduce: the
 * array is split into N chunks; the page does not say how when N does not
 * divide P). */
typedef enum {
    RAR_CHUNK_BALANCED = 0, /* sizes differ by at most 1, larger chunks first */
    RAR_CHUNK_CEIL = 1,     /* ceil(P/N) each; the tail takes the rest (may be short or empty) */
    RAR_CHUNK_ALIGN16 = 2   /* ceil(P/N) rounded up to whole 16-byte groups; tail as CEIL */
} rar_chunking;

typedef enum {
    RAR_ALGO_FUSED = 0, /* one pass: reads every rank once, writes every rank once */
    RAR_ALGO_RING = 1,  /* the 2(N-1) ring steps of [Gibiansky], one kernel per step */
    RAR_ALGO_NAIVE = 2  /* prior art: rank 0 reduces all and sends back ([Gibiansky]
                           §The communication problem); its own summation order */
} rar_algo;

typedef enum {
    RAR_OK = 0,
    RAR_EINVAL = -1,    /* bad argument */
    RAR_EMISMATCH = -2, /* P differs from the plan's P */
    RAR_EALIGN = -3,    /* a device pointer is not 16-byte aligned */
    RAR_ENOMEM = -4,    /* host or device allocation failed */
    RAR_EHIP = -5,      /* a HIP runtime call or kernel launch failed */
    RAR_ETOOLARGE = -6  /* P exceeds the static workspace (rar_allreduce_ring_noalloc) */
} rar_status;

/* ---------------------------------------------------------------------- */
/* Plans                                                                   */
/* ---------------------------------------------------------------------- */

/* Create a plan for N ranks (1..RAR_MAX_RANKS) of P >= 0 elements of dtype,
 * cut into chunks by `chunking` ([Gibiansky] §Scatter-reduce).  Host memory
 * only; no HIP call.  *out receives the plan (NULL on error).  The algorithm
 * starts as RAR_ALGO_FUSED. */
rar_status rar_plan(int N, int64_t P, rar_dtype dtype, rar_chunking chunking, rar_plan_t *out);

/* Not an operation of the pages: layout advice for callers that place the N
 * logical ranks of one device in a single allocation (rank n at base +
 * n * stride, base 16-byte aligned):
 * *stride_bytes receives the smallest stride >= P * element size that is
 * 2 MiB modulo 4 MiB.  Where rank buffers start matters on MI355X; measured
 * for the fused pass, 10 ranks x 300M fp32 with SGD, one process per box:
 * this stride 4.17-4.39 ms; separately allocated buffers (which lie a
 * multiple of 4 MiB apart) 4.28-4.59 ms; a stride of 1 or 3 MiB modulo
 * 4 MiB 4.40-4.80 ms.  40 ranks x 100M bf16: 2.92 ms against 3.12 ms for
 * separate buffers.  The rule does not hold for every shape: at 8 ranks x
 * 735M fp32 these strides are the slowest (8.1-8.4 ms against 7.5 ms for
 * multiples of 8 MiB), because which strides are fast follows a hash of
 * higher address bits; rar_rank_stride_tune measures instead.  Results never
 * depend on the layout.  Host only, no HIP call.  RAR_EINVAL: NULL
 * stride_bytes, unknown dtype, P < 0, or P so large that the stride
 * overflows. */
rar_status rar_rank_stride(int64_t P, rar_dtype dtype, int64_t *stride_bytes);

/* The stride candidates rar_rank_stride_tune times, so that a caller can size
 * its pool: *stride_bytes receives candidate k (0 <= k <
 * RAR_MAX_STRIDE_CANDIDATES) for ranks of P elements of dtype.  With s0 the
 * smallest multiple of 2 MiB >= P * element size, candidates 0..31 are s0,
 * s0 + 2 MiB, ..., s0 + 62 MiB, and candidates 32..63 are the multiples of
 * 8 MiB from the first one >= s0 + 64 MiB, 8 MiB apart.  They increase with
 * k; rar_rank_stride's stride is candidate 0 or 1.  A pool for the first K
 * candidates needs (N-1) * candidate(K-1) + P * element size bytes.  Host
 * only, no HIP call.  RAR_EINVAL: NULL stride_bytes, unknown dtype, P < 0, k
 * out of range, or P too large. */
rar_status rar_rank_stride_candidate(int64_t P, rar_dtype dtype, int k, int64_t *stride_bytes);

/* Not an operation of the pages either: measured layout advice for the same
 * single-allocation placement.  Times the fused mean over N ranks carved
 * from `pool` (device, 16-byte aligned, pool_bytes long) at the strides
 * rar_rank_stride_candidate gives, the first max_candidates
 * (1..RAR_MAX_STRIDE_CANDIDATES) of them for which (N-1) * stride + P *
 * element size <= pool_bytes, and returns the fastest in *stride_bytes.
 * Two stages, each in rounds that visit the candidates
 * forward and backward in turn, one untimed and two timed calls per
 * candidate and round: four rounds over every candidate, then eight more
 * over the finalists, the four with the smallest medians so far and the
 * stride rar_rank_stride gives when it is a candidate (24 timings each).
 * The finalist with the smallest median wins, ties to the smaller stride --
 * except that rar_rank_stride's stride is kept if its median exceeds the
 * winner's by no more than a third of the finalists' typical spread (the
 * median of their spreads, each the range of the middle three quarters of
 * its timings), about two standard errors of a difference of two such
 * medians: on MI355X the fast strides lie within about 1% of each other,
 * about as much as single calls vary.  Fast strides also lie beyond the
 * first few: at 10 x 300M fp32 the best of a sweep from 1146 to 1658 MiB
 * were 1280 and 1368 MiB, the SGD call 1% faster there than at the best
 * stride within 1146-1272 MiB and 2.5% faster than at the static rule's
 * 1146 MiB (one box, interleaved rounds).  The
 * pool's contents are overwritten; the call enqueues on `stream` and waits
 * for it, so it must not run under graph capture.  N == 1 or P == 0 returns
 * s0 without device work.  Which strides are fast differs by shape (see
 * rar_rank_stride); measured on MI355X, 8 ranks x 735M fp32: 7.50-7.57 ms at
 * the pick against 7.86 ms for separate allocations and 8.35 ms for
 * rar_rank_stride.  RAR_EINVAL: NULL stride_bytes or pool, N outside
 * 1..RAR_MAX_RANKS, P < 0, unknown dtype, max_candidates out of range, or a
 * pool too small for even s0.  RAR_EALIGN: pool not 16-byte aligned.
 * RAR_EHIP / RAR_ENOMEM: a HIP call failed. */
rar_status rar_rank_stride_tune(int N, int64_t P, rar_dtype dtype, void *pool, int64_t pool_bytes,
                                int max_candidates, void *stream, int64_t *stride_bytes);

/* rar_rank_stride_tune, also reporting what it measured: *n_candidates
 * receives K, the number of candidates timed (0 when N == 1 or P == 0), and
 * for k < K cand_stride[k], median_ms[k] and spread_ms[k], over all of
 * candidate k's timings (8, or 24 for a finalist; the spread is the range of
 * their middle three quarters).  The arrays hold max_candidates entries; any
 * of these outputs may be NULL. */
rar_status rar_rank_stride_tune_stats(int N, int64_t P, rar_dtype dtype, void *pool, int64_t pool_bytes,
                                      int max_candidates, void *stream, int64_t *stride_bytes,
                                      int *n_candidates, int64_t cand_stride[], float median_ms[],
                                      float spread_ms[]);

/* Free the plan and its workspace (if any).  Waits for the device to finish
 * work that may use the workspace.  NULL is accepted. */
rar_status rar_plan_destroy(rar_plan_t plan);

/* Select the algorithm used by rar_allreduce_mean / rar_allreduce_sgd.
 * For a bf16 plan, RAR_ALGO_RING allocates the binary32 workspace (4*P
 * bytes, chunk-indexed: it carries the running partial sum of each chunk
 * between ring steps); RAR_ENOMEM if that fails.  RAR_ALGO_NAIVE is
 * supported for RAR_F32 only. */
rar_status rar_plan_set_algo(rar_plan_t plan, rar_algo algo);

/* Kernel launch shape: at most max_blocks workgroups per launch (0 = the
 * library's choice).  Results do not depend on it. */
rar_status rar_plan_set_grid(rar_plan_t plan, int max_blocks);

/* Chunk c: element offset and length, and the rank that holds the finished
 * chunk after scatter-reduce, (c-1) mod N (derived from [Gibiansky]
 * §Scatter-reduce, and the step-1 table of §Allgather where GPU n starts by
 * sending chunk n+1).  Any output pointer may be NULL. */
rar_status rar_plan_chunk(rar_plan_t plan, int c, int64_t *offset, int64_t *length, int *owner_rank);

/* Elements rank `rank` sends and receives in the ring schedule (N-1
 * scatter-reduce plus N-1 all-gather transfers, [Gibiansky] §Allreduce
 * communication cost): 2P - |C(rank+1)| - |C(rank+2)| sent and
 * 2P - |C(rank)| - |C(rank+1)| received, i.e. 2(N-1)P/N when N divides P. */
rar_status rar_plan_traffic(rar_plan_t plan, int rank, int64_t *sent_elems, int64_t *recv_elems);

/* ---------------------------------------------------------------------- */
/* All-reduce                                                              */
/* ---------------------------------------------------------------------- */

/* In place: every bufs[n] (n < N; device, P elements of the plan's dtype)
 * ends holding the element-wise mean of the N inputs.  bufs is a host
 * array of N device pointers; it is copied, so it need not outlive the
 * call.  The N buffers must not overlap.  P must equal the plan's P (it is
 * passed again as a check: RAR_EMISMATCH).  P == 0 is a no-op. */
rar_status rar_allreduce_mean(rar_plan_t plan, void *const bufs[], int64_t P, void *stream);

/* As rar_allreduce_mean, then the synchronous SGD step on the binary32
 * weights w (device, P floats, must not overlap any buffer):
 * w[e] = w[e] - lr * mean[e] ([Gibiansky] §The communication problem;
 * [TrainMGPU] §Training Process, step 3; [DDPpage] §DDP). */
rar_status rar_allreduce_sgd(rar_plan_t plan, void *const bufs[], float *w, float lr, int64_t P,
                             void *stream);

/* Scatter-reduce with the owner's update, then an all-gather of weights (the
 * sharded shape of [DDPpage] §FSDP: gradients are reduce-scattered and each
 * rank updates only the part it owns).  After the call:
 *   - the owner of chunk c, (c-1) mod N, holds mean[C_c] in bufs[owner][C_c];
 *     other parts of the gradient buffers hold ring partial sums (unspecified);
 *   - every weight replica w_reps[n] (device, P floats each) holds
 *     w_reps[owner][e] - lr*mean[e] for every element e, i.e. the same bits
 *     rar_allreduce_sgd gives when all replicas start equal.
 * Only RAR_F32 plans; the algorithm selected by set_algo is ignored (this
 * call is always the ring: N-1 scatter-reduce steps, N-1 all-gather steps). */
rar_status rar_reduce_scatter_sgd_allgather(rar_plan_t plan, void *const bufs[],
                                            float *const w_reps[], float lr, int64_t P,
                                            void *stream);

/* For callers that cannot allocate device memory: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc.  The ring
 * algorithm of rar_allreduce_mean (w == NULL) or rar_allreduce_sgd (w != NULL)
 * with the same arguments, results and checks, whatever algorithm the plan
 * has selected, and with no device allocation, free or memset: a bf16 plan's
 * binary32 partial sums go to a workspace the library holds in a static device
 * array of RAR_STATIC_WS_ELEMS floats instead of one the plan allocates
 * (binary32 plans need none).  Each device keeps its own copy of that array
 * until the process ends; its address is looked up once per device, on the
 * first call there.  Every element of the workspace that a call reads was
 * written earlier in the same call, so nothing is cleared between calls.  All
 * calls on one device share the array: calls on that device that overlap in
 * time (other streams, other host threads) race and must be serialised by the
 * caller.  `stream` must belong to the current device (RAR_EINVAL otherwise).
 * RAR_ETOOLARGE: a bf16 plan with N > 1 and P > RAR_STATIC_WS_ELEMS. */
rar_status rar_allreduce_ring_noalloc(rar_plan_t plan, void *const bufs[], float *w, float lr, int64_t P,
                                      void *stream);

/* ---------------------------------------------------------------------- */
/* Buckets: a ragged list of per-layer gradients reduced in fixed-size     */
/* buckets ([Gibiansky] §Applying allreduce to deep learning: the          */
/* all-reduce can run on a subset of the parameters, and output-layer      */
/* gradients are ready first).                                             */
/* ---------------------------------------------------------------------- */

/* Lay n_tensors tensors (numel[t] elements each, listed in the order
 * back-propagation produces them) end to end and cut the stream into
 * buckets of bucket_bytes / sizeof(dtype) elements; a tensor that crosses a
 * boundary is split.  Host memory only. */
rar_status rar_bucket_plan(int n_tensors, const int64_t numel[], rar_dtype dtype, int64_t bucket_bytes,
                           rar_buckets_t *out);

rar_status rar_bucket_destroy(rar_buckets_t b);

/* Number of buckets and the largest bucket's element count. */
rar_status rar_bucket_count(rar_buckets_t b, int *n_buckets, int64_t *max_bucket_elems);

/* Bucket `bucket`: its first element in the concatenated stream, its element
 * count and its number of segments.  Any output may be NULL. */
rar_status rar_bucket_info(rar_buckets_t b, int bucket, int64_t *stream_offset, int64_t *elems,
                           int *n_segments);

/* Segment `seg` of a bucket: tensor index, offset inside that tensor, offset
 * inside the bucket, length (elements).  Any output may be NULL. */
rar_status rar_bucket_segment(rar_buckets_t b, int bucket, int seg, int *tensor, int64_t *tensor_offset,
                              int64_t *bucket_offset, int64_t *length);

/* Copy the bucket's segments of every rank's tensors into bucket_bufs[n]
 * (device, >= the bucket's elements).  tensors is a host array of N*n_tensors
 * device pointers, rank-major: tensors[n*n_tensors + t].  The N ranks' copies
 * of a segment, and the bucket's elements of the N bucket buffers, must all be
 * disjoint memory (RAR_EINVAL otherwise). */
rar_status rar_bucket_pack(rar_buckets_t b, int bucket, int N, void *const tensors[],
                           void *const bucket_bufs[], void *stream);

/* The reverse copy, from bucket_bufs[n] back into the tensors (same checks). */
rar_status rar_bucket_unpack(rar_buckets_t b, int bucket, int N, void *const bucket_bufs[],
                             void *const tensors[], void *stream);

/* Every bucket in order, all-reduce-mean in place in the tensors.  Element e
 * of a bucket ends bit-identical to what rar_allreduce_mean gives for that
 * bucket alone (chunk table of the bucket's size, `chunking`).
 * With RAR_ALGO_FUSED and N in {2, 4, 8, 10, 16, 40} the reduction reads and
 * writes the tensors directly (each bucket segment cut at the bucket's chunk
 * boundaries, and the pieces of consecutive tensors in one chunk joined
 * where every rank's tensors are adjacent in memory; 2*N*size bytes moved
 * per bucket) and bucket_bufs may be NULL.
 * The jobs of consecutive buckets then share launches, so all N*n_tensors
 * tensors must be pairwise disjoint memory (RAR_EINVAL otherwise).
 * With RAR_ALGO_RING, RAR_F32 and N >= 2 the 2(N-1) ring steps of
 * [Gibiansky] §Scatter-reduce and §Allgather run on those same pieces in
 * place (5*(N-1)*size*4 bytes moved per bucket, no packing); each step is
 * a few launches over the pieces of every bucket, so the tensors must again
 * be pairwise disjoint, and bucket_bufs may be NULL.  When every rank's
 * tensors lie end to end in the plan's order (views of one flat buffer per
 * rank, 16-byte aligned, with 16-byte aligned bucket starts), the call runs
 * as rar_bucket_allreduce_arena over those buffers, also for bf16 with
 * RAR_ALGO_RING (no packing; binary32 partial sums in a workspace kept with
 * the bucket handle).
 * Otherwise each bucket is packed into bucket_bufs[n] (N device buffers of at
 * least max_bucket_elems elements, 16-byte aligned, reused by every bucket,
 * overlapping neither each other nor the tensors: RAR_EINVAL), reduced with
 * `algo`, and unpacked. */
rar_status rar_bucket_allreduce_mean(rar_buckets_t b, int N, rar_chunking chunking, rar_algo algo,
                                     void *const tensors[], void *const bucket_bufs[], void *stream);

/* Every bucket in order, in place over per-rank flat arenas, each bucket
 * starting only once its gradients exist ([Gibiansky] §Applying allreduce to
 * deep learning: back-propagation produces the output layers' gradients
 * first, so their reduction can overlap the rest of the backward pass).
 * arenas[n] (device, 16-byte aligned) holds rank n's tensors end to end in
 * the plan's order, so bucket k is the slice [stream_offset, +elems) of every
 * arena and needs no packing.  ready_events is a host array of n_buckets
 * hipEvent_t (as void*), or NULL: before bucket k the call makes `stream`
 * wait for ready_events[k] (a NULL entry waits for nothing).  The producer
 * records the events on its own stream; the waits are enqueued, the call
 * does not block the host.  Every bucket start must be 16-byte aligned
 * (RAR_EALIGN otherwise; a bucket size that is a multiple of 16 bytes gives
 * that), and the N arenas (total elements each) must not overlap
 * (RAR_EINVAL).  With RAR_ALGO_FUSED and N in {2, 4, 8, 10, 16, 40}, and
 * with RAR_ALGO_RING and N >= 2 (each ring step over every chunk of those
 * buckets at once; bf16 keeps the binary32 partial sums in a workspace of one
 * float per element, allocated on the first such call and kept with the
 * bucket handle), the buckets between two ready events share launches.
 * Results are bit-identical to rar_allreduce_mean on each slice. */
rar_status rar_bucket_allreduce_arena(rar_buckets_t b, int N, rar_chunking chunking, rar_algo algo,
                                      void *const arenas[], void *const ready_events[], void *stream);

/* ---------------------------------------------------------------------- */
/* Producers of the gradients: the embedding, the linear layer and 8-bit   */
/* activation checkpoints.  These make the tensors whose gradients the     */
/* calls above reduce: a Transformer's embedding table and its projections */
/* W (in x out) with biases.                                               */
/*                                                                         */
/* Matrices are row-major with a leading dimension in elements (ld >= the  */
/* row length, at most 2^22; K, N, D at most 2^20; T at most 2^24; of a    */
/* linear layer T x K, T x N and K x N at most 2^37 elements).             */
/* Matrices in the operator's type need element alignment only; a linear   */
/* layer's products read rows of whole 16-byte groups at 16-byte aligned   */
/* addresses directly and copy others into the workspace first, in every   */
/* call.  Outputs must not overlap inputs or each other, unless a call     */
/* says so (RAR_EINVAL); two views of one leading dimension with disjoint  */
/* columns do not overlap.  Device buffers belong to the current device.   */
/*                                                                         */
/* Workspaces are the caller's: `ws` is device memory, 16-byte aligned, of */
/* at least the bytes the matching query gives (RAR_EINVAL otherwise); it  */
/* holds nothing between calls and need not be cleared.  Calls that may    */
/* overlap in time (other streams, other graphs) need workspaces of their  */
/* own.  Nothing is allocated, so every call can be captured.              */
/*                                                                         */
/* Numerics: bf16 operands are widened exactly; products, sums and         */
/* activations are binary32; each output is rounded once, to nearest even. */
/* gelu and its derivative are good to 2^-20 (1 + |z|) in a binary32 layer */
/* and to 2^-18 (1 + |z|), far inside its rounding, in a bf16 one; db,     */
/* which sums the unrounded dz, inherits that.  Accumulation in bf16       */
/* rounds the running sum to bf16 in every call.                           */
/* Results depend on the inputs and the sizes only, not on timing: no      */
/* floating-point atomics.  NaN and infinity propagate.                    */
/* ---------------------------------------------------------------------- */

typedef struct rar_linear_s *rar_linear_t;

typedef enum {
    RAR_ACT_NONE = 0,
    RAR_ACT_RELU = 1, /* max(z, 0); derivative 0 at 0 */
    RAR_ACT_GELU = 2  /* z * Phi(z), Phi the normal distribution function (the erf form) */
} rar_act;

/* Values of a row that share one scale in an 8-bit checkpoint. */
#define RAR_CKPT_GROUP 32

/* Embedding lookup: out[t] = scale * table[ids[t]] for t < T.  table is V x D
 * (contiguous), ids T int64, out T x D with leading dimension ldo.  An id
 * outside 0..V-1 (padding) gives a row of zeros.  T == 0 is a no-op. */
rar_status rar_embed_lookup(int64_t V, int64_t D, rar_dtype dtype, const void *table, int64_t T,
                            const int64_t *ids, float scale, void *out, int64_t ldo, void *stream);

/* Workspace of rar_embed_grad. */
rar_status rar_embed_grad_workspace(int64_t V, int64_t D, int64_t T, int64_t *bytes);

/* Gradient of the lookup: grad[v] = scale * (sum of dy[t] over the t with
 * ids[t] == v), for every v < V: rows that no token names become zero.  With
 * accumulate != 0 the sum is added to grad instead, and rows that no token
 * names are not touched.  dy is T x D with leading dimension lddy, grad V x D
 * contiguous.  Ids outside 0..V-1 are skipped.  Terms are added in an order
 * that the ids alone determine. */
rar_status rar_embed_grad(int64_t V, int64_t D, rar_dtype dtype, int64_t T, const int64_t *ids, const void *dy,
                          int64_t lddy, float scale, int accumulate, void *grad, void *ws, int64_t ws_bytes,
                          void *stream);

/* A linear layer of K inputs and N outputs: host memory only, immutable, any
 * number of threads and streams. */
rar_status rar_linear_plan(int64_t K, int64_t N, rar_dtype dtype, rar_act act, rar_linear_t *out);

rar_status rar_linear_destroy(rar_linear_t plan);

/* Workspaces of a forward and of a backward call on T rows, for matrices at any
 * address and of any leading dimension: copies of x and w are counted also
 * where a call reads them directly.  Either output may be NULL. */
rar_status rar_linear_workspace(rar_linear_t plan, int64_t T, int64_t *forward_bytes, int64_t *backward_bytes);

/* z = x W + bias, y = act(z) + residual.  x is T x K, w K x N contiguous, bias
 * N or NULL, residual T x N or NULL (it may be y itself), y T x N.  pre (or
 * NULL) receives z for the backward pass: in the layer's type with leading
 * dimension ldp, or, with pre_scales, as an 8-bit checkpoint (the one
 * rar_ckpt_store makes of z rounded to the layer's type; ldp is ignored).  The
 * activation is taken of the unrounded z.  T == 0 is a no-op. */
rar_status rar_linear_forward(rar_linear_t plan, int64_t T, const void *x, int64_t ldx, const void *w,
                              const void *bias, const void *residual, int64_t ldr, void *y, int64_t ldy, void *pre,
                              int64_t ldp, uint8_t *pre_scales, void *ws, int64_t ws_bytes, void *stream);

/* With dz = dy * act'(z):  dx = dz W^T,  dw = x^T dz,  db = column sums of dz.
 * dx (T x K), dw (K x N contiguous) and db (N) may each be NULL.  With
 * accumulate != 0 dw and db are added to (dx is not).  x and w are the
 * forward call's; x may be NULL without dw, w without dx.  pre is z as the
 * forward call wrote it; it is ignored, and may be NULL, for RAR_ACT_NONE.
 * With x_scales, x holds the codes of an 8-bit checkpoint of x (ldx ignored),
 * with pre_scales pre holds those of z.  dz is rounded to the layer's type
 * for the two products; db sums it unrounded.  The residual's gradient is dy. */
rar_status rar_linear_backward(rar_linear_t plan, int64_t T, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                               const uint8_t *x_scales, const void *w, const void *pre, int64_t ldp,
                               const uint8_t *pre_scales, void *dx, int64_t lddx, void *dw, void *db, int accumulate,
                               void *ws, int64_t ws_bytes, void *stream);

/* An 8-bit checkpoint of a T x D matrix: e4m3 codes, T rows of *pitch bytes (D
 * rounded up to whole groups of RAR_CKPT_GROUP; the codes behind D are zero),
 * and one scale byte a group, T rows of *groups bytes. */
rar_status rar_ckpt_size(int64_t D, int64_t *pitch, int64_t *groups);

/* For every group of a row: e is the smallest exponent >= -126 with max|x| <=
 * 448 * 2^e over the group's finite values, the scale byte e + 127, and each
 * code x / 2^e rounded to the nearest e4m3 value (ties to even).  NaN and
 * infinities become NaN.  x is T x D with leading dimension ldx; codes must be
 * 16-byte aligned (RAR_EALIGN). */
rar_status rar_ckpt_store(int64_t T, int64_t D, rar_dtype dtype, const void *x, int64_t ldx, uint8_t *codes,
                          uint8_t *scales, void *stream);

/* y = act(code * 2^(scale - 127)), T x D with leading dimension ldy: the stored
 * activation again, or the activation function of a stored z.  (A stored value
 * may have rounded up to 2^128: it loads as infinity.) */
rar_status rar_ckpt_load(int64_t T, int64_t D, rar_dtype dtype, const uint8_t *codes, const uint8_t *scales,
                         rar_act act, void *y, int64_t ldy, void *stream);

/* ---------------------------------------------------------------------- */
/* Between the linear layers and behind them: the norms around a block,     */
/* dropout, cross attention and the loss.  The rules of the operators above */
/* on matrices, leading dimensions, overlap, workspaces, capture and        */
/* numerics hold here too.  Matrices need element alignment only.           */
/* Exponentials under 2^-126 count as zero.                                 */
/* ---------------------------------------------------------------------- */

/* ---- the norms before and after a block, with its gate and residual ---- */

typedef struct rar_norm_s *rar_norm_t;

typedef enum {
    RAR_NORM_NONE = 0,  /* v itself; its weight and bias are ignored */
    RAR_NORM_LAYER = 1, /* w (v - mean) / sqrt(var + eps) + b, var = mean of (v - mean)^2 */
    RAR_NORM_RMS = 2    /* w v / sqrt(mean of v^2 + eps) + b */
} rar_norm_kind;

/* What stands between two blocks of D columns: `post` norms a block's output,
 * `pre` the next block's input.  eps > 0.  Host memory only, immutable, any
 * number of threads and streams. */
rar_status rar_norm_plan(int64_t D, rar_dtype dtype, rar_norm_kind post, rar_norm_kind pre, float eps,
                         rar_norm_t *out);

rar_status rar_norm_destroy(rar_norm_t plan);

/* Workspace of a backward call on T rows; it serves calls on fewer rows too. */
rar_status rar_norm_workspace(rar_norm_t plan, int64_t T, int64_t *bytes);

/* n = post(o),  h = a x + s (gate . n),  u = pre(h), all T x D.
 * x is the residual stream, o the block's output or NULL (h = a x: the norm
 * before the first block).  gate and the norms' weights and biases are vectors
 * of D or NULL (gate and weights one, biases zero).  h may be x itself, or NULL
 * when only u is wanted; u may be NULL.  u is the norm of the unrounded h.
 * T == 0 is a no-op. */
rar_status rar_norm_forward(rar_norm_t plan, int64_t T, const void *x, int64_t ldx, const void *o, int64_t ldo,
                            const void *post_w, const void *post_b, const void *gate, float a, float s,
                            const void *pre_w, const void *pre_b, void *h, int64_t ldh, void *u, int64_t ldu,
                            void *stream);

/* The gradients, from o and h as the forward call read and wrote them (the
 * statistics are made again from the rows, nothing else is kept):
 *   g = dh + pre'(du; h),  dx = a g,  do = post'(s gate . g; o)
 *   dpre_w = sum du . h^, dpre_b = sum du, dgate = sum s g . n,
 *   dpost_w = sum s gate . g . o^, dpost_b = sum s gate . g   (sums over rows,
 *   of the unrounded g; h^ and o^ the normalised rows without weight and bias)
 * dh, the gradient that reaches h from further on, may be NULL (zero), and so
 * may du; of a plan with RAR_NORM_NONE before the block pre(h) is h.  Every
 * output may be NULL.  With o NULL there are no do, dgate and dpost_* (they
 * must be NULL).  dpost_* need a post norm, dpre_* a pre norm (RAR_EINVAL).  dx
 * may be dh itself and do may be o itself.  With accumulate != 0 the five
 * vectors are added to (dx and do are not). */
rar_status rar_norm_backward(rar_norm_t plan, int64_t T, const void *dh, int64_t lddh, const void *du, int64_t lddu,
                             const void *o, int64_t ldo, const void *h, int64_t ldh, const void *post_w,
                             const void *post_b, const void *gate, float a, float s, const void *pre_w, void *dx,
                             int64_t lddx, void *d_o, int64_t lddo, void *dpost_w, void *dpost_b, void *dgate,
                             void *dpre_w, void *dpre_b, int accumulate, void *ws, int64_t ws_bytes, void *stream);

/* ---- dropout ------------------------------------------------------------ */

/* y = r + keep . x / (1 - p), T x D; r NULL stands for zero.  The mask is a
 * function of its place, the seed and the step, and is never stored: element
 * (t, c) is kept when the 16-bit draw c % 8 of Philox4x32-10 (Salmon et al.,
 * 2011) with key (seed low, seed high) and counter (g low, g high, step low,
 * step high), g = t * ceil(D / 8) + c / 8, is at least round(65536 p).  (Draw i
 * is the half i % 2, lower first, of word i / 2.)  1 - p is taken as kept draws
 * over 65536, so the mean is exact; p = 1 keeps nothing.  A dropped element
 * counts as zero whatever it holds.  step is one int64 on the device (a captured
 * call reads it in every replay) or NULL for zero.  The backward pass is the
 * same call on dy without r.  y may be x or r itself.  0 <= p <= 1.  T == 0 is a
 * no-op. */
rar_status rar_dropout(int64_t T, int64_t D, rar_dtype dtype, float p, uint64_t seed, const int64_t *step,
                       const void *x, int64_t ldx, const void *r, int64_t ldr, void *y, int64_t ldy, void *stream);

/* ---- cross attention ---------------------------------------------------- */

typedef struct rar_attn_s *rar_attn_t;

#define RAR_ATTN_MAX_WIDTH 128

/* Attention of H query heads of dh columns (1..RAR_ATTN_MAX_WIDTH) to an
 * encoder's states projected to Hkv key and value heads; Hkv divides H, and H /
 * Hkv neighbouring query heads share one.  H dh at most 2^20.  scale, 2^-100 to
 * 2^100, multiplies the scores.  Host memory only, immutable, any number of threads
 * and streams. */
rar_status rar_attn_plan(int64_t H, int64_t Hkv, int64_t dh, rar_dtype dtype, float scale, rar_attn_t *out);

rar_status rar_attn_destroy(rar_attn_t plan);

/* Workspaces of a forward and of a backward call on B sequences of Tq queries
 * and Tk keys, for matrices at any address and of any leading dimension.  B is at
 * most 65535, B Tq and B Tk at most 2^24; a launch's 2^32 lanes allow less than
 * 2^23 of B Hkv ceil(Tq H / (128 Hkv)) and of B H ceil(Tq / 64), and less than
 * 2^24 of B Hkv ceil(Tk / 128).  Either output may be NULL.  A forward call of at
 * most four rows a key head (Tq H / Hkv: a decoding step) reads its matrices as
 * they stand and needs no more than the parts that its keys are cut into.  Where
 * a query gives zero, ws may be NULL.  A workspace serves every call of fewer
 * sequences, queries or keys too. */
rar_status rar_attn_workspace(rar_attn_t plan, int64_t B, int64_t Tq, int64_t Tk, int64_t *forward_bytes,
                              int64_t *backward_bytes);

/* o = softmax(scale q k^T) v for every sequence and head.  q and o are B Tq rows
 * of H heads side by side, k and v B Tk rows of Hkv heads: what the linear layers
 * write.  qlen and klen are B int64 on the device or NULL (whole): of sequence b
 * the first qlen[b] queries and klen[b] keys count, taken into 0..Tq and 0..Tk.
 * What lies behind them is not used, whatever it holds.  o and lse of queries
 * behind qlen, and of queries that no key is left for (klen 0, or every score
 * -infinity), are zero and -infinity.  lse (B Tq x H binary32, contiguous, or
 * NULL) receives the logarithm of the sum of the scores' exponentials, which the
 * backward call reads.  bf16: the weights are rounded to bf16 for their product
 * with v, their sum is not.  B Tq == 0 is a no-op. */
rar_status rar_attn_forward(rar_attn_t plan, int64_t B, int64_t Tq, int64_t Tk, const void *q, int64_t ldq,
                            const void *k, int64_t ldk, const void *v, int64_t ldv, const int64_t *qlen,
                            const int64_t *klen, void *o, int64_t ldo, float *lse, void *ws, int64_t ws_bytes,
                            void *stream);

/* The gradients of q, k and v, given d_o and the forward call's inputs, o and
 * lse.  Rows of dq behind qlen and of dk and dv behind klen become zero, and so do
 * rows of dq of queries that no key is left for; shared heads' gradients are
 * summed in a fixed order.  (An infinity within the lengths counts as in the
 * formula: a weight of zero times an infinite key, query or d_o is NaN in the
 * gradient that it belongs to.)  dq, dk and dv may each be NULL.
 * bf16: weights and score gradients are rounded to bf16 for their products. */
rar_status rar_attn_backward(rar_attn_t plan, int64_t B, int64_t Tq, int64_t Tk, const void *d_o, int64_t lddo,
                             const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                             const int64_t *qlen, const int64_t *klen, const void *o, int64_t ldo, const float *lse,
                             void *dq, int64_t lddq, void *dk, int64_t lddk, void *dv, int64_t lddv, void *ws,
                             int64_t ws_bytes, void *stream);

/* ---- the loss ----------------------------------------------------------- */

#define RAR_LOGPROB_MAX_TOP 32

/* With z = scale * logits (T x V, 0 < scale <= 2^126) and p = softmax(z) of a row:
 *   logp[t]    = log p at targets[t]; zero for a target outside 0..V-1 (padding)
 *   entropy[t] = -sum p log p
 *   top_ids[t][k], top_logp[t][k], k < K: the K largest logits in falling order,
 *                ties to the lowest index, and their log probabilities
 * (T binary32, T binary32, T x K int64 and binary32, all contiguous; each may be
 * NULL, targets too when logp is).  0 <= K <= RAR_LOGPROB_MAX_TOP; K > 0 needs
 * top_ids and top_logp.  A logit of -infinity is masked: p = 0, and no
 * alternative; where fewer than K are left the rest are -1 and -infinity.  A row
 * that has nothing left gives logp -infinity and entropy zero.  A NaN or
 * +infinity in a row makes its log probabilities and entropy NaN (its
 * alternatives -1 and NaN).  T == 0 is a no-op. */
rar_status rar_logprob(int64_t T, int64_t V, rar_dtype dtype, const void *logits, int64_t ldz, float scale,
                       const int64_t *targets, float *logp, float *entropy, int K, int64_t *top_ids, float *top_logp,
                       void *stream);

/* The gradient of sum_t dlogp[t] logp[t] + dentropy[t] entropy[t] in the logits:
 *   dz[t][j] = scale (dlogp [j = target] - p (dlogp + dentropy (log p + entropy)))
 * dlogp and dentropy are T binary32 or NULL (zero); targets may be NULL without
 * dlogp.  dz may be the logits themselves.  logp and entropy, or NULL, receive
 * what rar_logprob gives: a loss whose dlogp is known beforehand (-1 / T of a
 * mean) needs this call only.  A row that has nothing left has a gradient of
 * zero.  dlogp of a padded target is ignored. */
rar_status rar_logprob_grad(int64_t T, int64_t V, rar_dtype dtype, const void *logits, int64_t ldz, float scale,
                            const int64_t *targets, const float *dlogp, const float *dentropy, float *logp,
                            float *entropy, void *dz, int64_t lddz, void *stream);

/* ---------------------------------------------------------------------- */

/* Static description of a status code; never NULL. */
const char *rar_strerror(rar_status s);

/* Library version as major*10000 + minor*100 + patch (0.2.0 = 200 adds
 * rar_rank_stride, 0.3.0 = 300 rar_rank_stride_tune, 0.4.0 = 400
 * rar_allreduce_ring_noalloc, 0.5.0 = 500 rar_rank_stride_tune_stats,
 * 0.6.0 = 600 rar_rank_stride_candidate and the wider stride search,
 * 0.7.0 = 700 rar_embed_*, rar_linear_* and rar_ckpt_*, 0.8.0 = 800
 * rar_norm_*, rar_dropout, rar_attn_* and rar_logprob*). */
int rar_version(void);

#ifdef __cplusplus
}
#endif

#endif /* RAR_H */
