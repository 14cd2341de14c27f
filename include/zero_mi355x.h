/*
 * zero_mi355x.h -- C ABI of the ZeRO partitioned mixed-precision Adam step on
 * one data-parallel rank's flat shard, for AMD Instinct MI355X (gfx950).
 *
 * The model state the pages fix (ZeRO paper card, section "Bottleneck"):
 * fp16 parameters and fp16 gradients plus fp32 master parameters, fp32
 * momentum and fp32 variance -- 16 bytes per parameter.  ZeRO partitions that
 * state across the Nd data-parallel ranks instead of replicating it (paper
 * card, "Method": stage 1 optimizer state, stage 2 gradients, stage 3
 * parameters).  One rank therefore steps only its own contiguous slice of n
 * parameters: this library is that step.
 *
 * The step is three calls, all asynchronous on one HIP stream, with no host
 * synchronisation between them:
 *   1. zero_flatten_bucket      pack per-layer fp16 gradient tensors into the
 *                               rank's contiguous gradient partition
 *                               (contiguous, defragmented buffers: paper card,
 *                               "Method", ZeRO-R paragraph);
 *   2. zero_shard_norm_overflow exact squared L2 norm + inf/NaN flag of that
 *                               partition, then the step decision (dynamic
 *                               loss scale, skip, clip factor, bias
 *                               corrections) kept in device memory;
 *   3. zero_shard_adam_step     one fused pass: unscale + clip + Adam with
 *                               bias correction and decoupled weight decay,
 *                               fp32 master/momentum/variance update and the
 *                               fp16 parameter copy (28 bytes per parameter).
 * zero_state_bytes gives the per-rank model-state bytes for each ZeRO stage.
 *
 * Two further forms of the same step:
 *   - fused: zero_flatten_norm_bucket computes the exact-norm partials while
 *     it flattens and zero_shard_decide folds them, so the norm needs no
 *     second pass over the partition;
 *   - gradient accumulation (the DeepSpeed article leaves gradient
 *     accumulation to the library): micro-batch fp16 gradients are added
 *     into an fp32 partition (zero_flatten_bucket with ZERO_F32, or the
 *     fused zero_flatten_norm_bucket_f32 for the last micro-batch), and the
 *     *_f32 reduction and update read that fp32 gradient (30 bytes per
 *     parameter in the update);
 *   - 1-bit Adam (DeepSpeed article): zero_onebit_step runs ordinary steps
 *     for a warm-up, then compresses the momentum to one bit per element
 *     with error feedback and updates with the frozen variance;
 *   - host step (ZeRO-Offload, in the DeepSpeed article: ZeRO-2 plus CPU
 *     memory): the fp32 master parameters, momentum and variance live in host
 *     memory and the CPU steps them (zero_host_*, zero_offload_step), with
 *     the fp16 gradient partition copied down and the fp16 parameters copied
 *     back up.
 *
 * Next to the step stand the layer operators that produce a block's small
 * parameter gradients: dropout whose mask is recomputed instead of stored,
 * layer norm with the gradients of its weights, and the two joined around a
 * residual sum (zero_dropout_*, zero_layernorm_*, zero_dropout_layernorm_*).
 * Their weight and bias gradients go to a per-layer tensor the flatten packs,
 * or straight to their place in the fp16 or fp32 partition.
 *
 * Conventions for every entry point:
 *   - pointers named dev_* or documented as device memory are HIP device
 *     pointers; everything else is host memory;
 *   - the caller owns and allocates every buffer; the library allocates
 *     nothing and keeps no pointer to a caller's buffer after a call
 *     returns.  Two exceptions, both owned by the library: a host context
 *     (zero_host_create: its worker threads and, after zero_offload_step,
 *     HIP events), and the fixed device array of
 *     zero_shard_norm_overflow_noalloc (4 KiB per GPU, held until the
 *     process ends);
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream);
 *     device work is enqueued there and the call returns without waiting;
 *   - return value: ZERO_OK (0) or a negative ZERO_E* code; argument errors
 *     are detected on the host before any device work is enqueued; a fault
 *     inside a kernel surfaces at the caller's next synchronisation;
 *   - calls on different streams with disjoint buffers may run concurrently;
 *     two calls that share a zero_step_state_t must be ordered on one stream.
 */
#ifndef ZERO_MI355X_H
#define ZERO_MI355X_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes --------------------------------------------------- */
#define ZERO_OK       0
#define ZERO_EINVAL  (-1)   /* null pointer, bad dtype/stage/hyperparameter */
#define ZERO_EALIGN  (-2)   /* a buffer is not aligned as required */
#define ZERO_ERANGE  (-3)   /* a size or segment is out of the allowed range */
#define ZERO_EHIP    (-4)   /* the HIP runtime refused a launch or a copy */
#define ZERO_ENOTSUP (-5)   /* the host CPU lacks an instruction set the host step needs */
#define ZERO_ENOMEM  (-6)   /* out of host memory */

/* Human-readable text for a status code (static storage; never NULL).
 * For ZERO_EHIP the text of the last HIP error seen by this thread. */
const char* zero_status_string(int code);

/* ---- element types of a flatten destination ------------------------- */
#define ZERO_F16 1          /* IEEE binary16, stored as uint16_t bit patterns */
#define ZERO_F32 2          /* IEEE binary32 */
#define ZERO_BF16 3         /* bfloat16 (layer operators only) */

/* One piece of a per-layer gradient tensor that lands in the partition:
 * count elements from src[src_off ...] go to dst[dst_off ...].
 * src is a DEVICE pointer to binary16 data; offsets and count are elements. */
typedef struct {
    const uint16_t* src;
    uint64_t src_off;
    uint64_t dst_off;
    uint64_t count;
} zero_segment_t;

/* Hyperparameters of one step (host struct, passed by pointer).
 * lr, beta1, beta2, eps, weight_decay: AdamW (Kingma & Ba 2015 with the
 *   decoupled decay of Loshchilov & Hutter 2019, schedule multiplier = lr);
 * max_grad_norm: clip threshold on the unscaled gradient norm, <= 0 = off;
 * backoff, growth, growth_interval, min_scale: dynamic loss scaling
 *   (Micikevicius et al. 2018) -- on an inf/NaN gradient the step is skipped
 *   and S <- max(S*backoff, min_scale); after growth_interval consecutive
 *   clean steps S <- S*growth (growth_interval <= 0: never grow). */
typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    double max_grad_norm;
    double backoff, growth, min_scale;
    int32_t growth_interval;
    int32_t reserved;
} zero_hparams_t;

/* Step state in DEVICE memory (128 bytes, 8-byte aligned).  Initialise it
 * with zero_step_state_init.  It carries the loss scaler and the Adam step
 * count between steps, and the last decision from zero_shard_norm_overflow to
 * zero_shard_adam_step.  The caller may copy it to the host to read it (after
 * synchronising the stream) and may save/restore it bytewise. */
typedef struct {
    /* carried from step to step */
    double   loss_scale;        /* S: gradients arrive multiplied by S */
    double   beta1_pow;         /* beta1^t, running binary64 product */
    double   beta2_pow;         /* beta2^t */
    int64_t  step;              /* t: applied (not skipped) steps */
    int32_t  good_steps;        /* clean steps since the last scale change */
    int32_t  skipped_total;     /* skipped steps so far */
    /* written by the last reduction (zero_shard_norm_overflow, its fp32
       form, or zero_shard_decide) */
    double   sumsq;             /* exact sum of squares of the scaled
                                   gradient, rounded once to binary64;
                                   +inf when overflow is set */
    double   grad_norm;         /* sqrt(sumsq) / S (unscaled norm); +inf on overflow */
    int32_t  overflow;          /* 1 if the gradient holds an inf or NaN */
    int32_t  skip;              /* 1 if this step is skipped (== overflow,
                                   or while wide_pending) */
    float    gmul;              /* fp32(coef / S): unscale and clip factor */
    float    bc1, bc2;          /* fp32(1 - beta1^t), fp32(1 - beta2^t) */
    float    lr, beta1, beta2;  /* fp32 hyperparameters of this step */
    float    omb1, omb2;        /* fp32(1 - beta1), fp32(1 - beta2) */
    float    eps, wd;
    uint32_t done_blocks;       /* internal arrival counter; 0 between calls */
    uint32_t wide_pending;      /* internal: 1 while an fp32 reduction waits
                                   for its wide pass (see
                                   zero_shard_norm_overflow_f32); 0 after it */
    uint64_t sumsq_units[2];    /* the exact sum in units of 2^-48 (low,
                                   high) when it is a whole number of them
                                   below 2^128 (always, for binary16
                                   gradients); otherwise both words are
                                   all ones */
} zero_step_state_t;

/* ---- model-state arithmetic (host only, no device work) ------------- */

/* Per-rank model-state bytes for a model of psi parameters over nd
 * data-parallel ranks, with k optimizer bytes per parameter (k = 12 for the
 * fp32 master, momentum and variance of mixed-precision Adam; paper card,
 * "Bottleneck").  A rank owns P = ceil(psi/nd) parameters.
 *   stage 0 (plain data parallel): (2 + 2 + k) * psi
 *   stage 1 (optimizer state):     4 * psi + k * P
 *   stage 2 (+ gradients):         2 * psi + (2 + k) * P
 *   stage 3 (+ parameters):        (2 + 2 + k) * P
 * (paper card, "Method": 4x, 8x and Nd-proportional reductions; "Evidence":
 * 1T parameters -> about 16 TB, about 16 GB per GPU over 1024 GPUs.)
 * Errors: ZERO_EINVAL (out_bytes NULL, nd == 0, stage not 0..3),
 *         ZERO_ERANGE (the result does not fit in 64 bits). */
int zero_state_bytes(uint64_t psi, uint32_t nd, uint32_t k, int stage, uint64_t* out_bytes);

/* Cut a segment list (sorted or not) to the destination window
 * [begin, end): every part of a segment whose dst range falls inside the
 * window is written to out (host array of cap entries), in input order.
 * This is how a partition is flattened in fixed-size buckets (paper card,
 * "Method": temporary buffers sized to balance memory and throughput).
 * Errors: ZERO_EINVAL (NULL pointers, begin > end), ZERO_ERANGE (more than
 * cap pieces; *out_n then holds the number needed). */
int zero_bucket_segments(const zero_segment_t* segs, uint32_t nsegs, uint64_t begin,
                         uint64_t end, zero_segment_t* out, uint32_t cap, uint32_t* out_n);

/* ---- device step ----------------------------------------------------- */

/* Enqueue the initialisation of a step state: loss_scale = initial_scale,
 * beta powers 1, step and all counters 0.  dev_state: device, 8-byte aligned.
 * Errors: ZERO_EINVAL (NULL, initial_scale not finite and > 0),
 *         ZERO_EALIGN, ZERO_EHIP. */
int zero_step_state_init(zero_step_state_t* dev_state, double initial_scale, void* stream);

/* Flatten: for each segment, dst[dst_off + i] <- src[src_off + i], i < count.
 *   dst_dtype ZERO_F16, accumulate 0: bit copy of the binary16 values;
 *   dst_dtype ZERO_F16, accumulate 1: dst = fp16(dst + src) (correctly
 *                                     rounded binary16 addition);
 *   dst_dtype ZERO_F32, accumulate 0: dst = fp32(src) (exact);
 *   dst_dtype ZERO_F32, accumulate 1: dst = dst + fp32(src) (binary32 add).
 * segs: HOST array of nsegs entries (the src pointers inside are device
 * pointers); dst: device, dst_len elements, 16-byte aligned.  Destination
 * elements no segment covers are not touched.  Segment destinations must not
 * overlap each other (the result of overlapping segments is unspecified).
 * Any number of segments; the library may split them over several launches.
 * Errors: ZERO_EINVAL (NULL dst/segs with nsegs > 0, NULL src, bad dtype),
 *         ZERO_ERANGE (dst_off + count > dst_len), ZERO_EALIGN (dst base or
 *         a src pointer not 2-byte aligned, dst base not 16-byte aligned),
 *         ZERO_EHIP. */
int zero_flatten_bucket(const zero_segment_t* segs, uint32_t nsegs, void* dst, uint64_t dst_len,
                        int dst_dtype, int accumulate, void* stream);

/* ---- fused flatten + norm (the norm without a second pass) ----------- */

/* Bytes of one per-workgroup partial of the exact sum (opaque contents). */
#define ZERO_NORM_PARTIAL_BYTES 16

/* Number of partials zero_flatten_norm_bucket writes for this segment list
 * (one per workgroup it launches; host only, no device work).  0 for NULL. */
uint64_t zero_flatten_norm_partials(const zero_segment_t* segs, uint32_t nsegs);

/* The fp16 flatten of zero_flatten_bucket (bit copy, or fp16 accumulate),
 * which also computes, for every value it stores, the exact square and the
 * inf/NaN test, and writes one partial per workgroup to partials[0 ..
 * zero_flatten_norm_partials(segs, nsegs)).  For a step flattened in several
 * buckets, give each call its own stretch of one partials buffer and fold all
 * of them with zero_shard_decide.  The norm so obtained covers exactly the
 * elements the segments write (the whole partition when the segments cover
 * it, as in a ZeRO shard; paper card, "Method": contiguous buffers).
 * dst: device binary16, dst_len elements, 16-byte aligned; partials: device,
 * 16-byte aligned, partials_capacity entries of ZERO_NORM_PARTIAL_BYTES.
 * Errors: those of zero_flatten_bucket, and ZERO_EINVAL (NULL partials),
 *         ZERO_EALIGN, ZERO_ERANGE (partials_capacity too small). */
int zero_flatten_norm_bucket(const zero_segment_t* segs, uint32_t nsegs, uint16_t* dst, uint64_t dst_len,
                             int accumulate, void* partials, uint64_t partials_capacity, void* stream);

/* The fp32 flatten of zero_flatten_bucket (dst = fp32(src), or with
 * accumulate dst = dst + fp32(src) in binary32), which also computes the
 * exact-norm partials of every fp32 value it stores, under the rules of
 * zero_shard_norm_overflow_f32.  Used for the last micro-batch of a
 * gradient-accumulation step: the partials it writes, folded by
 * zero_shard_decide, give exactly the decision zero_shard_norm_overflow_f32
 * takes on the finished partition.  It writes
 * zero_flatten_norm_partials(segs, nsegs) partials, like the fp16 form.
 * dst: device binary32, dst_len elements, 16-byte aligned; the rest as for
 * zero_flatten_norm_bucket.  Errors: as zero_flatten_norm_bucket. */
int zero_flatten_norm_bucket_f32(const zero_segment_t* segs, uint32_t nsegs, float* dst, uint64_t dst_len,
                                 int accumulate, void* partials, uint64_t partials_capacity, void* stream);

/* Several buckets of one step in one call: the same stores (and, with
 * partials, the same partials) as calling zero_flatten_bucket -- or
 * zero_flatten_norm_bucket / zero_flatten_norm_bucket_f32 when partials is
 * not NULL -- once per bucket, in order, each bucket's partials right after
 * the previous bucket's (paper card, "Method": the partition is one
 * contiguous buffer; the buckets are windows of it).  The first launch waits
 * for the work queued earlier on the stream, like any launch; the launches
 * between the first and the last are issued without the dispatch barrier,
 * so consecutive buckets overlap on the GPU instead of draining it between
 * them; the last keeps the barrier, so its completion implies every
 * earlier one's and anything queued or waiting on the stream after the call
 * (kernels, copies, events, synchronisation) sees all of them.  That is only safe
 * because no two buckets touch a common element: every segment's
 * destination range must be disjoint from every other's, and the call
 * checks it.
 * segs: HOST array of the buckets' segment lists, one after another;
 * bucket_nsegs: HOST array of nbuckets counts; dst: device, binary16 or
 * binary32 (dst_dtype), dst_len elements, 16-byte aligned; partials: NULL
 * (no norm) or device, 16-byte aligned, partials_capacity entries of
 * ZERO_NORM_PARTIAL_BYTES, at least zero_flatten_norm_partials(segs, total
 * segments) of them.  dst_dtype and accumulate as for zero_flatten_bucket.
 * Errors: those of zero_flatten_bucket and zero_flatten_norm_bucket;
 *         ZERO_EINVAL also for NULL bucket_nsegs with nbuckets > 0 and for
 *         two segments whose destination ranges overlap; ZERO_ERANGE for
 *         more than 2^32 - 1 segments in all; ZERO_ENOMEM if the host
 *         cannot allocate the overlap check's list.  No device work is
 *         queued when an argument error is returned. */
int zero_flatten_buckets(const zero_segment_t* segs, const uint32_t* bucket_nsegs, uint32_t nbuckets, void* dst,
                         uint64_t dst_len, int dst_dtype, int accumulate, void* partials,
                         uint64_t partials_capacity, void* stream);

/* Bytes of device workspace zero_shard_decide needs to fold `count` partials. */
size_t zero_decide_workspace_bytes(uint64_t count);

/* Folds `count` partials written by zero_flatten_norm_bucket into the
 * exact sum and overflow flag, then takes exactly the decision that
 * zero_shard_norm_overflow takes (same fields of dev_state, bit for bit).
 * Partials of zero_flatten_norm_bucket_f32 go to zero_shard_decide_f32:
 * folded here, a partition off the fast path (see
 * zero_shard_norm_overflow_f32) leaves the step pending and skipped with
 * the loss scale and counters untouched.
 * partials, workspace: device, 16-byte aligned; hp: host; workspace of at
 * least zero_decide_workspace_bytes(count).
 * Errors: as zero_shard_norm_overflow (ZERO_ERANGE: count > 2^30 or
 *         workspace too small). */
int zero_shard_decide(const void* partials, uint64_t count, const zero_hparams_t* hp,
                      zero_step_state_t* dev_state, void* workspace, size_t workspace_bytes, void* stream);

/* The decision over the partials of zero_flatten_norm_bucket_f32 calls that
 * together wrote the fp32 partition grad32[0..n): the fold of
 * zero_shard_decide, then the wide pass over grad32 when the fold left the
 * step pending.  The result is exactly zero_shard_norm_overflow_f32's on
 * the same partition, bit for bit.  grad32: device, 4-byte aligned (NULL
 * allowed when n = 0); the rest as zero_shard_decide.
 * Errors: those of zero_shard_decide, and ZERO_ERANGE (n > 2^40). */
int zero_shard_decide_f32(const void* partials, uint64_t count, const float* grad32, uint64_t n,
                          const zero_hparams_t* hp, zero_step_state_t* dev_state, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Bytes of device workspace zero_shard_norm_overflow needs for n elements
 * (per-block partial sums; fixed for a given n). */
size_t zero_norm_workspace_bytes(uint64_t n);

/* Reduce and decide.  Over the n binary16 gradient elements at grad16:
 *   overflow = 1 if any element has an all-ones exponent (inf or NaN);
 *   sumsq    = the exact sum of squares, rounded once to binary64
 *              (+inf on overflow);
 * then, from the state in dev_state and the hyperparameters in hp:
 *   overflow -> skip = 1, S <- max(S*backoff, min_scale), good_steps <- 0;
 *   otherwise -> skip = 0, t += 1, beta powers advance,
 *               grad_norm = sqrt(sumsq)/S,
 *               coef = grad_norm > max_grad_norm > 0 ? max_grad_norm/grad_norm : 1,
 *               gmul = fp32(coef/S), bc1/bc2 = fp32(1 - beta^t),
 *               good_steps += 1 and S <- S*growth every growth_interval.
 * All of it is written into dev_state for zero_shard_adam_step.  Result bits
 * do not depend on the launch configuration (the sum is exact).
 * grad16: device, 16-byte aligned; n may be 0; hp: host;
 * dev_state: device, 8-byte aligned, initialised by zero_step_state_init;
 * workspace: device, 16-byte aligned, >= zero_norm_workspace_bytes(n),
 * contents need no initialisation.
 * Errors: ZERO_EINVAL (NULL, hyperparameters out of range: lr < 0,
 *         beta not in [0,1), eps <= 0, weight_decay < 0, backoff not in
 *         (0,1], growth < 1, min_scale <= 0, any non-finite value),
 *         ZERO_EALIGN, ZERO_ERANGE (workspace too small, n > 2^40),
 *         ZERO_EHIP. */
int zero_shard_norm_overflow(const uint16_t* grad16, uint64_t n, const zero_hparams_t* hp,
                             zero_step_state_t* dev_state, void* workspace,
                             size_t workspace_bytes, void* stream);

/* zero_shard_norm_overflow without the workspace argument, for callers that
 * cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc).  Same reduction, same kernels,
 * same result bits and errors, except:
 *   - the per-workgroup partials live in a fixed device array inside the
 *     library (256 partials, 4 KiB), which each GPU the library runs on holds
 *     from the first call on that GPU until the process ends; its device
 *     address is looked up once per GPU, on that call, with that GPU current;
 *   - hence n <= 2^30 (ZERO_ERANGE above; the largest n whose grid of at
 *     most 256 workgroups fits the array);
 *   - every call on one GPU shares that array, and each call leaves its
 *     partials there: calls that overlap in time on one GPU (on different
 *     streams, or from different host threads) race and give undefined
 *     results -- order them on one stream.  Nothing in the array needs to
 *     start at zero (every partial a call reads, the same call wrote).
 * The call allocates nothing (no hipMalloc/hipFree, no allocating library
 * routine).  The stream must belong to the current device. */
int zero_shard_norm_overflow_noalloc(const uint16_t* grad16, uint64_t n, const zero_hparams_t* hp,
                                     zero_step_state_t* dev_state, void* stream);

/* Reduce and decide over an fp32 gradient partition (gradient
 * accumulation: a binary32 sum of micro-batch fp16 gradients).
 *   overflow = 1 if any element is inf or NaN;
 *   sumsq    = the exact sum of the squares of all n values, rounded once
 *              to binary64 (any finite binary32 values);
 * then the same decision as zero_shard_norm_overflow.  Two kernels: the
 * fast reduction sums exactly when every value is a multiple of 2^-24 below
 * 2^24 in magnitude (true of any binary32 sum of at most 256 binary16
 * values); when one is not, it leaves the decision pending
 * (wide_pending = 1) and the wide pass that follows sums the squares of any
 * binary32 values exactly (slower: LDS-atomic bound) and decides.  On the
 * fast path the wide pass returns at once.  sumsq_units holds the exact sum
 * in 2^-48 units when it is a whole number of them below 2^128, else all
 * ones.  grad32: device, 16-byte aligned; everything else as for
 * zero_shard_norm_overflow, including the workspace size
 * (zero_norm_workspace_bytes(n), which covers both kernels) and the
 * errors. */
int zero_shard_norm_overflow_f32(const float* grad32, uint64_t n, const zero_hparams_t* hp,
                                 zero_step_state_t* dev_state, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* The fused element update, in binary32 with one rounding per operation and
 * this order (unless dev_state says skip, in which case nothing is written):
 *   g  = fp32(grad16[i]) * gmul
 *   m  = beta1*m32[i] + omb1*g
 *   v  = beta2*v32[i] + omb2*(g*g)
 *   u  = (m/bc1) / (sqrt(v/bc2) + eps) + wd*p32[i]
 *   p  = p32[i] - lr*u
 *   m32[i] = m; v32[i] = v; p32[i] = p; p16[i] = fp16(p) (round to nearest even)
 * It reads 2 + 12 bytes and writes 12 + 2 bytes per parameter.
 * All five arrays: device, n elements, 16-byte aligned, index-aligned with
 * each other and with the grad16 the decision was made on; n may be 0.
 * Placement (performance only): the five arrays are streamed together; on
 * MI355X the update is 1-5% faster when they share one allocation with array
 * k (p32, m32, v32, grad16, p16) starting at a 2 MiB boundary plus k * 64 KiB,
 * as the Python binding's StateArena lays them out.
 * dev_state: as left by zero_shard_norm_overflow (read only here).
 * Errors: ZERO_EINVAL (NULL), ZERO_EALIGN, ZERO_ERANGE (n above about 2^42:
 *         more than 2^31 - 1 workgroups of 2048 parameters), ZERO_EHIP. */
int zero_shard_adam_step(uint16_t* p16, float* p32, float* m32, float* v32,
                         const uint16_t* grad16, uint64_t n,
                         const zero_step_state_t* dev_state, void* stream);

/* The same update reading an fp32 gradient (gradient accumulation):
 *   g = grad32[i] * gmul, then exactly as zero_shard_adam_step.
 * It reads 4 + 12 bytes and writes 12 + 2 bytes per parameter (30).
 * dev_state: as left by zero_shard_norm_overflow_f32, or by
 * zero_shard_decide over zero_flatten_norm_bucket_f32 partials.
 * grad32: device, n elements, 16-byte aligned; the rest and the errors as
 * for zero_shard_adam_step. */
int zero_shard_adam_step_f32(uint16_t* p16, float* p32, float* m32, float* v32,
                             const float* grad32, uint64_t n,
                             const zero_step_state_t* dev_state, void* stream);

/* ---- 1-bit Adam, compression stage ------------------------------------ */

/* State of the compression stage in DEVICE memory (72 bytes, 8-byte
 * aligned; initialise with zero_onebit_state_init).  After each step it
 * holds the two scales and their exact sums. */
typedef struct {
    float    scale_w, scale_s;  /* worker and server scales of the last step */
    double   sumsq_w, sumsq_s;  /* the exact sums of squares, rounded once to binary64 */
    int32_t  qexp_w, qexp_s;    /* diagnostics of the fast windowed sums: the */
    uint32_t done_blocks;       /*   final window's unit 2^qexp; internal
                                     arrival counter (0 between calls) */
    uint32_t wide_pending;      /* internal: bit 0 / bit 1 while the worker /
                                   server scale waits for its wide pass */
    uint64_t units_w[2];        /* the windowed sums as integers of 2^qexp */
    uint64_t units_s[2];        /* units (low, high), before the wide pass */
} zero_onebit_state_t;

/* Enqueue the zeroing of a compression-stage state.
 * Errors: ZERO_EINVAL (NULL), ZERO_EALIGN, ZERO_EHIP. */
int zero_onebit_state_init(zero_onebit_state_t* dev_onebit, void* stream);

/* Bytes of device workspace zero_onebit_step needs for n elements. */
size_t zero_onebit_workspace_bytes(uint64_t n);

/* One step of 1-bit Adam (the DeepSpeed article: 1-bit Adam cuts
 * communication up to 5x with Adam-like convergence; the algorithm is Tang
 * et al. 2021, Algorithm 1), after zero_shard_decide (or
 * zero_shard_norm_overflow) has decided it.  The device chooses the stage
 * from the applied-step count in dev_state, so the host never reads it back
 * and one captured graph can cross from one stage to the other:
 *   warm-up (the applied steps before this one number fewer than `warmup`,
 *   i.e. dev_state->step <= warmup after the decision): the ordinary update
 *   of zero_shard_adam_step, which also builds the variance v32;
 *   compression stage (otherwise): v32 frozen, and with the decision in
 *   dev_state (gmul, beta1, lr, eps, wd), on this rank, its own server:
 *     g = fp32(grad16)*gmul;  m = beta1*m + (1-beta1)*g
 *     x = m + err_w;  s_w = S(x);  bits_w = sgn(x);  err_w = x - s_w*sgn(x)
 *     u = s_w*sgn(x) + err_s;  s_s = S(u);  bits_s = sgn(u)
 *     m = s_s*sgn(u);  err_s = u - m
 *     p = p - lr*(m/(sqrt(v)+eps) + wd*p);  p16 = fp16(p)
 * A skipped step (overflow) changes nothing, errors and bits included; the
 * kernels of the stage not taken return at once, before any load.
 * sgn(x) = +1 for x >= 0 (zeros too), -1 otherwise; bit k of byte j of a
 * bits array is element 8j+k, 1 for +1.  S(x) = fp32(sqrt(sum/n)) with the
 * sum of squares exact and rounded once to binary64.  The fast sum works in
 * windows: each workgroup of 4096 elements rounds its squares to multiples
 * of 2^(2E_b-80), 2^E_b <= its max|x| < 2^(E_b+1), and a fold moves those
 * integer sums onto the window of the largest E_b, rounding each to the
 * nearest unit; it keeps the result when the binary64 rounding is the same
 * at both ends of the error interval this leaves, and otherwise hands the
 * sum to a wide pass that is exact for any binary32 values.
 * Every elementwise operation is one binary32 operation in the order
 * above.  Results do not depend on the launch configuration.
 * p16, p32, m32, v32, err_w, err_s, grad16: device, n elements, 16-byte
 * aligned; bits_w, bits_s: device, (n+7)/8 bytes; workspace: device,
 * 256-byte aligned, >= zero_onebit_workspace_bytes(n).
 * Errors: ZERO_EINVAL (NULL, warmup < 0), ZERO_EALIGN, ZERO_ERANGE
 *         (n > 2^40, workspace too small), ZERO_EHIP. */
int zero_onebit_step(uint16_t* p16, float* p32, float* m32, float* v32, float* err_w, float* err_s,
                     const uint16_t* grad16, uint64_t n, uint8_t* bits_w, uint8_t* bits_s,
                     const zero_step_state_t* dev_state, zero_onebit_state_t* dev_onebit, int64_t warmup,
                     void* workspace, size_t workspace_bytes, void* stream);

/* ---- host step (ZeRO-Offload form) ----------------------------------- */

/* A host context: a pool of worker threads (and, once zero_offload_step has
 * run, the HIP events it pipelines with).  Calls that share a context must
 * not overlap; different contexts are independent.  Every zero_host_* call
 * runs on the calling thread plus the pool and returns when it is done. */
typedef struct zero_host_ctx zero_host_ctx_t;

/* Create a context with `threads` workers in all (the calling thread counts
 * as one; <= 0: every CPU this process may run on).
 * Errors: ZERO_EINVAL (out NULL), ZERO_ENOTSUP (the CPU lacks AVX-512 F, BW,
 *         VL, DQ, F16C or FMA), ZERO_ERANGE (threads > 1024), ZERO_ENOMEM. */
int zero_host_create(int threads, zero_host_ctx_t** out);

/* Stop the workers and free the context (NULL is allowed). */
void zero_host_destroy(zero_host_ctx_t* ctx);

/* Number of workers of a context (0 for NULL). */
int zero_host_threads(const zero_host_ctx_t* ctx);

/* zero_step_state_init for a step state in HOST memory (no device work).
 * Errors: ZERO_EINVAL (NULL, initial_scale not finite and > 0). */
int zero_host_state_init(zero_step_state_t* state, double initial_scale);

/* zero_shard_norm_overflow on the CPU: over the n binary16 values at grad16
 * (host memory, any alignment), the same overflow test and the same exact
 * sum of squares, then the same decision into the HOST step state, bit for
 * bit (one source for the decision; the sum is exact on both).
 * Errors: ZERO_EINVAL (NULL, hyperparameters out of range as for
 *         zero_shard_norm_overflow). */
int zero_host_norm_overflow(zero_host_ctx_t* ctx, const uint16_t* grad16, uint64_t n, const zero_hparams_t* hp,
                            zero_step_state_t* state);

/* zero_shard_adam_step on the CPU: the same element update, each operation
 * one binary32 round-to-nearest-even operation in the same order, the fp16
 * copy rounded to nearest even -- bit-identical to the device kernel.  All
 * arrays are host memory of n elements; any alignment works, and when p32,
 * m32, v32 are 64-byte aligned and p16 32-byte aligned at the same index the
 * stores bypass the caches.  Nothing is written when state->skip is set.
 * Errors: ZERO_EINVAL (NULL). */
int zero_host_adam_step(zero_host_ctx_t* ctx, uint16_t* p16, float* p32, float* m32, float* v32,
                        const uint16_t* grad16, uint64_t n, const zero_step_state_t* state);

/* The whole offloaded step for a partition whose fp16 gradient and fp16
 * parameters live on the device and whose fp32 master parameters, momentum
 * and variance live in host memory.  Two ways to decide:
 *   dev_state NULL: the CPU decides.  dev_grad16 is copied to host_grad16
 *     in chunks on `stream`, each chunk reduced on the CPU as soon as it has
 *     landed; then the decision into the host `state` (as
 *     zero_host_norm_overflow; `hp` is required);
 *   dev_state given: the device has already decided on `stream`
 *     (zero_shard_decide over zero_flatten_norm_bucket partials, or
 *     zero_shard_norm_overflow), bit-identically to the CPU's decision.  The
 *     128-byte device state is copied into `state` first, then the gradient
 *     chunks, and the CPU updates each chunk as soon as it has landed
 *     (`hp` is not used and may be NULL).
 * Unless the step is skipped, each chunk is updated on the CPU (as
 * zero_host_adam_step, fp16 parameters into host_p16) and its copy
 * host_p16 -> dev_p16 is enqueued on `stream` right away.  The call returns
 * once every update is done; copies may still be in flight on `stream`
 * (later work on `stream` sees them; the host must not touch host_grad16
 * or host_p16 before they complete).  host_grad16, host_p16 and `state`
 * should be pinned host memory (hipHostMalloc) for the copies to overlap.
 * chunk_elems is the largest chunk; the first chunks ramp up from
 * chunk_elems/16 (at least 64) by doubling and the last ones ramp down the
 * same way, so the CPU starts once a small chunk has landed and the last
 * parameters go up right after their update; every chunk boundary but n is a
 * multiple of 64 elements.  The results do not depend on the chunking.
 * dev_grad16, dev_p16, dev_state: device; the other arrays host memory.
 * Errors: ZERO_EINVAL (NULL, hyperparameters out of range), ZERO_EALIGN
 *         (chunk_elems 0 or not a multiple of 64, dev_state not 8-byte
 *         aligned), ZERO_ERANGE (n above 4096 * chunk_elems), ZERO_EHIP (a copy,
 *         event or synchronisation failed). */
int zero_offload_step(zero_host_ctx_t* ctx, const uint16_t* dev_grad16, uint16_t* dev_p16, uint16_t* host_grad16,
                      uint16_t* host_p16, float* p32, float* m32, float* v32, uint64_t n,
                      const zero_hparams_t* hp, zero_step_state_t* state, const zero_step_state_t* dev_state,
                      uint64_t chunk_elems, void* stream);

/* A streaming copy of `bytes` host bytes (dst, src 64-byte aligned, bytes a
 * multiple of 64) on the context's workers: the host memory bandwidth
 * reference next to the host step.  Errors: ZERO_EINVAL, ZERO_EALIGN. */
int zero_host_stream_copy(zero_host_ctx_t* ctx, void* dst, const void* src, uint64_t bytes);

/* ---- layer operators ---------------------------------------------------
 *
 * The operators below work on matrices of `rows` rows (tokens) of `cols`
 * elements (the hidden size), ld elements from one row to the next: element
 * (i, j) of x is x[i * ld_x + j].  Common to all of them:
 *   - dtype is the type of every matrix: ZERO_F16, ZERO_BF16 or ZERO_F32.
 *     vec_dtype is the type of w, b and bias, grad_dtype that of dw, db and
 *     dbias: dtype or ZERO_F32, and not looked at when all of them are NULL;
 *   - arithmetic and sums are binary32; a stored value is rounded once, to
 *     nearest even;
 *   - matrices and vectors are device memory, aligned to their element and no
 *     more (a vector may be a slice of the flat partition at any offset); ld
 *     >= cols, and the elements between two rows are neither read nor written
 *     (one row: ld is not looked at);
 *   - an output matrix may be one of the call's input matrices (the same
 *     address and ld); two outputs must differ, and any other overlap of an
 *     output with another argument gives undefined results;
 *   - the stream belongs to the current device, and so does every pointer;
 *   - rows may be 0 (then the row sums dw, db, dbias are sums of nothing: 0, or
 *     with accumulate left as they are);
 *   - results do not depend on timing: equal calls give equal bits.
 * Errors of all of them: ZERO_EINVAL (a required pointer NULL with rows > 0,
 * a bad type, two equal outputs (mean and rstd among them), eps not finite and
 * > 0 in binary32, p not in [0, 1]), ZERO_EALIGN, ZERO_ERANGE (rows > 2^40,
 * cols > 2^30, cols = 0 for a norm, with rows > 1 ld < cols, ld > 2^50 or
 * rows * ld > 2^56, a workspace too small), ZERO_EHIP. */

/* The state of the dropout generator in DEVICE memory (16 bytes, 8-byte
 * aligned).  The mask of a call is a function of (seed, step, site, rows'
 * index, column, cols): keep it unchanged between a forward pass and its
 * backward (or recomputed forward) pass, and advance it after each backward
 * pass, so once per micro-batch where a training step accumulates over
 * several: two that share a step share their masks too.  For the same reason
 * ranks that train on different data need different seeds.  Being in device
 * memory, it lets a captured graph draw new masks at every replay. */
typedef struct {
    uint64_t seed;
    uint32_t step;              /* forward/backward passes so far */
    uint32_t reserved;          /* 0 */
} zero_rng_t;

/* Enqueue the initialisation of a generator: this seed, step 0.
 * Errors: ZERO_EINVAL (NULL), ZERO_EALIGN, ZERO_EHIP. */
int zero_rng_init(zero_rng_t* dev_rng, uint64_t seed, void* stream);

/* Enqueue step += 1 (modulo 2^32).  Errors: as zero_rng_init. */
int zero_rng_advance(zero_rng_t* dev_rng, void* stream);

/* Dropout, with the bias before it and the residual sum after it:
 *   out = residual + D(x + bias),   D(v) = kept ? v * s : 0
 * (residual and bias NULL: left out).  The mask is never stored: it is the
 * counter-based generator Philox4x32-10 (Salmon et al. 2011) with
 *   key     = (seed low, seed high),
 *   counter = (g low, g high, site, step), g = i * ceil(cols / 8) + j / 8,
 * of whose 128 output bits element (i, j) takes the 16-bit word j % 8 (low
 * half of an output first).  The element is dropped when that word is below
 *   t = floor(65536 p + 1/2);   s = fp32(65536 / (65536 - t)),
 * so the drop probability is p to the nearest 2^-16 and the expectation is
 * kept exactly for it; t = 0 draws nothing (dev_rng may then be NULL), t =
 * 65536 drops everything.  A dropped element is 0 whatever it held, inf and
 * NaN too.  site tells apart the dropouts of one pass (layer and place).
 * dev_rng: device, 8-byte aligned, read when the kernel runs. */
int zero_dropout_fwd(void* out, uint64_t ld_out, const void* x, uint64_t ld_x, const void* residual,
                     uint64_t ld_residual, const void* bias, int bias_dtype, uint64_t rows, uint64_t cols, int dtype,
                     double p, const zero_rng_t* dev_rng, uint32_t site, void* stream);

/* Bytes of device workspace the backward passes below need for this shape
 * (any of them, any type); 0 for an empty or refused shape. */
size_t zero_layer_workspace_bytes(uint64_t rows, uint64_t cols);

/* The backward pass of zero_dropout_fwd for the same generator state, site
 * and p:  dx = D(dout);  dbias[j] = sum over the rows of D(dout) (binary32,
 * of the unrounded values), stored, or with accumulate added to what dbias
 * holds, then rounded once to grad_dtype.  dbias may be NULL (no sum; then
 * no workspace is needed).  The residual's gradient is dout itself.
 * workspace: device, 16-byte aligned, >= zero_layer_workspace_bytes(rows,
 * cols); contents need no initialisation; calls that share it must be
 * ordered. */
int zero_dropout_bwd(void* dx, uint64_t ld_dx, void* dbias, int grad_dtype, int accumulate, const void* dout,
                     uint64_t ld_dout, uint64_t rows, uint64_t cols, int dtype, double p, const zero_rng_t* dev_rng,
                     uint32_t site, void* workspace, size_t workspace_bytes, void* stream);

/* Layer norm (Ba, Kiros and Hinton 2016) over each row:
 *   mean = sum(x) / cols,  var = sum((x - mean)^2) / cols,
 *   rstd = 1 / sqrt(var + eps),  y = (x - mean) * rstd * w + b
 * (w NULL: 1; b NULL: 0).  mean and rstd (binary32, one per row, kept for the
 * backward pass) may be NULL. */
int zero_layernorm_fwd(void* y, uint64_t ld_y, float* mean, float* rstd, const void* x, uint64_t ld_x, const void* w,
                       const void* b, int vec_dtype, uint64_t rows, uint64_t cols, int dtype, double eps,
                       void* stream);

/* The backward pass of zero_layernorm_fwd, from the mean and rstd it stored:
 *   h = (x - mean) * rstd,  g = dy * w,
 *   dx = rstd * (g - sum(g)/cols - h * sum(g*h)/cols) + dres
 *   dw[j] = sum over the rows of dy * h,  db[j] = sum over the rows of dy
 * dres (NULL: none) is the gradient that reaches x past the norm (the residual
 * stream of a pre-norm block).  dw and db may be NULL; they are stored, or
 * with accumulate added to what is there, then rounded once to grad_dtype: a
 * binary16 gradient too large for it becomes inf, which the step's decision
 * finds.  workspace: as for zero_dropout_bwd (always needed). */
int zero_layernorm_bwd(void* dx, uint64_t ld_dx, void* dw, void* db, int grad_dtype, int accumulate, const void* dy,
                       uint64_t ld_dy, const void* dres, uint64_t ld_dres, const void* x, uint64_t ld_x,
                       const float* mean, const float* rstd, const void* w, int vec_dtype, uint64_t rows,
                       uint64_t cols, int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* The two joined, as a transformer block has them between two sublayers:
 *   r = residual + D(x + bias)  (rounded to dtype and stored),
 *   y = layer norm of that r.
 * Equal to zero_dropout_fwd followed by zero_layernorm_fwd on its output, in
 * one pass.  residual and bias may be NULL. */
int zero_dropout_layernorm_fwd(void* r, uint64_t ld_r, void* y, uint64_t ld_y, float* mean, float* rstd, const void* x,
                               uint64_t ld_x, const void* residual, uint64_t ld_residual, const void* bias,
                               const void* w, const void* b, int vec_dtype, uint64_t rows, uint64_t cols, int dtype,
                               double eps, double p, const zero_rng_t* dev_rng, uint32_t site, void* stream);

/* The backward pass of zero_dropout_layernorm_fwd, from the r, mean and rstd
 * it stored.  dy is y's gradient, dres (NULL: none) the gradient that reaches
 * r from where else it is used:
 *   e  = rstd * (g - sum(g)/cols - h * sum(g*h)/cols) + dres  (as above, at r)
 *   dr = e (the residual's gradient),  dx = D(e),
 *   dw, db as in zero_layernorm_bwd,  dbias[j] = sum over the rows of D(e)
 * with D of the unrounded e.  dw, db and dbias may be NULL.  workspace: as
 * for zero_layernorm_bwd. */
int zero_dropout_layernorm_bwd(void* dx, uint64_t ld_dx, void* dr, uint64_t ld_dr, void* dw, void* db, void* dbias,
                               int grad_dtype, int accumulate, const void* dy, uint64_t ld_dy, const void* dres,
                               uint64_t ld_dres, const void* r, uint64_t ld_r, const float* mean, const float* rstd,
                               const void* w, int vec_dtype, uint64_t rows, uint64_t cols, int dtype, double p,
                               const zero_rng_t* dev_rng, uint32_t site, void* workspace, size_t workspace_bytes,
                               void* stream);

/* ---- attention operators -------------------------------------------------
 *
 * The attention side of a transformer block, beside the layer operators: the
 * norms of queries and keys with the position rotation, and causal attention
 * with a window, first tokens that stay visible and a learned bias.  Common to
 * them:
 *   - tokens are packed: those of a batch's sequences one after another.  An
 *     activation is tokens x heads x dim elements, (i, h, d) at
 *     i * ld + h * hs + d: ld and hs of at least dim take a slice of a joint
 *     projection's output, heads before or after queries, keys and values;
 *   - the elements between are neither read nor written;
 *   - arithmetic and sums are binary32, a stored value is rounded once, to
 *     nearest even; what the matrix units take in between is named below;
 *   - pointers are device memory, aligned to their element and no more;
 *   - the stream belongs to the current device, and so does every pointer;
 *   - tokens may be 0 (weight gradients are then sums of nothing: 0, or with
 *     accumulate left as they are);
 *   - results do not depend on timing: equal calls give equal bits. */

/* The norms of queries and keys over each head, with the position rotation in
 * the same pass.  For each token and head of x (q: tokens x heads x dim, k:
 * tokens x kv_heads x dim), over the head's elements:
 *   rstd = 1 / sqrt(mean(x^2) + eps),  u = x * rstd * w  (w NULL: 1),
 *   out = u with its first `rot` elements turned in pairs: for the pair p <
 *   rot / 2 with the position's (cos, sin),
 *     (a, b) -> (a cos - b sin, b cos + a sin),
 *   elements (p, p + rot / 2), or with interleaved (2p, 2p + 1).
 * The sum of squares is binary32's: of 2^128 or more it makes rstd 0.
 * dtype: ZERO_F16, ZERO_BF16 or ZERO_F32; wq and wk: dim elements of vec_dtype,
 * dtype or ZERO_F32.  dim even and at most 256, rot even and at most dim (0:
 * no rotation, table not looked at).  kv_heads may be 0 (k, k_out and wk NULL).
 * table: device, table_rows x rot / 2 x (cos, sin) binary32, 16-byte aligned
 * (zero_rope_table).  A token's position is dev_positions[i] (device), or where
 * that is NULL i mod period (period 0: i); one not in the table gives NaN.
 * An output may be its own input (the same address, ld and hs).
 * Errors: ZERO_EINVAL (NULL, a type, heads = 0, dim or rot odd or 0, rot > dim,
 *         eps not finite and > 0 in binary32, rot without a table, q_out ==
 *         k_out, k's arguments without kv_heads), ZERO_EALIGN, ZERO_ERANGE (dim
 *         > 256, more than 2^30 tokens or table rows, 65535 heads or 2^34 heads
 *         of all tokens, ld or hs < dim or > 2^50, an extent > 2^56), ZERO_EHIP. */
int zero_qk_norm_rope_fwd(void* q_out, uint64_t ld_q_out, uint64_t hs_q_out, void* k_out, uint64_t ld_k_out,
                          uint64_t hs_k_out, const void* q, uint64_t ld_q, uint64_t hs_q, const void* k, uint64_t ld_k,
                          uint64_t hs_k, const void* wq, const void* wk, int vec_dtype, uint64_t tokens, uint32_t heads,
                          uint32_t kv_heads, uint32_t dim, int dtype, double eps, const float* table,
                          uint64_t table_rows, uint32_t rot, int interleaved, const int32_t* dev_positions,
                          uint64_t period, void* stream);

/* Bytes of device workspace zero_qk_norm_rope_bwd needs (any type and rot); 0
 * for no tokens or a refused shape. */
size_t zero_qk_workspace_bytes(uint64_t tokens, uint32_t heads, uint32_t kv_heads, uint32_t dim);

/* The backward pass, from the x of the forward pass (q, k) and the gradients
 * at its outputs:
 *   g' = the gradient turned back,  h = x * rstd,  g = g' * w,
 *   dx = rstd * (g - h * mean(g * h)),
 *   dw = sum over tokens and heads of g' * h (of the unrounded values)
 * dwq and dwk (NULL: not wanted): dim elements of grad_dtype, dtype or
 * ZERO_F32, stored, or with accumulate added to what is there, then rounded
 * once.  dq may be dq_out or q, dk likewise (the same address, ld and hs).
 * workspace: device, 16-byte aligned, >= zero_qk_workspace_bytes(...), not
 * looked at where neither dwq nor dwk is wanted; contents need no
 * initialisation; calls that share it must be ordered. */
int zero_qk_norm_rope_bwd(void* dq, uint64_t ld_dq, uint64_t hs_dq, void* dk, uint64_t ld_dk, uint64_t hs_dk, void* dwq,
                          void* dwk, int grad_dtype, int accumulate, const void* dq_out, uint64_t ld_dq_out,
                          uint64_t hs_dq_out, const void* dk_out, uint64_t ld_dk_out, uint64_t hs_dk_out, const void* q,
                          uint64_t ld_q, uint64_t hs_q, const void* k, uint64_t ld_k, uint64_t hs_k, const void* wq,
                          const void* wk, int vec_dtype, uint64_t tokens, uint32_t heads, uint32_t kv_heads,
                          uint32_t dim, int dtype, double eps, const float* table, uint64_t table_rows, uint32_t rot,
                          int interleaved, const int32_t* dev_positions, uint64_t period, void* workspace,
                          size_t workspace_bytes, void* stream);

/* Enqueue the angles of positions 0 ... positions-1: table[t][p] = (cos, sin) of
 * t * base^(-2p / rot), p < rot / 2, formed in binary64 and rounded once.
 * table: device, positions x rot / 2 x 2 binary32, 16-byte aligned.
 * Errors: ZERO_EINVAL (NULL, base not finite and > 0, rot odd), ZERO_EALIGN,
 *         ZERO_ERANGE (positions > 2^30, rot > 256), ZERO_EHIP. */
int zero_rope_table(float* table, uint64_t positions, uint32_t rot, double base, void* stream);

#define ZERO_MAX_BUCKETS 64

/* What a model's attention is, the same for every call. */
typedef struct {
    uint32_t heads;             /* of queries; a multiple of kv_heads, <= 65535 */
    uint32_t kv_heads;          /* of keys and values: query head h reads h / (heads / kv_heads) */
    uint32_t dim;               /* elements of a head: a multiple of 8, <= 128 */
    uint32_t sinks;             /* first tokens of a sequence that stay visible */
    uint64_t window;            /* keys a query sees: itself and window - 1 before it; 0: no limit */
    double scale;               /* > 0 */
    uint32_t buckets;           /* of the bias; 0: no bias; <= ZERO_MAX_BUCKETS */
    uint32_t reserved;          /* 0 */
    uint32_t starts[ZERO_MAX_BUCKETS]; /* bucket b holds the distances starts[b] ... starts[b+1]-1, the last all beyond; ascending, starts[0] = 0 */
} zero_attention_t;

/* The usual borders for `buckets` buckets, into starts[buckets]: with half =
 * buckets / 2 the first half one distance each, 0 ... half-1, and bucket
 * half + b from the distance half * (max_distance / half)^(b / (buckets -
 * half)) on, rounded up (a whole number stays; at least one past the bucket
 * before).  Compared in whole numbers, so a distance on a border is in the
 * bucket that begins there.  Host only.
 * Errors: ZERO_EINVAL (NULL, buckets = 0, max_distance <= half for more than
 *         one bucket), ZERO_ERANGE (too many, max_distance > 2^30), ZERO_ENOMEM. */
int zero_attention_buckets(uint32_t* starts, uint32_t buckets, uint32_t max_distance);

/* Causal attention.  Token i of a sequence sees token j of the same where
 * j <= i and (i - j < window or j < sinks):
 *   s = scale * q_i . k_j (+ bias[h][bucket(i - j)]),   p = softmax(s),
 *   o_i = sum over j of p v_j,   lse[h][i] = log of the sum over j of exp(s)
 * q and o: tokens x heads x dim; k and v: tokens x kv_heads x dim; all of type
 * dtype, ZERO_F16 or ZERO_BF16.  lse: binary32, heads x tokens (NULL: not
 * kept; the backward pass needs it).  bias: heads x buckets of dtype or
 * ZERO_F32 (vec_dtype); NULL exactly where buckets is 0.
 * A bucket is masked by a bias of -inf or of any value far below the others';
 * a token that sees masked buckets alone gets NaN from -inf, and from finite
 * ones what binary32 leaves of scores so far from 0.  (They are formed in units
 * of log 2: of 2^127 log 2 or more in size, 1.18e38, a finite one counts as infinite.)
 * dev_offsets: device, sequences + 1 ascending token indices: sequence n is
 * the tokens dev_offsets[n] ... dev_offsets[n+1]-1 (its length may be 0); rows
 * of o and lse outside all sequences stay as they are.  NULL: sequences of
 * equal length, tokens / sequences.  (Indices out of order or range are
 * clamped to the tensors; which rows are then computed is undefined.)
 * What rows hold that a token does not see, inf and NaN too, changes its result by
 * roundings at most; an inf or NaN that it sees gives what its sums of products give.
 * The unnormalised weights are rounded to dtype for the product with v.
 * o must not overlap an input.
 * Errors: ZERO_EINVAL (NULL, a type, heads, dim or scale out of the above,
 *         sequences = 0 with tokens, tokens not a multiple of sequences
 *         without offsets, starts not ascending from 0, bias without buckets
 *         or the other way round), ZERO_EALIGN, ZERO_ERANGE (more than 2^30
 *         tokens or sequences, heads * (tokens / 128 + sequences) >= 2^24 - 8
 *         (without offsets: heads times the sequences' pieces of 128 tokens),
 *         ld or hs < dim or > 2^50, an extent > 2^56, dim > 128), ZERO_EHIP. */
int zero_attention_fwd(void* o, uint64_t ld_o, uint64_t hs_o, float* lse, const void* q, uint64_t ld_q, uint64_t hs_q,
                       const void* k, uint64_t ld_k, uint64_t hs_k, const void* v, uint64_t ld_v, uint64_t hs_v,
                       const void* bias, int vec_dtype, const zero_attention_t* params, uint64_t tokens,
                       const int32_t* dev_offsets, uint64_t sequences, int dtype, void* stream);

/* Enqueue 0 in the rows of x (tokens x heads x dim elements of dtype, ZERO_F16,
 * ZERO_BF16 or ZERO_F32) that are in no sequence: those before dev_offsets[0]
 * and from dev_offsets[sequences] on, which zero_attention_fwd and
 * zero_attention_bwd leave as they are.
 * Errors: ZERO_EINVAL (NULL, a type, heads = 0, dim no multiple of 8),
 *         ZERO_EALIGN, ZERO_ERANGE (dim > 128, more than 65535 heads or 2^30
 *         tokens or sequences, ld or hs < dim or > 2^50, an extent > 2^56),
 *         ZERO_EHIP. */
int zero_attention_clear_rows(void* x, uint64_t ld, uint64_t hs, uint64_t tokens, uint32_t heads, uint32_t dim,
                              int dtype, const int32_t* dev_offsets, uint64_t sequences, void* stream);

/* Bytes of device workspace zero_attention_bwd needs for these or fewer tokens
 * in these or fewer sequences; 0 for no tokens or a refused shape. */
size_t zero_attention_workspace_bytes(const zero_attention_t* params, uint64_t tokens, uint64_t sequences);

/* The backward pass of zero_attention_fwd, from the o and lse it stored:
 *   p = exp(s - lse),   ds = p * (do_i . v_j - do_i . o_i),
 *   dq_i = scale * sum over j of ds k_j,   dk_j = scale * sum over i of ds q_i,
 *   dv_j = sum over i of p do_i,   dbias[h][b] = sum of ds over the pairs of b
 * p is off relatively by about 2^-22 |lse|, so little is left of it in a row
 * whose every score is far from 0, as by a bias of -1e9 at all that it sees.
 * dk and dv are sums over the query heads that share a key head, too.  p and
 * ds are rounded to dtype for the products (ds for binary16 in units that go
 * by the sizes of do, o and v, so that it does not overflow); dbias is a sum of
 * the unrounded ds.  dbias (NULL: not wanted): heads x buckets of grad_dtype,
 * dtype or ZERO_F32, stored, or with accumulate added to what is there, then
 * rounded once.  An inf or NaN anywhere in a sequence may reach all gradients of
 * that sequence, and dbias, as an overflowed backward pass does; other sequences'
 * rows take nothing from it.
 * dq, dk and dv must not overlap an input or each other.  Rows outside all
 * sequences stay as they are.  workspace: device, 16-byte aligned, >=
 * zero_attention_workspace_bytes(params, tokens, sequences); contents need no
 * initialisation; calls that share it must be ordered.
 * Errors: as for zero_attention_fwd, and ZERO_ERANGE for a workspace too small,
 *         or where first tokens are seen by so many queries behind the window
 *         that kv_heads * (tokens / 128 + tokens / 1024 + 2 * sequences) >=
 *         2^24 - 8, or 2^21 sequences or more have such queries. */
int zero_attention_bwd(void* dq, uint64_t ld_dq, uint64_t hs_dq, void* dk, uint64_t ld_dk, uint64_t hs_dk, void* dv,
                       uint64_t ld_dv, uint64_t hs_dv, void* dbias, int grad_dtype, int accumulate, const void* dout,
                       uint64_t ld_dout, uint64_t hs_dout, const void* o, uint64_t ld_o, uint64_t hs_o,
                       const float* lse, const void* q, uint64_t ld_q, uint64_t hs_q, const void* k, uint64_t ld_k,
                       uint64_t hs_k, const void* v, uint64_t ld_v, uint64_t hs_v, const void* bias, int vec_dtype,
                       const zero_attention_t* params, uint64_t tokens, const int32_t* dev_offsets, uint64_t sequences,
                       int dtype, void* workspace, size_t workspace_bytes, void* stream);

/* ---- measurement reference ------------------------------------------ */

/* A plain streaming copy of `bytes` bytes (dst and src device, 16-byte
 * aligned, bytes a multiple of 16), used to measure the attainable HBM
 * bandwidth next to the step's kernels.  Errors: ZERO_EINVAL, ZERO_EALIGN,
 * ZERO_ERANGE (more than 2^31 - 1 workgroups), ZERO_EHIP. */
int zero_stream_copy(void* dst, const void* src, uint64_t bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_MI355X_H */
