/*
 * mpt.h -- libmpt: the loss-scaled FP32-master SGD-momentum optimizer step of
 * mixed-precision training, on one NVIDIA B200 (sm_100a).
 *
 * What one step computes (Micikevicius et al., "Mixed Precision Training",
 * as explained by the paper-graph-ui.vercel.app analysis, section 3.4,
 * "The Integrated Training Procedure (Figure 1)", Steps 5-7, and the
 * azimuth.plus tutorial, "Loss scaling: why gradients vanish in FP16"):
 *
 *   given FP16 weight gradients g16 of a list of tensors, computed from a loss
 *   multiplied by S, and per-parameter FP32 state (master w, momentum v):
 *     1. found_inf = any g16 is +-inf or NaN, over the whole list   (Step 6)
 *     2. g   = fp32(g16) * (1/S)                                     (Step 5)
 *     3. norm = sqrt(sum g^2) over the whole list (binary64);
 *        if clip > 0 and norm > clip: g = g * (clip / norm)  (global-L2 clip,
 *        after unscaling: "Summary of Design Choices")
 *     4. if found_inf: leave w, v and the FP16 copy untouched, S = S*beta
 *                                                   (Step 6, Method 3)
 *        else, per element, every operation rounded to binary32:
 *          d = g + lambda*w        ("A subtle interaction: weight decay")
 *          v = mu*v + d            (Step 7)
 *          w = w - eta*v           (Step 7)
 *          w16 = round_to_nearest_even_fp16(w)   (Step 1 of the next pass)
 *     5. after N consecutive clean steps, S = S*alpha (dynamic scaling,
 *        "Choosing the Loss Scaling Factor", Method 3)
 *
 * Conventions for every call:
 *   - Every function returns an int status: MPT_OK (0) or a negative
 *     MPT_ERR_* code.  No call aborts, throws, traps or prints.
 *   - A handle is used by one host thread at a time.
 *   - "device pointer" means memory of the CUDA device that is current when
 *     mpt_create is called; every later call must run with that device current.
 *   - cuda_stream arguments are cudaStream_t values passed as void*; NULL is
 *     the legacy default stream.
 *   - After MPT_ERR_CUDA the handle is broken: every later call except
 *     mpt_stats, mpt_error_string and mpt_destroy returns MPT_ERR_BROKEN.
 */
#ifndef LIBMPT_MPT_H
#define LIBMPT_MPT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------- */
#define MPT_OK 0
#define MPT_ERR_INVALID_ARG (-1)  /* null or odd pointer, n <= 0, size <= 0,
                                     S not finite or <= 0, lr / momentum /
                                     weight decay / clip not finite          */
#define MPT_ERR_WORKSPACE (-2)    /* workspace too small, not 256-B aligned,
                                     or not device memory of this device    */
#define MPT_ERR_CUDA (-3)         /* a CUDA runtime call failed             */
#define MPT_ERR_DEVICE_CHECK (-4) /* checked mode found a work-table entry out
                                     of bounds; that entry was not touched   */
#define MPT_ERR_BROKEN (-5)       /* the handle saw MPT_ERR_CUDA earlier     */
#define MPT_ERR_TOO_LARGE (-6)    /* input longer than MPT_NOALLOC_MAX_ELEMS
                                     (mpt_check_flat_noalloc only)           */

/* ---- configuration ------------------------------------------------------ */
#define MPT_FLAG_CHECKED 0x1u     /* kernels validate every work-table entry
                                     against the tensor sizes and arenas     */
#define MPT_FLAG_COUNT_STALE 0x2u /* count elements whose master moved but
                                     whose FP16 copy did not                 */
#define MPT_FLAG_GRAD_STATS 0x4u  /* the check pass also finds the largest
                                     |g16| and counts the gradients per
                                     binary16 exponent field (see
                                     mpt_grad_histogram); implied by
                                     MPT_SCALER_DIRECT                      */

/* Loss-scale modes ("Choosing the Loss Scaling Factor").  Both skip the
 * update and multiply S by backoff on overflow.
 *   DYNAMIC (Method 3): after growth_interval consecutive clean steps,
 *     multiply S by growth.
 *   DIRECT (Method 2): after every clean step set S = 65504 / (margin *
 *     max|g|), max|g| being that step's largest unscaled finite gradient
 *     (binary64, rounded to binary32, clamped to [min_scale, max_scale]);
 *     a step whose gradients are all zero keeps S. */
#define MPT_SCALER_DYNAMIC 0
#define MPT_SCALER_DIRECT 1

/* Update rule of the FP32 master (every operation rounded to binary32; d is
 * the unscaled, clipped gradient plus weight decay, d = g + lambda*w):
 *   MOMENTUM (default; Step 7): v = mu*v + d;  w = w - eta*v
 *   NESTEROV (the pages' speech models): v = mu*v + d;  w = w - eta*(d + mu*v)
 *   ADAGRAD (the pages' bigLSTM): v = v + d*d;  w = w - eta*d/(sqrt(v) + eps)
 *     -- the momentum arena holds the running sum of squares (zero at
 *     creation) and the momentum argument of the step is ignored. */
#define MPT_OPT_MOMENTUM 0
#define MPT_OPT_NESTEROV 1
#define MPT_OPT_ADAGRAD 2

typedef struct {
    float backoff;            /* beta: S multiplier on overflow (default 0.5)      */
    float growth;             /* alpha: S multiplier after N clean steps (2.0)     */
    int32_t growth_interval;  /* N; 0 = constant S (an overflow still backs off) */
    float min_scale;          /* lower bound of S after a backoff (2^-24)          */
    float max_scale;          /* upper bound of S after a growth (2^24)            */
    uint32_t flags;           /* MPT_FLAG_* (default 0)                            */
    int32_t check_chunk_elems;  /* elements per work bin (one CTA) of the check
                                   pass: a multiple of 2048 in [2048, 2^20];
                                   0 = default: 65536, halved down to 2048
                                   while the list gives fewer than 592 bins */
    int32_t scaler_mode;      /* MPT_SCALER_DYNAMIC (default) or _DIRECT           */
    float direct_margin;      /* direct mode: margin > 0 (default 2: one bit of
                                 headroom, as the pages suggest)                   */
    int32_t optimizer;        /* MPT_OPT_MOMENTUM (default), _NESTEROV, _ADAGRAD   */
    float eps;                /* Adagrad denominator term (default 1e-10)          */
    int32_t update_chunk_elems; /* the same for the update pass; 0 = default
                                   (4096)                                         */
} mpt_config;

/* ---- results ------------------------------------------------------------ */
typedef struct {
    int32_t found_inf;     /* 1: some gradient was +-inf/NaN; the update was
                              skipped and the state is bitwise unchanged        */
    int32_t clipped;       /* 1: clip > 0 and grad_norm > clip                  */
    float new_scale;       /* S to use for the next step                        */
    int32_t clean_run;     /* consecutive clean steps after this one            */
    double grad_norm;      /* global L2 norm of the unscaled, unclipped
                              gradients; +inf when found_inf                    */
    float clip_coef;       /* clip / grad_norm when clipped, else 1             */
    float max_abs_grad;    /* MPT_FLAG_GRAD_STATS / direct mode, else 0: the
                              largest unscaled finite |g|, fp32(max|g16|)*(1/S) */
    uint64_t n_zero;       /* FP16 gradients equal to +-0 (counted by the check
                              pass, so overflow steps report them too)         */
    uint64_t n_subnormal;  /* FP16 gradients with 0 < |g16| < 2^-14             */
    uint64_t n_nonfinite;  /* FP16 gradients that are +-inf or NaN              */
    uint64_t n_fp16_stale; /* MPT_FLAG_COUNT_STALE only, else 0: elements whose
                              master changed while the rounded copy did not     */
} mpt_step_result;

typedef struct {
    uint64_t steps;           /* steps completed on the device                  */
    uint64_t skipped;         /* of which were skipped on overflow              */
    float scale;              /* current S (last new_scale, or the value set)   */
    int32_t clean_run;        /* current clean-step counter                     */
    mpt_step_result last;     /* result of the last completed step              */
    uint64_t n_fp16_stale_total; /* MPT_FLAG_COUNT_STALE: n_fp16_stale summed
                              over every step since creation, queued ones
                              included (summed on the device)                 */
    uint64_t timed_steps;     /* steps timed while mpt_set_timing was on        */
    double check_ms_total;    /* summed CUDA-event durations of the check       */
    double update_ms_total;   /* kernel and of the update kernel over them      */
} mpt_stats_t;

typedef struct mpt_handle mpt_handle;  /* opaque */

/* ---- calls -------------------------------------------------------------- */

/* Fill *cfg with the defaults listed in mpt_config.
 * Errors: MPT_ERR_INVALID_ARG (cfg NULL). */
int mpt_config_init(mpt_config* cfg);

/* Bytes of device workspace mpt_create needs for n tensors with the given
 * element counts (host array sizes[n]); cfg NULL = defaults.  The workspace
 * holds the FP32 master arena, the FP32 momentum arena and the FP16
 * working-copy arena (each tensor at a 16-element-aligned offset) plus the
 * work tables and a small control block.
 * Errors: MPT_ERR_INVALID_ARG (a pointer NULL, n <= 0, a size <= 0, bad cfg). */
int mpt_workspace_bytes(const int64_t* sizes, int32_t n, const mpt_config* cfg,
                        size_t* bytes);

/* Create a handle over a caller-owned device workspace d_workspace of
 * ws_bytes bytes (256-byte aligned, at least mpt_workspace_bytes).  Builds and
 * uploads the work tables and zeroes the three arenas and the control block,
 * synchronously.  The caller then writes the initial master weights through
 * mpt_tensor_views and calls mpt_refresh_half.  The workspace and the
 * gradient buffers belong to the caller and must outlive the handle; the
 * library owns only host tables and two small pinned host buffers.  The loss
 * scale starts at 1 with a clean-step counter of 0 (mpt_set_scaler_state).
 * Errors: MPT_ERR_INVALID_ARG, MPT_ERR_WORKSPACE, MPT_ERR_CUDA. */
int mpt_create(const int64_t* sizes, int32_t n, const mpt_config* cfg,
               void* d_workspace, size_t ws_bytes, mpt_handle** out);

/* Device pointers to tensor i's slices of the arenas: FP32 master, FP32
 * momentum and FP16 working copy (binary16, sizes[i] elements each, 64-byte
 * aligned).  Any output pointer may be NULL.
 * Errors: MPT_ERR_INVALID_ARG (h NULL, i out of range). */
int mpt_tensor_views(const mpt_handle* h, int32_t i, float** master,
                     float** momentum, void** w16_half);

/* Rewrite every FP16 working copy from its FP32 master: w16 = RNE_fp16(w)
 * (Step 1 of the training iteration).  Asynchronous on cuda_stream.
 * Errors: MPT_ERR_INVALID_ARG, MPT_ERR_CUDA, MPT_ERR_BROKEN. */
int mpt_refresh_half(mpt_handle* h, void* cuda_stream);

/* The loss-scale state (S and the clean-step counter) lives in the
 * workspace and is advanced on the device by every step, so steps can be
 * queued without the host waiting; the handle keeps a host mirror that every
 * waiting call (mpt_step, mpt_wait, mpt_set_scaler_state) refreshes. */

/* One optimizer step.  d_grads_half is a HOST array of n DEVICE pointers, the
 * FP16 (binary16) gradients of the n tensors, computed from a loss multiplied
 * by `scale` (any 2-byte alignment; contents are only read).  lr, momentum
 * and weight_decay are eta, mu and lambda; clip <= 0 disables clipping.
 * Work is queued on cuda_stream and the call waits for it (it reads the
 * 384-byte control block back).  The scale state advances from `scale`:
 * out->new_scale is the S for the next step.  On overflow the arenas are
 * untouched.  Errors: MPT_ERR_INVALID_ARG, MPT_ERR_CUDA,
 * MPT_ERR_DEVICE_CHECK (checked mode; the bins that passed their check were
 * updated), MPT_ERR_BROKEN; on an argument error nothing is queued. */
int mpt_step(mpt_handle* h, const void* const* d_grads_half, float scale,
             float lr, float momentum, float weight_decay, float clip,
             void* cuda_stream, mpt_step_result* out);

/* The same step, queued on cuda_stream without waiting: S is the device
 * scale state (see mpt_device_scale), the gradients must have been computed
 * from a loss multiplied by that device value, and the step advances the
 * state on the device.  Nothing is read back; call mpt_wait for the result
 * of the last queued step.  The gradient buffers must stay unchanged until
 * the queued work has run.
 * Gradient-pointer tables: the handle keeps device copies of the last four
 * distinct tables passed to its steps (in its workspace).  A step whose
 * d_grads_half equals one of them queues exactly the two kernel launches (no
 * copy, no host synchronisation); a new table is copied from pinned host
 * memory into the least recently used copy first, ordered on the step's
 * stream after the steps queued before it.  So queue a handle's steps on one
 * stream (or order its streams yourself).
 * CUDA graphs: a step whose table is already held queues only the two
 * kernel launches, so it can be captured into a CUDA graph (kernel timing
 * off); capture only after a first, uncaptured step with the same table (a
 * new table's copy must not be recorded).  Each replay reads the gradients
 * its buffers hold at replay time, the pointer copy that the capture used,
 * and reads and advances the device scale state; mpt_wait on the replay
 * stream returns the replayed step's result.  A later step with a fifth
 * distinct table may rewrite that copy: replay a captured step only while
 * its table is among the last four used.
 * Errors: MPT_ERR_INVALID_ARG, MPT_ERR_CUDA, MPT_ERR_BROKEN. */
int mpt_step_async(mpt_handle* h, const void* const* d_grads_half, float lr,
                   float momentum, float weight_decay, float clip, void* cuda_stream);

/* Wait for the work queued on cuda_stream and return the result of the last
 * step (out may be NULL); refreshes the host mirror of the scale state and
 * the counters.  Errors: MPT_ERR_INVALID_ARG, MPT_ERR_CUDA,
 * MPT_ERR_DEVICE_CHECK, MPT_ERR_BROKEN. */
int mpt_wait(mpt_handle* h, void* cuda_stream, mpt_step_result* out);

/* Device address of the binary32 loss scale S that the next
 * mpt_step_async uses (inside the workspace): a training loop multiplies its
 * loss by it on the device.  Errors: MPT_ERR_INVALID_ARG. */
int mpt_device_scale(const mpt_handle* h, float** d_scale);

/* ---- sharded step (optimizer state split across the ranks of a data-
 * parallel group) ---------------------------------------------------------
 *
 * The flat parameter list (all tensors concatenated, P elements) is cut into
 * `world` equal contiguous shards of mpt_shard_len(P, world) elements (the
 * last one padded with elements whose gradient is always zero).  Rank r
 * creates an ordinary handle over ONE tensor of shard_len elements: it owns
 * the FP32 master, FP32 momentum and FP16 copy of flat elements
 * [r*shard_len, (r+1)*shard_len).  Per step, with the loss scale on the
 * device (as mpt_step_async):
 *   1. the caller reduce-scatters the FP16 gradients so that each rank holds
 *      the summed gradients of its shard (an FP16 sum can itself overflow;
 *      step 2 catches it like any other inf);
 *   2. mpt_step_partial queues the check pass over the shard and returns the
 *      device address of its 32-byte record (MPT_PARTIAL_BYTES: binary64 sum
 *      of squares, non-finite count, largest finite |g16|, error bits);
 *   3. the caller all-gathers the records of all ranks, in rank order, into
 *      one device array (16-byte aligned);
 *   4. mpt_step_finish queues the update of the shard, which first adds the
 *      records in rank order (so every rank gets bit-identical totals and the
 *      same next S) and finishes the step;
 *   5. the caller all-gathers the FP16 copies of the shards.
 * Only 32 bytes per rank cross between the two kernels of a step.  The
 * halves are not timed by mpt_set_timing; mpt_wait returns the last result:
 * found_inf, n_nonfinite, grad_norm, the clip coefficient and the scale are
 * those of the whole list (equal on every rank), n_zero, n_subnormal and the
 * histogram those of this rank's shard. */
#define MPT_PARTIAL_BYTES 32

/* shard_len = ceil(total / world) rounded up to a multiple of 16.
 * Errors: MPT_ERR_INVALID_ARG. */
int mpt_shard_len(int64_t total, int32_t world, int64_t* shard_len);

/* Phase 2: queue the check pass over the handle's gradients (a host array of
 * its tensors' device pointers, as for mpt_step) with S from the device
 * state; *d_partial receives the device address of this rank's record
 * (valid until the next call on the handle).  Errors: MPT_ERR_INVALID_ARG,
 * MPT_ERR_CUDA, MPT_ERR_BROKEN. */
int mpt_step_partial(mpt_handle* h, const void* const* d_grads_half, void* cuda_stream,
                     void** d_partial);

/* Phase 4: d_partials = device array of `world` records in rank order;
 * queues the update over the gradients of the preceding mpt_step_partial,
 * which first adds the records and finishes the step (norm, clip
 * coefficient, loss-scale state).
 * Errors: MPT_ERR_INVALID_ARG (no check pass queued, misaligned records),
 * MPT_ERR_CUDA, MPT_ERR_BROKEN. */
int mpt_step_finish(mpt_handle* h, const void* d_partials, int32_t world, float lr,
                    float momentum, float weight_decay, float clip, void* cuda_stream);

/* Statistics mode: counts[e] = number of gradients of the last step whose
 * binary16 exponent field is e (e = 0: zeros and subnormals; e = 31: inf and
 * NaN; otherwise |g16| in [2^(e-15), 2^(e-14))), as of the last waiting
 * call; all zero without statistics.  Errors: MPT_ERR_INVALID_ARG. */
int mpt_grad_histogram(const mpt_handle* h, uint64_t counts[32]);

/* Counters and the last result, as of the last waiting call.
 * Errors: MPT_ERR_INVALID_ARG. */
int mpt_stats(const mpt_handle* h, mpt_stats_t* out);

/* Read the host mirror of the loss-scale state (as of the last waiting
 * call) / set the state on the device and the host (checkpoint and resume;
 * synchronous, call it with no step in flight).  set requires a finite
 * scale > 0 and clean_run >= 0.  Errors: MPT_ERR_INVALID_ARG, MPT_ERR_CUDA,
 * MPT_ERR_BROKEN. */
int mpt_get_scaler_state(const mpt_handle* h, float* scale, int32_t* clean_run);
int mpt_set_scaler_state(mpt_handle* h, float scale, int32_t clean_run);

/* Time both kernels of every `every`-th following step (the first step
 * queued after the call, then every `every`-th; 1 = every step) with CUDA
 * events recorded on the step's stream before the check kernel, between the
 * two kernels and after the update kernel.  The durations are summed into
 * mpt_stats_t at the next waiting call, or when 256 timed steps are pending.
 * The events cost time of their own (the update of a timed step cannot start
 * early, and three more stream operations sit in each timed step), so a
 * throughput measurement should sample: every = 10 keeps that cost to a
 * tenth.  every = 0 turns timing off (and waits for the pending events).
 * Whole steps only: the halves of a sharded step are not timed.
 * Errors: MPT_ERR_INVALID_ARG (h NULL, every < 0), MPT_ERR_CUDA. */
int mpt_set_timing(mpt_handle* h, int32_t every);

/* Test hook (the pages have no counterpart): the next step of this handle --
 * mpt_step, mpt_step_async, mpt_step_partial or mpt_step_finish -- fails as
 * if its kernel launch had failed: it queues nothing, returns MPT_ERR_CUDA,
 * and the handle becomes unusable (every later call returns MPT_ERR_BROKEN),
 * exactly as after a real CUDA error.  No CUDA call is made and no GPU fault
 * is involved; it exists so that a caller's error path can be tested.
 * Errors: MPT_ERR_INVALID_ARG (h NULL). */
int mpt_debug_fail_next_step(mpt_handle* h);

/* Release the handle's host resources.  The workspace is the caller's and is
 * not freed.  NULL is accepted. */
int mpt_destroy(mpt_handle* h);

/* Static description of a status code (never NULL). */
const char* mpt_error_string(int code);

/* ---- allocation-free check of one flat gradient buffer ------------------ */

/* The paper has no counterpart to this call: it serves callers of this
 * library, not a step of the method.
 *
 * Some callers cannot allocate device memory: a library loaded into a host
 * program whose memory pool already owns the device (a cudaMalloc there
 * fails, or takes memory the host program has counted on), and code whose
 * step loop must never enter the CUDA allocator (cudaMalloc and cudaFree can
 * synchronize the device and stall every stream).  mpt_step needs a
 * workspace allocated up front; this call needs none.  It runs the overflow
 * check and the global norm of the step (found_inf, the L2 norm of the
 * unscaled gradients, the clip coefficient, the count of +-inf/NaN) over ONE
 * contiguous FP16 buffer, keeping its scratch (one binary64 partial per
 * 32768 elements and two counters, about 256 KiB) in a fixed array inside the
 * library that every GPU which loads the library holds until the process
 * exits.
 *
 *   d_grads_half  device pointer to n binary16 gradients (2-byte aligned),
 *                 scaled by `scale`; only read
 *   n             1 <= n <= MPT_NOALLOC_MAX_ELEMS; longer inputs return
 *                 MPT_ERR_TOO_LARGE before any CUDA call
 *   scale, clip   as in mpt_step (clip <= 0: no clipping, coefficient 1)
 *   d_result      device pointer (8-byte aligned) that receives the
 *                 mpt_check_result when the queued work completes
 *   cuda_stream   stream to queue on; the call returns without waiting
 *
 * The first successful call on each device sets that device up, with it
 * current: it looks up the device address of the scratch array and loads the
 * call's kernels (both of its variants, for power-of-two and other S), so no
 * later call loads code.  Make that first call before any stream capture; a
 * set-up that fails (inside a capture, say) returns MPT_ERR_CUDA, keeps
 * nothing, and the next call tries again.  Every call on a device shares the
 * one scratch array, which keeps the last call's contents; each call clears
 * the counters it needs before its kernel runs.  Calls whose work overlaps on
 * the GPU (other streams, other host threads) race on that array and give
 * wrong results: serialize them.  The call checks the status each CUDA call
 * returns; it clears the runtime's last-error state only after a failure of
 * its own, so an error left pending by earlier work stays for the caller.
 * Errors: MPT_ERR_INVALID_ARG, MPT_ERR_TOO_LARGE, MPT_ERR_CUDA. */
#define MPT_NOALLOC_MAX_ELEMS (((int64_t)1) << 30)

typedef struct {
    int32_t found_inf;     /* 1: some gradient was +-inf/NaN                     */
    int32_t clipped;       /* 1: clip > 0 and grad_norm > clip                   */
    double grad_norm;      /* L2 norm of the unscaled gradients; +inf if found   */
    float clip_coef;       /* clip / grad_norm when clipped, else 1              */
    int32_t reserved;
    uint64_t n_nonfinite;  /* gradients that are +-inf or NaN                    */
} mpt_check_result;

int mpt_check_flat_noalloc(const void* d_grads_half, int64_t n, float scale, float clip,
                           mpt_check_result* d_result, void* cuda_stream);

/* ---- gradient lists: global norm and clipping ----------------------------
 *
 * The norm and the clipping of mpt_step for gradients that do not go (or not
 * at once) through mpt_step: lists of FP16, BF16 or FP32 tensors, mixed as
 * they come, of any element-aligned address and any size, zero included.
 *
 *   s_i  = sum of g^2 over tensor i           (binary64)
 *   norm = sqrt(sum of s_i) / S               tensor norm i = sqrt(s_i) / S
 *   coef = clip / norm, rounded to binary32, when clip > 0, every gradient is
 *          finite and norm > clip; else 1
 *   out  = T(fp32(g) * coef), or with MPT_LIST_UNSCALE
 *          T(fp32(g) * fp32(1/S) * coef); each product rounded to binary32,
 *          T = the output type's round-to-nearest-even
 *
 * A gradient that is +-inf or NaN makes found_inf 1, the norm (and its
 * tensor's norm) +inf and the coefficient 1: the outputs are then the
 * gradients themselves (unscaled if asked), so a following mpt_step sees the
 * overflow and skips.  The sums' order depends on the list alone: the same
 * gradients give the same bits. */
#define MPT_F16 0   /* binary16 */
#define MPT_BF16 1  /* bfloat16 */
#define MPT_F32 2   /* binary32 */

#define MPT_LIST_TENSOR_NORMS 0x1u /* also write every tensor's own norm       */
#define MPT_LIST_UNSCALE 0x2u      /* mpt_list_clip: outputs divided by S      */

typedef struct mpt_list mpt_list;  /* opaque */

/* Bytes of device workspace for a list of n tensors: sizes[n] element counts
 * (>= 0), types[n] of MPT_F16 / MPT_BF16 / MPT_F32, out_types[n] the types
 * that mpt_list_clip writes (NULL: the gradients' own).  All host arrays.
 * Errors: MPT_ERR_INVALID_ARG. */
int mpt_list_workspace_bytes(const int64_t* sizes, const int32_t* types, const int32_t* out_types,
                             int32_t n, size_t* bytes);

/* Create a list over a caller-owned device workspace (256-byte aligned, at
 * least mpt_list_workspace_bytes), synchronously, after all work queued on the
 * device (so not while a stream is captured); the workspace must outlive the
 * list.  Errors: MPT_ERR_INVALID_ARG, MPT_ERR_WORKSPACE, MPT_ERR_CUDA. */
int mpt_list_create(const int64_t* sizes, const int32_t* types, const int32_t* out_types, int32_t n,
                    void* d_workspace, size_t ws_bytes, mpt_list** out);

/* Queue the norm of the gradients at d_grads (a HOST array of n DEVICE
 * pointers, as for mpt_step; the pointer of an empty tensor is not looked
 * at).  S is *d_scale, read on the device when the work runs, or `scale`
 * where d_scale is NULL (a device S is not checked: it must be finite and
 * > 0, as mpt_device_scale's always is).  flags: MPT_LIST_TENSOR_NORMS.
 * The results are written to the workspace (mpt_list_views): result record,
 * and the tensor norms if asked.  Queues two kernels and returns.
 * Queue a list's calls on one stream, or order the streams: they share the
 * workspace.  Pointer tables and CUDA graphs: as for mpt_step_async, with
 * one difference: a table that a capture has used is kept for good, so four
 * captured tables leave no room for a fifth table.
 * Errors: MPT_ERR_INVALID_ARG (also: another device is current; a capture
 * with a table that no earlier call has used; no table is free),
 * MPT_ERR_CUDA, MPT_ERR_BROKEN; on an argument error nothing is queued. */
int mpt_list_norm(mpt_list* h, const void* const* d_grads, float scale, const float* d_scale, float clip,
                  uint32_t flags, void* cuda_stream);

/* Queue the norm and the scaling of the gradients into d_out (a HOST array of
 * n DEVICE pointers).  d_out[i] may be d_grads[i] where the types are the
 * same (in place); apart from that no output may touch a gradient or another
 * output.  In place and without MPT_LIST_UNSCALE gradients within the limit
 * are left as they are.  Otherwise as mpt_list_norm.
 * Errors: as mpt_list_norm, and MPT_ERR_INVALID_ARG for outputs that
 * overlap. */
int mpt_list_clip(mpt_list* h, const void* const* d_grads, void* const* d_out, float scale,
                  const float* d_scale, float clip, uint32_t flags, void* cuda_stream);

/* Device addresses, inside the workspace, of the result record of the last
 * call and of the n tensor norms.  Either may be NULL.
 * Errors: MPT_ERR_INVALID_ARG. */
int mpt_list_views(const mpt_list* h, mpt_check_result** d_result, double** d_tensor_norms);

/* Wait for the work queued on cuda_stream and return the last result (out
 * may be NULL).  Errors: MPT_ERR_INVALID_ARG (also: another device is current;
 * cuda_stream is being captured), MPT_ERR_CUDA, MPT_ERR_BROKEN. */
int mpt_list_wait(mpt_list* h, void* cuda_stream, mpt_check_result* out);

/* Release the list's host resources (NULL is accepted), once the copies of
 * pointer tables that its calls have queued are done.  The workspace has to stay
 * until the kernels are. */
int mpt_list_destroy(mpt_list* h);

/* ---- softmax cross entropy of a head, with loss-scaled gradients ---------
 *
 * The start of the backward pass: the loss that S multiplies.  For n rows of
 * hidden (n x d), a head's weight (v x d) and one target class per row,
 *
 *   z      = hidden weight^T
 *   loss_i = log(sum_u exp(z_iu)) - z_it        (0 where t == ignore_index)
 *   loss   = sum of loss_i, or that divided by the number of rows that are
 *            not ignored (MPT_XENT_MEAN; 0 where every row is)
 *   grad_hidden = S dloss/dhidden,  grad_weight = S dloss/dweight
 *
 * FP16 or BF16 operands and gradients of the same type; products are summed
 * in binary32 (in parts of 512 for a logit, of at most 16384 for a gradient;
 * the tensor cores truncate, so that a logit whose products have one sign is low
 * by 2.4e-6 of itself), exponentials and their sums are binary32, the gradient of
 * the logits is rounded to 16 bits once (scaled so that it does not underflow),
 * and S/n is applied in binary32 before the gradients are rounded: a value
 * beyond FP16's range becomes inf there, which mpt_step finds and skips on.
 * A target that is neither ignored nor a class makes the loss and the
 * gradients NaN (and nothing out of range is read), and so does a logit of
 * +inf or NaN, as an overflow in the layers below leaves it; one of -inf is a
 * class of probability 0 (as target: a loss of +inf).  An infinite or NaN
 * operand also spoils the gradient values that it is a factor of, by 0 too:
 * rows that are ignored have to be finite.  Each result depends on
 * the call's arguments alone, bit for bit: no sum's order depends on timing. */
/* Memory: no buffer holds all logits of a large call.  Their gradient is held for
 * a piece of the vocabulary at a time, at most 256 MB in 16 bits; the logits of
 * a call are kept only where all of them take at most 256 MB in binary32 and
 * moving them is quicker than multiplying again.  The row statistics take a 64th
 * of the logits in binary32, grad_hidden a binary32 copy for each part that its
 * sums are cut into, and grad_weight, from 16385 rows on, one of a piece's
 * classes.  The workspace does not always grow with n: ask for every size that
 * is used. */
#define MPT_XENT_MEAN 0
#define MPT_XENT_SUM 1

typedef struct {
    int32_t type;             /* MPT_F16 or MPT_BF16                             */
    int32_t target_bytes;     /* 4 (int32) or 8 (int64, default)                  */
    int64_t n, v, d;          /* rows (>= 0), classes (>= 1), width (a multiple
                                 of 8)                                            */
    const void* hidden;       /* n rows of d, ld_hidden elements apart: 16-byte
                                 aligned, ld a multiple of 8                      */
    int64_t ld_hidden;
    const void* weight;       /* v rows of d, likewise                            */
    int64_t ld_weight;
    const void* targets;      /* n integers                                       */
    int64_t ignore_index;     /* rows with this target do not count (-100)        */
    int32_t reduction;        /* MPT_XENT_MEAN (default) or MPT_XENT_SUM          */
    float scale;              /* S (default 1), or                                */
    const float* d_scale;     /* S on the device, read when the work runs         */
    float* loss;              /* out: 1 value                                     */
    float* token_loss;        /* out: n values, or NULL                           */
    float* lse;               /* out: n values, log sum exp z, or NULL            */
    int64_t* n_valid;         /* out: rows that are not ignored, or NULL          */
    void* grad_hidden;        /* out: n rows of d, or NULL                        */
    int64_t ld_grad_hidden;
    void* grad_weight;        /* out: v rows of d, or NULL                        */
    int64_t ld_grad_weight;
} mpt_xent_args;

/* Fill *args with zeros and the defaults named above.
 * Errors: MPT_ERR_INVALID_ARG. */
int mpt_xent_args_init(mpt_xent_args* args);

/* Bytes of device workspace for these sizes and these outputs (which of
 * grad_hidden and grad_weight are asked for; addresses are not looked at
 * otherwise).  Errors: MPT_ERR_INVALID_ARG. */
int mpt_xent_workspace_bytes(const mpt_xent_args* args, size_t* bytes);

/* Queue the loss and the gradients asked for on cuda_stream and return.  All
 * pointers are device pointers of the current device; the address ranges of
 * the gradients may not meet those of hidden, weight or each other.  The
 * workspace (256-byte aligned) holds nothing between calls: calls that may
 * overlap on the GPU need one each.  Can be captured into a CUDA graph; the
 * first call on a device loads the kernels, so make one before any capture.
 * No wait inside a kernel is without a limit (some seconds, where none takes a
 * millisecond): should one run out, the work still ends, the loss is NaN, and so
 * is a value at least of every gradient that is not whole, so that mpt_step
 * skips on it.
 * Errors: MPT_ERR_INVALID_ARG, MPT_ERR_WORKSPACE, MPT_ERR_CUDA; on an
 * argument error nothing is queued. */
int mpt_xent(const mpt_xent_args* args, void* d_workspace, size_t ws_bytes, void* cuda_stream);

/* Test hook: in the next mpt_xent that this thread queues, the blocks of the
 * named passes' product kernels stop loading after up to eight steps and give
 * up the waits for what does not come, as they do after some seconds otherwise.
 * Errors: MPT_ERR_INVALID_ARG. */
#define MPT_XENT_PASS_LOSS 0x1 /* products of the loss (from five rows on)           */
#define MPT_XENT_PASS_DZ 0x2   /* logits multiplied again (where they are not kept)  */
#define MPT_XENT_PASS_GRAD 0x4 /* products of the gradients                          */
int mpt_debug_xent_give_up(int32_t passes);

#ifdef __cplusplus
}
#endif
#endif
