/*
 * dszero.h -- C ABI of the MI355X (gfx950) ZeRO mixed-precision optimizer step.
 *
 * One GPU's share of ZeRO data-parallel training: the optimizer step that each
 * rank runs on its own contiguous 1/N partition of the model state, gated by
 * dynamic loss scaling and fed by fp16 gradient accumulation into an fp32
 * buffer.
 *
 * Pages cited (by title and section):
 *   [Guide]    "DeepSpeed complete guide" (youngju.dev, Japanese)
 *   [Overview] "DeepSpeed" project overview (aibars.net, Japanese), core features
 *
 * Model state per element of a partition ([Guide] section 2, memory table):
 * fp16 parameter copy (p16), fp16 gradient, fp32 master parameter, fp32 Adam
 * first moment (m), fp32 Adam second moment (v).  In bf16 mode ([Guide]
 * section 4.2, bf16 settings) the 16-bit parameter copy and gradients are
 * bf16 instead and no loss scaling is applied (a static scale of 1).  With
 * ZeRO-1/2 each rank owns a contiguous 1/N range of these arrays and updates
 * only that range ([Guide] sections 2.1 and 2.2).
 *
 * Conventions shared by every entry point:
 *  - Memory.  Array arguments are DEVICE pointers owned by the caller; the
 *    library never allocates, frees or keeps them.  Work is enqueued
 *    asynchronously on `stream` (a hipStream_t; NULL is the default stream)
 *    and uses the buffers until the stream reaches it.
 *  - Layout.  Arrays are flat and contiguous, element i of every array belongs
 *    to the same parameter.  16-bit values are bit patterns (uint16_t) of IEEE
 *    binary16 (DS_FP16) or bf16 (DS_BF16: the upper half of an IEEE binary32);
 *    fp32 values are IEEE binary32.
 *  - Alignment.  Every array pointer must be 16-byte aligned; a ds_scaler
 *    pointer must be 8-byte aligned.
 *  - Errors.  Every call validates all arguments before any device work, so a
 *    call that returns an error has had no effect.  n < 0, or n > 2^40
 *    (more elements than any device holds) -> DS_ERR_SIZE;
 *    n == 0 -> DS_OK and nothing is launched; a NULL array with n > 0 ->
 *    DS_ERR_NULL; a misaligned pointer -> DS_ERR_ALIGN; overlapping arrays ->
 *    DS_ERR_ALIAS; an unknown dtype -> DS_ERR_DTYPE; an out-of-range
 *    hyperparameter -> DS_ERR_HPARAM; a failed HIP launch or copy ->
 *    DS_ERR_HIP (the enqueue failed; earlier work is unaffected).
 *  - Data is not an error: inf/NaN gradients set the overflow flag.
 *  - Per-step order on one stream: all ds_accumulate calls, then any number of
 *    ds_check_overflow calls (disjoint ranges), then any number of
 *    ds_adam_step calls (disjoint ranges, all reading the same state), then
 *    exactly one ds_update_loss_scale; or, for a partition updated by a
 *    single call, one ds_adam_step_fused in place of both.  No host
 *    synchronisation is needed inside a step: the skip decision is taken on
 *    the device.
 *  - Thread safety: the library keeps no mutable global state.  Calls that
 *    share a ds_scaler must be ordered on one stream.
 *  - Launch-shape knobs, read from the environment at each call (for tests
 *    and tuning; results are bit-identical under every setting):
 *    DSZERO_GRID=<blocks> pins the block count of every kernel of the call
 *    (the kernels loop over their tiles or chunks); DSZERO_UNROLL=2 halves
 *    the tile of ds_adam_step to 2048 elements (256 lanes x 2 quads; by
 *    default 4096 elements as 256 lanes x 4 quads, or 512 x 2 for
 *    ds_adam_step_fused without non-temporal hints); DSZERO_NT=0|1 turns the
 *    non-temporal load/store hints of the read/write kernels off or on
 *    (default: on above 2^24 elements, off at and below, where the state
 *    stays in the Infinity Cache between steps).
 */
#ifndef DSZERO_H
#define DSZERO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
/* A C caller may pass any int where an enum is expected; giving the enums a
 * fixed underlying type makes every such value representable in C++ (so the
 * library can reject it as DS_ERR_DTYPE and the like) with the same 4-byte
 * layout as the C enums. */
#define DS_ENUM_BASE : int32_t
#else
#define DS_ENUM_BASE
#endif

typedef enum ds_status DS_ENUM_BASE {
    DS_OK = 0,
    DS_ERR_NULL = 1,
    DS_ERR_SIZE = 2,
    DS_ERR_ALIGN = 3,
    DS_ERR_DTYPE = 4,
    DS_ERR_HPARAM = 5,
    DS_ERR_ALIAS = 6,
    DS_ERR_HIP = 7
} ds_status;

/* DS_FP8: 8-bit floats with a scale per 256 elements, for the states of a
 * ds_tensor_list only (every other call refuses it). */
typedef enum ds_dtype DS_ENUM_BASE { DS_FP16 = 1, DS_FP32 = 2, DS_BF16 = 3, DS_FP8 = 4 } ds_dtype;

/*
 * Per-step device state, 128 bytes, kept in caller-owned DEVICE memory so that
 * the kernels read the scale, the overflow flag and the gradient norm without
 * a host sync.  The loss-scaler fields follow the fp16 block of ds_config.json
 * ([Guide] section 4.2: loss_scale 0 = dynamic, initial scale
 * 2^initial_scale_power, loss_scale_window = successful steps before the scale
 * grows, hysteresis = overflows before it shrinks, min_loss_scale = floor).
 * grad_sumsq accumulates the sum of squares of the step's (still scaled)
 * gradient for global-norm clipping ([Guide] section 4.1 gradient_clipping).
 */
typedef struct ds_scaler {
    float scale;                    /* S: loss scale the next step unscales by        */
    float min_scale;                /* floor of S (min_loss_scale)                    */
    int32_t growth_window;          /* W: successful steps before S doubles           */
    int32_t growth_count;           /* successful steps since last overflow or growth */
    int32_t hysteresis;             /* H: overflows needed before S halves            */
    int32_t hysteresis_left;        /* overflows still tolerated before S halves      */
    int32_t dynamic;                /* 1: dynamic scaling; 0: static S                */
    uint32_t overflow;              /* OR of non-finite findings of the current step  */
    int64_t step;                   /* applied Adam steps (t of the last update)      */
    int64_t iter;                   /* all steps, applied or skipped                  */
    int64_t skipped;                /* skipped steps                                  */
    int32_t consecutive_hysteresis; /* 1: a successful step refills hysteresis_left   */
    uint32_t last_overflow;         /* overflow flag consumed by the last update      */
    double grad_sumsq;              /* sum of squares of the step's gradient so far   */
    double last_grad_sumsq;         /* grad_sumsq consumed by the last update         */
    uint32_t blocks_done;           /* ds_adam_step_fused: blocks finished (0 between steps) */
    uint32_t sumsq_blocks_done;     /* sum-of-squares second pass: blocks finished (0 between calls) */
    uint32_t current;               /* ds_adam_step_double_buffered: copy holding the state (0 or 1) */
    uint32_t reserved0;             /* zero                                           */
    uint64_t db_tickets;            /* ds_adam_step_double_buffered: blocks finished (low 32 bits) and
                                       blocks that found a non-finite gradient (high 32 bits); 0 between steps */
    uint8_t reserved[24];           /* zero                                           */
} ds_scaler;

/* sizeof(ds_scaler) as compiled into the library (128). */
size_t ds_scaler_size(void);

/*
 * Initialise a scaler ([Guide] section 4.2).  init_scale = 2^initial_scale_power,
 * min_scale = min_loss_scale, growth_window = loss_scale_window, hysteresis,
 * consecutive_hysteresis, dynamic = (loss_scale == 0); for a static scale pass
 * the fixed scale as init_scale and dynamic = 0.  Sets step = iter = skipped = 0
 * and clears the flag and the gradient sum of squares.  Asynchronous (a
 * one-thread kernel writes the struct).
 * DS_ERR_HPARAM: init_scale or min_scale not finite or <= 0, growth_window < 1,
 * hysteresis < 1.
 */
ds_status ds_state_init(ds_scaler* st, float init_scale, float min_scale, int32_t growth_window,
                        int32_t hysteresis, int32_t consecutive_hysteresis, int32_t dynamic,
                        void* stream);

/* Copy the device state into *host_out (host memory) and synchronise `stream`. */
ds_status ds_state_read(const ds_scaler* st, ds_scaler* host_out, void* stream);

/* Overwrite the device state with *host_in (resume from a snapshot).  The
 * struct is passed by value to a one-thread kernel, so host_in may be freed as
 * soon as the call returns. */
ds_status ds_state_write(ds_scaler* st, const ds_scaler* host_in, void* stream);

/*
 * Gradient accumulation ([Overview] core features: accumulating micro-batch
 * gradients emulates a larger batch; [Guide] section 5.1: backward handles
 * the accumulation; section 4.3: gradient_accumulation_steps).
 *   overwrite != 0 : acc[i] = float(g16[i])            (first micro-batch)
 *   overwrite == 0 : acc[i] = acc[i] + float(g16[i])   (later micro-batches, in order)
 * acc: fp32[n], g16: 16-bit[n] of type gdt (DS_FP16 or DS_BF16; the widening
 * is exact).  If st is not NULL the same pass ORs "acc[i] is not finite" into
 * st->overflow (use it on the last micro-batch: the check of the step then
 * costs no extra pass).  Errors: see the conventions; acc, g16 and st must not
 * overlap; gdt other than DS_FP16/DS_BF16 -> DS_ERR_DTYPE.
 */
ds_status ds_accumulate(float* acc, const uint16_t* g16, ds_dtype gdt, int64_t n, int32_t overwrite,
                        ds_scaler* st_or_null, void* stream);

/*
 * Overflow check ([Overview] core features: dynamic loss scaling; [Guide]
 * section 13.1, gradient overflow in fp16): ORs "some grad[i] is +-inf or NaN"
 * into st->overflow.  grad: fp16[n] (dt = DS_FP16), bf16[n] (DS_BF16) or
 * fp32[n] (DS_FP32).  The largest finite value (65504 in fp16) is not an
 * overflow.  Does nothing more once the flag is already set for this step.
 */
ds_status ds_check_overflow(ds_scaler* st, const void* grad, ds_dtype dt, int64_t n, void* stream);

/*
 * Fused mixed-precision Adam step over n elements ([Guide] section 2: fp32
 * master, first and second moments, fp16 parameter copy; section 4.1:
 * optimizer AdamW with lr, betas, eps, weight_decay; section 5.1: step()).
 * If st->overflow is set the kernel writes nothing (the step is skipped).
 * Otherwise, with S = st->scale, K = accum_steps and t = st->step + 1:
 *   g      = grad[i] / (S*K)                     (unscale; grad fp16 or fp32)
 *            (with max_grad_norm > 0 the multiplier 1/(S*K) is scaled by the
 *             global-norm clipping coefficient below)
 *   m[i]   = beta1*m[i] + (1-beta1)*g
 *   v[i]   = beta2*v[i] + (1-beta2)*g*g
 *   master = master - lr*weight_decay*master     (only if weight_decay != 0)
 *   master = master - lr/(1-beta1^t) * m[i] / (sqrt(v[i])/sqrt(1-beta2^t) + eps)
 *   p16[i] = fp16(master[i]) or bf16(master[i])  (pdt; round to nearest even)
 * in IEEE fp32, one rounding per operation; the two bias-correction factors
 * are evaluated in fp64 and rounded once.  master/m/v: fp32[n] in place;
 * p16: 16-bit[n] out, of type pdt (DS_FP16 or DS_BF16); grad: [n] in, of
 * type dt (DS_FP16, DS_BF16, or DS_FP32 for the accumulation buffer).  st is
 * read only (t and S advance in ds_update_loss_scale).
 * Global-norm clipping ([Guide] sections 4.1 and 5.4 gradient_clipping,
 * section 5.1 step() includes clipping): with max_grad_norm > 0, using the
 * step's st->grad_sumsq (filled by ds_check_overflow_sumsq or
 * ds_accumulate_sumsq over the whole partition) and inv = fp32(1/(S*K)):
 *   norm = sqrt(grad_sumsq) * inv                         (fp64)
 *   coef = min(1, max_grad_norm / (norm + 1e-6))          (fp64)
 *   the multiplier of the gradient becomes fp32(inv * coef)
 * max_grad_norm = 0 disables clipping (the multiplier is inv).
 * DS_ERR_HPARAM: lr, weight_decay or max_grad_norm negative or not finite,
 * beta1 or beta2 outside [0, 1), eps not finite or <= 0, accum_steps < 1.
 */
ds_status ds_adam_step(const ds_scaler* st, float* master, float* m, float* v, uint16_t* p16,
                       ds_dtype pdt, const void* grad, ds_dtype dt, int64_t n, float lr, float beta1,
                       float beta2, float eps, float weight_decay, float max_grad_norm,
                       int32_t accum_steps, void* stream);

/*
 * Learning-rate schedules ([Guide] section 4.1: the scheduler block of the
 * base ds_config.json, WarmupLR; section 4.4: WarmupDecayLR with
 * warmup_min_lr, warmup_max_lr, warmup_num_steps, total_num_steps and a
 * linear warmup).  The pages give the parameters, not the formula; the
 * schedule read here: with it = st->step, the count of Adam steps applied
 * before this one (a fresh run starts at 0; a skipped step does not advance
 * it, so the schedule stays on the device and resumes with the state),
 *   gamma = it / warmup_num_steps                    while it < warmup_num_steps
 *         = 1                                        afterwards, DS_LR_WARMUP
 *         = max(0, (total - it) / max(1, total - warmup_num_steps))
 *                                                    afterwards, DS_LR_WARMUP_DECAY
 *   lr    = warmup_min_lr + (warmup_max_lr - warmup_min_lr) * gamma
 * in fp64, rounded once to fp32; that lr then enters the step like a
 * constant lr.  A host struct, read during the call and not kept.
 * Valid: kind one of the two below, both rates finite and >= 0,
 * warmup_num_steps >= 0, and for DS_LR_WARMUP_DECAY total_num_steps >=
 * warmup_num_steps; anything else is DS_ERR_HPARAM.
 */
typedef enum ds_lr_kind DS_ENUM_BASE { DS_LR_WARMUP = 1, DS_LR_WARMUP_DECAY = 2 } ds_lr_kind;

typedef struct ds_lr_schedule {
    int32_t kind;             /* ds_lr_kind */
    int32_t reserved;         /* set to 0 */
    int64_t warmup_num_steps; /* applied steps of the linear rise */
    int64_t total_num_steps;  /* DS_LR_WARMUP_DECAY: where the fall ends; else ignored */
    float warmup_min_lr;      /* lr of the first step, and the end of the fall */
    float warmup_max_lr;      /* the peak, reached after the warmup */
} ds_lr_schedule;

/*
 * ds_adam_step with the learning rate taken from `sched` (a HOST pointer) at
 * the device's applied-step count, so a whole step, schedule included, runs
 * without a host round trip (and can be captured once into a graph and
 * replayed).  Every other argument, the arithmetic and the errors are those
 * of ds_adam_step; sched NULL is DS_ERR_NULL, an invalid schedule
 * DS_ERR_HPARAM.
 */
ds_status ds_adam_step_sched(const ds_scaler* st, float* master, float* m, float* v, uint16_t* p16,
                             ds_dtype pdt, const void* grad, ds_dtype dt, int64_t n,
                             const ds_lr_schedule* sched, float beta1, float beta2, float eps,
                             float weight_decay, float max_grad_norm, int32_t accum_steps,
                             void* stream);

/*
 * ds_adam_step (sched_or_null NULL: constant lr) or ds_adam_step_sched
 * (sched_or_null: a host ds_lr_schedule, lr ignored) followed by
 * ds_update_loss_scale, in one kernel: for a partition updated by a single
 * call per step, which then calls no ds_update_loss_scale of its own.  Each
 * block of the kernel, when done, takes a ticket from st->blocks_done (one
 * atomic add); the block with the last ticket advances the scaler exactly as
 * ds_update_loss_scale does and sets the count back to 0.  Arithmetic,
 * results and errors are those of the two calls it replaces; with n == 0
 * only the scaler advances.  st is read and written.
 */
ds_status ds_adam_step_fused(ds_scaler* st, float* master, float* m, float* v, uint16_t* p16, ds_dtype pdt,
                             const void* grad, ds_dtype dt, int64_t n, float lr,
                             const ds_lr_schedule* sched_or_null, float beta1, float beta2, float eps,
                             float weight_decay, float max_grad_norm, int32_t accum_steps, void* stream);

/*
 * A whole step for a caller that keeps two copies (0 and 1) of the fp32
 * master, m and v arrays and of the 16-bit parameter copy (30 bytes of device
 * memory per element instead of 16), in one HBM pass: the overflow check of
 * the gradient is fused into the Adam pass ([Guide] section 2, section 4.2
 * dynamic loss scaling, section 5.1 step()).  st->current names the copy that
 * holds the state.  The kernel reads the gradient and the current copy once,
 * tests whether some gradient value is +-inf or NaN, and writes the Adam
 * update of every element (the arithmetic of ds_adam_step) into the other
 * copy; each block's finding travels in its ticket (st->db_tickets), and the
 * last block to finish advances the scaler as ds_update_loss_scale does with
 * the OR of all findings and st->overflow and, if the step applied (no
 * overflow), makes the other copy current.  A skipped step leaves the current
 * copy bit-identical (only the other copy, which holds no state, is written)
 * and t unchanged.
 * The step moves 28 bytes per element with an fp16 gradient instead of the
 * 30 of ds_check_overflow + ds_adam_step_fused.  Call it once per step for the
 * whole partition, in place of ds_check_overflow and ds_adam_step_fused (a flag
 * already raised earlier in the step, e.g. by a fused accumulation check, also
 * skips it).  No gradient clipping (it needs the whole gradient's norm before
 * the update).
 * master2, m2, v2: HOST arrays of 2 DEVICE pointers to fp32[n]; p16_2: HOST
 * array of 2 DEVICE pointers to 16-bit[n] of type pdt; the eight arrays, grad
 * and st must not overlap.  lr / sched_or_null, betas, eps, weight_decay,
 * accum_steps, grad and dt: as for ds_adam_step_fused.  With n == 0 only the
 * scaler advances (and the copies swap if the step applied).  The copy that
 * is current after a call is read back with ds_state_read (st.current).
 * Errors: as for ds_adam_step_fused; a NULL host array -> DS_ERR_NULL.
 */
ds_status ds_adam_step_double_buffered(ds_scaler* st, float* const* master2, float* const* m2, float* const* v2,
                                       uint16_t* const* p16_2, ds_dtype pdt, const void* grad, ds_dtype dt,
                                       int64_t n, float lr, const ds_lr_schedule* sched_or_null, float beta1,
                                       float beta2, float eps, float weight_decay, int32_t accum_steps,
                                       void* stream);

/*
 * The last micro-batches of a step folded into the double-buffered Adam pass
 * ([Guide] section 4.3 gradient accumulation, [Overview] gradient
 * accumulation; [Guide] section 4.2 dynamic loss scaling, section 5.1
 * step()).  The gradient of element i is the fp32 sum, in micro-batch order,
 * of acc_or_null[i] (the running sum of the step's earlier micro-batches as
 * ds_accumulate / ds_accumulate_multi leave it; NULL when grads are all of the
 * step's micro-batches, the first of them then starting the sum) and of
 * grads[0][i] .. grads[count-1][i]: the sum ds_accumulate would have formed,
 * which is used, not stored.  The pass ORs "some sum is +-inf or NaN" into
 * st->overflow and writes the Adam update of every element of [0, n) (the
 * arithmetic of ds_adam_step with that sum as the fp32 gradient) into the copy
 * of master, m, v and the 16-bit copy that does not hold the state
 * (st->current names the one that does); nothing else in st changes.  Call it
 * once for the partition, or once per bucket (disjoint ranges, each with its
 * own offsets into every array), then ds_update_loss_scale_double_buffered
 * exactly once.  The step's earlier micro-batches go through ds_accumulate
 * (with st_or_null NULL or not: a flag raised there also skips the step).
 * Bytes per element: 2 * count + 30 with the running sum (read only), 2 *
 * count + 26 without, against 2 * count + 8 (or + 4) for the fold and 30 for
 * the Adam pass done separately.  No gradient clipping (it needs the whole
 * gradient's norm before the update).
 * master2, m2, v2, p16_2, pdt, lr / sched_or_null, betas, eps, weight_decay,
 * accum_steps (K, the unscale divisor), stream: as for
 * ds_adam_step_double_buffered.  grads: HOST array of count (1-8) DEVICE
 * pointers to 16-bit[n] of format gdt (fp16 or bf16); they may repeat but
 * must not overlap acc, st or the eight state arrays, which must not overlap
 * one another.  acc_or_null: DEVICE fp32[n] or NULL.
 * Errors: count outside 1..8 -> DS_ERR_SIZE; gdt or pdt not a 16-bit format ->
 * DS_ERR_DTYPE; acc_or_null NULL with count != accum_steps, or non-NULL with
 * count >= accum_steps -> DS_ERR_HPARAM; otherwise as for
 * ds_adam_step_double_buffered.  With n == 0 nothing is launched.
 */
ds_status ds_accumulate_adam_double_buffered(ds_scaler* st, float* const* master2, float* const* m2,
                                             float* const* v2, uint16_t* const* p16_2, ds_dtype pdt,
                                             const float* acc_or_null, const uint16_t* const* grads, int32_t count,
                                             ds_dtype gdt, int64_t n, float lr, const ds_lr_schedule* sched_or_null,
                                             float beta1, float beta2, float eps, float weight_decay,
                                             int32_t accum_steps, void* stream);

/*
 * End of a double-buffered step taken with ds_accumulate_adam_double_buffered
 * ([Guide] section 4.2): advance the scaler by the step's flag as
 * ds_update_loss_scale does and, if the step applied (no overflow), make the
 * other copy current (st->current ^= 1).  Call exactly once per step.
 * Errors: st NULL -> DS_ERR_NULL; st not 8-byte aligned -> DS_ERR_ALIGN.
 */
ds_status ds_update_loss_scale_double_buffered(ds_scaler* st, void* stream);

/*
 * End of a step: advance the scaler by the step's overflow flag, then clear
 * the flag ([Guide] section 4.2).  Overflow: skipped += 1, growth_count = 0;
 * if dynamic, one more overflow is charged to the hysteresis and, when it is
 * used up, S = max(S/2, min_scale) and the hysteresis restarts.  No overflow:
 * step += 1; if dynamic, growth_count += 1 and at growth_window S doubles and
 * growth_count restarts (consecutive_hysteresis refills the hysteresis).
 * iter += 1, last_overflow = flag and last_grad_sumsq = grad_sumsq in both
 * cases; grad_sumsq restarts at 0.  Call exactly once per step.
 */
ds_status ds_update_loss_scale(ds_scaler* st, void* stream);

/*
 * Gradient sum of squares for global-norm clipping, fused into the passes
 * that already read the gradient.  Both add sum(x_i^2) over their n values
 * (the stored, still loss-scaled gradient: fp16 values, or the fp32
 * accumulation) into st->grad_sumsq, in fp64.  The sum is taken over fixed
 * chunks of consecutive elements (8192 for the check, 1024 for the
 * accumulation), each reduced in a fixed order, then over groups of 4096
 * chunk sums and the group sums, each in a fixed order, so the result does
 * not depend on the launch shape.  Several calls per step (disjoint ranges,
 * e.g. buckets) add up in call order.
 *
 * workspace: caller-owned DEVICE scratch of at least
 * ds_sumsq_workspace_bytes(n) bytes (one fp64 partial sum per chunk and per
 * group), 8-byte aligned, no initial contents needed.  Each call is two
 * kernels: the pass over the data writes the chunk sums, a second pass adds
 * them by groups, and its last block to finish adds the group sums (taking
 * one ticket per block from st->sumsq_blocks_done, which it leaves at 0).
 * One workspace serves every call on one stream (calls that may run at the
 * same time need their own).
 * Errors as for the plain entry points; DS_ERR_NULL / DS_ERR_SIZE /
 * DS_ERR_ALIGN / DS_ERR_ALIAS also cover the workspace.
 */
size_t ds_sumsq_workspace_bytes(int64_t n);

/* ds_check_overflow plus the sum of squares of grad (fp16, bf16 or fp32), one pass. */
ds_status ds_check_overflow_sumsq(ds_scaler* st, const void* grad, ds_dtype dt, int64_t n,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * ds_check_overflow_sumsq without a caller workspace, for callers that cannot
 * allocate device memory: code under stream or graph capture, tight serving
 * loops, harnesses that forbid allocation.  The call allocates nothing: the
 * chunk and group sums go to a scratch array of 2^21 fp64 values (16 MiB)
 * that the library holds in each device's memory until the process ends.
 * Flag and sum of squares are bit-identical to those of
 * ds_check_overflow_sumsq.  n may be at most DS_NOALLOC_MAX_ELEMS (2,096,640
 * chunks of 8192 elements); a larger n is DS_ERR_SIZE.  The first call on a
 * device (the device of `stream`, or the current one for the null stream)
 * looks up the address of that device's array and keeps it; DS_ERR_HIP if
 * that fails.  Every call on one device shares that device's array, which
 * keeps the last call's contents: calls that may run at the same time on one
 * device (other streams, other threads) race and give wrong sums, so order
 * them on one stream.  Nothing in the array needs to start at zero: every
 * chunk and group sum is written before it is read.
 */
#define DS_NOALLOC_MAX_ELEMS 17175674880LL
ds_status ds_check_overflow_sumsq_noalloc(ds_scaler* st, const void* grad, ds_dtype dt, int64_t n, void* stream);

/* ds_accumulate with the fused overflow check (st required) plus the sum of
 * squares of the accumulated values, one pass: use it for the last
 * micro-batch of a clipped step. */
ds_status ds_accumulate_sumsq(float* acc, const uint16_t* g16, ds_dtype gdt, int64_t n,
                              int32_t overwrite, ds_scaler* st, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * Several micro-batch gradients folded into the accumulation buffer in one
 * pass (gradient accumulation as for ds_accumulate: [Overview] core features;
 * [Guide] sections 4.3 and 5.1):
 *   acc[i] = (overwrite ? float(g_0[i]) : acc[i] + float(g_0[i]))
 *            + float(g_1[i]) + ... + float(g_{count-1}[i])
 * with every add an fp32 add in this order, so the result is bit for bit that
 * of `count` consecutive ds_accumulate calls.  A caller that can hold `count`
 * 16-bit micro-batch gradients at once (grads[k] is the k-th in micro-batch
 * order) moves 2 * count + 8 bytes per element (2 * count + 4 when
 * overwriting) instead of 10 bytes per micro-batch.
 * grads: HOST array of `count` (1..8) DEVICE pointers to 16-bit[n] arrays of
 * type gdt; they may repeat or overlap one another but not acc, st or the
 * workspace.  st_or_null: as for ds_accumulate (the fused inf/NaN check of the
 * result).  workspace_or_null: as for ds_accumulate_sumsq (requires st; adds
 * the sum of squares of the result to st->grad_sumsq, same chunks, so the
 * value equals that of a ds_accumulate_sumsq pass producing the same acc).
 * Errors: count outside 1..8 -> DS_ERR_SIZE; otherwise as ds_accumulate and
 * ds_accumulate_sumsq.
 */
ds_status ds_accumulate_multi(float* acc, const uint16_t* const* grads, int32_t count, ds_dtype gdt, int64_t n,
                              int32_t overwrite, ds_scaler* st_or_null, void* workspace_or_null,
                              size_t workspace_bytes, void* stream);

/*
 * The bias-correction scalars the next applied step will use, evaluated on
 * the device exactly as ds_adam_step does (t = st->step + 1):
 * out2[0] = fp32(lr / (1 - beta1^t)), out2[1] = fp32(1 / sqrt(1 - beta2^t)).
 * out2: device float[2].  For diagnostics and tests.
 */
ds_status ds_adam_bias_scalars(const ds_scaler* st, float lr, float beta1, float beta2,
                               float* out2, void* stream);

/*
 * The scheduled learning rate and bias-correction scalars the next applied
 * step will use, evaluated on the device exactly as ds_adam_step_sched does:
 * out3[0] = lr, out3[1] = fp32(lr / (1 - beta1^t)),
 * out3[2] = fp32(1 / sqrt(1 - beta2^t)), t = st->step + 1.
 * sched: host struct; out3: device float[3].  For diagnostics and tests.
 */
ds_status ds_lr_scalars(const ds_scaler* st, const ds_lr_schedule* sched, float beta1, float beta2,
                        float* out3, void* stream);

/*
 * Flat layout of ragged tensors in contiguous buffers with greedy buckets
 * ([Guide] sections 2.2 and 4.1: contiguous_gradients, reduce_bucket_size and
 * allgather_bucket_size of 2e8 elements).  Host-only, no device work.
 * Tensors keep their order; tensor i starts at offsets[i], a multiple of
 * `align` elements.  A tensor joins the open bucket if the bucket, padded to
 * `align`, then holds at most `cap` elements; otherwise the bucket closes and
 * the tensor opens the next one (a tensor larger than cap gets its own
 * bucket).  Outputs (host arrays of `count` entries, caller-owned): offsets,
 * bucket_of; bucket_start and bucket_size (first *n_buckets entries used);
 * *total = padded length of the flat array.  DS_ERR_SIZE: count < 0, a
 * negative size, cap < 1, align < 1, cap or align above 2^40, or sizes whose
 * sum plus count * (align - 1) exceeds 2^40 (nothing is written then).
 */
ds_status ds_layout_greedy(const int64_t* numels, int32_t count, int64_t cap, int64_t align,
                           int64_t* offsets, int32_t* bucket_of, int64_t* bucket_start,
                           int64_t* bucket_size, int32_t* n_buckets, int64_t* total);

/*
 * ZeRO partition of a flat array of `total` elements over `world` ranks
 * ([Guide] sections 2.1 and 2.2: each rank owns a contiguous 1/N share):
 * rank r gets [r*per, min((r+1)*per, total)) with per = ceil(total/world)
 * rounded up to `align`.  Host-only.  DS_ERR_SIZE: total outside
 * [0, 2^40], world < 1, rank outside [0, world), align outside [1, 2^40].
 */
ds_status ds_partition_range(int64_t total, int32_t world, int32_t rank, int64_t align,
                             int64_t* start, int64_t* count);

/*
 * ---------------------------------------------------------------------------
 * The optimizer step over a list of tensors
 * ---------------------------------------------------------------------------
 * For parameters that are not one flat partition: expert groups, norms and
 * biases with a decay of their own, fp32 parameters beside 16-bit ones.  One
 * call covers every tensor of the list, gated by the same ds_scaler; the two
 * Adam states are held in 32 bits (DS_FP32: the arithmetic of ds_adam_step) or
 * in 8 (DS_FP8: as below).
 *
 * 8-bit states.  Element i of a tensor belongs to block i / 256 of that tensor
 * (the last block may be short).  m is stored as e4m3 codes (sign, 4 exponent
 * bits with bias 7, 3 mantissa bits; no infinity, 0x7F is NaN, the largest
 * value 448), v as e5m2 codes (5 exponent bits with bias 15, 2 mantissa bits;
 * the largest finite value 57344, 0x7F is NaN), with one fp32 scale per block
 * and state; a code of value c stands for c * scale.  A step decodes m and v
 * and updates them in fp32 as ds_adam_step does.  The parameter moves by the new
 * m and v before they are rounded, in fp32, but with the hardware's square root
 * and reciprocal (each within 1 unit in the last place) and fused multiply-adds:
 *   p = p - lr_j weight_decay p
 *   p = p - step_size (m (1 / max(sqrt(v) rbc2 + eps, 2^-126)))
 * (step_size = lr_j / (1 - beta1^t), rbc2 = 1 / sqrt(1 - beta2^t)), so it is
 * within a few units of ds_adam_step's, not its bits.  Then x = m, v
 * are encoded, with max = 448, 57344:
 *   top   = max |x| over the block, at most 2^126
 *   scale = top / max,  a = min(|x| * (max * (1 / top)), max)
 *           (top < 2^-110: scale 0 and a = 0)
 *   code  = floor(a / ulp + u) steps of ulp: 2^(max(floor(log2 a), -6) - 3)
 *           for m, 2^(max(floor(log2 a), -14) - 2) for v
 * with u = 1/2 (DS_ROUND_NEAREST) or a dither in [0, 1) (DS_ROUND_DITHER).
 * A positive v never becomes code 0 but code 1, since 0 would leave a zero
 * denominator under a moment that is not zero (under a scale of 0 code 1 stands
 * for 0 too).  A NaN is kept as a NaN code.  Why a
 * dither: v moves by (1 - beta2) of itself or less per step, far below half a
 * step of its code, so rounding to nearest would hold it where it is; with
 * the dither the expected value of the stored state is the fp32 one (a
 * positive v below the smallest code aside).
 * The dither is fixed by (seed, t, tensor index, block, element), so a
 * repeated step gives the same bits.  With all arithmetic modulo 2^32,
 * G = 0x9E3779B9 and mix(x): x ^= x >> 16, x *= 0x6A09E667, x ^= x >> 15,
 * x *= 0xBB67AE85, x ^= x >> 16:
 *   k = mix(mix(seed >> 32) ^ seed);  k = mix(k + t * G);
 *   k = mix(k + tensor * G);          k = mix(k + block * G)
 *   u of m = ((k + (i % 256) * G) >> 12) / 2^20
 *   u of v = ((mix(k ^ 0xBB67AE85) + (i % 256) * G) >> 11) / 2^21
 */
typedef enum ds_rounding DS_ENUM_BASE { DS_ROUND_NEAREST = 0, DS_ROUND_DITHER = 1 } ds_rounding;

/* Elements that share one scale of an 8-bit state. */
#define DS_STATE_BLOCK 256

/* One tensor of a list (host memory; the arrays are device memory). */
typedef struct ds_tensor {
    float* master;       /* fp32[n], in and out */
    uint16_t* p16;       /* 16-bit[n] out, of type pdt; NULL with pdt DS_FP32 */
    void* m;             /* fp32[n], or e4m3 codes [n] */
    void* v;             /* fp32[n], or e5m2 codes [n] */
    float* m_scale;      /* fp32[ceil(n / 256)] for 8-bit states, else NULL */
    float* v_scale;      /* likewise */
    const void* grad;    /* [n] of type gdt */
    int64_t n;           /* elements; 0 is allowed (the pointers may be NULL then) */
    float weight_decay;  /* this tensor's */
    float lr_scale;      /* multiplies the learning rate for this tensor */
    ds_dtype pdt;        /* DS_FP16, DS_BF16, or DS_FP32: the master is the parameter */
    ds_dtype gdt;        /* DS_FP16, DS_BF16 or DS_FP32 */
} ds_tensor;

/* A list as the calls below take it (host memory, filled by
 * ds_tensor_list_write, passed back unchanged). */
typedef struct ds_tensor_list {
    void* table;         /* the device table */
    int64_t tiles;       /* tiles of 4096 elements over all tensors */
    int64_t elems;       /* elements over all tensors */
    int32_t count;       /* tensors */
    ds_dtype sdt;        /* DS_FP32 or DS_FP8 */
} ds_tensor_list;

/* Device bytes of the table of a list of `count` tensors (0 for count < 0). */
size_t ds_tensor_list_bytes(int32_t count);

/*
 * Describe `count` tensors to the device: validates them, writes the table
 * (caller-owned device memory of at least ds_tensor_list_bytes(count) bytes,
 * 16-byte aligned) with kernels that carry the descriptors as arguments, so
 * it can be captured and `tensors` may be freed on return, and fills *list.
 * Write it again when an address changes (new gradient tensors); steps already
 * enqueued on the same stream use the table as it was.  The arrays need the
 * alignment of their element type only; whole 4096-element tiles whose arrays
 * are 16-byte (16-bit arrays 8-byte, codes 4-byte) aligned move in vectors.
 * Errors: count < 0 or above 2^20, some n < 0, or more than 2^40 elements in
 * all -> DS_ERR_SIZE, likewise a short table; list NULL, or (count > 0) tensors
 * or table NULL, or a NULL array of a tensor with n > 0 -> DS_ERR_NULL; sdt not
 * DS_FP32 / DS_FP8, or an unknown pdt or gdt -> DS_ERR_DTYPE; p16 given with
 * pdt DS_FP32 or a scale array given with 32-bit states, weight_decay or
 * lr_scale negative or not finite -> DS_ERR_HPARAM; a misaligned pointer ->
 * DS_ERR_ALIGN; a written array that overlaps any other array or the table ->
 * DS_ERR_ALIAS (gradients may overlap one another).
 */
ds_status ds_tensor_list_write(ds_tensor_list* list, void* table, size_t table_bytes, const ds_tensor* tensors,
                               int32_t count, ds_dtype sdt, void* stream);

/* Workspace of ds_check_overflow_list with the sum of squares: one fp64 per
 * group of tiles (of one tile up to 2048 of them, of four above) and per 4096
 * groups (0 for list NULL). */
size_t ds_tensor_list_workspace_bytes(const ds_tensor_list* list);

/*
 * ds_check_overflow over every gradient of the list, and with a workspace
 * (device, 8-byte aligned, no initial contents) also the sum of squares as
 * ds_check_overflow_sumsq: per tile (per four of a list of more than 2048) in a
 * fixed order, then per 4096 of those sums, so the result depends on the list
 * alone.  It adds to st->grad_sumsq, so a flat partition checked in the same
 * step is clipped by the joint norm.  An empty list launches nothing.  Errors as for ds_check_overflow_sumsq, but that the
 * scaler and the workspace are compared with the table and with one another
 * only: the addresses of the list's arrays are on the device, and the caller
 * keeps both apart from them (so too in the two calls below).  A list that
 * ds_tensor_list_write has not filled -> DS_ERR_NULL / DS_ERR_SIZE.
 */
ds_status ds_check_overflow_list(ds_scaler* st, const ds_tensor_list* list, void* workspace_or_null,
                                 size_t workspace_bytes, void* stream);

/*
 * The gated Adam step over every tensor of the list in one kernel, with the
 * arithmetic above (lr / sched_or_null, eps, max_grad_norm and accum_steps as
 * in ds_adam_step) and lr_j = lr * lr_scale (fp32) and weight_decay of
 * each tensor.  The betas come in 64 bits: 1 - beta is formed there and then
 * rounded (1 - 0.999f in fp32 is 4.7e-5 off 0.001, as much as 8-bit codes can
 * see); with 32-bit states, betas that fp32 holds give the bits of
 * ds_adam_step.  end_step != 0 also advances the scaler, as
 * ds_adam_step_fused does; 0 leaves that to a later call of the same step
 * (another list, or a flat partition's ds_adam_step_fused).  rounding and seed:
 * of 8-bit states (ignored with 32-bit ones).  An empty list only advances the
 * scaler, if asked.  Errors as for ds_adam_step_fused; an unknown rounding ->
 * DS_ERR_HPARAM.
 */
ds_status ds_adam_step_list(ds_scaler* st, const ds_tensor_list* list, float lr,
                            const ds_lr_schedule* sched_or_null, double beta1, double beta2, float eps,
                            float max_grad_norm, int32_t accum_steps, ds_rounding rounding, uint64_t seed,
                            int32_t end_step, void* stream);

/*
 * A whole step over one list: ds_check_overflow_list, then ds_adam_step_list
 * with end_step, to the same bits.  Short lists take fewer launches: one up to
 * 8 tiles, where every block of the update checks the whole list itself, and
 * with a workspace two up to 2048 tiles, where every block adds the check's
 * partial sums itself.  What was checked before in the same step (a flat partition,
 * another list) counts here as for ds_adam_step_list.  Without a workspace this
 * list's squares are not summed: max_grad_norm > 0 then clips by what other calls
 * of the step have summed (by nothing, if none has).  Errors as for the two calls;
 * refused as a whole.
 */
ds_status ds_step_list(ds_scaler* st, const ds_tensor_list* list, void* workspace_or_null, size_t workspace_bytes,
                       float lr, const ds_lr_schedule* sched_or_null, double beta1, double beta2, float eps,
                       float max_grad_norm, int32_t accum_steps, ds_rounding rounding, uint64_t seed, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Balance loss of a mixture-of-experts router, counts per expert, gradient
 * ---------------------------------------------------------------------------
 * logits: [tokens] rows of `experts` values of type dt (DS_FP16, DS_BF16 or
 * DS_FP32), row t starting row_stride elements after row t - 1.  A row is used
 * if mask is NULL or mask[t] != 0, and some logit is above -infinity; T' is
 * the number of used rows (*used).  Over used rows, with p = softmax(row):
 *   counts[e] = rows in which e is among the k largest logits (of equal logits
 *               the lowest index first; a logit of -infinity is never chosen)
 *   f_e = counts[e] / (k T'),  mean_prob[e] = sum_t p_te / T'
 *   loss = coef * experts * sum_e f_e mean_prob[e]
 * and, f being constant,
 *   d loss / d logit_tj = coef * experts / T' * p_tj (f_j - sum_e f_e p_te)
 * T' = 0: mean_prob, loss and the gradient are 0.  Rows that are not used have
 * gradient 0, whatever they hold.  A used row with a NaN or +infinity makes
 * mean_prob, the loss and its own gradient NaN and counts nothing.  fp32
 * arithmetic per row; sums over rows in fp32 for some thousand rows at most,
 * over these in fp64, in a fixed order (the same bits every call).
 */
#define DS_MAX_EXPERTS 512
#define DS_MAX_EXPERT_CHOICES 16

/* Device scratch of ds_balance_loss (0 for sizes out of range). */
size_t ds_balance_workspace_bytes(int64_t tokens, int32_t experts);

/*
 * counts: int32[experts], mean_prob: fp32[experts], loss: fp32[1], used:
 * int32[1], all device, all written.  workspace: device, 8-byte aligned,
 * cleared to zero once before its first call (it holds a count of finished
 * blocks that every call leaves at zero; later calls may have other sizes, but
 * not run at the same time).  tokens may be 0 (logits may be NULL then).
 * Errors: tokens outside [0, 2^30], experts outside 1..512, k outside
 * 1..min(experts, 16), row_stride < experts, a short workspace -> DS_ERR_SIZE;
 * coef not finite or negative -> DS_ERR_HPARAM; else as in the conventions
 * (logits need the alignment of their type).
 */
ds_status ds_balance_loss(const void* logits, ds_dtype dt, int64_t tokens, int32_t experts, int64_t row_stride,
                          const uint8_t* mask_or_null, int32_t k, float coef, int32_t* counts, float* mean_prob,
                          float* loss, int32_t* used, void* workspace, size_t workspace_bytes, void* stream);

/*
 * The gradient, from the same logits and mask and the counts and *used that
 * ds_balance_loss left on the device: dlogits (type dt, row stride
 * grad_stride) = S * d loss / d logits, with S = st->scale read on the device
 * (st_or_null NULL: 1), so that it joins a loss-scaled backward pass.
 * accumulate != 0 adds to what dlogits holds (the sum in fp32, rounded once;
 * rows that are not used stay as they are); 0 overwrites.  dlogits, from its
 * first to its last element, must not overlap any other array.  Errors as for
 * ds_balance_loss.
 */
ds_status ds_balance_loss_grad(const ds_scaler* st_or_null, const void* logits, ds_dtype dt, int64_t tokens,
                               int32_t experts, int64_t row_stride, const uint8_t* mask_or_null, int32_t k,
                               float coef, const int32_t* counts, const int32_t* used, void* dlogits,
                               int64_t grad_stride, int32_t accumulate, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Tokens sorted by expert, moved there and back, with the gradients
 * ---------------------------------------------------------------------------
 * chosen: [tokens] rows of k expert numbers (int32 or int64: index_bytes 4 or
 * 8), rows row_stride elements apart.  A number outside 0..experts-1 drops its
 * choice (a token over an expert's capacity).  The pairs p = t k + j that are
 * not dropped are sorted by expert, and by p inside an expert: pair p has slot
 * place[p] (dropped: -1), slot q holds pair source[q] (behind the last one: -1),
 * and expert e has the slots offsets[e] .. offsets[e + 1] - 1.  The same expert
 * twice in a row is two pairs.
 *
 * The moves take rows of `width` values of type dt (DS_FP16, DS_BF16, DS_FP32):
 *   gather        out[place[t k + j]] = x[t]
 *   gather_grad   dx[t] = sum_j dout[place[t k + j]]
 *   combine       out[t] = sum_j gate_tj rows[place[t k + j]]
 *   combine_grad  drows[place[t k + j]] = gate_tj dout[t],
 *                 dgate_tj = sum_d dout[t]_d rows[place[t k + j]]_d
 * over the choices that are not dropped (a token without any: 0; a dropped
 * choice's gate is not read, its dgate is 0).  Sums in fp32 in a fixed order (j
 * ascending), rounded once.  Rows of the sorted side behind the last slot are
 * left as they are, and a slot of place at or past the sorted side's row count
 * is passed over.  Gates and their gradients have the type gdt, any of the
 * three.  Every array needs the alignment of its type only.
 * Limits: experts 1..512, k 1..16, tokens k < 2^31, width 1..2^24.  Errors:
 * sizes, strides smaller than a row or a short workspace -> DS_ERR_SIZE;
 * an unknown dt, gdt or index_bytes -> DS_ERR_DTYPE; else as in the conventions.
 */

/* Device scratch of ds_dispatch_sort (0 for sizes out of range); what serves many tokens serves fewer. */
size_t ds_dispatch_workspace_bytes(int64_t tokens, int32_t experts, int32_t k);

/* offsets: int32[experts + 1], place and source: int32[tokens k], all written.
 * workspace: device, 4-byte aligned, no initial contents. */
ds_status ds_dispatch_sort(const void* chosen, int32_t index_bytes, int64_t tokens, int32_t experts, int32_t k,
                           int64_t row_stride, int32_t* offsets, int32_t* place, int32_t* source, void* workspace,
                           size_t workspace_bytes, void* stream);

ds_status ds_dispatch_gather(const void* x, ds_dtype dt, int64_t tokens, int32_t k, int64_t width, int64_t x_stride,
                             const int32_t* place, void* out, int64_t out_stride, int64_t out_rows, void* stream);

ds_status ds_dispatch_gather_grad(const void* dout, ds_dtype dt, int64_t tokens, int32_t k, int64_t width,
                                  int64_t dout_stride, int64_t dout_rows, const int32_t* place, void* dx,
                                  int64_t dx_stride, void* stream);

ds_status ds_dispatch_combine(const void* rows, ds_dtype dt, int64_t tokens, int32_t k, int64_t width, int64_t rows_stride,
                              int64_t rows_count, const int32_t* place, const void* gates, ds_dtype gdt,
                              int64_t gates_stride, void* out, int64_t out_stride, void* stream);

ds_status ds_dispatch_combine_grad(const void* dout, ds_dtype dt, int64_t tokens, int32_t k, int64_t width,
                                   int64_t dout_stride, const void* rows, int64_t rows_stride, int64_t rows_count,
                                   const int32_t* place, const void* gates, ds_dtype gdt, int64_t gates_stride, void* drows,
                                   int64_t drows_stride, void* dgates, int64_t dgates_stride, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Distillation from a teacher's top logits, with the gradient
 * ---------------------------------------------------------------------------
 * logits: the student's, [tokens] rows of `vocab` values of type dt, row_stride
 * apart.  teacher, index: [tokens] rows of k of the teacher's logits (type tdt)
 * and their places in the vocabulary (int32 or int64: index_bytes 4 or 8), in
 * any order; a negative place is an absent entry, so that rows may have
 * different numbers of them; the same place twice adds up.  A row is used if
 * mask is NULL or mask[t] != 0, it has an entry above -infinity, and some logit
 * is above -infinity; T' is the number of used rows (*used).  With q the softmax
 * of the row's entries / temperature and p that of its logits / temperature:
 *   token_loss[t] = temperature^2 sum_j q_j (log q_j - log p_place(j))
 *   loss = coef / T' sum over used rows of token_loss[t]
 *   dlogits_tv = S coef temperature / T' (p_v - sum of q_j with place(j) = v)
 * with S = st->scale read on the device (st_or_null NULL: 1).  Entries with q_j
 * = 0 add nothing.  token_loss and the gradient of rows that are not used are 0,
 * whatever they hold; T' = 0: loss 0.  A used row with a NaN or +infinity, or
 * with a place at or past vocab, has a NaN loss and a gradient of NaN.  fp32
 * arithmetic per row, rounded once; the mean over rows in fp64 in a fixed order.
 * dlogits_or_null (type dt, rows grad_stride apart) may be the logits
 * themselves, with the same stride; else it overlaps no other array.
 * accumulate != 0 adds to what it holds (in fp32, rounded once; rows that are
 * not used stay as they are).  token_loss: fp32[tokens], loss: fp32[1], used:
 * int32[1].  workspace: device, 8-byte aligned, cleared to zero once before its
 * first call (every call leaves its count at zero; calls that share it must not
 * run at the same time).  Arrays need the alignment of their type only.
 * Errors: tokens outside [0, 2^30], vocab outside [1, 2^30], k outside 1..1024,
 * a stride smaller than a row, a short workspace -> DS_ERR_SIZE; a temperature
 * outside [2^-10, 2^10], coef negative or not finite, accumulate without
 * dlogits -> DS_ERR_HPARAM; an unknown dt, tdt or index_bytes -> DS_ERR_DTYPE;
 * else as in the conventions.
 */
#define DS_MAX_TEACHER_LOGITS 1024

/* Device scratch of ds_distill_loss (0 for sizes out of range). */
size_t ds_distill_workspace_bytes(int64_t tokens);

ds_status ds_distill_loss(const ds_scaler* st_or_null, const void* logits, ds_dtype dt, int64_t tokens, int64_t vocab,
                          int64_t row_stride, const void* teacher, ds_dtype tdt, int64_t teacher_stride, const void* index,
                          int32_t index_bytes, int64_t index_stride, int32_t k, const uint8_t* mask_or_null,
                          float temperature, float coef, float* token_loss, float* loss, int32_t* used,
                          void* dlogits_or_null, int64_t grad_stride, int32_t accumulate, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * ---------------------------------------------------------------------------
 * Cross entropy over a large vocabulary from hidden states, with the gradient
 * ---------------------------------------------------------------------------
 * hidden: [tokens] rows of `width` values, weight: [vocab] rows of `width`
 * values, both of type dt (DS_FP16 or DS_BF16), rows hidden_stride and
 * weight_stride apart; targets: [tokens] (int32 or int64: index_bytes 4 or 8).
 * A row is used if mask is NULL or mask[t] != 0, and its target is not negative;
 * T' is the number of used rows (*used).  With z = hidden weight^T (fp32 sums),
 * never kept:
 *   token_loss[t] = log sum_v exp(z_tv) - z_t,target
 *   loss = coef / T' sum over used rows of token_loss[t]
 *   dz_tv = S coef / T' (exp(z_tv) / sum_u exp(z_tu) - [v = target])
 *   dhidden = dz weight,  dweight = dz^T hidden
 * with S = st->scale read on the device (st_or_null NULL: 1).  Rows that are not
 * used have token_loss and dhidden 0 and reach nothing else, whatever they hold;
 * T' = 0: loss and gradients are 0.  A target at or past vocab makes its row's
 * loss and gradient, and with them dweight, NaN.  exp(z) / sum - [v = target] is
 * rounded to dt (in fp16 times 2^15) before the two products of the gradient,
 * which sum in fp32 and are rounded once.  dhidden_or_null: type dt;
 * dweight_or_null: type dwdt, dt or DS_FP32 (without both: the loss alone).
 * accumulate != 0 adds to dweight (in fp32, rounded once).
 * workspace: device, 256-byte aligned, no initial contents; calls that share it
 * must not run at the same time.  It holds a piece of the vocabulary's dz, 512
 * MiB at most for up to 131072 tokens.  Arrays need the alignment of their type
 * only; a weight whose rows are 16-byte aligned and a multiple of 64 values
 * wide is read where it lies, any other copied piece by piece.
 * Errors: tokens outside [0, 2^24], vocab outside [1, 2^24], width outside
 * [1, 65536], a stride smaller than a row, a short workspace -> DS_ERR_SIZE;
 * dt not 16-bit, dwdt another type, an unknown index_bytes -> DS_ERR_DTYPE; coef
 * negative or not finite, accumulate without dweight -> DS_ERR_HPARAM; else as
 * in the conventions.
 */

/* Device scratch of ds_vocab_ce (0 for sizes out of range). */
size_t ds_vocab_ce_workspace_bytes(int64_t tokens, int64_t vocab, int64_t width);

ds_status ds_vocab_ce(const ds_scaler* st_or_null, const void* hidden, int64_t hidden_stride, const void* weight,
                      int64_t weight_stride, ds_dtype dt, const void* targets, int32_t index_bytes, int64_t tokens,
                      int64_t vocab, int64_t width, const uint8_t* mask_or_null, float coef, float* token_loss, float* loss,
                      int32_t* used, void* dhidden_or_null, int64_t dhidden_stride, void* dweight_or_null, ds_dtype dwdt,
                      int64_t dweight_stride, int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream);

/* Static string naming a status code. */
const char* ds_status_string(ds_status s);

#ifdef __cplusplus
}
#endif

#endif /* DSZERO_H */
