/*
 * zeroadam.h -- C ABI of libzeroadam.so: the ZeRO stage-1/2 mixed-precision
 * Adam step and the ZeRO-3 unit gather on one GB300 (sm_103a), and the rest of
 * a training step around them: a unit's linear maps forward and backward, the
 * global gradient norm, and AdamW over a list of tensors.
 *
 * The method is the one in "ZeRO and FSDP: partitioning the optimizer states,
 * the gradients and the parameters" (AI infra handbooks): the parameters are
 * one flat vector of numel elements, zero-padded to world*shard with
 * shard = ceil(numel/world); rank r owns [r*shard, (r+1)*shard).  One step of
 * rank r ("Implementing ZeRO's Adam from scratch", ZeroAdam.step):
 *   1. reduce-scatter the world ranks' gradients and average them,
 *   2. Adam with bias correction on rank r's fp32 master/m/v shard,
 *   3. all-gather the updated shard back into the full parameters.
 * Here the ranks are buffers in one GPU's memory: step 1 reads the world
 * gradient buffers directly, and step 3 writes rank r's shard, cast to bf16,
 * straight into the flat bf16 parameter buffer.  One kernel does all three.
 *
 * Conventions for every call:
 *   - Status: 0 (ZERO_OK) or a negative ZERO_E_* code.  Nothing is launched
 *     when a call returns an error.  No call aborts or allocates device
 *     memory; none synchronises except zero_device_status; the only state kept
 *     between calls is a per-device status word that a kernel sets only if one
 *     of its bounded waits gives up (see zero_device_status).  Faults inside a
 *     launched kernel surface, as for any CUDA work, at the caller's next sync.
 *   - Tracing: every call that launches work, and zero_device_status,
 *     opens an NVTX range
 *     named after the function for the duration of the call (visible to
 *     Nsight tools and any NVTX injection library; free when none is
 *     attached).
 *   - Calls on different streams may run concurrently when their output
 *     buffers are disjoint; a sequence of calls may be captured into a CUDA
 *     graph after each kernel's first call on the device (which does one-time
 *     set-up outside any capture).
 *   - Device pointers are in the current CUDA device's address space; the
 *     stream argument is a cudaStream_t passed as void* (NULL = the legacy
 *     default stream) and must belong to the current device.
 *   - bf16 buffers are arrays of IEEE bfloat16 bit patterns (uint16_t).
 *   - The caller owns every buffer.  Host pointer arrays (grad_ptrs,
 *     shard_ptrs) are read before the call returns.
 *   - Alignment: bf16 pointers must be 2-byte and fp32 pointers 4-byte
 *     aligned (ZERO_E_ALIGN otherwise).  16-byte alignment is not required,
 *     but the fast vectorised path runs only where the buffers can be
 *     accessed 16 bytes at a time together (always so for buffers from the
 *     PyTorch/cudaMalloc allocator used as whole flat vectors).
 */
#ifndef ZEROADAM_H
#define ZEROADAM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ----------------------------------------------------------------- status */

#define ZERO_OK 0
#define ZERO_E_NULLPTR (-1) /* a required pointer is NULL                          */
#define ZERO_E_WORLD (-2)   /* world < 1 or world > ZERO_MAX_WORLD                  */
#define ZERO_E_NUMEL (-3)   /* numel < 1, or world*shard overflows int64           */
#define ZERO_E_RANK (-4)    /* rank not in [0, world) and not ZERO_ALL_RANKS        */
#define ZERO_E_STEP (-5)    /* t < 1 (t is the 1-based step count after increment)  */
#define ZERO_E_ALIGN (-6)   /* bf16 pointer odd, or fp32 pointer not 4-byte aligned */
#define ZERO_E_HPARAM (-7)  /* lr/eps (weight_decay, max_norm) < 0 or not finite; beta not in [0, 1);
                               scale, alpha not finite */
#define ZERO_E_LAYOUT (-8)  /* unknown layout, activation, norm or flag, a shard layout with ALL_RANKS,
                               or a tensor that the norm's kind does not have */
#define ZERO_E_PLAN (-9)    /* the plan's fields are not those zero_plan computes   */
#define ZERO_E_ALIAS (-10)  /* an output buffer overlaps another buffer             */
#define ZERO_E_LAUNCH (-11) /* the CUDA launch failed; see zero_strerror            */
#define ZERO_E_DEVICE (-12) /* no usable CUDA device                                */
#define ZERO_E_RANGE (-13)  /* zero_adam_step_range: begin < 0 or end < begin       */
#define ZERO_E_SHAPE (-14)  /* a tensor count, size or pitch is out of the call's range */
#define ZERO_E_TIMEOUT (-15) /* a kernel gave up a bounded wait (zero_device_status) */
#define ZERO_E_HOOK (-16)    /* a test hook was called without ZEROADAM_TEST_HOOKS=1 */
#define ZERO_E_WORKSPACE (-17) /* the workspace is NULL, misaligned or too small     */

/* Largest tensor count of one zero3_unit_gather_rows unit. */
#define ZERO_MAX_UNIT_TENSORS 256

/* Largest world (number of emulated data-parallel ranks) accepted. */
#define ZERO_MAX_WORLD 1024

/* rank argument: step every rank's shard in one launch. */
#define ZERO_ALL_RANKS (-1)

/* grad_layout: one layout, optionally OR-ed with the flags below */
#define ZERO_GRAD_FULL 0   /* grad_ptrs[k]: rank k's whole padded flat gradient (>= numel elements) */
#define ZERO_GRAD_SHARD 1  /* grad_ptrs[k]: rank k's gradient slice of THIS rank's shard (shard elements); single rank only */
#define ZERO_GRAD_WINDOW 2 /* zero_adam_step_range only: grad_ptrs[k][i - begin], the window's gradients alone */
#define ZERO_GRAD_LAYOUT_MASK 0x0f
#define ZERO_GRAD_F32 0x10 /* flag: gradient buffers hold fp32 (default: bf16) */
#define ZERO_ACC_BF16 0x20 /* flag: round the running sum over ranks to bf16 after every addition */
#define ZERO_GRAD_ACCUMULATE 0x40 /* gradients of weights (dw, dbias, dtable, ...): add to them instead of writing */

/* param_layout */
#define ZERO_PARAM_FULL 0  /* param_bf16: the whole flat parameter buffer (>= numel elements) */
#define ZERO_PARAM_SHARD 1 /* param_bf16: this rank's shard only (shard elements; ZeRO-3); single rank only */

/* act: the activation of a linear map's epilogue */
#define ZERO_ACT_NONE 0
#define ZERO_ACT_RELU 1 /* max(z, 0); its derivative at 0 is 0                          */
#define ZERO_ACT_GELU 2 /* z/2 (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))), the tanh form */
#define ZERO_ACT_SILU 3 /* z / (1 + exp(-z))                                            */

/* zero_linear_workspace */
#define ZERO_LINEAR_BACKWARD 1
#define ZERO_LINEAR_ALIGNED 2
#define ZERO_LINEAR_PLAIN 4

/* flag: token ids and targets are int32 (default: int64) */
#define ZERO_IDS_I32 0x100

/* kinds of norm of zero_block_norm_* */
#define ZERO_NORM_NONE 0
#define ZERO_NORM_RMS 1   /* x / sqrt(mean(x^2) + eps) * weight                      */
#define ZERO_NORM_LAYER 2 /* (x - mean(x)) / sqrt(var(x) + eps) * weight + bias      */

/* zero_adamw_step */
#define ZERO_STATE_8BIT 0x80   /* flag: m and v are held as 8-bit codes with block scales */
#define ZERO_MOMENT_BLOCK 256  /* elements that share one scale of an 8-bit moment        */
#define ZERO_MAX_LIST 65536    /* largest number of tensors of one list                   */

/* ------------------------------------------------------------------- plan */

/*
 * Layout and per-card memory of a flat vector of numel parameters on world
 * data-parallel ranks.
 *
 *   shard  = ceil(numel / world), pad = world*shard - numel, padded = world*shard
 *            ("Implementing ZeRO's Adam from scratch": shard size and _flatten's
 *            zero padding).
 *   bytes_* : model-state bytes per card with the padded shard: DP 16*numel,
 *            ZeRO-1 4*numel + 12*shard, ZeRO-2 2*numel + 14*shard,
 *            ZeRO-3 16*shard (mixed-precision Adam: bf16 parameter 2 B, bf16
 *            gradient 2 B, fp32 master/m/v 12 B; "The three stages" table).
 *   formula_*: the same table's real-valued expressions 16 Psi, 4 Psi + 12 Psi/N,
 *            2 Psi + 14 Psi/N, 16 Psi/N (equal to bytes_* when pad == 0).
 *   state_bytes_rank: fp32 master + m + v bytes one rank holds, 12*shard
 *            (ZeroAdam.state_bytes).
 *   comm_*: bytes sent per card per step for the bf16 gradients/parameters
 *            ("The three stages" table, last column, and "Exercises": a ring
 *            all-reduce sends 2(N-1)/N of the gradient size; ZeRO-1/2 send the
 *            same as a reduce-scatter plus an all-gather; ZeRO-3 adds one more
 *            parameter all-gather, 1.5x): comm_dp = comm_z1 = comm_z2 =
 *            2 * (N-1)/N * 2*padded, comm_z3 = 3 * (N-1)/N * 2*padded.
 *
 * Host only; no CUDA call.  Errors: ZERO_E_NULLPTR, ZERO_E_WORLD, ZERO_E_NUMEL.
 */
typedef struct {
  int64_t numel, world, shard, pad, padded;
  uint64_t bytes_dp, bytes_z1, bytes_z2, bytes_z3;
  double formula_dp, formula_z1, formula_z2, formula_z3;
  uint64_t state_bytes_rank;
  double comm_dp, comm_z1, comm_z2, comm_z3;
} zero_plan_t;

int zero_plan(int64_t numel, int32_t world, zero_plan_t* out);

/* ------------------------------------------------------------------- step */

/*
 * One ZeRO-1/2 Adam step ("Implementing ZeRO's Adam from scratch",
 * ZeroAdam.step) for rank `rank`, or for all ranks (ZERO_ALL_RANKS), on the
 * ranks' shards of the flat vector described by plan (from zero_plan).
 *
 * For every global flat index i < numel that the stepped rank(s) own:
 *   g    = (((float)g_0[i] + (float)g_1[i]) + ... + (float)g_{N-1}[i]) / N
 *          (reduce_scatter_tensor, then g /= world; fp32 sum in rank order)
 *   m    = m*b1 + (1-b1)*g ;  v = v*b2 + ((1-b2)*g)*g
 *   w    = w - (lr * (m / (1-b1^t))) / (sqrt(v / (1-b2^t)) + eps)
 *   p[i] = bf16 round-to-nearest-even of w   (all_gather_into_tensor + copy
 *          into the parameters)
 * Each operation is one IEEE binary32 operation rounded to nearest even (no
 * FMA contraction, denormals kept); the scalars 1-b1, 1-b2, 1-b1^t, 1-b2^t,
 * b1, b2, lr, eps, N are formed in double and rounded to binary32 once.
 * Indices >= numel (the zero padding) are neither read nor written.
 *
 *   plan        from zero_plan(numel, world); checked (ZERO_E_PLAN).
 *   rank        in [0, world), or ZERO_ALL_RANKS.
 *   grad_ptrs   host array of world device pointers, bf16 (fp32 with ZERO_GRAD_F32).
 *               ZERO_GRAD_FULL : grad_ptrs[k][i] for global index i.
 *               ZERO_GRAD_SHARD: grad_ptrs[k][i - rank*shard] (single rank).
 *               (ZERO_GRAD_WINDOW is zero_adam_step_range's; here ZERO_E_LAYOUT.)
 *   master,m,v  device fp32, read and written in place.
 *               ALL_RANKS: padded elements, index i (the ranks' shards back to
 *               back); single rank: shard elements, index i - rank*shard.
 *   param_bf16  device bf16, written only.
 *               ZERO_PARAM_FULL : index i, buffer of >= numel elements.
 *               ZERO_PARAM_SHARD: index i - rank*shard (single rank).
 *   lr, beta1, beta2, eps  Adam hyper-parameters (lr, eps >= 0; 0 <= beta < 1).
 *   t           1-based step number after the increment (ZeroAdam.step's
 *               self.t += 1 happens before the moments are used).
 *   stream      cudaStream_t as void*.
 * The gradient buffers must not overlap any output; master, m, v and
 * param_bf16 must not overlap one another (ZERO_E_ALIAS).
 */
int zero_adam_step(const zero_plan_t* plan, int32_t rank, const void* const* grad_ptrs,
                   int32_t grad_layout, float* master, float* m, float* v, void* param_bf16,
                   int32_t param_layout, double lr, double beta1, double beta2, double eps,
                   int64_t t, void* stream);

/*
 * The same step restricted to the global flat window [begin, end) (clipped to
 * the stepped rank's real elements): ZeRO-2's bucketed schedule ("Implementing
 * ZeRO's Adam from scratch", closing note: real ZeRO-2 reduce-scatters bucket
 * by bucket during the backward pass and frees each full-gradient bucket once
 * it has gone out).  With ZERO_GRAD_WINDOW each grad_ptrs[k] holds only the
 * bucket, element i at grad_ptrs[k][i - begin], so the full gradient never
 * needs to exist; ZERO_GRAD_FULL and ZERO_GRAD_SHARD address as in
 * zero_adam_step.  master/m/v and param_bf16 are addressed as in
 * zero_adam_step.  Buckets that tile the flat vector give exactly the result
 * of one zero_adam_step (the step is elementwise).  Errors: those of
 * zero_adam_step, and ZERO_E_RANGE.
 *
 * Gradient variants (flags in grad_layout, both calls): ZERO_GRAD_F32 takes
 * fp32 gradient buffers (the page's runnable demo keeps fp32 gradients);
 * ZERO_ACC_BF16 rounds the running sum over ranks to bf16 after every
 * addition, the result a reduce-scatter on bf16 buffers delivers (a
 * sensitivity variant, not the method).
 */
int zero_adam_step_range(const zero_plan_t* plan, int32_t rank, int64_t begin, int64_t end,
                         const void* const* grad_ptrs, int32_t grad_layout, float* master,
                         float* m, float* v, void* param_bf16, int32_t param_layout, double lr,
                         double beta1, double beta2, double eps, int64_t t, void* stream);

/* ------------------------------------------------------------ ZeRO-3 gather */

/*
 * ZeRO-3 unit all-gather ("ZeRO-3 and FSDP": before a unit is used in the
 * forward or backward pass its complete parameters are all-gathered):
 *   full_bf16[r*shard + j] = shard_ptrs[r][j]  for r < world, j < shard,
 *                                              r*shard + j < numel,
 * where unit_plan = zero_plan(U, world) of the unit's U elements.  The copy is
 * bit-exact; the padded tail of the last shard is not copied.
 *
 *   shard_ptrs  host array of world device pointers to bf16 shards of
 *               unit_plan->shard elements each.
 *   full_bf16   device bf16 buffer of >= numel elements, written only; must not
 *               overlap a shard (ZERO_E_ALIAS).
 *
 * When shard is a multiple of 8 elements and every buffer is 16-byte aligned
 * (whole cudaMalloc/PyTorch buffers) the copy runs on the TMA engine, whose
 * waits are bounded (see zero_device_status); otherwise a load/store kernel.
 */
int zero3_unit_gather(const zero_plan_t* unit_plan, const void* const* shard_ptrs,
                      void* full_bf16, void* stream);

/*
 * FSDP2-style unit gather ("ZeRO-3 and FSDP": FSDP2 represents every parameter
 * as a DTensor sharded along dimension 0, so each rank holds a block of rows of
 * each tensor).  The unit is ntensors row-major bf16 tensors, tensor i of
 * rows[i] x cols[i] elements.  With R_i = ceil(rows[i] / world), rank r holds
 * rows [r*R_i, min((r+1)*R_i, rows[i])) of tensor i, stored as R_i x cols[i]
 * elements (rows past the tensor's end are padding and are not copied); its
 * shard buffer is those blocks for i = 0..ntensors-1 back to back
 * (sum_i R_i*cols[i] elements).  The gathered unit full_bf16 is the tensors
 * back to back (sum_i rows[i]*cols[i] elements).  Bit-exact copy.  For one
 * tensor whose rows divide by world this is zero3_unit_gather's layout.
 *
 *   rows, cols  host arrays of ntensors positive sizes, read before return.
 *   shard_ptrs  host array of world device pointers (bf16 shards).
 * Errors: ZERO_E_SHAPE (ntensors not in [1, ZERO_MAX_UNIT_TENSORS], a size < 1,
 * or the unit's element count overflows), ZERO_E_WORLD, ZERO_E_NULLPTR,
 * ZERO_E_ALIGN (odd pointer), ZERO_E_ALIAS (output overlaps a shard),
 * ZERO_E_LAUNCH.
 *
 * When every tensor's offset in the unit and every R_i*cols[i] is a multiple of
 * 8 elements and every buffer is 16-byte aligned (e.g. a Llama layer's weights
 * from whole cudaMalloc/PyTorch buffers) the copy runs on the TMA engine, whose
 * waits are bounded (see zero_device_status); otherwise a load/store kernel.
 */
int zero3_unit_gather_rows(int32_t ntensors, const int64_t* rows, const int64_t* cols,
                           int32_t world, const void* const* shard_ptrs, void* full_bf16,
                           void* stream);

/*
 * One ZeRO-3 unit's gather and one rank's step in a single launch ("ZeRO-3 and
 * FSDP": a unit's parameters are all-gathered from the ranks' shards before
 * the unit is used, and each rank updates only its own shard).  The result is
 * exactly that of
 *   zero3_unit_gather(unit_plan, shard_ptrs, full_bf16, stream);
 *   zero_adam_step(unit_plan, rank, grad_ptrs, grad_layout, master, m, v,
 *                  param_bf16, param_layout, lr, beta1, beta2, eps, t, stream);
 * with the same arguments, layouts and errors as those two calls.  The step
 * does not read the gathered unit, so the two parts run side by side in one
 * grid instead of one after the other (one launch, overlapped ramps: the
 * page's small units are latency-bound).  Because they overlap, the buffers
 * of the two parts must be disjoint: full_bf16 must not overlap any gradient
 * or any step output, and no shard may overlap a step output (ZERO_E_ALIAS).
 * To update the rank's own bf16 shard in place (param_bf16 inside
 * shard_ptrs[rank]) call the two functions in sequence instead.
 *
 * When the shard is a multiple of 8 elements, every buffer of both parts is
 * 16-byte aligned at its first element, the gradients are bf16, the sum is
 * fp32 and the unit moves at most 512 MiB (gather 4 bytes per unit element +
 * step (2*world + 26) bytes per stepped element), the single launch runs (bulk copies on the TMA engine, bounded waits reported by
 * zero_device_status); otherwise the two kernels are launched in order on the
 * stream (larger units stream as fast that way, with the launch cost
 * amortised).  Errors: those of zero3_unit_gather and
 * zero_adam_step (ZERO_GRAD_WINDOW is not accepted: ZERO_E_LAYOUT).
 */
int zero3_unit_step(const zero_plan_t* unit_plan, int32_t rank, const void* const* shard_ptrs,
                    void* full_bf16, const void* const* grad_ptrs, int32_t grad_layout,
                    float* master, float* m, float* v, void* param_bf16, int32_t param_layout,
                    double lr, double beta1, double beta2, double eps, int64_t t, void* stream);

/* ------------------------------------------------------------- linear maps */

/*
 * Sizes of one linear map y = x W^T of `rows` tokens from `in` to `out`
 * features, and the row pitches (leading dimensions, in elements) of its
 * matrices.  Every matrix is row-major with unit column stride: x and dx are
 * rows x in, W and dw out x in, y, dy, residual and pre rows x out, pre_in
 * rows x in.  A pitch is at least the matrix's width; pitches of matrices that
 * a call does not use are not read.  1 <= in, out; 0 <= rows; in, out and
 * rows below 2^31.
 */
typedef struct {
  int64_t rows, in, out;
  int64_t ldx, ldw, ldy;      /* x, W, y (forward) or dy (backward)  */
  int64_t ldr, ldp;           /* residual, pre                       */
  int64_t ldpi, lddx, lddw;   /* pre_in, dx, dw                      */
} zero_linear_t;

/*
 * Forward: with z = x W^T + bias (fp32 sums),
 *   y   = bf16(act(z) + residual),   pre = bf16(z).
 * A unit's maps on its gathered weights ("ZeRO-3 and FSDP": the complete
 * parameters are used in the forward pass, then freed).  The activation and
 * the residual take z in fp32; each output is rounded to bf16 once.
 *
 *   x, w        bf16, read.
 *   bias        bf16, `out` elements, or NULL.
 *   act         ZERO_ACT_*.
 *   residual    bf16, or NULL.  It may be y itself (same pitch): in place.
 *   pre         bf16, written, or NULL: what the backward pass takes.
 *   y           bf16, written.
 *   workspace   device memory of zero_linear_workspace bytes,
 *               16-byte aligned (NULL where that is 0), free again once the
 *               call's work has run.
 * rows = 0 is valid and launches nothing (matrices of no rows may be NULL).  Any
 * alignment of 2 bytes and any pitch is taken; x and w whose base is 16-byte
 * aligned and whose pitch is a multiple of 8, and a bias on a 16-byte boundary,
 * are read in place, others are laid out anew in the workspace first.  Results
 * do not depend on the run: every sum has a fixed order for given sizes.
 * Results in bf16 (here and in the backward) are sums in one chain on the tensor
 * cores, which cut off what does not fit 24 bits: 1e-9 of the sum a step of the
 * reduction, a hundredth of the last rounding at 16,384 steps and in proportion.
 * Errors: ZERO_E_NULLPTR, ZERO_E_SHAPE, ZERO_E_LAYOUT (unknown act),
 * ZERO_E_ALIGN, ZERO_E_ALIAS (y or pre overlaps another matrix),
 * ZERO_E_WORKSPACE, ZERO_E_LAUNCH, ZERO_E_DEVICE.
 */
int zero_linear_forward(const zero_linear_t* shape, const void* x, const void* w,
                        const void* bias, int32_t act, const void* residual, void* pre, void* y,
                        void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Backward of y = act(x W^T + bias): with dz = dy * act'(pre),
 *   dx    = bf16((dz W) * act_in'(pre_in)),
 *   dw    = dz^T x          (added to dw with ZERO_GRAD_ACCUMULATE),
 *   dbias = sum over rows of dz (likewise),
 * in fp32 sums.  act_in / pre_in are the activation that made x, and what it
 * was given: dx is then the gradient of the map before it, ready to be that
 * map's dy with act NONE.  A residual's gradient is dy itself.
 *
 *   dy          bf16, read.
 *   act, pre    the map's activation and the `pre` its forward wrote (NULL
 *               with ZERO_ACT_NONE).  With an activation dz is rounded to
 *               bf16 before the products (the tensor cores' operand type);
 *               dbias sums it unrounded.
 *   act_in, pre_in  as above; ZERO_ACT_NONE and NULL to leave dx as it is.
 *   x, w        bf16, read (x only for dw, w only for dx; else may be NULL).
 *   dx, dw, dbias  each written, or NULL to skip it.  dw and dbias are bf16,
 *               or fp32 with ZERO_GRAD_F32: a tensor's place in a rank's flat
 *               gradient buffer can be passed as it is.
 *   flags       ZERO_GRAD_F32, ZERO_GRAD_ACCUMULATE.  Added to fp32 what comes
 *               to less than 2^-126 may be held as 0.
 *   workspace   zero_linear_workspace bytes with ZERO_LINEAR_BACKWARD.
 * rows = 0 writes zeros to dw and dbias (or leaves them, accumulating).
 * Errors: as zero_linear_forward (ZERO_E_LAYOUT also for unknown flags).
 */
int zero_linear_backward(const zero_linear_t* shape, const void* dy, const void* x, const void* w,
                         int32_t act, const void* pre, int32_t act_in, const void* pre_in,
                         void* dx, void* dw, void* dbias, int32_t flags, void* workspace,
                         int64_t workspace_bytes, void* stream);

/* Bytes of workspace that suffice for zero_linear_forward, or with
 * ZERO_LINEAR_BACKWARD for zero_linear_backward, of this shape; 0 for a forward
 * of at most 16 rows.  ZERO_LINEAR_ALIGNED: every matrix's base, and a
 * forward's bias, will be on a 16-byte boundary and every pitch a multiple of 8,
 * so none is laid out anew
 * (a call whose matrices are not so needs the figure without it).
 * ZERO_LINEAR_PLAIN: a backward with ZERO_ACT_NONE.  Negative: the ZERO_E_* code
 * of a bad shape or flag.  Host only. */
int64_t zero_linear_workspace(const zero_linear_t* shape, int32_t flags);

/* ------------------------------------------------- AdamW over a list of tensors */

/*
 * Global norm of a list of gradients, and the factor that clips it:
 *   out[0] = sqrt(sum over tensors and elements of g^2)
 *   out[1] = min(1, max_norm / (out[0] + 1e-6))   (NaN if the norm is NaN)
 * Squares and each thread's run of up to 64 of them are summed in fp32, all
 * else in fp64; the order is fixed, so equal inputs give equal bits.
 *
 *   grads, numels  host arrays of ntensors device pointers and sizes (>= 0).
 *   flags       ZERO_GRAD_F32 for fp32 gradients (default bf16).
 *   out         device, two fp32.
 *   workspace   device memory of zero_grad_norm_workspace() bytes, 16-byte
 *               aligned.  Set to zero once before its first use; every call
 *               leaves it ready for the next.  One call at a time may use it.
 * Errors: ZERO_E_SHAPE (ntensors not in [0, ZERO_MAX_LIST], or a size < 0),
 * ZERO_E_NULLPTR, ZERO_E_LAYOUT, ZERO_E_ALIGN, ZERO_E_HPARAM (max_norm not
 * finite or < 0), ZERO_E_WORKSPACE, ZERO_E_LAUNCH, ZERO_E_DEVICE.
 */
int zero_grad_norm(int32_t ntensors, const void* const* grads, const int64_t* numels,
                   int32_t flags, double max_norm, float* out, void* workspace,
                   int64_t workspace_bytes, void* stream);
int64_t zero_grad_norm_workspace(void);

/* One tensor of an AdamW list.  m_scale and v_scale are used with
 * ZERO_STATE_8BIT only (ceil(numel / ZERO_MOMENT_BLOCK) fp32 each). */
typedef struct {
  int64_t numel;        /* >= 0                                              */
  const void* grad;     /* bf16, or fp32 with ZERO_GRAD_F32                   */
  float* master;        /* fp32 weights, in place                            */
  void* param_bf16;     /* bf16 copy of the new weights, written; or NULL     */
  void* m;              /* fp32, or 8-bit codes; in place                    */
  void* v;
  float* m_scale;
  float* v_scale;
  double weight_decay;  /* >= 0, finite                                      */
} zero_adamw_tensor_t;

/*
 * One AdamW step (Adam with bias correction and decoupled weight decay) over a
 * list of tensors: the optimizer of FSDP2-style shards, where a rank holds a
 * block of rows of every tensor instead of a slice of one flat vector.  With
 * c = *grad_scale (1 if NULL), for every element:
 *   g = c * grad
 *   m = m*b1 + (1-b1)*g ;  v = v*b2 + ((1-b2)*g)*g
 *   w = w*(1 - lr*weight_decay) - (lr/(1-b1^t)) * m / (sqrt(v)/sqrt(1-b2^t) + eps)
 *   p = bf16 round-to-nearest-even of w
 * m and v are computed in binary32, one rounding per operation, exactly as
 * zero_adam_step does; the update of w takes them before they are encoded, and
 * its square root and quotient are good to a few ulp of binary32.
 *
 * 8-bit moments (ZERO_STATE_8BIT): a tensor's elements are cut into blocks of
 * ZERO_MOMENT_BLOCK from its first one.  A block's scale is the power of two
 * 2^e of its largest magnitude after that is rounded up to 4 significant bits
 * (e in [-126, 126]).  Codes keep 3 mantissa bits with gradual underflow, f
 * the low 3 bits and x the exponent bits above them:
 *   |value| = scale * (1 + f/8) 2^(x-top), or scale * f/8 2^(1-top) for x = 0;
 *   m: sign in bit 7, 4 exponent bits (top = 15); v: 5 (top = 31), no sign.
 * Rounding is stochastic: 16 random bits r of each element are added to the
 * dropped 20 (as 16 r + 8) before the cut, so the expected value is the moment
 * itself; a moving average that moves less than half a step at a time would
 * stand still under rounding to nearest.  The scales are powers of two so that
 * a value that has not changed is held exactly.  r comes from a hash: with
 * h the 32-bit permuted congruential generator's step, k = h(h(seed) + index
 * in the list) and u = h(k + element), m takes u >> 16 and v takes u & 0xffff
 * (element counted within the tensor; beyond 2^32 of them k adds
 * 0x9E3779B9 per 2^32).  A new seed every step; the same seed, the same bits.
 * A block with an infinity or NaN gets the scale NaN and codes 0: it reads as
 * NaN from then on.  All-zero codes and scales are zero moments.
 *
 *   tensors     host array, read before the call returns.
 *   flags       ZERO_GRAD_F32, ZERO_STATE_8BIT.
 *   grad_scale  device fp32 (zero_grad_norm's out + 1, say), or NULL.
 *   seed        of the rounding; unused with fp32 moments.
 * Lists of any length take one launch per 384 tensors.  Tensors of no elements
 * are skipped.  Any alignment of the element type is taken; tensors whose
 * buffers all begin the same number of elements (0 to 7) past a 16-byte boundary,
 * as where all are packed in flat vectors alike, go in 16-byte accesses (8-bit
 * codes that begin on an 8-byte boundary, at a lower rate unless that number is 0).
 * Errors: ZERO_E_SHAPE, ZERO_E_NULLPTR, ZERO_E_LAYOUT (unknown flags),
 * ZERO_E_HPARAM, ZERO_E_STEP, ZERO_E_ALIGN, ZERO_E_ALIAS (within a tensor:
 * master, m, v, param, grad or scales overlap; tensors of one list are not
 * compared with each other and must not share memory that is written),
 * ZERO_E_LAUNCH, ZERO_E_DEVICE.
 */
int zero_adamw_step(int32_t ntensors, const zero_adamw_tensor_t* tensors, int32_t flags,
                    double lr, double beta1, double beta2, double eps, int64_t t,
                    const float* grad_scale, uint32_t seed, void* stream);

/*
 * The values of 8-bit moments, as fp32 (for a checkpoint, or to go on with
 * fp32 moments): m_out[i] and v_out[i] are device buffers of tensors[i].numel
 * fp32, written; either array may be NULL.  Only numel, m, v and the scales of
 * each tensor are read.  Errors: as zero_adamw_step.
 */
int zero_adamw_state_f32(int32_t ntensors, const zero_adamw_tensor_t* tensors,
                         float* const* m_out, float* const* v_out, void* stream);

/* ------------------------------------------- the two ends of a model, and norms */

/*
 * Sizes of a table of `vocab` rows of `width` elements looked up by `rows` ids,
 * and the pitches (elements) of the table (or of its gradient) and of the rows
 * looked up (or of their gradient).  1 <= width, vocab; 0 <= rows; all below 2^31 - 1.
 */
typedef struct {
  int64_t rows, width, vocab;
  int64_t ldt, ldy;
} zero_embedding_t;

/*
 * Embedding: y[i] = bf16(scale * table[ids[i]]), the product in fp32.
 *   table, y    bf16, any pitch and 2-byte address.
 *   ids         int64, or int32 with ZERO_IDS_I32.  A row whose id is not in
 *               [0, vocab) is NaN: nothing is read for it.
 *   flags       ZERO_IDS_I32.
 * Errors: ZERO_E_NULLPTR, ZERO_E_SHAPE, ZERO_E_LAYOUT (unknown flags),
 * ZERO_E_HPARAM (scale not finite), ZERO_E_ALIGN, ZERO_E_ALIAS, ZERO_E_LAUNCH,
 * ZERO_E_DEVICE.
 */
int zero_embedding_forward(const zero_embedding_t* shape, const void* table, const void* ids,
                           int32_t flags, double scale, void* y, void* stream);

/*
 * Its gradient: dtable[v] = scale * (sum of dy[i] over the rows i with id v), in
 * fp32 in an order that follows from the ids alone, and rounded once.  Rows of no
 * token are set to zero; with ZERO_GRAD_ACCUMULATE sums are added to what is there
 * and rows of no token are left alone.
 *   dy          bf16.
 *   padding     an id whose rows have no gradient (-1: none).  Rows whose id is
 *               not in [0, vocab) have none either.
 *   dtable      bf16, or fp32 with ZERO_GRAD_F32.  Added to fp32 what comes to
 *               less than 2^-126 may be held as 0.
 *   flags       ZERO_IDS_I32, ZERO_GRAD_F32, ZERO_GRAD_ACCUMULATE.
 * No workspace.  Errors: as zero_embedding_forward.
 */
int zero_embedding_backward(const zero_embedding_t* shape, const void* dy, const void* ids,
                            int32_t flags, double scale, int64_t padding, void* dtable,
                            void* stream);

/*
 * Sizes of a linear map of `rows` tokens from `width` features onto a vocabulary,
 * and the pitches (elements) of x, w and their gradients.  1 <= width, vocab;
 * 0 <= rows; all below 2^31 - 1.
 */
typedef struct {
  int64_t rows, width, vocab;
  int64_t ldx, ldw, lddx, lddw;
} zero_cross_entropy_t;

/*
 * Softmax cross entropy of z = x W^T against a target each row, and its gradient,
 * without keeping z:
 *   losses[i] = log(sum over j of exp(z[i][j])) - z[i][targets[i]]
 *   total     = sum over i of c[i] * losses[i]
 *   dz[i][j]  = c[i] * (exp(z[i][j] - log(sum ...)) - (j == targets[i]))
 *   dx = bf16(dz W),   dw = dz^T x  (added to dw with ZERO_GRAD_ACCUMULATE).
 * c[i] is scale[i], or without scale 1 / (number of rows that are not ignored): the
 * mean.  An ignored row's loss and dx are 0 and it adds nothing to total and dw,
 * whatever is in its x; if every row is ignored total and all gradients are 0.
 *
 *   x, w        bf16, read; any pitch and 2-byte address.
 *   targets     int64, or int32 with ZERO_IDS_I32.  Rows whose target is
 *               ignore_index are ignored.  Any other target that is not in
 *               [0, vocab) is an error of the data: its row's loss is NaN, and so
 *               are then total and the gradients.
 *   scale       device, fp32, one a row; or NULL.
 *   losses      fp32, one a row, written, or NULL.
 *   total       fp32, one, written, or NULL.
 *   dx, dw      written, or NULL to skip (both NULL: the loss alone, a third of the
 *               work).  dw is bf16, or fp32 with ZERO_GRAD_F32.
 *   flags       ZERO_IDS_I32, ZERO_GRAD_F32, ZERO_GRAD_ACCUMULATE.
 *   workspace   zero_linear_cross_entropy_workspace bytes, 16-byte aligned.
 * Sums are fp32.  The products' operands are bf16 (the tensor cores' type): the
 * exponentials, and then dz, each rounded once; of more than 2^25 values (rows *
 * vocab) the exponentials alone, and x times its row's factor for dw, whose rounding
 * averages out over a token's rows (the factor is within 2^-9 of its value, so that
 * the target's term is exact).  Exponentials below exp(-87) of the target's (of the
 * largest, in a row whose loss is above 44) are 0 in dz.  Rows that are ignored are
 * left out of the products.  The loss alone takes other kernels than the loss with
 * gradients, and may differ from it in its last bits.  Rows go in pieces whose
 * exponentials take at most 1 GiB of the workspace.  Results do not depend on the run.
 * rows = 0: total is 0, and dw is too (or is left, accumulating).
 * Errors: ZERO_E_NULLPTR, ZERO_E_SHAPE, ZERO_E_LAYOUT, ZERO_E_ALIGN, ZERO_E_ALIAS
 * (an output overlaps another buffer), ZERO_E_WORKSPACE, ZERO_E_LAUNCH, ZERO_E_DEVICE.
 */
int zero_linear_cross_entropy(const zero_cross_entropy_t* shape, const void* x, const void* w,
                              const void* targets, int64_t ignore_index, const float* scale,
                              float* losses, float* total, void* dx, void* dw, int32_t flags,
                              void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that suffice for zero_linear_cross_entropy of this shape;
 * flags: ZERO_LINEAR_BACKWARD if dx or dw is wanted, ZERO_GRAD_F32 if dw is fp32,
 * ZERO_LINEAR_ALIGNED if w's base is on a 16-byte boundary and its pitch a multiple
 * of 8 (else it is laid out anew).  Negative: the ZERO_E_* code.  Host only. */
int64_t zero_linear_cross_entropy_workspace(const zero_cross_entropy_t* shape, int32_t flags);

/*
 * The norms before and after a block, its gate and its residual scale: a model's
 * residual stream r takes the output h of a block, and the next block gets y,
 *   s = r + alpha * gate * P(h),   y = N(s)
 * with P of kind `post` (NONE: h itself) and N of kind `kind` (RMS or LAYER), each
 * row by itself.  Pitches in elements, below 2^31; ldg = 0: gate is one vector for all
 * rows.  1 <= width <= ZERO_MAX_NORM_WIDTH; 0 <= rows < 2^31 - 1.
 */
#define ZERO_MAX_NORM_WIDTH 32768
typedef struct {
  int64_t rows, width;
  int32_t post, kind;
  double alpha, eps;
  int64_t ldr, ldh, ldg, lds, ldy;        /* r, h, gate, s, y              */
  int64_t lddy, ldds, lddr, lddh, lddg;   /* dy, ds, dr, dh, dgate         */
} zero_block_norm_t;

/*
 * Forward.  Everything is bf16 in memory and fp32 within: y takes s unrounded.
 *   r           read.
 *   h           read, or NULL: no block yet, s = r (post is NONE, gate NULL).
 *   post_weight, post_bias   `width` elements each, or NULL for 1 and 0 (post_bias
 *               is LAYER's alone); weight, bias likewise for N.
 *   gate        a vector (ldg = 0), a matrix of rows x width, or NULL for 1.
 *   s           written, or NULL; it may be r itself (same pitch): in place.
 *   y           written.
 * Errors: ZERO_E_NULLPTR, ZERO_E_SHAPE, ZERO_E_LAYOUT (unknown kind, or a weight,
 * bias or gate that its kind or h does not have), ZERO_E_HPARAM (alpha not finite,
 * eps < 0 or not finite), ZERO_E_ALIGN, ZERO_E_ALIAS, ZERO_E_LAUNCH, ZERO_E_DEVICE.
 */
int zero_block_norm_forward(const zero_block_norm_t* shape, const void* r, const void* h,
                            const void* post_weight, const void* post_bias, const void* gate,
                            const void* weight, const void* bias, void* s, void* y, void* stream);

/*
 * Backward: from dy and the gradient ds that reaches s from elsewhere (NULL: 0),
 *   dr = ds + N's gradient of dy,   dh, dgate, and the weights' and biases' sums.
 * Statistics are computed anew from s and h as they are here.
 *   dy, s       read.   h: read, or NULL as in the forward.
 *   dr          written, or NULL; it may be ds itself (same pitch).
 *   dh          written, or NULL.  With post NONE, no gate and alpha 1 it is dr.
 *   dgate       NULL, or with ldg = 0 a vector, its sum over rows, else (lddg) a
 *               matrix, bf16.
 *   dpost_weight, dpost_bias, dweight, dbias   sums over rows; NULL to skip.  They
 *               and a vector dgate are bf16, or fp32 with ZERO_GRAD_F32, and added
 *               to what is there with ZERO_GRAD_ACCUMULATE.
 *   workspace   zero_block_norm_workspace bytes, 16-byte aligned; free again once
 *               the call's work has run.
 * Sums are fp32 in an order that follows from the sizes alone.  rows = 0 writes zeros
 * to the sums (or leaves them, accumulating).
 * Errors: as the forward, and ZERO_E_WORKSPACE.
 */
int zero_block_norm_backward(const zero_block_norm_t* shape, const void* dy, const void* ds,
                             const void* s, const void* h, const void* post_weight,
                             const void* post_bias, const void* gate, const void* weight,
                             void* dr, void* dh, void* dgate, void* dpost_weight,
                             void* dpost_bias, void* dweight, void* dbias, int32_t flags,
                             void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that suffice for zero_block_norm_backward.  Negative: the
 * ZERO_E_* code of a bad shape.  Host only. */
int64_t zero_block_norm_workspace(const zero_block_norm_t* shape);

/* ------------------------------------------------------------------ misc */

/*
 * Device-side status of the library's kernels on the current device.  Some
 * launches stage data through shared memory with asynchronous bulk copies and
 * wait on hardware barriers; every such wait is bounded, and a wait that gives
 * up (one second without progress, by the GPU's global timer) ends the launch
 * early, leaving that step's outputs incomplete, and records the fact in a
 * per-device status word.
 * The call first synchronises the current device (cudaDeviceSynchronize),
 * so every kernel launched before it, on any stream of the device, has
 * finished; then it reads and clears the words with one atomic exchange on the
 * GPU each, so a word set while the call runs is reported now or by the next
 * call, never lost.  Returns ZERO_OK if no wait has given up since the previous
 * call, else ZERO_E_TIMEOUT.  ZERO_E_DEVICE if there is no usable device or the
 * synchronisation reports an error (an earlier asynchronous fault; its CUDA
 * text is in zero_strerror).  It launches a one-thread kernel on the legacy
 * default stream, so it must not be called while a stream capture is open.
 */
int zero_device_status(void);

/*
 * Test hook for the bounded waits; the pages' method has no counterpart.
 * While `on` is nonzero, every step launch that uses a TMA-staged kernel
 * (world >= 5, bf16 gradients, fp32 sum, all buffers 16-byte aligned at the
 * stepped range's first element), every zero3_unit_gather or
 * zero3_unit_gather_rows that uses the TMA copy (see those calls), every
 * zero3_unit_step that runs as a single launch, and every product of
 * zero_linear_forward (more than 16 rows), zero_linear_backward and
 * zero_linear_cross_entropy tells its producers to issue no copies.  Every wait then runs out after its limit (about one second),
 * the outputs of the parts that wait are not written (at world <= 4 the
 * unit step's step part reads its gradients without staging and completes),
 * and zero_device_status reports ZERO_E_TIMEOUT; the device and its context
 * stay usable.  Launches of the other kernels are unaffected (they do not
 * wait).  The setting is process-wide and read when a call launches.  Returns
 * the previous
 * setting (0 or 1).  It exists so that tests can exercise the timeout path
 * without faulting or hanging a GPU; production code never calls it.  It is
 * off unless the environment variable ZEROADAM_TEST_HOOKS is "1" when it is
 * called; otherwise it changes nothing and returns ZERO_E_HOOK.
 */
int zero_test_withhold_copies(int on);

/* Text for a status code.  For ZERO_E_LAUNCH it includes the CUDA error text
   of this thread's last failed launch.  The pointer stays valid until this
   thread's next call into the library. */
const char* zero_strerror(int status);

/* Library version, e.g. 0x000100 for 0.1.0. */
int zero_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ZEROADAM_H */
