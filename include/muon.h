/*
 * muon.h -- C ABI of the MI355X (gfx950) Muon optimizer-step library.
 *
 * The operation (sources: Keller Jordan's "new optimizer" X thread,
 * xunroll.com/thread/1842300916864844014, tweets 2/8, 5/8 and 6/8; the
 * momentum convention from "07. Training neural networks", section
 * "Momentum"):
 *
 *   for every 2-D parameter matrix W (rows x cols, fp32) with gradient G and
 *   momentum buffer M:
 *     M  <- beta * M + G                      SGD momentum buffer
 *     U  <- G + beta * M                      Nesterov look-ahead
 *     X0 <- bf16( U / (||U||_F + 1e-7) )      transposed first if rows > cols
 *     repeat ns_steps times (quintic Newton-Schulz, in bfloat16):
 *        A <- bf16(X X^T);  B <- bf16(b A + c A A);  X <- bf16(a X + B X)
 *     W  <- W - lr * X                        (X transposed back)
 *
 * The thread states the design: orthogonalise each parameter's update after
 * Nesterov momentum, with a quintic Newton-Schulz iteration run in bfloat16,
 * whose coefficients maximise the slope at zero at the cost of exact
 * convergence.  The normalisation, the epsilon, the coefficient values and the
 * bf16 storage points are readings of those statements, not quotes: every
 * product accumulates in fp32 from bf16 operands; A, B and each new X are
 * rounded to bf16 (round to nearest even); the epilogue combinations
 * b*A + c*(AA) and a*X + (BX) are two fp32 products and one fp32 sum, not
 * fused.  No weight decay (the thread's replies report it as worse).  Only
 * 2-D matrices belong here; 1-D parameters go to another optimizer.
 *
 * Conventions for every entry point:
 *   - All matrix pointers are device pointers (HIP device memory, e.g. from
 *     PyTorch), row-major, contiguous, 4-byte aligned, caller-owned, and do
 *     not alias one another.  Arrays of pointers and shapes are host arrays,
 *     read only during the call.
 *   - Work is enqueued on `stream` and the call returns without waiting.
 *     Kernel faults surface at the caller's next synchronisation.  The
 *     calls made on one device must be ordered on the GPU: make them on one
 *     stream, or order the streams yourself (events).  They share the
 *     library's workspace and plan tables, which each call writes in its
 *     stream's order.
 *   - Plans are cached per device and keyed on the shapes (and the entry
 *     point), not on the pointers.  The first call with a set of shapes
 *     builds its plan: it allocates the plan's device table block
 *     (descriptors and work lists, a few hundred KB at most for GPT-2-sized
 *     sets) and enqueues its upload; it does not synchronise.  A call whose
 *     pointers differ from the previous call's on that plan enqueues one
 *     small kernel per 40 matrices that writes them into the descriptors;
 *     otherwise a call only enqueues the step's kernels.  Up to 8 plans are
 *     kept; evicting the least recently used one, or growing the library's
 *     workspace, waits for the device (hipDeviceSynchronize).
 *   - HIP graph capture: a call made while `stream` is capturing must find
 *     its plan and a large enough workspace already there (make one call
 *     with the same shapes first; otherwise it fails with MUON_EINVAL and
 *     enqueues nothing).  It allocates nothing and records only kernel
 *     launches: the pointer write and the step.  Its plan, and the workspace
 *     that plan uses, are then kept until muon_release(): neither eviction
 *     nor a later, larger call frees them, so the graph can be replayed
 *     between other calls.  Graphs must not be replayed after
 *     muon_release(), or after muon_set_workspace() replaced a caller-owned
 *     workspace they use.
 *   - Arguments are validated on the host before any HIP call; on failure
 *     the call returns a negative code, enqueues nothing and
 *     muon_last_error() describes the problem.
 *   - Return codes: MUON_OK (0), MUON_EINVAL (bad argument), MUON_ENOMEM
 *     (workspace allocation failed or caller workspace too small),
 *     MUON_EHIP (a HIP runtime call or launch failed; the HIP error string is
 *     in muon_last_error()).
 */
#ifndef MUON_H_
#define MUON_H_

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MUON_OK 0
#define MUON_EINVAL (-1)
#define MUON_ENOMEM (-2)
#define MUON_EHIP (-3)

/* Largest accepted ns_steps and matrix count per call. */
#define MUON_MAX_NS_STEPS 64
#define MUON_MAX_MATRICES 65536

/* Matrix shape in the caller's orientation. */
typedef struct {
  int64_t rows;
  int64_t cols;
} muon_shape_t;

/*
 * One Muon step over n independent matrices.
 *   params[i]   fp32 rows x cols, updated in place
 *   grads[i]    fp32 rows x cols, read only
 *   momentum[i] fp32 rows x cols, updated in place (zero before the first step)
 *   shapes[i]   rows, cols >= 1; rows * cols < 2^31
 *   lr          finite
 *   beta        in [0, 1)
 *   ns_steps    0 .. MUON_MAX_NS_STEPS (0 applies the normalised bf16 X0)
 *   coeffs      host array {a, b, c}, finite; the same triple every iteration
 * n == 0 is a no-op.  A zero gradient with a zero buffer leaves W unchanged.
 * NaN/Inf in the inputs propagate; nothing checks for them.
 */
int muon_step(float* const* params, const float* const* grads, float* const* momentum,
              const muon_shape_t* shapes, int n, float lr, float beta, int ns_steps,
              const float* coeffs, hipStream_t stream);

/*
 * Same as muon_step, and additionally writes the bf16 update X (the value
 * applied as W -= lr * X) to updates[i] (uint16 bf16 bit patterns,
 * rows x cols, caller orientation).  updates may be NULL, or any element may
 * be NULL, to skip that output.
 */
int muon_step_ex(float* const* params, const float* const* grads, float* const* momentum,
                 const muon_shape_t* shapes, int n, float lr, float beta, int ns_steps,
                 const float* coeffs, uint16_t* const* updates, hipStream_t stream);

/*
 * muon_step for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation.
 * Same arguments, same kernels and bit-identical results as muon_step, but
 * the workspace and the plan tables live in a static device array of
 * MUON_NOALLOC_SCRATCH_BYTES (128 MiB) that every device the library runs on
 * holds from the library's load until the process ends; no hipMalloc,
 * hipFree, pinned host memory or copy-engine transfer is used (the tables
 * and pointers reach the device as kernel arguments; host bookkeeping uses
 * the C++ heap).  A call whose workspace and tables exceed the array (one
 * GPT-2-124M block, 55.4 MiB, fits; the whole 48-matrix hidden set does not)
 * fails with MUON_ENOMEM and enqueues nothing.  Every call on a device
 * shares that device's array and leaves its contents behind; no call
 * depends on them (every value a kernel reads there was written earlier in
 * the same call), but calls whose GPU work overlaps in time on one device
 * race on the array: order them (one stream).
 */
#define MUON_NOALLOC_SCRATCH_BYTES (128u * 1024u * 1024u)
int muon_step_noalloc(float* const* params, const float* const* grads, float* const* momentum,
                      const muon_shape_t* shapes, int n, float lr, float beta, int ns_steps,
                      const float* coeffs, hipStream_t stream);

/*
 * muon_step_ex with a coefficient schedule: coeffs is a host array of
 * 3 * ns_steps floats, iteration k (0-based) using coeffs[3k .. 3k+2] as
 * {a, b, c}; all must be finite; it may be NULL when ns_steps = 0.  (The
 * thread's tweet 6/8 presents the coefficients as a trade-off between the
 * slope at zero and closeness to 1; a schedule makes that choice per
 * iteration.)  A schedule repeating one triple gives exactly muon_step_ex's
 * result.  updates as in muon_step_ex (may be NULL).
 */
int muon_step_sched(float* const* params, const float* const* grads, float* const* momentum,
                    const muon_shape_t* shapes, int n, float lr, float beta, int ns_steps,
                    const float* coeffs, uint16_t* const* updates, hipStream_t stream);

/*
 * The Newton-Schulz core alone: out[i] = iterate(x[i]) with the same
 * storage points as muon_step, no normalisation, no momentum.  x[i] and out[i]
 * are bf16 bit patterns (uint16), rows x cols in the caller's orientation
 * (tall matrices are transposed internally); out may equal x.  ns_steps = 0
 * copies.
 */
int muon_newton_schulz(const uint16_t* const* x, uint16_t* const* out, const muon_shape_t* shapes,
                       int n, int ns_steps, const float* coeffs, hipStream_t stream);

/* muon_newton_schulz with a coefficient schedule (3 * ns_steps floats, as in
 * muon_step_sched). */
int muon_newton_schulz_sched(const uint16_t* const* x, uint16_t* const* out, const muon_shape_t* shapes,
                             int n, int ns_steps, const float* coeffs, hipStream_t stream);

/*
 * Multi-tensor AdamW step, for the parameters that are not hidden 2-D
 * matrices (embeddings, biases, norm gains).  The update (the "07. Training
 * neural networks" page, section "Adam, weight decay and AdamW" and its
 * derivation of the bias correction and of the decoupled decay), for every
 * element of tensor i, with t = step:
 *   p <- p * (1 - lr * weight_decay[i])           decay first (decoupled)
 *   u <- beta1 * u + (1 - beta1) * g
 *   v <- beta2 * v + (1 - beta2) * g * g
 *   p <- p - lr * (u / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * fp32 throughout, one IEEE rounding per operation in the order written
 * (no fused multiply-add; division and square root correctly rounded);
 * 1 - beta_k and 1 - beta_k^t are evaluated in double from the fp32
 * arguments and rounded once to fp32; the decay factor is
 * fp32(1 - fp32(lr * weight_decay[i])).
 *   params[i], exp_avg[i], exp_avg_sq[i]  fp32, numels[i] contiguous elements,
 *               updated in place (exp_avg, exp_avg_sq zero before step 1)
 *   grads[i]    fp32, numels[i] elements, read only
 *   numels[i]   >= 0; a tensor with 0 elements is skipped (its pointers may be NULL)
 *   weight_decay  host array of n finite values >= 0, or NULL for 0 everywhere
 *   lr          finite;  beta1, beta2 in [0, 1);  eps finite, >= 0
 *   step        >= 1 (t of the bias corrections: 1 on the first step)
 * Pointers as for muon_step (device, 4-byte aligned, no two arrays
 * overlapping).  n == 0 is a no-op; n <= MUON_ADAMW_MAX_TENSORS.  Uses no
 * workspace; its work list is cached per pointer set like the Muon plans.
 * lr, the betas, eps and step are launch arguments, and so is the first
 * non-zero weight_decay value, shared by every tensor that uses it: a
 * schedule of those values reuses the cached list.  Only a tensor whose
 * non-zero lambda differs from that shared value has its lambda cached with
 * the list.
 */
#define MUON_ADAMW_MAX_TENSORS 65536
int muon_adamw_step(float* const* params, const float* const* grads, float* const* exp_avg,
                    float* const* exp_avg_sq, const int64_t* numels, const float* weight_decay, int n,
                    float lr, float beta1, float beta2, float eps, int64_t step, hipStream_t stream);

/*
 * Delayed untying of a shared parameter (the "nanoGPT Speedrun Techniques:
 * How Delayed Untying Solves the Sparse Gradient Problem" page, section
 * "Option B: Delayed Untying"): the parameter and both of its AdamW moments
 * (rows x cols fp32 each, row-major) are copied into new buffers, so that the
 * new parameter's trajectory continues from the shared point instead of
 * restarting its moments.  transpose = 1 writes the copies as cols x rows
 * (an output layer stored d_model x vocab against a vocab x d_model
 * embedding); transpose = 0 copies as is.  rows, cols >= 1 with
 * rows * cols <= 2^40; all six pointers device, 4-byte aligned, no
 * destination overlapping another array.  Bit-exact copies.
 */
int muon_adamw_untie(const float* param, const float* exp_avg, const float* exp_avg_sq, float* new_param,
                     float* new_exp_avg, float* new_exp_avg_sq, int64_t rows, int64_t cols, int transpose,
                     hipStream_t stream);

/*
 * Global gradient norm and clipping ("Let's reproduce GPT-2 (124M)" clips the
 * global norm at 1.0 before every optimizer step).  Over every element of
 * every tensor of the call, with g the gradients:
 *   norm   = scale * sqrt(sum of g^2)
 *   c      = min(1, max_norm / (norm + 1e-6)), 1 when max_norm = inf
 *   factor = scale * c
 * and the clipped gradient is g' = fp32(fp32(g) * factor), one rounding.  The
 * sum is held in fp64 in a fixed order, so equal calls give equal bits; norm
 * and factor are each rounded once, to fp32.  `scale` serves gradient
 * accumulation (1 / micro-batches) and loss scaling (1 / loss scale).
 * An infinity among the gradients gives norm = inf and factor = 0 (under a
 * finite max_norm), a NaN gives NaN for both; a norm beyond the fp32 range
 * reads as inf.
 *
 * The result is a record of MUON_CLIP_RECORD_FLOATS floats on the device,
 * {norm, factor}.  Steps on clipped gradients (muon_step_clip,
 * muon_adamw_step_clip) read it there, so the gradients are never written
 * back and the host never waits.  A step whose record's norm is not finite
 * changes nothing: parameters, momentum and moments keep their bits.
 *
 * Arguments shared by the calls below:
 *   dtypes      host array: element type of each tensor, MUON_FP32, MUON_BF16
 *               or MUON_FP16, mixed as needed
 *   numels      host array: contiguous elements of each tensor, 0 .. 2^35; a
 *               tensor with 0 elements takes no part (its pointer may be NULL)
 *   n           0 .. MUON_GRAD_MAX_TENSORS; with no elements at all the norm is 0
 *   max_norm    >= 0, or inf;  scale finite, > 0
 *   record      device, MUON_CLIP_RECORD_FLOATS floats, 4-byte aligned
 *   workspace   device, MUON_GRAD_WORKSPACE_BYTES bytes, 16-byte aligned, all
 *               zero before its first use; a call that finishes leaves it ready for the
 *               next.  Calls that share a workspace must be ordered on the GPU;
 *               calls with workspaces and records of their own may overlap.
 * Tensors are aligned to their element type only.  These calls use none of
 * the library's workspace or plan tables: they allocate nothing, cache
 * nothing, and can be captured without an earlier call.
 */
#define MUON_FP32 0
#define MUON_BF16 1
#define MUON_FP16 2
#define MUON_GRAD_MAX_TENSORS 65536
#define MUON_CLIP_RECORD_FLOATS 2
#define MUON_GRAD_WORKSPACE_BYTES 16640

/* The record of the gradients' norm.  Gradients are read only, and may share
 * memory with one another (each is counted). */
int muon_grad_norm(const void* const* grads, const int64_t* numels, const int* dtypes, int n, float max_norm,
                   float scale, float* record, void* workspace, hipStream_t stream);

/*
 * The record, and the clipped gradients g' rounded once (nearest even) to
 * out_dtypes[i] in outs[i]: other tensors, of the gradients' types or not
 * (16-bit gradients into fp32 ones), or the gradients themselves
 * (outs[i] = grads[i], same type).  In place a factor of 1 writes nothing.
 * No out may overlap another array of the call.
 */
int muon_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes,
                   const int* out_dtypes, int n, float max_norm, float scale, float* record, void* workspace,
                   hipStream_t stream);

/*
 * muon_adamw_step on the clipped gradients g' of the record, which may be of
 * 16-bit types.  Same arithmetic on g', same argument rules, no cached work
 * list; record may be NULL (factor 1: on fp32 gradients, muon_adamw_step's
 * bits).  The gradients may share memory with one another.
 */
int muon_adamw_step_clip(float* const* params, const void* const* grads, const int* grad_dtypes,
                         float* const* exp_avg, float* const* exp_avg_sq, const int64_t* numels,
                         const float* weight_decay, int n, float lr, float beta1, float beta2, float eps,
                         int64_t step, const float* record, hipStream_t stream);

/*
 * muon_step_sched (3 * ns_steps coefficients) on the clipped gradients g' of
 * the record; record may be NULL (factor 1: muon_step_sched's bits).  Under a
 * norm that is not finite `updates` receives zeros.
 */
int muon_step_clip(float* const* params, const float* const* grads, float* const* momentum,
                   const muon_shape_t* shapes, int n, float lr, float beta, int ns_steps, const float* coeffs,
                   uint16_t* const* updates, const float* record, hipStream_t stream);

/*
 * Products of the hidden layers, whose weights muon_step takes: the forward
 * product with bias, activation, dropout and residual in its epilogue, and the
 * two products of its backward pass ("Let's reproduce GPT-2 (124M)": a block's
 * linear layers, its MLP with the tanh form of GELU and its residual path).
 * For a layer z = x w + bias, y = residual + drop(act(z)):
 *   x m x k, w k x n, bias n;  z, y m x n
 *   muon_linear      y, and z itself on request (for the backward pass)
 *   muon_linear_dx   dx = residual + drop(dz w^T) act'(preact), m x k: the
 *                    gradient of the layer's input, carried on through the
 *                    dropout and activation of the layer below (preact is that
 *                    layer's z) where they are given
 *   muon_linear_dw   dw = x^T dz, or dw + x^T dz;  dbias likewise from the sums
 *                    of dz over its rows
 * Operands are bf16 or fp16; weights may also be fp32 (the master weights
 * that muon_step steps) and are then rounded to x's type, nearest even.
 * Everything else is fp32: the products' sums, bias, activation, its slope and
 * the residual's sum; y, dx and z are each rounded once, nearest even.  dw and
 * dbias are fp32.  Equal calls give equal bits.
 *   act     MUON_ACT_GELU  z / (1 + exp(-2u)), u = sqrt(2/pi) (z + 0.044715 z^3)
 *           MUON_ACT_RELU  max(z, 0);  MUON_ACT_RELU2  max(z, 0)^2
 *           act' of relu is 0 for z <= 0 and 1 above, of relu2 2 max(z, 0).  A NaN z
 *           has a NaN act and act', in every activation
 *   drop    with t = min(65535, floor(2^16 dropout + 1/2)): an element whose 16 random
 *           bits are at least t is kept, times 2^16 / (2^16 - t); the others become 0,
 *           whatever they were (an infinity or NaN too).  So `dropout` acts in steps
 *           of 2^-16.  The bits of element (r, c): of the 128 bits that Philox 4x32
 *           (Salmon, Moraes, Dror and Shaw, SC'11) with 7 rounds makes of the
 *           counter (c / 8, r, site, step) under the key (seed low, seed high), bits
 *           16 (c mod 8) and up.  The mask is never stored: muon_linear_dx and
 *           muon_dropout make it anew from the same numbers, for a matrix of the
 *           same width.  site tells a model's dropouts apart, step the training steps.
 *           r counts the rows of the call: calls that take other rows of one batch
 *           (micro-batches, ranks) need a step or seed of their own, or they drop the
 *           same places.
 *
 * Fields of muon_linear_t (for muon_linear_dx x is dz, m x n, y is dx, m x k,
 * residual is m x k and preact, read, m x k):
 *   m, k, n   m 0 .. MUON_LINEAR_MAX_ROWS; k, n 1 .. MUON_LINEAR_MAX_WIDTH;
 *             m = 0 does nothing.  Outputs of 2^23 tiles of 256 x 256
 *             and more (over 500 GB) are refused
 *   x, w, residual, y, preact  device; elements of a row adjacent, rows ldx, ldw,
 *             ldr, ldy, ldp elements apart, any alignment of the element
 *             type.  w_transposed = 1: w is stored n x k (ldw from row to row of k).
 *             Rows that are read may overlap (a distance of 0 repeats one); rows that are
 *             written may not.  The fastest kernels read matrices
 *             whose base is 16-byte aligned and whose rows are a multiple of 8
 *             elements apart (at most MUON_LINEAR_MAX_WIDTH) and long.  Others, and fp32
 *             weights, are read through registers by small products and copied to the workspace
 *             first by large ones: x costs that pass once more.
 *   x_type    MUON_BF16 or MUON_FP16, also the type of preact
 *   w_type, bias_type   x_type or MUON_FP32
 *   y_type    x_type or MUON_FP32, also the type of residual
 *   bias, residual, preact   may be NULL; muon_linear_dx takes no bias, and
 *             preact if and only if act is not MUON_ACT_NONE
 *   dropout   in [0, 1)
 *   rng       NULL, or two int64 on the device, 8-byte aligned: {seed, step}, read
 *             when the call runs, in the place of seed and step (a captured
 *             training step counts its step there); their bits are taken modulo
 *             2^64 and 2^32
 * y may be the residual itself, and for muon_linear_dx the preact (same
 * pointer, distance and type); no other array may overlap a written one, except
 * as column ranges of one buffer of rows.
 * workspace: device, 16-byte aligned, of at least the bytes that the
 * _workspace_bytes function gives for the same arguments (0: NULL will do).  Its contents
 * mean nothing before or after a call; calls that share it must be ordered on
 * the GPU.  The calls use none of the library's own workspace or plans: they
 * allocate nothing, cache nothing, and can be captured without an earlier call.
 */
#define MUON_ACT_NONE 0
#define MUON_ACT_GELU 1
#define MUON_ACT_RELU 2
#define MUON_ACT_RELU2 3
#define MUON_LINEAR_MAX_ROWS (1 << 30)
#define MUON_LINEAR_MAX_WIDTH (1 << 22)

typedef struct {
  int64_t m, k, n;
  const void* x;
  const void* w;
  const void* bias;
  const void* residual;
  void* y;
  void* preact;
  const int64_t* rng;
  int64_t ldx, ldw, ldr, ldy, ldp;
  uint64_t seed;
  uint32_t step, site;
  float dropout;
  int x_type, w_type, w_transposed, bias_type, y_type;
  int act;
} muon_linear_t;

int muon_linear(const muon_linear_t* layer, void* workspace, size_t workspace_bytes, hipStream_t stream);
int muon_linear_dx(const muon_linear_t* layer, void* workspace, size_t workspace_bytes, hipStream_t stream);
/* backward: 0 for muon_linear, 1 for muon_linear_dx.  0 is also given for
 * sizes, types and distances of x and w that the call refuses.  Of pointers only the
 * alignment of x and w counts; what overlaps is not looked at. */
size_t muon_linear_workspace_bytes(const muon_linear_t* layer, int backward);

/*
 * dw is k x n (dw_transposed = 1: stored n x k), rows lddw elements apart; dbias
 * may be NULL.  accumulate = 1 adds to what dw and dbias hold (the
 * micro-batches of a step).  m = 0 writes zeros, or adds nothing.
 */
typedef struct {
  int64_t m, k, n;
  const void* x;
  const void* dz;
  float* dw;
  float* dbias;
  int64_t ldx, lddz, lddw;
  int type, dw_transposed, accumulate;
} muon_linear_dw_t;

int muon_linear_dw(const muon_linear_dw_t* layer, void* workspace, size_t workspace_bytes, hipStream_t stream);
size_t muon_linear_dw_workspace_bytes(const muon_linear_dw_t* layer);

/*
 * Dropout by itself: y = residual + drop(x) act'(preact), m x n, with the mask,
 * the fields and the rules of muon_linear_t.  Without preact this is dropout and
 * its gradient (the same call on dy); with it, the gradient dz of a layer's z.
 * x_type any of the three types, also that of preact; y_type any, also that of
 * residual; n up to MUON_DROPOUT_MAX_COLS, and up to about 2^35 elements in all (2^24 blocks
 * of 256 groups of 8).  y may be x, preact or residual itself.
 */
#define MUON_DROPOUT_MAX_COLS ((int64_t)1 << 34)
typedef struct {
  int64_t m, n;
  const void* x;
  const void* residual;
  void* y;
  const void* preact;
  const int64_t* rng;
  int64_t ldx, ldr, ldy, ldp;
  uint64_t seed;
  uint32_t step, site;
  float dropout;
  int x_type, y_type;
  int act;
} muon_dropout_t;

int muon_dropout(const muon_dropout_t* args, hipStream_t stream);

/* Thread-local description of the last failing call on this thread ("" if none). */
const char* muon_last_error(void);

/*
 * Device workspace bytes a call over these shapes needs (bf16 iterates,
 * Gram and polynomial matrices, norm partials, fp32 partial tiles when a
 * long-K Gram product is cut into K chunks).  The plan's table block
 * (descriptors and work lists) is not part of it: each cached plan holds
 * its own small device allocation.  Pure host computation.  Returns 0 and
 * sets the error text for invalid shapes.
 */
size_t muon_workspace_bytes(const muon_shape_t* shapes, int n);

/*
 * Hand the library a caller-owned device workspace for the current device
 * (NULL/0 returns to library-owned workspace, allocated at the next call).
 * The caller keeps it alive until muon_release() or another
 * muon_set_workspace() call; calls that need more than `bytes` fail with
 * MUON_ENOMEM.  Waits for the device; plans on the previous workspace that
 * no captured graph uses are dropped.
 */
int muon_set_workspace(void* dev_ptr, size_t bytes);

/* Free the library's cached workspace and plans on all devices (synchronises). */
void muon_release(void);

/*
 * Counters of the current device's plan cache since it was created (or
 * since muon_release()), for diagnostics: out[0] plans built, out[1] table
 * uploads, out[2] pointer-write launches, out[3] device synchronisations,
 * out[4] plans evicted, out[5] workspace allocations.  out is a host array
 * of 6.  Never touches the device.
 */
int muon_plan_stats(int64_t out[6]);

/*
 * Concurrency of one call (1 .. 4, default 1; the setting is process-wide).
 * Matrices of one canonical shape (m x n, m <= n) form a group; with more
 * than one lane the groups are spread over up to `lanes` lanes, and each
 * lane runs its matrices' whole step on an internal stream of the library,
 * forked from the caller's stream (after everything enqueued there before the
 * call) and joined back to it, so that one group's kernels fill the GPU while
 * another's tail off.  1 keeps every kernel on the caller's stream.  Results
 * are bit-identical for any setting; under graph capture the lanes run one
 * after another on the capturing stream.  Kernel timing (below) brackets
 * each lane's launches on that lane's stream.
 */
int muon_set_lanes(int lanes);

/*
 * Kernel timing for measurement.  muon_timing_enable(k) brackets every
 * subsequent launch of kernel family k with HIP events on the launch stream;
 * k = -1 stops.  muon_timing_read waits for the recorded events and returns
 * the summed kernel time and the number of launches since the last read.
 */
#define MUON_KERNEL_MOMENTUM 0 /* momentum update + norm partial sums */
#define MUON_KERNEL_CAST 1     /* normalise + transpose + cast to bf16 */
#define MUON_KERNEL_GRAM 2     /* A = X X^T */
#define MUON_KERNEL_POLY 3     /* B = b A + c A A */
#define MUON_KERNEL_UPDATE 4   /* X <- a X + B X */
#define MUON_KERNEL_APPLY 5    /* W -= lr X */
#define MUON_KERNEL_ADAMW 6    /* multi-tensor AdamW (muon_adamw_step, muon_adamw_step_clip) */
#define MUON_KERNEL_GRAD_NORM 7 /* global gradient norm */
#define MUON_KERNEL_GRAD_CLIP 8 /* clipped gradients of muon_grad_clip */
#define MUON_KERNEL_LINEAR 9    /* muon_linear, muon_linear_dx, with their operands' copies */
#define MUON_KERNEL_LINEAR_DW 10 /* muon_linear_dw, likewise */
#define MUON_KERNEL_DROPOUT 11  /* muon_dropout */
int muon_timing_enable(int kernel);
int muon_timing_read(double* total_ms, int64_t* launches);

#ifdef __cplusplus
}
#endif

#endif /* MUON_H_ */
