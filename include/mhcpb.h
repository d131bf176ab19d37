/*
 * mhcpb -- mHC projection/RMS backward for GB300 (sm_103a), C ABI.
 *
 * The operation (cuDNN frontend page "DSv4.1 mHC projection/RMS backward",
 * intro):
 *
 *     P  = grad_proj[:, :24]
 *     dX = P @ W + grad_r / (r * K) * X          (stored BF16)
 *     dW = P^T @ X                                (stored FP32)
 *
 * Both matrix products use operands converted to TF32 (round to nearest,
 * ties away) with FP32 accumulation; the RMS term is FP32 arithmetic.  dW is
 * summed over tokens in an order fixed in advance and with no atomic adds, so it is bitwise
 * reproducible for a given (T, K) on any GB300.  Outputs are overwritten,
 * never accumulated into.  grad_proj's columns 24..31 are not read at all.
 *
 * The caller-facing shape of the API follows the same page's "Prepared class
 * API": a plan is created once per shape, reports its scratch size, and each
 * execute launches two kernels on the caller's stream (a streaming kernel
 * that writes dX and per-chunk dW partials into the workspace, then a
 * fixed-order reduction of the partials into dW) and makes no allocation.
 *
 * Layouts (all compact row-major, the page's "Requirements and tensor
 * contract"):
 *     x            BF16 [T, K]
 *     w            FP32 [24, K]
 *     grad_proj    FP32 [T, 32]     columns 24..31 ignored, even NaN/Inf
 *     grad_r, r    FP32 [T]         ([T,1] column vectors); r > 0 required
 *     dx           BF16 [T, K]      output, overwritten
 *     dw           FP32 [24, K]     output, overwritten
 *     grad_x_addend BF16 [T, K]     optional; dX = bf16(fp32(bf16(core)) + fp32(addend)),
 *                                   the value a separate BF16 add would give
 *                                   (prime-kernels PR #15, "fused mHC stream gradient")
 * K counts n_streams * hidden (4 * 5120 = 20480 in the training profile).
 *
 * Ownership: the caller owns every buffer and the stream.  The library keeps
 * no pointer past the return of mhcpb_execute; buffers must stay alive until
 * the enqueued work completes (and for every replay of a captured graph).
 * Executions that may overlap on the GPU need their own workspace and outputs.
 *
 * Errors: every function returns a status.  On any error nothing is enqueued.
 * A wait inside a kernel that runs out of time (about one second) ends the
 * kernel early and records MHCPB_ERR_DEVICE_TIMEOUT in the plan's device
 * status word, read with mhcpb_get_device_status; the outputs of that
 * execution are then undefined but the CUDA context stays usable.
 *
 * Thread safety: a plan may be used from several host threads; executions on
 * one plan share its device status word only.
 */
#ifndef MHCPB_H
#define MHCPB_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct mhcpb_plan_s* mhcpb_plan_t;

typedef enum {
    MHCPB_OK = 0,
    MHCPB_ERR_INVALID_ARG = 1,        /* NULL plan/pointer, addend presence disagreeing with the plan */
    MHCPB_ERR_UNSUPPORTED_SHAPE = 2,  /* a size, count or stride outside the call's limits: T < 0, a plan's K
                                         not a positive multiple of 8, above the maxima below */
    MHCPB_ERR_MISALIGNED = 3,         /* a pointer not aligned as the call requires (a plan's calls: 16 bytes,
                                         4 for the gate operands) */
    MHCPB_ERR_ALIASING = 4,           /* two operands (or workspace) share bytes */
    MHCPB_ERR_WRONG_DEVICE = 5,       /* a pointer not in device memory of the plan's device, or without a
                                         plan of the current device */
    MHCPB_ERR_TF32_NOT_ALLOWED = 6,   /* flags lack MHCPB_ALLOW_TF32 */
    MHCPB_ERR_WORKSPACE_TOO_SMALL = 7,
    MHCPB_ERR_CUDA = 8,               /* a CUDA runtime/driver call failed (see mhcpb_last_cuda_error) */
    MHCPB_ERR_DEVICE_TIMEOUT = 9,     /* reported by mhcpb_get_device_status */
    MHCPB_ERR_UNSUPPORTED_DEVICE = 10, /* device is not compute capability 10.3 (GB300) */
    MHCPB_ERR_SCRATCH_TOO_SMALL = 11  /* mhcpb_execute_static_scratch: the shape needs more
                                         than MHCPB_STATIC_SCRATCH_BYTES of dW partials */
} mhcpb_status_t;

/* Plan flags. */
enum {
    /* Required: the caller accepts TF32 operands in the matrix products (the
     * page makes allow_tf32=True mandatory). */
    MHCPB_ALLOW_TF32 = 1u,
    /* Executions pass a BF16 grad_x_addend that is added into dX. */
    MHCPB_HAS_ADDEND = 2u,
    /* Use the FP32-FMA (CUDA-core) streaming kernel instead of the tensor-core
     * one.  Same results within tolerance, same determinism; kept as the
     * measured control for the tensor-core kernel. */
    MHCPB_FMA_KERNEL = 4u,
    /* Compensated dW reduction: the second kernel sums each element's S chunk
     * partials in the same fixed order, but with an error-free transformation
     * at every addition (TwoSum: s + p = s' + e exactly) and the errors e
     * accumulated beside the sum, then rounds once to FP32: dW = fl(s + E).
     * This is Ogita, Rump and Oishi's cascaded summation (Sum2): as accurate
     * as summing the partials in twice the working precision and rounding
     * once, instead of S - 1 FP32 roundings.  Within a
     * chunk the products are exact in either mode (TF32 x BF16 split into
     * BF16 pairs) and are accumulated by the tensor cores in FP32.  Same
     * determinism: bitwise reproducible and independent of the SM count.
     * The idea comes from the FlashInfer page on
     * cake_rmsnorm_det_train_backward (program windows), whose small-T dw
     * column sums keep exact products, accumulate with TwoSum and round to
     * FP32 once; here it is applied to the cross-chunk reduction.  Costs a
     * few FP32 operations per partial in the second kernel only. */
    MHCPB_COMPENSATED_DW = 8u,
    /* Accumulate dW into the caller's buffer instead of overwriting it:
     * dW_out = dW_in + D in FP32 (one rounding), where D is exactly what the
     * execute would write without this flag (plain or compensated).  For
     * callers that sum weight gradients over micro-batches in an FP32 buffer of
     * their own (prime-kernels PR #15 offers this for its FP8 expert weight
     * gradients; here it applies to dW).  dW must
     * then hold valid values before the execute; dX is unaffected. */
    MHCPB_ACCUMULATE_DW = 16u,
    /* Test hook for failure detection: in the tensor-core kernel the MMA
     * issuer first waits on a barrier that nothing completes, so the execute
     * ends by the in-kernel wait limit, records MHCPB_ERR_DEVICE_TIMEOUT in the
     * status word and leaves the context usable.  Outputs are undefined.  Not
     * for production use. */
    MHCPB_TEST_INJECT_STALL = 1u << 30
};

/* Shape limits (inclusive).  0 <= T <= MHCPB_MAX_T.  T = 0 (an empty batch)
 * is valid everywhere: dX, proj, r and the gate outputs are empty, dW (a sum
 * over no tokens) is written as zeros, or left as dW + 0 with
 * MHCPB_ACCUMULATE_DW, and the workspaces are 0 bytes.  An operand with no
 * elements needs no storage: its pointer may be NULL and is not checked;
 * every non-empty operand (W, dW, the gates' alpha and bias) is checked as
 * for T > 0. */
#define MHCPB_MAX_T (1 << 24)
#define MHCPB_MAX_K (1 << 20)
/* Number of projection columns used, stored width of grad_proj. */
#define MHCPB_NPROJ 24
#define MHCPB_GRAD_PROJ_COLS 32
/* Tokens per dW partial: the token reduction is split into
 * S = ceil(T / MHCPB_PARTIAL_TOKENS(T)) fixed chunks of 512 tokens, whatever
 * the GPU, so dW bits depend only on (T, K) and the inputs. */
#define MHCPB_PARTIAL_TOKENS(T) 512

/* Creates a plan for one shape on one device.  Checks the flags and shape
 * first (no CUDA call is made when they are rejected), then that `device` is
 * a compute-capability-10.3 GPU, loads both kernels and allocates the plan's
 * 4-byte device status word.  `*out` is set only on success. */
mhcpb_status_t mhcpb_plan_create(mhcpb_plan_t* out, int64_t T, int64_t K, int device,
                                 uint32_t flags);

/* Scratch bytes an execute needs: S * 24 * K * 4 with
 * S = ceil(T / MHCPB_PARTIAL_TOKENS(T)) (15,728,640 B at T=4096, K=20480).
 * Contents need no initialisation and are dead after the execute (the
 * reduction drops them from L2 without writing them back when the workspace
 * is 128-byte aligned). */
mhcpb_status_t mhcpb_workspace_bytes(mhcpb_plan_t plan, size_t* bytes);

/* Enqueues the backward on `stream` (a cudaStream_t; NULL is the legacy
 * default stream).  All pointers are device pointers on the plan's device,
 * 16-byte aligned and pairwise disjoint; `grad_x_addend` must be NULL unless
 * the plan has MHCPB_HAS_ADDEND, and non-NULL if it has.  Returns without
 * synchronising.  Capturable into a CUDA graph (no allocation, no host sync;
 * tensor maps travel by value in the kernel parameters).  Both kernels are
 * launched as programmatic dependents of the kernel before them in the
 * stream: they may be scheduled early but touch no global memory before it
 * has completed, so stream order holds as for ordinary launches. */
mhcpb_status_t mhcpb_execute(mhcpb_plan_t plan,
                             const void* x, const float* w, const float* grad_proj,
                             const float* grad_r, const float* r,
                             void* dx, float* dw,
                             void* workspace, size_t workspace_bytes,
                             const void* grad_x_addend, void* stream);

/* The same backward in two calls, so that a caller can start using dX (send
 * it, or run the next layer's backward) before dW exists -- the split
 * backward of the prime-kernels PR #15 (the input gradient first, the weight
 * gradients after), applied to this stage:
 *
 *   mhcpb_execute_dx: enqueues the streaming kernel only.  When it completes,
 *   dX is final and `workspace` holds the dW partials of these inputs.
 *   mhcpb_reduce_dw:  enqueues the reduction only: dW from the partials that
 *   the last mhcpb_execute_dx with this workspace left there (overwritten, or
 *   accumulated with MHCPB_ACCUMULATE_DW).  It only reads the workspace, so
 *   it may be repeated on the same partials (e.g. a retried step, or the same
 *   partials accumulated into two dW buffers); each call gives the same sum.
 *   (mhcpb_execute, which writes and reduces the partials in one call, may
 *   drop them from L2 once summed: after it the workspace holds nothing
 *   reusable.)
 *
 * Arguments, checks and status codes are those of mhcpb_execute for the
 * operands each call uses.  The caller orders the two (same stream, or an
 * event) and must not touch the workspace in between.  dX and dW are
 * bitwise identical to mhcpb_execute's. */
mhcpb_status_t mhcpb_execute_dx(mhcpb_plan_t plan,
                                const void* x, const float* w, const float* grad_proj,
                                const float* grad_r, const float* r, void* dx,
                                void* workspace, size_t workspace_bytes,
                                const void* grad_x_addend, void* stream);
mhcpb_status_t mhcpb_reduce_dw(mhcpb_plan_t plan, void* workspace, size_t workspace_bytes,
                               float* dw, void* stream);

/* mhcpb_execute with timing events for measurement tools: records
 * `ev_before` (a cudaEvent_t, may be NULL) before the streaming kernel,
 * `ev_between` after it and `ev_after` after the reduction kernel, all on
 * `stream`.  The recorded event between the kernels stops the reduction from
 * starting early, so use plain mhcpb_execute for end-to-end timing. */
mhcpb_status_t mhcpb_execute_profiled(mhcpb_plan_t plan,
                                      const void* x, const float* w, const float* grad_proj,
                                      const float* grad_r, const float* r,
                                      void* dx, float* dw,
                                      void* workspace, size_t workspace_bytes,
                                      const void* grad_x_addend, void* stream,
                                      void* ev_before, void* ev_between, void* ev_after);

/* Reads (and, if `clear` is nonzero, resets) the plan's device status word.
 * Synchronises with the device.  *status is MHCPB_OK or the first device-side
 * error recorded since the last clear (MHCPB_ERR_DEVICE_TIMEOUT). */
mhcpb_status_t mhcpb_get_device_status(mhcpb_plan_t plan, mhcpb_status_t* status, int clear);

/* Plan facts for tools and tests: which = 0 T, 1 K, 2 partial count S,
 * 3 grid size of the streaming kernel, 4 flags, 5 streaming-kernel dynamic
 * shared memory bytes, 6 token tile, 7 column strip width, 8 tokens per
 * dW partial. */
mhcpb_status_t mhcpb_plan_query(mhcpb_plan_t plan, int which, int64_t* value);

/* Bounds checks of a checked build.  A library compiled with -DMHCPB_CHECKED
 * checks every global-memory access its kernels make at a computed address
 * (tensor-map copies are bounded by their maps) against the extent of its
 * buffer, skips an access found outside and records the first such site of
 * each kernel family.  This call copies those records and clears them:
 * sites[5] = {tensor-core backward, FMA backward, dW reduction, forward, gate
 * kernels}, each 0 (none since the last call) or 1 + the site within that
 * family's source.  *checked is 1 for a checked build; a normal build sets
 * it to 0 and every site to 0 and makes no CUDA call.  NULL arguments:
 * MHCPB_ERR_INVALID_ARG.  The words are per device (the current one) and
 * shared by all plans. */
mhcpb_status_t mhcpb_debug_checked_sites(uint32_t* sites, int* checked);

/* Sets the bound on every wait inside the plan's kernels (default 1 s,
 * accepted range 1 ms .. 60 s).  A wait that runs out ends the kernel early
 * with MHCPB_ERR_DEVICE_TIMEOUT in the status word.  Applies to executes
 * enqueued after the call. */
mhcpb_status_t mhcpb_plan_set_wait_limit(mhcpb_plan_t plan, uint64_t nanoseconds);

/* Caps the persistent grids of the tensor-core backward kernel and of the
 * forward kernel at `max_ctas` CTAs (one per SM; 0 restores the default of
 * every SM), e.g. to leave SMs to kernels that run concurrently on other
 * streams.  Results are bitwise identical for every cap: the dW partition
 * depends only on T, the forward's only on K.  The backward of
 * MHCPB_FMA_KERNEL plans is not affected.  Applies to calls enqueued after
 * this one. */
mhcpb_status_t mhcpb_plan_set_max_ctas(mhcpb_plan_t plan, int max_ctas);

/* Size of the library's built-in scratch buffer (see below): 16 MiB. */
#define MHCPB_STATIC_SCRATCH_BYTES (16u << 20)

/* The backward for callers that cannot allocate device memory at all: code
 * running inside a host framework that owns every byte of the device heap
 * (its own caching allocator, no cudaMalloc allowed), or plugin code that is
 * handed its input and output buffers and nothing else.  Such a caller cannot
 * create a plan (mhcpb_plan_create allocates the plan's status word) nor pass a
 * workspace.  This entry point needs neither: it runs the same two kernels as
 * mhcpb_execute (tensor-core streaming kernel, then the fixed-order reduction)
 * with the dW partials kept in a buffer the library itself declares as a
 * file-scope __device__ array of MHCPB_STATIC_SCRATCH_BYTES.  No counterpart
 * on the pages: their API always takes a caller-allocated workspace.
 *
 *  - No cudaMalloc, cudaFree or other allocating call is made.  The buffer is
 *    part of the loaded module: every GPU that loads the library holds its
 *    16 MiB until the process exits.
 *  - Shapes needing more than that are rejected with
 *    MHCPB_ERR_SCRATCH_TOO_SMALL: S * 24 * K * 4 bytes with
 *    S = ceil(T / MHCPB_PARTIAL_TOKENS(T)), i.e. up to T = 4096 at K = 20480.
 *  - Runs on the calling thread's current device; all pointers must be device
 *    memory there, 16-byte aligned and disjoint (same contract and status codes
 *    as mhcpb_execute).  `flags` must contain MHCPB_ALLOW_TF32 and may contain
 *    MHCPB_HAS_ADDEND (then `grad_x_addend` is required), MHCPB_COMPENSATED_DW
 *    and MHCPB_ACCUMULATE_DW, nothing else.
 *  - The first call on a device does that device's set-up (looks up the
 *    buffer's device address, raises the kernels' shared-memory limit).  Make
 *    that first call before any stream capture.
 *  - Every call, on every stream, shares the one buffer.  Nothing in it needs
 *    to start at zero (each call overwrites every partial it reads) and
 *    nothing in it is meant to be read afterwards (the reduction may drop the
 *    partials from L2 once summed).  Calls that may overlap on the GPU race on
 *    the buffer: order them on one stream or with events.
 *  - Every wait inside the kernels is bounded by a fixed 1 s (there is no plan
 *    to set another limit on).  A wait that runs out leaves the outputs
 *    undefined and is recorded in a device word that the kernels only ever
 *    write: this entry point neither reports nor clears it, so a timeout is
 *    not visible to the caller beyond the wrong outputs. */
mhcpb_status_t mhcpb_execute_static_scratch(int64_t T, int64_t K, uint32_t flags,
                                            const void* x, const float* w, const float* grad_proj,
                                            const float* grad_r, const float* r,
                                            void* dx, float* dw,
                                            const void* grad_x_addend, void* stream);

/* ---------------------------------------------------------------------------
 * The forward of the stage (the step before the backward in the graph).
 * The prime-kernels PR #15 page describes its mhc_projection as the RMS of the
 * streams and the projection logits, both from a single pass over X; this stage's
 * backward (the cuDNN page above) receives the gradients of exactly these two
 * outputs, and its dX formula is their vector-Jacobian product:
 *
 *     proj[t, j] = sum_k X[t, k] * W[j, k]      j < 24, TF32 W (nearest, ties
 *                                                away), FP32 accumulation
 *     r[t]       = sqrt(sum_k X[t, k]^2 / K + eps)
 *
 * Layouts: x BF16 [T, K] and w FP32 [24, K] as for the backward; proj FP32
 * [T, 32] (overwritten; columns 24..31 written as zero, the layout the
 * backward reads grad_proj in); r FP32 [T] (overwritten).  One streaming
 * kernel (tensor cores for the projection, CUDA cores for the squares) and a
 * fixed-order reduction of per-512-column partials: bitwise reproducible and
 * independent of the SM count.  The stream collapse that the page's
 * forward also fuses is a call of its own here (mhcpb_collapse_norm_forward,
 * by the gates H_pre).
 *
 * Uses the plan's T and K (any flags).  `eps` must be finite and >= 0.
 * Workspace: mhcpb_forward_workspace_bytes (ceil(K/512) * 25 * T' * 4 bytes,
 * T' = T rounded up to 32; 16,384,000 B at T=4096, K=20480), no
 * initialisation needed.  Pointers 16-byte aligned, disjoint, on the plan's
 * device; the same status codes and device status word as mhcpb_execute. */
mhcpb_status_t mhcpb_forward_workspace_bytes(mhcpb_plan_t plan, size_t* bytes);
mhcpb_status_t mhcpb_forward(mhcpb_plan_t plan, const void* x, const float* w, float eps,
                             float* proj, float* r, void* workspace, size_t workspace_bytes,
                             void* stream);
/* mhcpb_forward with timing events for measurement tools (cudaEvent_t, each
 * may be NULL): recorded before the streaming kernel, between the two
 * kernels and after the reduction, on `stream`. */
mhcpb_status_t mhcpb_forward_profiled(mhcpb_plan_t plan, const void* x, const float* w, float eps,
                                      float* proj, float* r, void* workspace,
                                      size_t workspace_bytes, void* stream, void* ev_before,
                                      void* ev_between, void* ev_after);

/* The forward with the gate step fused into its second kernel (the
 * prime-kernels PR #15 page's mhc_projection fuses the gate activations,
 * sigmoid and Sinkhorn, into the projection): writes proj and r exactly as
 * mhcpb_forward does, and h [T, 24] from them exactly as mhcpb_gate_forward
 * (below) would from the stored proj and r with the same alpha, bias and
 * n_iter: the same bits, one kernel launch fewer.  alpha [3], bias [24] and
 * h follow mhcpb_gate_forward's rules (device memory of the plan's device,
 * 4-byte aligned; h overlaps no other operand), the rest mhcpb_forward's.
 * n_iter outside 1 .. MHCPB_GATE_MAX_ITER: MHCPB_ERR_UNSUPPORTED_SHAPE.  The
 * reduction always takes its line layout here. */
mhcpb_status_t mhcpb_forward_gates(mhcpb_plan_t plan, const void* x, const float* w, float eps,
                                   const float* alpha, const float* bias, int n_iter, float* proj,
                                   float* r, float* h, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* ---------------------------------------------------------------------------
 * The gate/normalisation step around the stage: the forward turns the
 * projection logits and r into the mHC gates; the backward turns the gates'
 * upstream gradients into this stage's inputs grad_proj and grad_r.  The
 * cuDNN page (intro) places "the gate and normalization derivatives" before
 * the stage and leaves "Sinkhorn, gate derivatives" to the caller; the
 * prime-kernels PR #15 page ("mhc_projection") fuses "gate activations
 * (sigmoid, Sinkhorn)" into the projection.  Neither page writes the
 * formulas; these calls compute this reading of them (n = 4 streams, so the
 * 24 projection columns are 2n + n^2 logits):
 *
 *     columns 0..3 pre, 4..7 post, 8..23 res (row-major 4 x 4: 8 + 4i + j)
 *     l[t, j]  = a_g(j) * proj[t, j] / r[t] + b[j]       a = (a_pre, a_post, a_res)
 *     H_pre    = sigmoid(l_pre)
 *     H_post   = 2 sigmoid(l_post)
 *     H_res    = Sinkhorn(exp(l_res)): n_iter times, every row divided by its
 *                sum, then every column divided by its sum
 *
 * and the backward, for upstream gradients G in H's layout, the exact chain
 * rule: dl = dL/dl, grad_proj[t, j] = dl[t, j] a_g(j) / r[t] (columns 24..31
 * written as zero), grad_r[t] = -sum_j dl[t, j] a_g(j) proj[t, j] / r[t]^2.
 * The parameter gradients of a and b stay with the caller (the cuDNN page
 * leaves parameter-gradient accumulation to it); `dlogits`, if not NULL,
 * receives dl [T, 24] for that.
 *
 * Layouts (all FP32, row-major): proj [T, 32] (columns 24..31 not read), r [T],
 * alpha [3], bias [24], h and grad_h [T, 24], grad_proj [T, 32], grad_r [T].
 * FP32 arithmetic; results within 1e-4 of each token's largest magnitude of
 * the exact values (the backward for logits spanning up to ~35; beyond ~70 the
 * FP32 backward through the unrolled iterations loses accuracy, though it
 * stays finite; the forward holds at any spread).  0 <= T <= MHCPB_MAX_T, 1 <= n_iter <= MHCPB_GATE_MAX_ITER
 * (else MHCPB_ERR_UNSUPPORTED_SHAPE).  No plan and no workspace: the calls
 * run on the calling thread's current device, where every pointer must be
 * device memory (MHCPB_ERR_WRONG_DEVICE), 4-byte aligned (MHCPB_ERR_MISALIGNED);
 * outputs may not overlap each other or any input (MHCPB_ERR_ALIASING).
 * Enqueued on `stream`; nothing is allocated; outputs are overwritten. */
#define MHCPB_GATE_MAX_ITER 64
mhcpb_status_t mhcpb_gate_forward(int64_t T, int n_iter, const float* proj, const float* r,
                                  const float* alpha, const float* bias, float* h, void* stream);
mhcpb_status_t mhcpb_gate_backward(int64_t T, int n_iter, const float* proj, const float* r,
                                   const float* alpha, const float* bias, const float* grad_h,
                                   float* grad_proj, float* grad_r, float* dlogits, void* stream);

/* ---------------------------------------------------------------------------
 * The operators around the stage: what a model needs between its token ids,
 * the residual streams X and a sublayer (n = 4 streams of hidden size D, so
 * K = 4 D):
 *
 *     mhcpb_embed_*          token ids -> X, and the embedding table's gradient
 *     mhcpb_layernorm_*      a norm of any [T, D] activations
 *     mhcpb_collapse_norm_*  X and the gates H_pre -> the sublayer's normalised input
 *     mhcpb_dropout          dropout without a stored mask
 *     mhcpb_update_*         X, H_res, H_post and the sublayer's output -> the next X
 *
 * One sublayer is mhcpb_forward_gates (proj, r and h from X), collapse_norm
 * (y), the caller's sublayer, update (the next X).  Its backward is
 * update_backward (the sublayer output's gradient and columns 4..23 of
 * grad_h), the caller's sublayer, collapse_norm_backward (columns 0..3 of
 * grad_h, and the part of dX that does not go through the projection),
 * mhcpb_gate_backward (grad_proj and grad_r from grad_h), and mhcpb_execute
 * with that part of dX as its grad_x_addend.
 *
 * Common rules.  No plan: the calls run on the calling thread's current
 * device, where every operand must be device memory
 * (MHCPB_ERR_WRONG_DEVICE).  Nothing is allocated and nothing synchronises;
 * the calls are enqueued on `stream` and can be captured into a CUDA graph.
 * FP32 arithmetic; each output is rounded once, to its own type.  Every result
 * is bitwise reproducible for the same sizes and alignment.  Outputs are
 * overwritten (parameter gradients are added to with MHCPB_ACCUMULATE_DW) and
 * overlap no other operand (MHCPB_ERR_ALIASING), except where "in place" is
 * said.  Layouts are compact and row-major unless a stride is given; a stride
 * counts elements between rows, at least the row's width (else
 * MHCPB_ERR_UNSUPPORTED_SHAPE) and at most 2^24.  Operands with the same stride
 * may lie in each other's gaps, as column slices of one buffer do; with other
 * operands the gaps count as the operand's own.  Pointers are aligned to
 * their element's size (MHCPB_ERR_MISALIGNED); streams, their gradients and
 * collapse_norm's and update's other BF16 operands, and workspaces, to 16
 * bytes.  Sizes that are multiples of 8, on 16-byte aligned pointers, run
 * fastest.  T = 0 is valid: there is nothing to write but the parameter
 * gradients, which are then 0 (or unchanged when accumulating); operands with
 * no elements may be NULL.  1 <= D, with D <= MHCPB_MAX_K for mhcpb_layernorm_*,
 * 4 D <= MHCPB_MAX_K for the streams, n_streams * D <= MHCPB_MAX_K for
 * mhcpb_embed_*; 0 <= T <= MHCPB_MAX_T (else MHCPB_ERR_UNSUPPORTED_SHAPE).
 * Unknown types or flags: MHCPB_ERR_INVALID_ARG.  Non-finite values propagate
 * as the formulas say and never leave their token (parameter gradients apart). */
enum {                      /* element types */
    MHCPB_BF16 = 0,
    MHCPB_FP16 = 1,
    MHCPB_FP32 = 2
};
#define MHCPB_MAX_VOCAB (1 << 24)
#define MHCPB_MAX_STREAMS 16

/* x[t, s, :] = bf16(scale * table[ids[t], :]) for each of n_streams streams s.
 * table: `type` [V, D]; ids: [T] signed integers of id_bytes = 4 or 8 bytes; x: BF16
 * [T, n_streams * D].  An id outside [0, V), such as a padding id of -1, gives
 * a row of zeros.  1 <= V <= MHCPB_MAX_VOCAB, 1 <= n_streams <= MHCPB_MAX_STREAMS. */
mhcpb_status_t mhcpb_embed_forward(int64_t T, int64_t V, int64_t D, int n_streams, int type,
                                   const void* table, const void* ids, int id_bytes, float scale,
                                   void* x, void* stream);
/* grad_table[v, :] = scale * sum over tokens t with ids[t] = v and streams s of
 * grad_x[t, s, :], FP32 [V, D]; rows no token names are written as zeros, or
 * left alone with MHCPB_ACCUMULATE_DW.  grad_x: BF16 [T, n_streams * D].  Ids
 * outside [0, V) contribute nothing.  The tokens are sorted by id and each
 * row is summed in a fixed order (no sum uses atomics). */
mhcpb_status_t mhcpb_embed_workspace_bytes(int64_t T, int64_t V, int64_t D, size_t* bytes);
mhcpb_status_t mhcpb_embed_backward(int64_t T, int64_t V, int64_t D, int n_streams,
                                    const void* grad_x, const void* ids, int id_bytes, float scale,
                                    uint32_t flags, float* grad_table, void* workspace,
                                    size_t workspace_bytes, void* stream);

/* Layer norm over the last axis of x: `type` [T, D] with a row stride:
 *     mean = sum x / D, rstd = 1 / sqrt(sum (x - mean)^2 / D + eps)
 *     y    = (x - mean) * rstd * gamma + beta
 * gamma, beta: FP32 [D], NULL for ones and zeros.  y: `type`.  mean and rstd:
 * FP32 [T], both NULL where no backward follows.  eps finite and >= 0. */
mhcpb_status_t mhcpb_layernorm_forward(int64_t T, int64_t D, int type, const void* x,
                                       int64_t x_stride, const float* gamma, const float* beta,
                                       float eps, void* y, int64_t y_stride, float* mean,
                                       float* rstd, void* stream);
/* Its gradient from x, grad_y (`type`) and the forward's mean and rstd, with
 * z = (x - mean) rstd, w = grad_y gamma:
 *     grad_x = rstd (w - sum w / D - z sum(w z) / D)           `type`
 *     grad_gamma = sum_t grad_y z,  grad_beta = sum_t grad_y   FP32 [D], each may be NULL
 * `workspace` is not looked at (and may be NULL) when both are. */
mhcpb_status_t mhcpb_layernorm_workspace_bytes(int64_t T, int64_t D, size_t* bytes);
mhcpb_status_t mhcpb_layernorm_backward(int64_t T, int64_t D, int type, const void* x,
                                        int64_t x_stride, const void* grad_y, int64_t grad_y_stride,
                                        const float* gamma, const float* mean, const float* rstd,
                                        void* grad_x, int64_t grad_x_stride, float* grad_gamma,
                                        float* grad_beta, uint32_t flags, void* workspace,
                                        size_t workspace_bytes, void* stream);

/* y[e] = x[e] / (1 - p) where element e is kept, else 0 (whatever x[e] holds).
 * The mask comes from a counter and is never stored: element e is kept when
 *     word e % 4 of Philox4x32-10(counter {e / 4, rng[1] + sequence}, key rng[0])
 * is at least floor(p 2^32 + 1/2).  (Philox: Salmon, Moraes, Dror, Shaw, SC
 * 2011; counter and key words low half first, sums modulo 2^64.)  rng: two
 * 64-bit integers in device memory, 8-byte aligned, read when the call runs,
 * so that a captured graph draws new masks when the caller advances rng[1]
 * between replays; `sequence` tells the dropouts of one step apart.  The
 * gradient is the same call on the gradient.  0 <= p < 1; with p = 0, rng is
 * not looked at and may be NULL.  y may be x (in place). */
mhcpb_status_t mhcpb_dropout(int64_t n, int type, const void* x, float p, const void* rng,
                             uint64_t sequence, void* y, void* stream);

/* The sublayer's input: u = sum_s h[t, s] X[t, s, :] over the four streams
 * (H_pre is columns 0..3 of h [T, 24]), kept in FP32, then the layer norm of u
 * as above.  x: BF16 [T, 4 D]; y: BF16 [T, D]; mean and rstd of u. */
mhcpb_status_t mhcpb_collapse_norm_forward(int64_t T, int64_t D, const void* x, const float* h,
                                           const float* gamma, const float* beta, float eps,
                                           void* y, float* mean, float* rstd, void* stream);
/* Its gradient, with the residual path's share of dX (u is formed again from X):
 *     du = the layer norm's grad_x of grad_y
 *     grad_x[t, j, :] = h[t, j] du + sum_i H_res[t][i][j] grad_x_out[t, i, :]
 *     grad_h[t, j]    = <X[t, j, :], du>    j < 4; columns 4..23 are not touched
 * grad_x_out: BF16 [T, 4 D], the gradient of the streams after the sublayer;
 * NULL leaves that sum out.  grad_x: BF16 [T, 4 D].  grad_gamma, grad_beta,
 * flags and workspace as for mhcpb_layernorm_backward. */
mhcpb_status_t mhcpb_collapse_norm_workspace_bytes(int64_t T, int64_t D, size_t* bytes);
mhcpb_status_t mhcpb_collapse_norm_backward(int64_t T, int64_t D, const void* x, const float* h,
                                            const void* grad_y, const float* gamma,
                                            const float* mean, const float* rstd,
                                            const void* grad_x_out, void* grad_x, float* grad_h,
                                            float* grad_gamma, float* grad_beta, uint32_t flags,
                                            void* workspace, size_t workspace_bytes, void* stream);

/* The streams after the sublayer, with dropout of its output y (as
 * mhcpb_dropout on y [T, D]; p = 0: none):
 *     x_out[t, i, :] = sum_j H_res[t][i][j] X[t, j, :] + H_post[t][i] drop(y)[t, :]
 * H_post is columns 4..7 of h [T, 24], H_res columns 8 + 4 i + j.  x, x_out:
 * BF16 [T, 4 D], x_out may be x (in place); y: BF16 [T, D]. */
mhcpb_status_t mhcpb_update_forward(int64_t T, int64_t D, const void* x, const void* y,
                                    const float* h, float p, const void* rng, uint64_t sequence,
                                    void* x_out, void* stream);
/* Its gradient but for X (mhcpb_collapse_norm_backward adds that):
 *     grad_y = drop(sum_i H_post[t][i] grad_x_out[t, i, :])                BF16 [T, D]
 *     grad_h[t, 4 + i]         = <grad_x_out[t, i, :], drop(y)[t, :]>
 *     grad_h[t, 8 + 4 i + j]   = <grad_x_out[t, i, :], X[t, j, :]>;  columns 0..3 are not touched */
mhcpb_status_t mhcpb_update_backward(int64_t T, int64_t D, const void* x, const void* y,
                                     const float* h, float p, const void* rng, uint64_t sequence,
                                     const void* grad_x_out, void* grad_y, float* grad_h,
                                     void* stream);

/* mhcpb_debug_checked_sites for the operators above: sites[3] = {embedding,
 * norms, dropout and update}, read and cleared apart from that call's words. */
mhcpb_status_t mhcpb_debug_checked_operator_sites(uint32_t* sites, int* checked);

/* ---------------------------------------------------------------------------
 * A sublayer, and the update of its weights: the gated feed-forward block with
 * its gradient, and the orthogonalised update of a matrix.  The common rules
 * above hold, with these of their own:
 *  - every pointer is aligned to 16 bytes (MHCPB_ERR_MISALIGNED);
 *  - a row stride is the row's width, or a larger multiple of 8 (else
 *    MHCPB_ERR_UNSUPPORTED_SHAPE);
 *  - matrix products take 16-bit operands with FP32 accumulators; what one product
 *    forms and another reads (a = act(g) u, dg, du; X, A, B) is rounded to 16 bits
 *    between the two, everything else once, at the output.  Up to 64 tokens what
 *    that rounding loses is kept beside it (of up to four, a is FP32), but for the
 *    weights' gradients.  With FP16 operands a, dg and du also have FP16's range:
 *    beyond 65,504 they are infinite (a from five tokens on), and what is below 2^-25
 *    is zero (2^-36 up to 64 tokens, but for the weights' gradients), with FP32
 *    gradients too: grad_y is to be scaled as for any gradient in FP16, and BF16
 *    taken where act(g) u grows that large;
 *  - the waits inside the kernels are bounded (1 s): one that runs out leaves wrong
 *    outputs and is reported by mhcpb_operators_device_status. */
enum {                      /* activations */
    MHCPB_SILU = 0,         /* act(g) = g / (1 + exp(-g)) */
    MHCPB_GELU = 1          /* act(g) = g (1 + erf(g / sqrt 2)) / 2 */
};

/* The gated feed-forward block:
 *     g = x Wg^T,  u = x Wu^T,  y = (act(g) u) Wd^T
 * x, y: `type` (BF16 or FP16) [T, D] with row strides; w_gate, w_up: `type`
 * [F, D]; w_down: `type` [D, F].  gate and up: `type` [T, F], receive g and u for
 * the backward; both NULL where none follows.  1 <= D, F <= MHCPB_MAX_K.  D and
 * F that are multiples of 8 run fastest (others are copied to padded rows in the
 * workspace).  Any number of tokens; for one or a few, the time is the weights'
 * way from memory. */
mhcpb_status_t mhcpb_ffn_forward_workspace_bytes(int64_t T, int64_t D, int64_t F, size_t* bytes);
mhcpb_status_t mhcpb_ffn_forward(int64_t T, int64_t D, int64_t F, int type, int activation,
                                 const void* x, int64_t x_stride, const void* w_gate,
                                 const void* w_up, const void* w_down, void* y, int64_t y_stride,
                                 void* gate, void* up, void* workspace, size_t workspace_bytes,
                                 void* stream);
/* Its gradient from the forward's inputs, gate and up, with da = grad_y Wd,
 * dg = da u act'(g), du = da act(g), a = act(g) u:
 *     grad_x = dg Wg + du Wu                                      `type` [T, D]
 *     grad_w_gate = dg^T x,  grad_w_up = du^T x                   `grad_type` [F, D]
 *     grad_w_down = grad_y^T a                                    `grad_type` [D, F]
 * Each output may be NULL and is then not computed.  grad_type: `type`, or
 * MHCPB_FP32 (a sum over micro-batches loses nothing there; dg, du and a are
 * still rounded to `type`, so one call's share has that type's precision).
 * flags: MHCPB_ACCUMULATE_DW adds to the weights' gradients;
 * MHCPB_TEST_INJECT_STALL makes a wait run out. */
mhcpb_status_t mhcpb_ffn_backward_workspace_bytes(int64_t T, int64_t D, int64_t F, size_t* bytes);
mhcpb_status_t mhcpb_ffn_backward(int64_t T, int64_t D, int64_t F, int type, int activation,
                                  const void* x, int64_t x_stride, const void* w_gate,
                                  const void* w_up, const void* w_down, const void* gate,
                                  const void* up, const void* grad_y, int64_t grad_y_stride,
                                  void* grad_x, int64_t grad_x_stride, int grad_type,
                                  void* grad_w_gate, void* grad_w_up, void* grad_w_down,
                                  uint32_t flags, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* The orthogonalised update: X = G / (|G|_F + eps), then `steps` times
 *     A = X X^T,  B = b A + c A^2,  X = a X + B X       (a, b, c) = (3.4445, -4.7750, 2.0315)
 * (for m > n the same by columns), and out = scale X: each singular value of X
 * goes through a s + b s^3 + c s^5, singular vectors stay.  g: `type` (BF16, FP16
 * or FP32) [m, n], out: BF16 [m, n], both with row strides.  1 <= m, n <=
 * MHCPB_MAX_K, 1 <= steps <= MHCPB_ORTH_MAX_STEPS, eps finite and >= 0 (a zero G
 * with eps = 0 gives NaN, else 0), scale finite.  A non-finite element makes all
 * of out NaN.  A short side of at most 32 takes a cluster of 16 blocks: MHCPB_ERR_CUDA
 * where a limit on the process's SMs leaves no place for one. */
#define MHCPB_ORTH_MAX_STEPS 32
mhcpb_status_t mhcpb_orthogonalize_workspace_bytes(int64_t m, int64_t n, size_t* bytes);
mhcpb_status_t mhcpb_orthogonalize(int64_t m, int64_t n, int type, const void* g, int64_t g_stride,
                                   int steps, float eps, float scale, void* out,
                                   int64_t out_stride, void* workspace, size_t workspace_bytes,
                                   void* stream);

/* MHCPB_OK, or MHCPB_ERR_DEVICE_TIMEOUT once a wait inside a kernel of the calls
 * of this section has run out on the calling thread's current device; `clear` sets
 * it back.  Waits for the device's work. */
mhcpb_status_t mhcpb_operators_device_status(mhcpb_status_t* status, int clear);

/* mhcpb_debug_checked_sites for the calls of this section: sites[2] =
 * {feed-forward, orthogonalisation}. */
mhcpb_status_t mhcpb_debug_checked_matrix_sites(uint32_t* sites, int* checked);

/* Releases the plan (and its status word).  Safe on NULL. */
mhcpb_status_t mhcpb_destroy(mhcpb_plan_t plan);

/* Static description of a status; never NULL. */
const char* mhcpb_status_string(mhcpb_status_t status);

/* The last CUDA error string seen by this thread inside the library (for
 * MHCPB_ERR_CUDA), or "" if none. */
const char* mhcpb_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MHCPB_H */
