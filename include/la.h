/*
 * la.h -- C ABI of the GB300 (sm_103a) fused linear-attention library (libla.so).
 *
 * The operation (module neuralops.core.triton_kernels.linear_attn, functions `fwd` and
 * `bwd`; feature list in that module's docstring: feature maps elu+1 and relu, chunked
 * causal streaming, bidirectional parallel reduction, cosFormer cos/sin modulation):
 *
 *   a_i^p = w_i^p phi(q_i),  b_j^p = w_j^p phi(k_j)
 *   S_i^p = sum_{j in J(i)} b_j^p v_j^T,  z_i^p = sum_{j in J(i)} b_j^p
 *   out_i = (sum_p (a_i^p)^T S_i^p) / (sum_p a_i^p . z_i^p + eps)
 *
 * J(i) = {j <= i} (causal) or all j (bidirectional); phi(x) = elu(x) + 1, relu(x) or x;
 * without position weights there is one term p with w = 1, with them there are two:
 * w^cos = cos_weight and w^sin = sin_weight.  la_bwd returns the exact gradient of la_fwd
 * (the page's `bwd` differentiates `fwd`).
 *
 * Grouped-query attention (module neuralops.core.triton_kernels.gqa, `fwd`/`bwd`): with
 * Hkv key/value heads and Hq = n_rep * Hkv query heads, query head h reads key/value head
 * h / n_rep, and dk, dv are the sums over the n_rep query heads of each group.  The
 * expanded key/value tensors are never formed.
 *
 * Layout: q, out, grad_out, dq are contiguous [B, Hq, N, D]; k, v, dk, dv are contiguous
 * [B, Hkv, N, D] (row-major, D fastest); la_fwd_strided and la_bwd_strided take inputs with
 * other strides (D still contiguous).  la_fwd_v and la_bwd_v take a value width Dv of its
 * own: v, dv [B, Hkv, N, Dv] and out, grad_out [B, Hq, N, Dv] (`fwd` takes v as a tensor of
 * its own and reads only q's head dimension; the state S = sum b v^T is then D x Dv).  Elements are float32 (LA_F32) or
 * bfloat16 (LA_BF16); outputs use the input type.  Arithmetic is float32 accumulation in
 * both cases (bfloat16 tensor-core operands on the LA_BF16 fast path).  cos_weight and
 * sin_weight are float32 device vectors of length N, indexed by position, applied to
 * phi(q_i) and phi(k_i); give both or neither.
 *
 * Ownership: every pointer is caller-owned device memory (except where a function says
 * host).  The library allocates no device memory: scratch comes from the caller's
 * workspace of at least la_workspace_size() bytes, 256-byte aligned.  Outputs are fully
 * overwritten, never accumulated into.  The workspace must not be shared by calls that
 * can run at the same time.
 *
 * Execution: la_fwd and la_bwd only enqueue kernels on `stream` (a cudaStream_t; NULL is
 * the legacy default stream) and return; they never synchronise.  Kernels are launched with
 * programmatic stream serialization, so a kernel's blocks may be placed while the previous
 * kernel's last blocks finish; each kernel waits for the work before it on the stream to
 * complete (griddepcontrol.wait) before it touches memory, so stream order holds as for
 * plain launches.  Their status covers
 * argument checks and launch errors.  Errors found by a kernel while it runs (a bounded
 * wait that ran out) are latched in a device word that la_get_status() reads.
 *
 * Errors: no exception crosses this ABI and no kernel traps.
 *   LA_ERR_ARG          null required pointer, B, Hq, Hkv, N or D <= 0, Hq % Hkv != 0,
 *                       eps negative or not finite, unknown dtype or phi, exactly one of
 *                       cos_weight / sin_weight given, sizes whose element count
 *                       overflows 64 bits
 *   LA_ERR_UNSUPPORTED  D (or Dv) not in {32, 64, 128}
 *   LA_ERR_ALIGN        a pointer that is not 16-byte aligned (workspace: 256-byte)
 *   LA_ERR_WORKSPACE    ws_bytes < la_workspace_size(...) or workspace NULL while needed;
 *                       (from la_get_status) la_bwd_from_fwd got a workspace that another
 *                       la_fwd call wrote
 *   LA_ERR_CUDA         a CUDA launch or runtime error (see la_last_cuda_error())
 *   LA_ERR_TIMEOUT      (from la_get_status) a kernel's bounded wait ran out
 * All argument checks run on the host before any CUDA call.
 */
#ifndef LA_H
#define LA_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    LA_OK = 0,
    LA_ERR_ARG = 1,
    LA_ERR_UNSUPPORTED = 2,
    LA_ERR_ALIGN = 3,
    LA_ERR_CUDA = 4,
    LA_ERR_TIMEOUT = 5,
    LA_ERR_WORKSPACE = 6
} la_status;

/* Feature map phi: elu(x) + 1 with alpha = 1, max(x, 0), or x itself (identity: the
 * caller's q and k are the features; the linear_attn page lists the maps as non-negative,
 * so identity expects non-negative q and k: with signed features the denominator can
 * vanish and the result is ill-conditioned or non-finite). */
typedef enum { LA_PHI_ELU1 = 0, LA_PHI_RELU = 1, LA_PHI_IDENTITY = 2 } la_phi;

/* Element type of q, k, v, grad_out and of every output. */
typedef enum { LA_F32 = 0, LA_BF16 = 1 } la_dtype;

/* Which kernel family a call with these arguments runs. */
typedef enum { LA_PATH_SIMT = 0, LA_PATH_TCGEN05 = 1 } la_path;

/* Element strides of a [B, H, N, D] input along B, H and N; its last dimension (D) is
 * contiguous.  E.g. q taken from a fused [B, N, 3, H, D] projection as qkv[:, :, 0]
 * permuted to [B, H, N, D]: b = 3 N H D, h = D, n = 3 H D. */
typedef struct {
    long long b, h, n;
} la_strides;

/* Bytes of workspace that la_fwd (is_bwd = 0) or la_bwd (is_bwd = 1) needs for these
 * sizes.  Host-only, never fails: returns 0 for arguments la_fwd / la_bwd would reject.
 * has_weights: 1 when cos_weight and sin_weight are given. */
size_t la_workspace_size(int B, int Hq, int Hkv, int N, int D, la_dtype dtype, int is_causal,
                         int has_weights, int is_bwd);

/* Kernel family chosen for these arguments (host-only; for tests and reports): the
 * tensor-core kernels (LA_PATH_TCGEN05) for bfloat16 at D = 64 or 128 with n_rep = Hq / Hkv
 * in {1, 2, 4, 8}, forward and backward (with cos/sin weights as two passes, one per term);
 * the CUDA-core kernels (LA_PATH_SIMT) otherwise. */
la_path la_kernel_path(int B, int Hq, int Hkv, int N, int D, la_dtype dtype, int is_causal,
                       int has_weights, int is_bwd);

/* la_workspace_size and la_kernel_path for a value width Dv (la_fwd_v, la_bwd_v).  Dv != D
 * runs on the CUDA-core kernels. */
size_t la_workspace_size_v(int B, int Hq, int Hkv, int N, int D, int Dv, la_dtype dtype, int is_causal,
                           int has_weights, int is_bwd);
la_path la_kernel_path_v(int B, int Hq, int Hkv, int N, int D, int Dv, la_dtype dtype, int is_causal,
                         int has_weights, int is_bwd);

/* Forward, `linear_attn.fwd(q, k, v, is_causal, phi, eps, cos_weight, sin_weight)`:
 * writes out [B, Hq, N, D]. */
la_status la_fwd(const void *q, const void *k, const void *v, void *out, int B, int Hq,
                 int Hkv, int N, int D, la_dtype dtype, int is_causal, la_phi phi, float eps,
                 const float *cos_weight, const float *sin_weight, void *workspace,
                 size_t ws_bytes, void *stream);

/* la_fwd on inputs with strides: q_strides, k_strides, v_strides (NULL: contiguous) give
 * each input's element strides; out is contiguous.  The strides are used as given (the
 * caller guarantees every element they reach lies in the input's allocation); negative
 * strides: LA_ERR_ARG.  On the tensor-core path (la_kernel_path) every stride must be a
 * multiple of 8 elements (TMA: 16-byte row strides), else LA_ERR_ALIGN; the CUDA-core
 * path takes any.  The gqa page's wrapper passes strides to its kernel in the same way. */
la_status la_fwd_strided(const void *q, const void *k, const void *v, void *out, int B, int Hq,
                         int Hkv, int N, int D, la_dtype dtype, int is_causal, la_phi phi,
                         float eps, const float *cos_weight, const float *sin_weight,
                         const la_strides *q_strides, const la_strides *k_strides,
                         const la_strides *v_strides, void *workspace, size_t ws_bytes,
                         void *stream);

/* Backward, `linear_attn.bwd(q, k, v, grad_out, is_causal, phi, eps, cos_weight,
 * sin_weight) -> (dq, dk, dv)`: writes dq [B, Hq, N, D] and the group-summed dk, dv
 * [B, Hkv, N, D].  Recomputes what it needs of the forward from q, k, v. */
la_status la_bwd(const void *q, const void *k, const void *v, const void *grad_out, void *dq,
                 void *dk, void *dv, int B, int Hq, int Hkv, int N, int D, la_dtype dtype,
                 int is_causal, la_phi phi, float eps, const float *cos_weight,
                 const float *sin_weight, void *workspace, size_t ws_bytes, void *stream);

/* The same backward (same operation, same results) for a caller that has just run la_fwd
 * on these inputs: fwd_workspace / fwd_ws_bytes are that call's workspace, still holding
 * what la_fwd left there: its scanned per-segment states S, z and, on the tensor-core path,
 * every row's denominator den_i = sum_p a_i^p . z_i^p + eps, a record of the call and, with
 * cos/sin weights, the output rows in float32.  When
 * the forward and the backward cut the sequence the same way (the same kernel family, chunk
 * and segments; true whenever both run on the tensor-core path) the backward reads those
 * instead of recomputing them, which saves the forward's pass over q, k and v (la_bwd on the
 * tensor-core path runs that forward itself, with dq as its output scratch); otherwise it
 * recomputes them and fwd_workspace is not read.  The pages' `bwd` recomputes the forward
 * through autograd; keeping the forward's context is this library's design.
 *
 * The caller guarantees that la_fwd ran with the same q, k, v (same buffers and values),
 * sizes, mode, phi, eps and weights, that its workspace was not written since, and that
 * the forward is ordered before this call (same stream, or an event).  On the tensor-core
 * path the backward checks the forward's record (sizes, mode, phi, eps, segments and the
 * q, k, v addresses): a workspace that another call wrote makes la_get_status() return
 * LA_ERR_WORKSPACE (the gradients of that call are then not valid).  Values changed in the
 * same buffers cannot be detected.  fwd_workspace is read only.  Errors as la_bwd;
 * LA_ERR_ARG if fwd_workspace is NULL. */
la_status la_bwd_from_fwd(const void *q, const void *k, const void *v, const void *grad_out,
                          void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int N, int D,
                          la_dtype dtype, int is_causal, la_phi phi, float eps,
                          const float *cos_weight, const float *sin_weight,
                          const void *fwd_workspace, size_t fwd_ws_bytes, void *workspace,
                          size_t ws_bytes, void *stream);

/* la_bwd (fwd_workspace NULL) or la_bwd_from_fwd (fwd_workspace given, from la_fwd_strided
 * with the same inputs and strides) on inputs with strides: q, k, v, grad_out strides as in
 * la_fwd_strided (NULL: contiguous); dq, dk, dv are contiguous.  Errors as la_fwd_strided
 * and la_bwd. */
la_status la_bwd_strided(const void *q, const void *k, const void *v, const void *grad_out,
                         void *dq, void *dk, void *dv, int B, int Hq, int Hkv, int N, int D,
                         la_dtype dtype, int is_causal, la_phi phi, float eps,
                         const float *cos_weight, const float *sin_weight,
                         const la_strides *q_strides, const la_strides *k_strides,
                         const la_strides *v_strides, const la_strides *g_strides,
                         const void *fwd_workspace, size_t fwd_ws_bytes, void *workspace,
                         size_t ws_bytes, void *stream);

/* la_fwd with a value width Dv in {32, 64, 128} of its own: q, k [.., N, D]; v [B, Hkv, N,
 * Dv]; writes out [B, Hq, N, Dv].  All contiguous.  The state S = sum_j b_j v_j^T is D x Dv;
 * Dv = D is la_fwd.  Workspace: la_workspace_size_v.  Errors as la_fwd. */
la_status la_fwd_v(const void *q, const void *k, const void *v, void *out, int B, int Hq, int Hkv, int N, int D,
                   int Dv, la_dtype dtype, int is_causal, la_phi phi, float eps, const float *cos_weight,
                   const float *sin_weight, void *workspace, size_t ws_bytes, void *stream);

/* la_bwd (fwd_workspace NULL) or la_bwd_from_fwd (fwd_workspace from la_fwd_v with the same
 * arguments) with a value width Dv: grad_out [B, Hq, N, Dv]; writes dq [B, Hq, N, D], dk
 * [B, Hkv, N, D] and dv [B, Hkv, N, Dv].  All contiguous.  Errors as la_bwd. */
la_status la_bwd_v(const void *q, const void *k, const void *v, const void *grad_out, void *dq, void *dk, void *dv,
                   int B, int Hq, int Hkv, int N, int D, int Dv, la_dtype dtype, int is_causal, la_phi phi, float eps,
                   const float *cos_weight, const float *sin_weight, const void *fwd_workspace, size_t fwd_ws_bytes,
                   void *workspace, size_t ws_bytes, void *stream);

/* Synchronises `stream`, then returns and clears the device-side error word of the
 * current device: LA_ERR_TIMEOUT if a kernel's bounded wait ran out since the last call,
 * LA_ERR_WORKSPACE if la_bwd_from_fwd was given a forward workspace that another call
 * wrote, LA_ERR_CUDA if the synchronisation failed, else LA_OK. */
la_status la_get_status(void *stream);

/* Static, NUL-terminated description of a status code (host). */
const char *la_status_str(la_status status);

/* Static description of the most recent CUDA error seen by this library on the calling
 * thread ("" if none). */
const char *la_last_cuda_error(void);

/* Kernel timing for reports.  Between la_trace_start() and la_trace_stop() the library
 * brackets each of its kernel launches with a pair of CUDA events recorded on the
 * launch's own stream (the kernels themselves are unchanged).  la_trace_collect()
 * waits for those events, folds them per kernel name, frees them and returns how many
 * distinct kernels ran; la_trace_kernel() then reads entry `index` (0-based): a static
 * name, the number of launches and their summed device time in milliseconds.  Host-side
 * state is process-wide and guarded by a mutex. */
la_status la_trace_start(void);
la_status la_trace_stop(void);
int la_trace_collect(void);
la_status la_trace_kernel(int index, const char **name, int *launches, double *total_ms);

/* Low-rank projection (module neuralops.core.triton_kernels.low_rank, `fwd`):
 *
 *   y = (x V^T) U^T + bias
 *
 * x [M, K_in], V [r, K_in], U [K_out, r], bias [K_out] (NULL: no bias), y [M, K_out]; every
 * tensor row-major and contiguous, bfloat16 (LA_BF16), on the device; the leading
 * dimensions of a caller's x (batch, sequence) are the M rows.  Arithmetic: float32
 * accumulation on the tensor cores; the bottleneck t = x V^T is rounded to bf16 once before
 * the second product (as a bf16 framework computes the two products).  One kernel does both
 * products per 128-row tile, so t never goes to memory.  No workspace.
 * Errors: LA_ERR_ARG for sizes <= 0, a null x, U, V or y or an unknown dtype;
 * LA_ERR_UNSUPPORTED for LA_F32, r > 256, or K_in, K_out or r not a multiple of 8 (rows
 * must start on 16-byte boundaries); LA_ERR_ALIGN for a pointer that is not 16-byte
 * aligned.  Asynchronous on `stream`, like la_fwd. */
la_status la_lowrank_fwd(const void *x, const void *U, const void *V, const void *bias, void *y, int M,
                         int K_in, int r, int K_out, la_dtype dtype, void *stream);

/* Bytes of workspace that la_lowrank_bwd (is_bwd = 1) needs; 0 for the forward or for
 * arguments the calls reject.  Host-only. */
size_t la_lowrank_workspace_size(int M, int K_in, int r, int K_out, la_dtype dtype, int is_bwd);

/* Backward of la_lowrank_fwd (the page's `bwd`: gradients for x, U, V and bias) for the
 * output gradient grad_out [M, K_out]:
 *   t = x V^T,  dt = grad_out U,  dx = dt V,  dU = grad_out^T t,  dV = dt^T x,
 *   dbias = sum over the M rows of grad_out.
 * Writes dx [M, K_in], dU [K_out, r], dV [r, K_in] and, when dbias is not NULL, dbias
 * [K_out] (bf16).  t and dt (bf16, rounded once like the forward's t) and the float32
 * partial sums of the row reductions live in the workspace (la_lowrank_workspace_size, 256-
 * byte aligned); the row reductions are summed in a fixed order, so results are
 * deterministic.  Errors as la_lowrank_fwd, plus LA_ERR_WORKSPACE. */
la_status la_lowrank_bwd(const void *x, const void *U, const void *V, const void *grad_out, void *dx, void *dU,
                         void *dV, void *dbias, int M, int K_in, int r, int K_out, la_dtype dtype,
                         void *workspace, size_t ws_bytes, void *stream);

/* la_lowrank_fwd that also writes the bottleneck t = x V^T (bf16, [M, r], rounded once: the
 * bits la_lowrank_bwd would recompute) to t_out, for la_lowrank_bwd_t.  LA_ERR_ARG if t_out
 * is NULL; otherwise as la_lowrank_fwd. */
la_status la_lowrank_fwd_t(const void *x, const void *U, const void *V, const void *bias, void *y,
                           void *t_out, int M, int K_in, int r, int K_out, la_dtype dtype,
                           void *stream);

/* la_lowrank_bwd given the t that la_lowrank_fwd_t wrote for these x and V (ordered before
 * this call): the same results, without the backward's own pass over x for t.  The caller
 * guarantees t matches x and V.  LA_ERR_ARG if t is NULL; otherwise as la_lowrank_bwd (the
 * workspace size is the same). */
la_status la_lowrank_bwd_t(const void *x, const void *U, const void *V, const void *t,
                           const void *grad_out, void *dx, void *dU, void *dV, void *dbias, int M,
                           int K_in, int r, int K_out, la_dtype dtype, void *workspace,
                           size_t ws_bytes, void *stream);

/* ---- decayed linear attention -------------------------------------------------------------
 *
 * Linear attention whose state of each key/value head decays by gamma = exp(log_decay[head])
 * with every token (a matrix-valued state S [D, Dv], float32):
 *
 *   S_i = gamma S_{i-1} + k_i v_i^T,      out_i = scale q_i^T S_i
 *
 * i.e. out_i = scale sum_{j <= i} gamma^(i-j) (q_i . k_j) v_j + scale gamma^(i+1) q_i^T S_0.  No
 * feature map and no denominator: q and k are used as given (see la_qk_norm_rope_fwd).  The
 * pages have no counterpart of these entry points; layouts, grouped heads, dtypes, ownership,
 * streams and errors are la_fwd's: q, out [B, Hq, N, D | Dv], k, v [B, Hkv, N, D | Dv], D and Dv
 * in {32, 64, 128}, query head h reads key/value head h / n_rep; inputs may be strided
 * (la_strides, NULL: contiguous; 0 along a broadcast dimension), outputs are contiguous and overlap
 * no input but for the states named below.
 *
 * log_decay [Hkv] is a float32 device vector, expected <= 0 (a non-finite -inf is gamma = 0:
 * each token sees itself alone); it gets no gradient.  Values above 0 grow the state by the
 * same formula.  scale: a normal float32 (finite, not 0, not subnormal); grad_final_state / scale has
 * to be within float32.
 *
 * Arithmetic.  float32 inputs: float32 throughout.  bfloat16 inputs on the tensor cores
 * (la_decay_kernel_path): float32 sums and states; each term of an output is rounded to bfloat16 once on its way
 * (as a decayed score, or as the decayed k (q, v) in the state that queries read) and the output once
 * more: 2.3e-3 (2-norm) from the exact ones, where rounding the outputs alone leaves 1.7e-3.  The states that are given
 * are read to 2^-17; those that go out are within 1e-6 (2-norm), 3e-7 as measured.  For float32
 * arithmetic throughout give float32 inputs.
 *
 * A NaN or infinity in a token's row reaches, besides the outputs that depend on it, at most
 * the other rows of the same 128-token chunk on the tensor cores (earlier ones among them: a weight of 0
 * is multiplied there), none on the CUDA cores. */

/* Bytes of workspace of la_decay_fwd (is_bwd = 0) or la_decay_bwd (is_bwd = 1, enough for the
 * forward too), with or without a state that goes out; 0 for arguments that they reject (and where
 * none is needed).  Host-only. */
size_t la_decay_workspace_size(int B, int Hq, int Hkv, int N, int D, int Dv, la_dtype dtype, int is_bwd);

/* Kernel family of la_decay_fwd and la_decay_bwd: LA_PATH_TCGEN05 for bfloat16 with D and Dv in
 * {64, 128}, any n_rep (every input stride must then be a multiple of 8 elements, else
 * LA_ERR_ALIGN); LA_PATH_SIMT (float32 arithmetic, any strides) otherwise. */
la_path la_decay_kernel_path(int B, int Hq, int Hkv, int N, int D, int Dv, la_dtype dtype, int is_bwd);

/* Chunked form, for prompts and training.  initial_state [B, Hkv, D, Dv] float32 or NULL (zeros);
 * final_state like it or NULL (not wanted), may be the same buffer.  lengths: NULL, or a device
 * vector of B int32: sequence b has min(max(lengths[b], 0), N) tokens.  Rows past a sequence's
 * length are never used, whatever they hold; their out rows are zeros and final_state is the
 * state after the last token (the initial state when there is none). */
la_status la_decay_fwd(const void *q, const void *k, const void *v, void *out, const float *log_decay,
                       const float *initial_state, float *final_state, const int *lengths, int B, int Hq, int Hkv,
                       int N, int D, int Dv, la_dtype dtype, float scale, const la_strides *q_strides,
                       const la_strides *k_strides, const la_strides *v_strides, void *workspace, size_t ws_bytes,
                       void *stream);

/* Exact gradient of la_decay_fwd (without lengths): writes dq [B, Hq, N, D], dk [B, Hkv, N, D],
 * dv [B, Hkv, N, Dv] (summed over each group's query heads) and, when given, grad_initial_state.
 * grad_final_state: the gradient of final_state, or NULL (zeros); both [B, Hkv, D, Dv] float32,
 * contiguous; grad_initial_state may overlap no input (LA_ERR_ARG where it is initial_state or
 * grad_final_state).  Nothing of the forward is needed: the states are recomputed. */
la_status la_decay_bwd(const void *q, const void *k, const void *v, const void *grad_out, void *dq, void *dk, void *dv,
                       const float *log_decay, const float *initial_state, const float *grad_final_state,
                       float *grad_initial_state, int B, int Hq, int Hkv, int N, int D, int Dv, la_dtype dtype,
                       float scale, const la_strides *q_strides, const la_strides *k_strides,
                       const la_strides *v_strides, const la_strides *g_strides, void *workspace, size_t ws_bytes,
                       void *stream);

/* Recurrent form, one token per sequence (q, out [B, Hq, 1, D | Dv], k, v [B, Hkv, 1, D | Dv]), on a
 * pool of `pool` states [pool, Hkv, D, Dv] float32: sequence b owns slot slots[b] (device int32;
 * NULL: slot b).  Its state becomes gamma S + k v^T, in state_out at the same slot (state_out may
 * be `state`: in place; slots that no sequence names are not touched), and out = scale q^T S of the new
 * state.  A sequence whose slot is outside [0, pool) is padding: its out rows are zeros and no
 * state changes.  Two sequences of one call must not name the same slot.  Any strides (n is not used). */
la_status la_decay_step(const void *q, const void *k, const void *v, void *out, const float *state, float *state_out,
                        const float *log_decay, const int *slots, int pool, int B, int Hq, int Hkv, int D, int Dv,
                        la_dtype dtype, float scale, const la_strides *q_strides, const la_strides *k_strides,
                        const la_strides *v_strides, void *stream);

/* ---- norm of queries and keys with the position rotation ------------------------------------
 *
 * One pass over q [B, Hq, N, D] and k [B, Hkv, N, D]: every head's row x becomes
 *
 *   y = Rot(x r w),   r = rsqrt(mean(x^2) + eps)
 *
 * normalize = 0 leaves out r and w (rotation alone).  q_weight, k_weight: NULL (ones) or D elements
 * of weight_dtype (LA_F32, or the inputs' type).  Rot turns pair p of the row's first `rot` elements
 * (rot a multiple of 16, <= D; 0: no rotation) by the angle positions[a][b][n] inv_freq[p], where a
 * is the axis that pair p belongs to: the first sections[0] pairs to axis 0, the next sections[1]
 * to axis 1 and so on (1 to 4 axes, e.g. time, height, width; sum of sections = rot / 2).  Pair p is
 * elements (p, p + rot / 2), or (2p, 2p + 1) with interleaved = 1; elements past rot are not turned.
 * positions: device int64 [axes, B, N] with element strides pos_strides[3] (0 broadcasts);
 * inv_freq: rot / 2 device float64; sections and pos_strides are host arrays.  Angles are reduced
 * in 64-bit integer turns: the reduction errs by |position| 2^-65 turns (inv_freq up to 1), which is
 * below float32's own error for positions up to 2^39, and 2^-15 turns at 2^50.
 *
 * Inputs may be strided (rows must start on 16-byte boundaries, else LA_ERR_ALIGN); outputs are
 * contiguous and may not overlap the inputs.  Float32 arithmetic, D in {32, 64, 128}.  The pages have no
 * counterpart of these entry points; errors and streams are la_fwd's. */
typedef struct {
    const void *q_weight, *k_weight;
    la_dtype weight_dtype;
    float eps;                       /* >= 0, finite */
    int normalize, interleaved;
    int rot, axes;
    const int *sections;             /* host, `axes` entries (NULL: one axis) */
    const long long *positions;      /* device */
    const long long *pos_strides;    /* host, 3 entries */
    const double *inv_freq;          /* device */
} la_qk_args;

la_status la_qk_norm_rope_fwd(const void *q, const void *k, void *q_out, void *k_out, int B, int Hq, int Hkv, int N,
                              int D, la_dtype dtype, const la_strides *q_strides, const la_strides *k_strides,
                              const la_qk_args *args, void *stream);

/* Gradient: from grad_q, grad_k (of q_out, k_out) and the forward's inputs, dq [B, Hq, N, D], dk [B, Hkv, N,
 * D] and, where not NULL, dq_weight and dk_weight (D elements of weight_dtype; they need normalize = 1).  The sums over rows
 * are taken in a fixed order.  Workspace: la_qk_norm_rope_workspace_size (256-byte aligned). */
size_t la_qk_norm_rope_workspace_size(int B, int Hq, int Hkv, int N, int D, la_dtype dtype);
la_status la_qk_norm_rope_bwd(const void *q, const void *k, const void *grad_q, const void *grad_k, void *dq, void *dk,
                              void *dq_weight, void *dk_weight, int B, int Hq, int Hkv, int N, int D, la_dtype dtype,
                              const la_strides *q_strides, const la_strides *k_strides, const la_strides *gq_strides,
                              const la_strides *gk_strides, const la_qk_args *args, void *workspace, size_t ws_bytes,
                              void *stream);

/* ---- short causal convolution ---------------------------------------------------------------
 *
 * Each channel e of x [B, N, E] alone, with W taps (2 to 4):
 *
 *   v_t = bias + sum_j weight[e][j] x_(t - W + 1 + j),    out_t = v_t sigmoid(v_t)   (silu = 0: v_t)
 *
 * Rows before the first token are the initial state's, [B, W - 1, E] of x's type, the oldest first (NULL:
 * zeros); the final state is the last W - 1 rows, of the initial state where there are fewer, and may be the
 * same buffer.  weight [E, W], bias [E] (NULL: none): float32, or x's type (weight_dtype).  E a multiple of 8, at most
 * 2^31 - 128.
 * lengths: NULL, or B device int32: sequence b has min(max(lengths[b], 0), N) tokens; rows past them are not
 * used, whatever they hold, and their out rows are zeros.  x may be strided (la_strides, h not used: NULL
 * contiguous; 16-byte rows, i.e. multiples of 8 bfloat16 or 4 float32 elements, else LA_ERR_ALIGN; 0 along a broadcast
 * dimension).  Outputs are contiguous and overlap no input but for the states named.  Float32 arithmetic, one
 * rounding of an output.  The pages have no counterpart of these entry points; ownership, streams and errors
 * are la_fwd's (LA_ERR_UNSUPPORTED: W or E); every pointer is 16-byte aligned, lengths and slots 4. */
la_status la_conv_fwd(const void *x, const void *weight, const void *bias, void *out, const void *initial_state,
                      void *final_state, const int *lengths, int B, int N, int E, int W, la_dtype dtype,
                      la_dtype weight_dtype, int silu, const la_strides *x_strides, void *stream);

/* Bytes of workspace of la_conv_bwd; 0 for arguments that it rejects.  Host-only. */
size_t la_conv_workspace_size(int B, int N, int E, int W, la_dtype dtype);

/* Exact gradient: dx [B, N, E] (rows past a length: zeros), dweight [E, W] and, where not NULL, dbias [E] (which needs a
 * bias), of the weight's type, and, where not NULL, grad_initial_state [B, W - 1, E] of x's type, which may be none of
 * the inputs (LA_ERR_ARG).  grad_final_state: the gradient of the final state, or NULL (zeros).  Sums over tokens are
 * taken in float32 in a fixed order. */
la_status la_conv_bwd(const void *x, const void *weight, const void *bias, const void *grad_out, void *dx, void *dweight,
                      void *dbias, const void *initial_state, const void *grad_final_state, void *grad_initial_state,
                      const int *lengths, int B, int N, int E, int W, la_dtype dtype, la_dtype weight_dtype, int silu,
                      const la_strides *x_strides, const la_strides *g_strides, void *workspace, size_t ws_bytes,
                      void *stream);

/* One token per sequence, x and out [B, 1, E], on a pool of states [pool, W - 1, E] of x's type: sequence b owns slot
 * slots[b] (device int32; NULL: slot b), whose rows move up by one into state_out at the same slot (which may be
 * `state`: in place; slots that no sequence names are not touched).  A slot outside [0, pool) is a padding row: out
 * zeros, no state touched.  Two sequences of one call must not name the same slot. */
la_status la_conv_step(const void *x, const void *weight, const void *bias, void *out, const void *state, void *state_out,
                       const int *slots, int pool, int B, int E, int W, la_dtype dtype, la_dtype weight_dtype, int silu,
                       const la_strides *x_strides, void *stream);

/* ---- selective state space scan ---------------------------------------------------------------
 *
 * Every channel e of x [B, N, E] has S states (8, 16, 32 or 64) that decay by a factor of their own with every token:
 *
 *   d_t = softplus(dt_t + dt_bias)            (softplus = 0: dt_t + dt_bias)
 *   h_t = exp(d_t A) h_(t-1) + d_t x_t B_t,   out_t = (C_t . h_t + skip x_t) z_t sigmoid(z_t)
 *
 * x, dt, z, out [B, N, E] (z NULL: no gate); B, C [B, N, G, S], read by the E / G channels of a group in turn (E / G a
 * multiple of 8); A [E, S], skip [E], dt_bias [E] float32 (skip, dt_bias NULL: zeros).  A is finite, expected < 0;
 * other values grow the states by the same formula (one token's exp(d A) is to be below 2^128).  Inputs may be strided (la_strides; h is the step of B's and C's groups, not
 * used by the others; every stride a multiple of 16 bytes, else LA_ERR_ALIGN); outputs are contiguous and overlap no
 * input but for the states named.  States are float32 [B, E, S]: initial_state (NULL: zeros) comes in, the final one,
 * after each sequence's last token, goes out and may be the same buffer.  lengths: as la_conv_fwd's.
 *
 * Arithmetic is float32 for both types, one rounding of an output; states and sums err by a few 2^-23 of their
 * terms for each token that they remember.  A NaN or infinity in a token reaches what depends on it alone.  The pages have
 * no counterpart of these entry points; ownership, streams and errors are la_fwd's (LA_ERR_UNSUPPORTED: S or E / G);
 * every pointer is 16-byte aligned but skip, dt_bias, lengths and slots (4 bytes). */
typedef struct {
    const void *x, *dt, *B, *C, *z;
    const float *A, *skip, *dt_bias, *initial_state;
    const int *lengths;
    const la_strides *x_strides, *dt_strides, *B_strides, *C_strides, *z_strides;   /* host; NULL: contiguous */
    int batch, N, E, S, G;
    la_dtype dtype;
    int softplus;
} la_ssm_args;

/* Bytes of workspace of la_ssm_fwd (is_bwd = 0) or la_ssm_bwd (is_bwd = 1, enough for the forward too), and bytes of
 * the states that a training forward keeps for its gradient (every eighth token's, float32); 0 for arguments that
 * they reject (and where none is needed).  Host-only. */
size_t la_ssm_workspace_size(int batch, int N, int E, int S, int G, la_dtype dtype, int is_bwd);
size_t la_ssm_states_size(int batch, int N, int E, int S);

/* Prompts and training.  out may be NULL where `states` is given: only these (and the final state) are computed.
 * states: NULL, or states_bytes >= la_ssm_states_size (else LA_ERR_WORKSPACE), for la_ssm_bwd. */
la_status la_ssm_fwd(const la_ssm_args *args, void *out, float *final_state, void *states, size_t states_bytes,
                     void *workspace, size_t ws_bytes, void *stream);

/* Exact gradient for grad_out [B, N, E] (strided like x) and grad_final_state [B, E, S] (NULL: zeros).  `states` are those
 * that la_ssm_fwd left for the same args.  All of dx, ddt, dz [B, N, E] (dz with z only; rows past a length: zeros), dB, dC
 * [B, N, G, S] and dA [E, S] are written; dskip, ddt_bias [E] and grad_initial_state [B, E, S] where not NULL (the first two need
 * skip and dt_bias).  dA, dskip, ddt_bias and grad_initial_state are float32, the last may be none of the inputs
 * (LA_ERR_ARG).  All sums are taken in float32 in a fixed order. */
typedef struct {
    void *dx, *ddt, *dB, *dC, *dz;
    float *dA, *dskip, *ddt_bias, *grad_initial_state;
} la_ssm_grads;
la_status la_ssm_bwd(const la_ssm_args *args, const void *grad_out, const la_strides *g_strides,
                     const float *grad_final_state, const void *states, size_t states_bytes, const la_ssm_grads *grads,
                     void *workspace, size_t ws_bytes, void *stream);

/* One token per sequence (args->N = 1; initial_state and lengths NULL) on a pool of states [pool, E, S]; slots, state_out
 * and padding as in la_conv_step. */
la_status la_ssm_step(const la_ssm_args *args, void *out, const float *state, float *state_out, const int *slots, int pool,
                      void *stream);

/* Forward for callers that cannot allocate device memory.
 *
 * Some callers have no way to obtain scratch memory on the GPU: a plugin host that hands
 * a kernel library only its input and output buffers, or a latency-critical loop that may
 * not call cudaMalloc/cudaFree because those can synchronise the whole device.  This entry
 * point computes exactly what la_fwd computes, with the same arguments minus the
 * workspace: its scratch lives in LA_STATIC_WS_BYTES bytes of static device memory inside
 * this library, which every GPU that loads the library holds until the process exits.
 * It calls no allocator (no cudaMalloc, cudaFree or allocating library routine).  The
 * pages have no counterpart of this entry point.
 *
 * - Sizes whose forward needs more scratch than LA_STATIC_WS_BYTES (see
 *   la_workspace_size(..., is_bwd = 0)) are rejected with LA_ERR_STATIC_WS_LIMIT before
 *   any CUDA call.
 * - The first call on each device looks up the device address of the static scratch
 *   (cudaGetSymbolAddress, with that device current); make that first call before any
 *   stream capture.
 * - All calls share the one scratch array, which keeps whatever the last call left in
 *   it; the forward writes every scratch word before reading it, so nothing needs
 *   clearing between calls.  Calls whose work can overlap on the GPU (different streams,
 *   or different host threads) race on the scratch and must be serialised by the caller.
 */
#define LA_STATIC_WS_BYTES (64u * 1024u * 1024u)
#define LA_ERR_STATIC_WS_LIMIT ((la_status)7)

la_status la_fwd_static_ws(const void *q, const void *k, const void *v, void *out, int B,
                           int Hq, int Hkv, int N, int D, la_dtype dtype, int is_causal,
                           la_phi phi, float eps, const float *cos_weight,
                           const float *sin_weight, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LA_H */
