/*
 * falcon.h -- C ABI of the GB300 (sm_103a) Falcon fast-weight attention
 * library: chunk-parallel forward of Falcon-1 and Falcon-1A and its backward
 * pass, the forward of Falcon-2 and Falcon-2A (per-column step sizes) and of
 * Falcon-3A (sliding window) in token-recurrent and chunk form, and the
 * single-token recurrent decode step.  Beside these, the operators of a
 * selective state space block (short causal convolution, selective scan,
 * clipping of a step's gradients) and those of a linear attention block (attention with
 * a fixed decay a head, gated norms), in parts of their own below.
 *
 * The operations are defined on the page hyper.ai/fr/papers/2608.27763
 * ("Fast Weight Attention for Continual Learning"):
 *   - causal write pair x_t = phi(k_{t-1}), y_t = v_t, boundary x_1 = 0 with
 *     eta_1 = 0, and the read after write o_t = S_t^T phi(q_t): Section 4,
 *     "Naming and formula summary", and Section 3 "Indexing and causality
 *     conventions";
 *   - Falcon-1: S_t = (1 - eta_t lambda_t) S_{t-1} + eta_t x_t r_t^T with
 *     r_t = v_t - S_{t-1}^T x_t: Section 3.1, Eq. (3.3);
 *   - Falcon-1A: S_t = (1 - eta_t lambda_t) S_{t-1} + eta_t x_t v_t^T:
 *     Section 4.3, Eq. (4.6);
 *   - step size eta_t = beta_t / (||x_t||^2 + lambda_t + eps), 0 when the
 *     denominator is 0: Section 3.1, Eq. (3.4) and Section 4.3, Eq. (4.8);
 *   - decay clamp alpha_t = min(eta_t lambda_t, 1 - eps_gamma),
 *     gamma_t = 1 - alpha_t, evaluated in log space: Section 4.3, "Decay
 *     positivity", and Section 4.4, Eq. (4.15)-(4.16).
 * phi is the identity or the l2 map u / max(||u||_2, 1e-12) ("QK-l2" of the
 * experiments).
 *
 * Conventions shared by every entry point
 *   - All pointers are DEVICE pointers owned by the caller.  The library keeps
 *     no pointer after a call returns and allocates no memory; scratch space,
 *     where needed, is the caller's `workspace`.
 *   - Every call is asynchronous on the caller's `stream` (0 = legacy default
 *     stream) and returns before the GPU work ends.  A nonzero return means
 *     nothing was launched (argument errors) or a launch failed (FALCON_ERR_CUDA).
 *   - A chunked call with few heads and many chunks runs part of its work on a
 *     second stream the library creates once per device (with its events):
 *     the call forks from the caller's stream and joins back to it by events,
 *     so later work on the caller's stream sees the call complete, and a
 *     stream capture of the call captures the fork and the join.
 *   - The chunked forwards launch their kernels as programmatic dependent
 *     launches, and their last kernel lets the next such launch on the
 *     stream begin early.  Each of the library's kernels waits for the grid
 *     before it (griddepcontrol.wait) before it reads or writes memory, so
 *     stream order holds for the library's own calls and for ordinary
 *     launches.  A kernel of the caller's that is launched right after one of
 *     these calls with programmatic stream serialization may start before the
 *     call ends, and must wait for it (cudaGridDependencySynchronize) before it
 *     reads the call's outputs, as every such launch must.
 *   - Tensors are dense, row-major, contiguous; [B,H,T,m] means element
 *     (b,h,t,i) is at ((b*H + h)*T + t)*m + i.
 *   - Every pointer must be 16-byte aligned (FALCON_ERR_MISALIGNED otherwise).
 *   - The library never prints, exits or traps.
 */
#ifndef FALCON_GB300_H
#define FALCON_GB300_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define FALCON_OK 0
#define FALCON_ERR_NULL_PTR (-1)   /* a required pointer is NULL */
#define FALCON_ERR_BAD_SHAPE (-2)  /* unsupported size (see each call) */
#define FALCON_ERR_BAD_DTYPE (-3)  /* dtype or phi code out of range */
#define FALCON_ERR_MISALIGNED (-4) /* a pointer is not 16-byte aligned */
#define FALCON_ERR_WORKSPACE (-5)  /* workspace NULL or smaller than required */
#define FALCON_ERR_CUDA (-6)       /* a CUDA launch or query failed */
#define FALCON_ERR_TIMEOUT (-7)    /* a device-side wait hit its limit */
#define FALCON_ERR_BAD_ARG (-8)    /* eps/eps_gamma (or another scalar argument) out of range */
#define FALCON_ERR_DEVICE (-9)     /* the current device is not sm_103 */
#define FALCON_ERR_SCRATCH_LIMIT (-10) /* needs more than FALCON_FIXED_SCRATCH_BYTES */

/* Size of the scratch array built into the library for
 * falcon1_fwd_chunked_fixed_scratch (held on every GPU that loads it). */
#define FALCON_FIXED_SCRATCH_BYTES (16u * 1024u * 1024u)

/* Element type of q, k, v and o.  beta, lambda, states and features are
 * always float32. */
#define FALCON_BF16 0
#define FALCON_F32 1

/* Feature map phi applied to q and k: the identity, the l2 map
 * u / max(||u||_2, 1e-12), or RMSNorm(u) = u / sqrt(||u||_2^2 / d + eps_rms)
 * with eps_rms = 1e-6 (Section 4.1, "Scaled features": the pages' default
 * feature map; they name eps_rms without a value). */
#define FALCON_PHI_IDENTITY 0
#define FALCON_PHI_L2 1
#define FALCON_PHI_RMS 2

/* Ridge parameterisation (Section 4.1, "Scaled DeltaNet and the common ridge
 * parameterization"): lambda as given, or a base ridge lambda_bar from which
 * the recurrence takes lambda_t = lambda_bar_t * ||x_t||^2. */
#define FALCON_RIDGE_GIVEN 0
#define FALCON_RIDGE_SCALED 1

/* Problem description for the chunked forward calls.
 *   B, H   batch and heads; the B*H heads are independent.
 *   T      tokens per head, T >= 0; T need not be a multiple of `chunk`
 *          (the last chunk is partial).
 *   m      feature dimension of q, k (and of the state's rows): 16, 32, 64
 *          or 128.
 *   dv     value dimension: 16, 32, 64 or 128.
 *   chunk  chunk length C used by the chunk-parallel form: 16, 32 or 64.  It
 *          changes only the rounding, never the result in exact arithmetic.
 *   dtype  FALCON_BF16 or FALCON_F32 (q, k, v, o).
 *   phi    FALCON_PHI_IDENTITY, FALCON_PHI_L2 or FALCON_PHI_RMS.
 *   eps    >= 0, the step-size stabiliser of Eq. (3.4).
 *   eps_gamma in (0, 1), the clamp margin: gamma_t >= eps_gamma.
 *   ridge  FALCON_RIDGE_GIVEN (lambda is lambda_t) or FALCON_RIDGE_SCALED
 *          (lambda is the base ridge; lambda_t = lambda_t(input) * ||x_t||^2). */
typedef struct {
  int64_t B, H, T;
  int32_t m, dv, chunk;
  int32_t dtype;
  int32_t phi;
  float eps;
  float eps_gamma;
  int32_t ridge;
} falcon_shape;

/* Bytes of device workspace a chunked forward call with this shape needs
 * (0 means the call accepts workspace = NULL).  Returns 0 for an invalid
 * shape as well; the forward call then reports the shape error. */
size_t falcon_workspace_bytes(const falcon_shape *shape);

/* Falcon-1 chunk-parallel forward (Section 3.1 Eq. (3.3) with Eq. (3.4)).
 *   q, k    [B,H,T,m]  dtype
 *   v       [B,H,T,dv] dtype
 *   beta    [B,H,T]    f32, the gain beta_t (the pages use beta in (0,2))
 *   lambda  [B,H,T]    f32, the ridge coefficient lambda_t >= 0
 *   S0      [B,H,m,dv] f32, state entering token 1; NULL means zeros
 *   x_prev  [B,H,m]    f32, write feature of token 1 (phi(k) of the token
 *           before this segment); NULL means a fresh sequence, where the
 *           boundary sentinel applies (x_1 = 0, eta_1 = 0)
 *   o       [B,H,T,dv] dtype, out: o_t = S_t^T phi(q_t)
 *   S_out   [B,H,m,dv] f32, out: S_T.  May alias S0.
 *   x_last  [B,H,m]    f32, out, nullable: phi(k_T) (x_prev of the next
 *           segment; left untouched when T = 0 and x_prev is NULL, copied
 *           from x_prev when T = 0 otherwise)
 *   workspace, workspace_bytes: device scratch of at least
 *           falcon_workspace_bytes(shape) bytes, 256-byte aligned; contents
 *           are overwritten.  Concurrent calls need separate workspaces.
 * Errors: FALCON_ERR_NULL_PTR, _BAD_SHAPE, _BAD_DTYPE, _MISALIGNED,
 * _WORKSPACE, _BAD_ARG, _DEVICE (nothing launched); _CUDA (launch failed). */
int falcon1_fwd_chunked(const falcon_shape *shape, const void *q, const void *k,
                        const void *v, const float *beta, const float *lambda,
                        const float *S0, const float *x_prev, void *o,
                        float *S_out, float *x_last, void *workspace,
                        size_t workspace_bytes, cudaStream_t stream);

/* falcon1_fwd_chunked for callers that cannot allocate device memory: the
 * paper has no counterpart; this is a library convenience.  It computes
 * exactly what falcon1_fwd_chunked computes, but takes no workspace: its
 * scratch is a fixed array of FALCON_FIXED_SCRATCH_BYTES inside the library
 * (held on every GPU that loads the library until the process exits), so the
 * call allocates nothing.  It serves callers that are handed only input and
 * output buffers (a C host program, a plugin interface), whose allocator is
 * out of reach at the call site, or that forbid allocation after start-up.
 *   - Shapes with falcon_workspace_bytes(shape) > FALCON_FIXED_SCRATCH_BYTES
 *     are rejected with FALCON_ERR_SCRATCH_LIMIT (nothing launched).
 *   - The first call on each device, with that device current, resolves the
 *     array's device address (cudaGetSymbolAddress); make that first call
 *     before any stream capture on the device.  A tensor-core shape with
 *     few heads and many chunks (the chunk-range pieces described above)
 *     also creates, on its first use on the device, the library's second
 *     stream and its events, as falcon1_fwd_chunked does; a warm-up call of
 *     such a shape does that set-up too.
 *   - All calls on a device share the array, which keeps the previous call's
 *     contents (nothing needs clearing: every scratch element read is written
 *     first by the same call).  Calls whose GPU work overlaps race on it: issue
 *     them on one stream.
 * Other arguments, layouts, ownership and errors are those of
 * falcon1_fwd_chunked. */
int falcon1_fwd_chunked_fixed_scratch(const falcon_shape *shape, const void *q,
                                      const void *k, const void *v,
                                      const float *beta, const float *lambda,
                                      const float *S0, const float *x_prev,
                                      void *o, float *S_out, float *x_last,
                                      cudaStream_t stream);

/* Falcon-1A chunk-parallel forward (Section 4.3 Eq. (4.6), step size
 * Eq. (4.8) with E_t = ||x_t||^2).  Arguments, layouts, ownership and errors
 * are those of falcon1_fwd_chunked. */
int falcon1a_fwd_chunked(const falcon_shape *shape, const void *q,
                         const void *k, const void *v, const float *beta,
                         const float *lambda, const float *S0,
                         const float *x_prev, void *o, float *S_out,
                         float *x_last, void *workspace, size_t workspace_bytes,
                         cudaStream_t stream);

/* Falcon-1A with the normalised read (Section 2.2, Eq. (2.1)-(2.3): the
 * normaliser z_t of linear attention on the shifted write stream):
 *     o_t = S_t^T phi(q_t) / (z_t^T phi(q_t) + eps_attn),
 *     z_t = gamma_t z_{t-1} + eta_t x_t,
 * with S_t the Falcon-1A state and z taking the same step size eta_t and
 * clamped decay gamma_t as the numerator.  The pages define z for plain linear
 * attention (lambda = 0, unit gain, where this is their Eq. (2.3) exactly) and
 * defer the Falcon-1A version to an appendix they do not include; this is the
 * plainest reading.  The denominator is not clamped away from zero (the pages
 * note that the normalised read is attention-like only for a nonnegative
 * normaliser): callers with signed features choose eps_attn accordingly.
 *   z0      [B,H,m] f32, normaliser entering token 1; NULL means zeros
 *   z_out   [B,H,m] f32, out, nullable: z_T (may alias z0)
 *   eps_attn >= 0 and finite (FALCON_ERR_BAD_ARG otherwise)
 *   workspace: at least falcon_normalized_workspace_bytes(shape) bytes.
 * Other arguments, layouts, ownership and errors are those of
 * falcon1a_fwd_chunked (o holds the normalised read).  The call runs the
 * Falcon-1A forward and then one to three plain kernels for the denominator
 * (ordinary launches: they start after the forward's kernels complete); on the
 * tensor-core path with m = 64 the forward's map launch also writes the
 * denominator's per-chunk terms to the workspace. */
size_t falcon_normalized_workspace_bytes(const falcon_shape *shape);
int falcon1a_fwd_chunked_normalized(const falcon_shape *shape, const void *q,
                                    const void *k, const void *v,
                                    const float *beta, const float *lambda,
                                    const float *S0, const float *z0,
                                    const float *x_prev, float eps_attn,
                                    void *o, float *S_out, float *z_out,
                                    float *x_last, void *workspace,
                                    size_t workspace_bytes,
                                    cudaStream_t stream);

/* Bytes of device workspace falcon1_bwd_chunked / falcon1a_bwd_chunked need
 * for this shape (0 for an invalid shape; the call then reports the error). */
size_t falcon_bwd_workspace_bytes(const falcon_shape *shape);
/* Backward pass of the Falcon-1 chunk-parallel forward: the gradient of
 *   L = <dO, o> + <dS_T, S_T> + <dx_last, x_last>
 * with respect to every input of falcon1_fwd_chunked.  The pages state that
 * training differentiates through the update, so that the slow weights that
 * produce q, k, v, beta and lambda learn (Section 3, "Implicit fast-memory
 * objective"), through the log-decay renormalisation and the normalised step
 * size (Section 4.6, "Backward pass"); this is the exact gradient of the
 * forward as computed, with two conventions: on the clamped branch of the
 * decay (eta_t lambda_t >= 1 - eps_gamma) gamma_t = eps_gamma is a constant,
 * and the boundary sentinel (eta_1 = 0) passes no gradient to beta_1,
 * lambda_1.  The call recomputes the forward (chunk maps and the state
 * entering every chunk) in its workspace; it needs none of the forward's
 * outputs.
 *   shape, q, k, v, beta, lambda, S0, x_prev: the forward's arguments
 *           (S0 and x_prev nullable as there)
 *   dO      [B,H,T,dv] dtype, the cotangent of o
 *   dS_T    [B,H,m,dv] f32, nullable (zero), the cotangent of S_T
 *   dx_last [B,H,m] f32, nullable (zero), the cotangent of x_last
 *   dq, dk  [B,H,T,m] dtype, out;   dv [B,H,T,dv] dtype, out
 *   dbeta, dlambda [B,H,T] f32, out (with FALCON_RIDGE_SCALED, dlambda is
 *           the gradient for the lambda input, the base ridge)
 *   dS0     [B,H,m,dv] f32, out, nullable (not written); may alias dS_T
 *   dx_prev [B,H,m] f32, out, nullable (not written); zeros when x_prev is
 *           NULL (the sentinel feature is a constant)
 *   workspace, workspace_bytes: at least falcon_bwd_workspace_bytes(shape)
 *           bytes, 256-byte aligned; contents are overwritten.
 * Every shape and dtype of falcon1_fwd_chunked is accepted (fp32 arithmetic
 * on CUDA cores).  Errors as for falcon1_fwd_chunked. */
int falcon1_bwd_chunked(const falcon_shape *shape, const void *q, const void *k,
                        const void *v, const float *beta, const float *lambda,
                        const float *S0, const float *x_prev, const void *dO,
                        const float *dS_T, const float *dx_last, void *dq, void *dk,
                        void *dv, float *dbeta, float *dlambda, float *dS0,
                        float *dx_prev, void *workspace, size_t workspace_bytes,
                        cudaStream_t stream);
/* The backward pass of falcon1a_fwd_chunked (Section 4.3 Eq. (4.6)).
 * Arguments, layouts, ownership and errors are those of falcon1_bwd_chunked. */
int falcon1a_bwd_chunked(const falcon_shape *shape, const void *q, const void *k,
                         const void *v, const float *beta, const float *lambda,
                         const float *S0, const float *x_prev, const void *dO,
                         const float *dS_T, const float *dx_last, void *dq, void *dk,
                         void *dv, float *dbeta, float *dlambda, float *dS0,
                         float *dx_prev, void *workspace, size_t workspace_bytes,
                         cudaStream_t stream);
/* Falcon-2 forward (per-column step sizes), token-recurrent form: every
 * column j of the state follows its own step size and clamped decay,
 *   eta_{j,t} = beta_{j,t} / (||x_t||^2 + lambda_t + eps)  (0 at the sentinel
 *   and when the denominator is 0), gamma_{j,t} = 1 - min(eta_{j,t} lambda_t,
 *   1 - eps_gamma), S_t[:, j] = gamma_{j,t} S_{t-1}[:, j] + eta_{j,t} x_t r_{t,j},
 *   r_t = v_t - S_{t-1}^T x_t,  o_t = S_t^T phi(q_t);
 * page hyper.ai/fr/papers/2608.27763, the regression-family display of
 * Section 3.1 and the per-column NLMS step sizes of Section 4.2.
 * Arguments, layouts, ownership and errors are those of falcon1_fwd_chunked
 * except:
 *   beta    [B,H,T,dv] f32: one gain per value column and token
 *   shape->chunk is checked (16, 32 or 64) but not used: the call runs the
 *           recurrence token by token, and needs no workspace.
 * One CTA per head and 32 value columns runs the tokens in order; the state
 * stays in registers. */
int falcon2_fwd_recurrent(const falcon_shape *shape, const void *q,
                          const void *k, const void *v, const float *beta,
                          const float *lambda, const float *S0,
                          const float *x_prev, void *o, float *S_out,
                          float *x_last, cudaStream_t stream);

/* Falcon-2A, the per-column inner-product rule (Section 4.3, "Falcon-2A:
 * per-column inner-product write"): as falcon2_fwd_recurrent with r_t
 * replaced by v_t and E_t = ||x_t||^2 in the step size. */
int falcon2a_fwd_recurrent(const falcon_shape *shape, const void *q,
                           const void *k, const void *v, const float *beta,
                           const float *lambda, const float *S0,
                           const float *x_prev, void *o, float *S_out,
                           float *x_last, cudaStream_t stream);

/* Falcon-3A forward, the sliding-window inner-product rule (Section 4.5),
 * token-recurrent form, for fresh sequences:
 *   for t >= 2 the window I_t of the last `window` write pairs (x_j, v_j),
 *   j >= 2, B_t = |I_t|: N_bar_t = (1/B_t) sum x_j v_j^T, E_bar_t =
 *   (1/B_t) sum ||x_j||^2, eta_t = beta_t / (E_bar_t + lambda_t + eps)
 *   (lambda_t = lambda_bar_t * E_bar_t with FALCON_RIDGE_SCALED), gamma_t =
 *   1 - min(eta_t lambda_t, 1 - eps_gamma), S_t = gamma_t S_{t-1} +
 *   eta_t N_bar_t; token 1 is the boundary (no update); o_t = S_t^T phi(q_t).
 *   window  1 .. 32 (window 1 is Falcon-1A); FALCON_ERR_BAD_ARG otherwise.
 * Arguments, layouts, ownership and errors are those of falcon1_fwd_chunked
 * except: no x_prev (the window does not reach into a previous segment: exact
 * continuation would need the last window - 1 pairs), no workspace, and
 * shape->chunk is checked but not used. */
int falcon3a_fwd_recurrent(const falcon_shape *shape, int32_t window,
                           const void *q, const void *k, const void *v,
                           const float *beta, const float *lambda,
                           const float *S0, void *o, float *S_out,
                           float *x_last, cudaStream_t stream);

/* Falcon-2A forward in chunk form: the same result as falcon2a_fwd_recurrent
 * (up to rounding).  Every value column j has its own step sizes and
 * decays, so within a chunk of 64 tokens o_{t,j} = e^{G_{j,t}} (Q S)_{t,j} +
 * sum_{s<=t} <phi(q_t), x_s> e^{G_{j,t} - G_{j,s}} eta_{j,s} v_{s,j} and the
 * state leaving it is S o e^{G_C} + X^T V' (G_{j,.} the chunk-local log
 * prefix of column j; no triangular solve: the inner-product rule writes the
 * target itself).  For bf16 q, k, v with m = dv = 64 and shape->chunk = 64
 * this runs on the tensor cores and needs a workspace of
 * falcon_workspace_bytes(shape) bytes (256-byte aligned); for every other
 * shape it runs falcon2a_fwd_recurrent and ignores the workspace.
 * Arguments, layouts and errors are those of falcon2a_fwd_recurrent, plus
 * workspace / workspace_bytes as in falcon1_fwd_chunked. */
/* Falcon-2 forward in chunk form: the same result as falcon2_fwd_recurrent
 * (up to rounding).  Every value column j runs its own scalar-step delta
 * rule on the shared write features (Section 3.1, regression display; Section
 * 4.2, per-column step sizes), so inside a chunk of 64 tokens the written
 * residuals u_{t,j} = eta_{j,t} r_{t,j} of column j solve a unit-lower system
 * built from the shared Gram <x_t, x_l> and the column's own decays: one
 * batched per-column triangular solve per chunk.  With E_{t,j} the product of
 * column j's gammas over the chunk up to token t and w = u / E, the solve is
 * u_t = eta_t v_t - eta_t E_{t-1} ((X S)_t + sum_{l<t} <x_t, x_l> w_l), the
 * output o_t = E_t ((Q S)_t + sum_{l<=t} <q_t, x_l> w_l) and the state leaving
 * the chunk E_C (S + X^T W); a chunk whose decay product falls below e^{-60}
 * in some column (clamped gammas) runs token by token instead.  The chunks of
 * a head are sequential (the per-column systems depend on the entering
 * state): one CTA per head.  For bf16 q, k, v with m = dv = 64 and
 * shape->chunk = 64 this runs on the tensor cores; for every other shape it
 * runs falcon2_fwd_recurrent.  Arguments, layouts, ownership and errors are
 * those of falcon2_fwd_recurrent; no workspace is needed. */
int falcon2_fwd_chunked(const falcon_shape *shape, const void *q,
                        const void *k, const void *v, const float *beta,
                        const float *lambda, const float *S0,
                        const float *x_prev, void *o, float *S_out,
                        float *x_last, cudaStream_t stream);
int falcon2a_fwd_chunked(const falcon_shape *shape, const void *q,
                         const void *k, const void *v, const float *beta,
                         const float *lambda, const float *S0,
                         const float *x_prev, void *o, float *S_out,
                         float *x_last, void *workspace, size_t workspace_bytes,
                         cudaStream_t stream);
/* Falcon-3A forward in chunk form: the same result as falcon3a_fwd_recurrent
 * (up to rounding), computed as the masked-attention form of Section 4.6:
 * within a chunk of 64 tokens the state after token t is e^{g_t} S plus the
 * write pairs of the chunk and of the B - 1 pairs before it, each weighted by
 * w_{t,j} = sum over the chunk's tokens s <= t whose window holds pair j of
 * e^{g_t - g_s} eta_s / B_s; the chunk maps are composed across chunks by the
 * tensor-core scan.  For bf16 q, k, v with m = dv = 64 and shape->chunk = 64
 * this runs on the tensor cores and needs a workspace of
 * falcon_workspace_bytes(shape) bytes (256-byte aligned); for every other
 * shape it runs falcon3a_fwd_recurrent and ignores the workspace.
 * Arguments, layouts and errors are those of falcon3a_fwd_recurrent, plus
 * workspace / workspace_bytes as in falcon1_fwd_chunked. */
int falcon3a_fwd_chunked(const falcon_shape *shape, int32_t window,
                         const void *q, const void *k, const void *v,
                         const float *beta, const float *lambda,
                         const float *S0, void *o, float *S_out,
                         float *x_last, void *workspace, size_t workspace_bytes,
                         cudaStream_t stream);
/* One recurrent token (read after write) for N independent states: the
 * Falcon-1 update of Section 3.1 Eq. (3.3), as in the one-step listing of page
 * rcap.io/posts/fast-weight-attention-for-continual-learning-2026-08-27.
 *   q, k    [N,m]  dtype;  v, o [N,dv] dtype;  beta, lambda [N] f32
 *   S       [N,m,dv] f32, updated in place to S_t
 *   x_prev  [N,m] f32: read as this token's write feature x_t, then
 *           overwritten with phi(k_t) for the next token
 *   fresh   [N] bytes, nullable: nonzero marks a state whose sequence starts
 *           at this token (sentinel: x_t = 0, eta_t = 0, so S is not
 *           decayed and o = S^T phi(q)); NULL means no state is fresh
 * phi and ridge as in falcon_shape.
 * m, dv in {16, 32, 64, 128}.  N >= 0 (N = 0 launches nothing).
 * Errors as for falcon1_fwd_chunked (no workspace). */
int falcon1_decode_step(int64_t N, int32_t m, int32_t dv, int32_t dtype,
                        int32_t phi, int32_t ridge, float eps, float eps_gamma,
                        const void *q,
                        const void *k, const void *v, const float *beta,
                        const float *lambda, float *S, float *x_prev,
                        const uint8_t *fresh, void *o, cudaStream_t stream);

/* The same single-token step for Falcon-1A (Section 4.3 Eq. (4.6)). */
int falcon1a_decode_step(int64_t N, int32_t m, int32_t dv, int32_t dtype,
                         int32_t phi, int32_t ridge, float eps, float eps_gamma,
                         const void *q,
                         const void *k, const void *v, const float *beta,
                         const float *lambda, float *S, float *x_prev,
                         const uint8_t *fresh, void *o, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * A selective state space block: the short causal convolution, the selective
 * scan, and the clipping of a training step's gradients.  The convolution is
 * also what the paper's layers put before q, k and v ("short conv" in the
 * experiment setup), so its tensors may be laid out head by head, ready for
 * the calls above.
 *
 * Conventions of these calls where they differ from the ones above
 *   - Activations are FALCON_BF16 or FALCON_F32, read and written through
 *     strides (in elements; consecutive channels are adjacent), so that parts
 *     of one projection's rows need no copy.  Parameters (filters, biases, A,
 *     D), scan states and their gradients are dense float32.  Arithmetic is
 *     float32; a result is rounded once, when it is stored.
 *   - Pointers need the alignment of their element only.  Calls whose pointers
 *     are 16-byte aligned, with sizes and strides that keep rows so, move
 *     several channels per access; others move one.
 *   - `lengths` [B] int32, nullable: row b holds tokens 0 .. lengths[b] - 1
 *     (clamped to 0 .. T).  Later tokens are not read; their outputs and
 *     gradients are written as zeros.  A row of length 0 passes its state on.
 *   - `slots` [N] int32, nullable: row i of a single-token step uses state
 *     slots[i] of a pool of `pool` states (NULL: state i).  A row whose slot is
 *     outside 0 .. pool - 1 touches no state and its output is zero.  Two rows
 *     of a call must not name the same slot.
 *   - `fresh` [N] bytes, nullable: nonzero marks a sequence that starts at this
 *     token: its old state counts as zero.
 *   - Outputs must not overlap inputs unless a call says so, nor themselves.  An
 *     output of the convolution that starts where an input does, or an output with
 *     a zero stride over more than one row, is FALCON_ERR_BAD_ARG. */

/* Element strides of a tensor [B,H,T,m] (or [B,T,D], [B,T,G,N]: `head` is then
 * unused, or the group's stride). */
typedef struct {
  int64_t batch, head, time;
} falcon_strides;

#define FALCON_ACT_IDENTITY 0
#define FALCON_ACT_SILU 1

/* B rows of T tokens with H*m channels; channel c = h*m + i has a filter of
 * `width` taps (2, 3 or 4).  H = 1 is the plain [B,T,m] layout. */
typedef struct {
  int64_t B, H, T;
  int32_t m, width, dtype, activation;
} falcon_conv_shape;

/* Depthwise causal convolution over time:
 *   y_t = act(bias + sum_{j < width} weight_j x_{t - width + 1 + j}),
 * act the identity or silu(p) = p / (1 + e^{-p}); the inputs before token 0
 * are the carried ones.
 *   x          [B,H,T,m] dtype, strides x_strides
 *   weight     [H*m, width] f32;  bias [H*m] f32, nullable (zeros)
 *   state      [B, width-1, H*m] dtype, nullable (zeros): the inputs before
 *              token 0, oldest first
 *   y          [B,H,T,m] dtype, out, strides y_strides
 *   state_out  [B, width-1, H*m] dtype, out, nullable: the last width-1 inputs of
 *              each row (the carried ones where the row is shorter)
 * Errors: FALCON_ERR_NULL_PTR, _BAD_SHAPE, _BAD_DTYPE, _MISALIGNED, _BAD_ARG
 * (activation code, negative stride), _DEVICE; _CUDA. */
int falcon_short_conv_fwd(const falcon_conv_shape *shape, const void *x,
                          const falcon_strides *x_strides, const float *weight,
                          const float *bias, const void *state,
                          const int32_t *lengths, void *y,
                          const falcon_strides *y_strides, void *state_out,
                          cudaStream_t stream);

/* Gradients of <dy, y> + <dstate_out, state_out> of the call above.
 *   dy [B,H,T,m] dtype;  dstate_out [B, width-1, H*m] dtype, nullable (zeros)
 *   dx [B,H,T,m] dtype, out;  dweight [H*m, width] f32, out;
 *   dbias [H*m] f32, out, nullable;  dstate [B, width-1, H*m] dtype, out, nullable
 *   workspace: at least falcon_short_conv_bwd_workspace_bytes(shape) bytes,
 *   16-byte aligned (per-block sums of dweight and dbias, added in a fixed order). */
size_t falcon_short_conv_bwd_workspace_bytes(const falcon_conv_shape *shape);
int falcon_short_conv_bwd(const falcon_conv_shape *shape, const void *x,
                          const falcon_strides *x_strides, const float *weight,
                          const float *bias, const void *state,
                          const int32_t *lengths, const void *dy,
                          const falcon_strides *dy_strides, const void *dstate_out,
                          void *dx, const falcon_strides *dx_strides,
                          float *dweight, float *dbias, void *dstate,
                          void *workspace, size_t workspace_bytes,
                          cudaStream_t stream);

/* One token of N sequences: x [N,C] dtype with row stride x_stride, y [N,C]
 * dtype dense, out; state [pool, width-1, C] dtype, updated in place (the oldest
 * input leaves, x enters). */
int falcon_short_conv_step(int64_t N, int32_t C, int32_t width, int32_t dtype,
                           int32_t activation, const void *x, int64_t x_stride,
                           const float *weight, const float *bias, void *state,
                           int64_t pool, const int32_t *slots,
                           const uint8_t *fresh, void *y, cudaStream_t stream);

/* B rows of T tokens, D channels in G groups (D a multiple of G) that share
 * their B and C vectors, N states a channel (1 .. 128), B at most 65535; softplus nonzero:
 * the step size is softplus(delta + delta_bias), otherwise their sum. */
typedef struct {
  int64_t B, T;
  int32_t D, G, N, dtype, softplus;
} falcon_scan_shape;

/* Selective scan: for channel d of group g,
 *   s_t = softplus(delta_t + delta_bias),
 *   h_t = exp(s_t A) h_{t-1} + s_t u_t Bm_t      (per state n)
 *   y_t = (<Cm_t, h_t> + Dskip u_t) silu(z_t).
 *   u, delta, z, y  [B,T,D] dtype (z nullable: no gate; `head` stride unused)
 *   Bm, Cm          [B,T,G,N] dtype (`head` is the group's stride)
 *   A               [D,N] f32 (an infinite rate counts as the largest number, so that
 *                   a step of zero leaves the state);  Dskip, delta_bias [D] f32,
 *                   nullable (zeros)
 *   h0              [B,D,N] f32, nullable (zeros);  h_out [B,D,N] f32, out, may
 *                   alias h0
 * No workspace.  Errors as for falcon_short_conv_fwd. */
int falcon_selective_scan_fwd(const falcon_scan_shape *shape, const void *u,
                              const falcon_strides *u_strides, const void *delta,
                              const falcon_strides *delta_strides, const float *A,
                              const void *Bm, const falcon_strides *B_strides,
                              const void *Cm, const falcon_strides *C_strides,
                              const float *Dskip, const void *z,
                              const falcon_strides *z_strides,
                              const float *delta_bias, const float *h0,
                              const int32_t *lengths, void *y,
                              const falcon_strides *y_strides, float *h_out,
                              cudaStream_t stream);

/* Gradients of <dy, y> + <dh_T, h_T> of the call above; the forward is
 * recomputed.  With g_t the adjoint of h_t (g_t = Cm_t dy_t + exp(s_{t+1} A)
 * g_{t+1}, dy_t after the gate): dC_t = sum_d dy_t h_t, dB_t = sum_d g_t s_t u_t,
 * du_t = s_t <g_t, Bm_t> + Dskip dy_t, ds_t = <g_t exp(s_t A) h_{t-1}, A> +
 * <g_t, Bm_t> u_t, dA = sum_t g_t exp(s_t A) h_{t-1} s_t.
 *   dy [B,T,D] dtype;  dh_T [B,D,N] f32, nullable (zeros)
 *   du, ddelta [B,T,D] dtype, dense, out;  dz [B,T,D] dtype, dense, out, given
 *   exactly where z is;  dB, dC [B,T,G,N] dtype, dense, out;  dA [D,N] f32, out;
 *   dDskip, ddelta_bias [D] f32, out, nullable;  dh0 [B,D,N] f32, out, nullable,
 *   may alias dh_T (not h0)
 *   workspace: at least falcon_selective_scan_bwd_workspace_bytes(shape) bytes,
 *   256-byte aligned: a state and an adjoint for every 32 tokens, and sums, of which
 *   those of dB and dC take 2 GB at most, or two fp32 copies of dB and dC where that
 *   is more.  Sums over tokens and channels run in a fixed order. */
size_t falcon_selective_scan_bwd_workspace_bytes(const falcon_scan_shape *shape);
int falcon_selective_scan_bwd(const falcon_scan_shape *shape, const void *u,
                              const falcon_strides *u_strides, const void *delta,
                              const falcon_strides *delta_strides, const float *A,
                              const void *Bm, const falcon_strides *B_strides,
                              const void *Cm, const falcon_strides *C_strides,
                              const float *Dskip, const void *z,
                              const falcon_strides *z_strides,
                              const float *delta_bias, const float *h0,
                              const int32_t *lengths, const void *dy,
                              const falcon_strides *dy_strides, const float *dh_T,
                              void *du, void *ddelta, float *dA, void *dB, void *dC,
                              float *dDskip, void *dz, float *ddelta_bias, float *dh0,
                              void *workspace, size_t workspace_bytes,
                              cudaStream_t stream);

/* One token of N sequences: u, delta, z [N,D] dtype with row strides, Bm, Cm
 * [N,G,S] dtype (`batch` the row's stride, `head` the group's), y [N,D] dtype
 * dense, out; h [pool,D,S] f32, updated in place.  S states a channel (1 .. 128),
 * D up to 262144. */
int falcon_selective_scan_step(int64_t N, int32_t D, int32_t G, int32_t S,
                               int32_t dtype, int32_t softplus, const void *u,
                               int64_t u_stride, const void *delta,
                               int64_t delta_stride, const float *A, const void *Bm,
                               const falcon_strides *B_strides, const void *Cm,
                               const falcon_strides *C_strides, const float *Dskip,
                               const void *z, int64_t z_stride,
                               const float *delta_bias, float *h, int64_t pool,
                               const int32_t *slots, const uint8_t *fresh, void *y,
                               cudaStream_t stream);

/* One gradient of a step: `count` elements at `grad`, scaled into `out`
 * (out == grad: in place). */
typedef struct {
  const void *grad;
  void *out;
  int64_t count;
  int32_t dtype; /* FALCON_BF16 or FALCON_F32 */
} falcon_grad;

/* Clips the gradients of a step by their global norm n = sqrt(sum g^2):
 *   out = g * min(1, max_norm / (n + eps)).
 *   grads  HOST array of `tensors` descriptions (read before the call returns);
 *          dense tensors of any size, element-aligned.  A result shares its place
 *          with no other result and no gradient but its own (so no gradient is
 *          named twice in place)
 *   norm   [1] f32, out: n (before clipping)
 * In place, gradients that need no scaling are not rewritten.  A norm that is
 * NaN makes every output NaN; an infinite gradient makes the norm infinite, becomes
 * NaN, and scales the others by 0.  Squares are summed in float32 within a thread
 * where that holds them, in float64 otherwise and across threads, so that sizes
 * whose squares leave float32 count as well; a finite norm beyond float32 comes out
 * infinite, the gradients being scaled by its value.
 *   workspace: at least falcon_clip_workspace_bytes(grads, tensors) bytes,
 *   16-byte aligned.
 * Errors: FALCON_ERR_NULL_PTR, _BAD_SHAPE (negative count), _BAD_DTYPE,
 * _MISALIGNED, _WORKSPACE, _BAD_ARG (max_norm or eps negative or NaN, results that
 * overlap), _DEVICE; _CUDA. */
size_t falcon_clip_workspace_bytes(const falcon_grad *grads, int64_t tensors);
int falcon_clip_grad_norm(const falcon_grad *grads, int64_t tensors, float max_norm,
                          float eps, float *norm, void *workspace,
                          size_t workspace_bytes, cudaStream_t stream);

/* ---------------------------------------------------------------------------
 * A linear attention block with a fixed decay for each head: the attention over
 * prompts, its gradient and its single-token step, and the norms around a block.
 *
 * The conventions are those of the selective state space block above (strides,
 * alignment, `lengths`, `slots`, `fresh`, overlap).  Strides of inputs may be zero
 * (a broadcast head or row); the gradient of a broadcast input is returned for every
 * head and row that reads it, to be summed by the caller. */

/* B rows of T tokens, H heads with keys of m and values of dv channels (1 .. 128
 * each); scale multiplies the reads. */
typedef struct {
  int64_t B, H, T;
  int32_t m, dv, dtype;
  float scale;
} falcon_decay_shape;

/* Attention with a decay: for each row and head, gamma = exp(log_decay),
 *   S_t = gamma S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
 *   q, k       [B,H,T,m] dtype;  v, o [B,H,T,dv] dtype
 *   log_decay  [H] f32, at most 0 (a positive one counts as 0, minus infinity as
 *              the lowest number: the state then holds the last token alone)
 *   S0         [B,H,m,dv] f32, nullable (zeros);  S_out [B,H,m,dv] f32, out,
 *              nullable, may be S0
 *   workspace: at least falcon_decay_attn_workspace_bytes(shape) bytes, 256-byte
 *   aligned: a state for every run of tokens that is worked on by itself.
 * A NaN or infinity in a token reaches the tokens behind it in its row and head, and
 * may reach those before it among the 128 that are worked on together.  Whether it still
 * reaches a state or a token where its weight is zero in float32 (gamma^n below 2^-149)
 * depends on how the row is split.
 *   Behind a call's first kernel, an ordinary launch, the others are programmatic
 * dependent ones; they read the call's inputs, not what its kernels write, before they
 * wait for the one before them.  What is said above of a caller's kernel launched in
 * that way behind a chunked forward holds behind these calls too.
 * Errors: FALCON_ERR_NULL_PTR, _BAD_SHAPE, _BAD_DTYPE, _MISALIGNED, _WORKSPACE,
 * _BAD_ARG (negative stride, o where an input starts or on itself, scale not
 * finite), _DEVICE; _CUDA. */
size_t falcon_decay_attn_workspace_bytes(const falcon_decay_shape *shape);
int falcon_decay_attn_fwd(const falcon_decay_shape *shape, const void *q,
                          const falcon_strides *q_strides, const void *k,
                          const falcon_strides *k_strides, const void *v,
                          const falcon_strides *v_strides, const float *log_decay,
                          const float *S0, const int32_t *lengths, void *o,
                          const falcon_strides *o_strides, float *S_out,
                          void *workspace, size_t workspace_bytes,
                          cudaStream_t stream);

/* Gradients of <dO, o> + <dS_T, S_T> of the call above (the decay is fixed and has
 * none).  With G_t the adjoint of S_t, G_t = scale q_t dO_t^T + gamma G_{t+1}:
 * dq_t = scale S_t dO_t, dk_t = G_t v_t, dv_t = G_t^T k_t, dS0 = gamma G_1.
 *   dO [B,H,T,dv] dtype;  dS_T [B,H,m,dv] f32, nullable (zeros)
 *   dq, dk [B,H,T,m] dtype, dv [B,H,T,dv] dtype, out;  dS0 [B,H,m,dv] f32, out,
 *   nullable, may be dS_T (not S0)
 *   workspace: at least falcon_decay_attn_bwd_workspace_bytes(shape) bytes, 256-byte
 *   aligned. */
size_t falcon_decay_attn_bwd_workspace_bytes(const falcon_decay_shape *shape);
int falcon_decay_attn_bwd(const falcon_decay_shape *shape, const void *q,
                          const falcon_strides *q_strides, const void *k,
                          const falcon_strides *k_strides, const void *v,
                          const falcon_strides *v_strides, const float *log_decay,
                          const float *S0, const int32_t *lengths, const void *dO,
                          const falcon_strides *dO_strides, const float *dS_T, void *dq,
                          const falcon_strides *dq_strides, void *dk,
                          const falcon_strides *dk_strides, void *dv,
                          const falcon_strides *dv_strides, float *dS0, void *workspace,
                          size_t workspace_bytes, cudaStream_t stream);

/* One token of N sequences: q, k [N,H,m], v [N,H,dv] dtype (`batch` the row's stride,
 * `head` the head's), o [N,H,dv] dtype dense, out; S [pool,H,m,dv] f32, updated in
 * place.  The shape's B is N; its T is not read. */
int falcon_decay_attn_step(const falcon_decay_shape *shape, const void *q,
                           const falcon_strides *q_strides, const void *k,
                           const falcon_strides *k_strides, const void *v,
                           const falcon_strides *v_strides, const float *log_decay,
                           float *S, int64_t pool, const int32_t *slots,
                           const uint8_t *fresh, void *o, cudaStream_t stream);

#define FALCON_ACT_SIGMOID 2 /* a gate of the norm below */

/* B rows of T tokens with H heads of m channels (H*m at most 8192), each head
 * normalised by itself; gate is the activation of z (FALCON_ACT_*), eps > 0 the norms'
 * stabiliser. */
typedef struct {
  int64_t B, H, T;
  int32_t m, dtype, gate;
  float eps;
} falcon_norm_shape;

/* The norm behind a block, its gate, its scale and the residual, and the norm before
 * the next block, in one pass over the rows:
 *   out  = x + scale act(z) n(h) weight,   n(h) = h / sqrt(mean_head h^2 + eps)
 *   next = out / sqrt(mean out^2 + eps) next_weight
 * next is taken from out before its rounding.  Squares are summed in float32: where the
 * sum leaves its range (values from about 1e19 on) n, or next, and what the gradient
 * passes back through it are zero.  Where h is NULL, out = x is not
 * written, and next alone is the norm before the first block.
 *   h           [B,H,T,m] dtype, any strides (an attention's head-major output, or
 *               rows of channels: H = 1, or `head` = m)
 *   z, x, out, next  [B,T,H*m] dtype (`head` unused)
 *   weight, scale, next_weight  [H*m] f32
 * Nullable: weight, scale (ones), z (no gate), x (zeros), next_weight together with
 * next (no next norm); h together with out, weight, scale and z.
 *   out may be x (with x's strides).
 * No workspace.  Errors as for falcon_decay_attn_fwd; _BAD_ARG also for a gate code
 * or eps out of range, and _NULL_PTR for a pointer without its partner. */
int falcon_gated_norm_fwd(const falcon_norm_shape *shape, const void *h,
                          const falcon_strides *h_strides, const float *weight,
                          const void *z, const falcon_strides *z_strides,
                          const float *scale, const void *x,
                          const falcon_strides *x_strides, const float *next_weight,
                          const int32_t *lengths, void *out,
                          const falcon_strides *out_strides, void *next,
                          const falcon_strides *next_strides, cudaStream_t stream);

/* Gradients of <dout, out> + <dnext, next> of the call above.
 *   out    [B,T,H*m] dtype: the stored output (where h is NULL: x); given where
 *          next_weight is
 *   dout, dnext  [B,T,H*m] dtype; dout nullable (zeros) where dnext is given, dnext
 *          given where next_weight is
 *   dx     [B,T,H*m] dtype, out, nullable: the gradient of x, may be dout (with
 *          dout's strides)
 *   dh     [B,H,T,m] dtype, out, given where h is;  dz [B,T,H*m] dtype, out, given
 *          where z is
 *   dweight, dscale, dnext_weight  [H*m] f32, out, nullable; dscale only where scale
 *          is given, dnext_weight only where next_weight is
 *   workspace: at least falcon_gated_norm_bwd_workspace_bytes(shape) bytes, 16-byte
 *   aligned (per-block sums of the parameters' gradients, added in a fixed order). */
size_t falcon_gated_norm_bwd_workspace_bytes(const falcon_norm_shape *shape);
int falcon_gated_norm_bwd(const falcon_norm_shape *shape, const void *h,
                          const falcon_strides *h_strides, const float *weight,
                          const void *z, const falcon_strides *z_strides,
                          const float *scale, const void *out,
                          const falcon_strides *out_strides, const float *next_weight,
                          const int32_t *lengths, const void *dout,
                          const falcon_strides *dout_strides, const void *dnext,
                          const falcon_strides *dnext_strides, void *dx,
                          const falcon_strides *dx_strides, void *dh,
                          const falcon_strides *dh_strides, void *dz,
                          const falcon_strides *dz_strides, float *dweight,
                          float *dscale, float *dnext_weight, void *workspace,
                          size_t workspace_bytes, cudaStream_t stream);

/* Waits for `stream`, then reads and clears the library's device error word
 * (set by a kernel whose bounded wait ran out).  Returns FALCON_OK,
 * FALCON_ERR_TIMEOUT, or FALCON_ERR_CUDA if the stream itself failed.
 * The error word is one per device, not one per call: every call on the
 * device writes the same word, so with calls in flight on several streams a
 * timeout in any of them is reported to whichever caller reads the word
 * first (and cleared for the others).  Callers that need a per-call status
 * synchronise their streams one at a time. */
int falcon_sync_check(cudaStream_t stream);

/* Diagnostic of the failure path (no counterpart in the paper): launches a
 * kernel whose threads wait on a barrier that nothing completes.  The wait
 * gives up after limit_us microseconds (1 .. 10^7) and records the expiry in
 * the device error word, exactly as the chunked kernels do when a wait is
 * lost; nothing traps and the CUDA context stays usable.  A following
 * falcon_sync_check(stream) returns FALCON_ERR_TIMEOUT (and clears the word).
 * Returns FALCON_ERR_BAD_ARG for limit_us out of range. */
int falcon_selftest_wait_timeout(uint32_t limit_us, cudaStream_t stream);

/* Static description of a return code. */
const char *falcon_strerror(int code);

/* Library version, major*10000 + minor*100 + patch. */
int falcon_version(void);

#ifdef __cplusplus
}
#endif
#endif /* FALCON_GB300_H */
