/*
 * msm.h -- C ABI of the Momentum-Mamba selective scan for AMD Instinct MI355X (gfx950).
 *
 * The operation (Momentum Mamba README, "Momentum Mamba Recurrence"; its plain-Mamba special
 * case beta = 0, alpha = 1 is "Standard Mamba Recurrence" on the same page).  For every batch
 * row b, channel d and state n, starting from v = h = 0:
 *
 *     a_t = exp(delta[b,t,d] * A[d,n])                               (exact Abar, first-order Bbar:
 *     v_t = beta * v_{t-1} + alpha * delta[b,t,d] * B[b,t,n] * x[b,t,d]   "Discretization Note")
 *     h_t = a_t * h_{t-1} + v_t
 *     y[b,t,d] = sum_n C[b,t,n] * h_t  (+ Dskip[d] * x[b,t,d] when Dskip is given)
 *
 * B and C carry N values per position shared by all channels, delta one value per channel and
 * A one value per (channel, state) -- the selection layout of "Mamba: Choosing What to Remember
 * Based on the Input", section "From input features to update coefficients".  The skip term is
 * the per-channel D weight of the Mamba block ("Where the state computation sits in a Mamba
 * block" on the same page); alpha does not scale it.
 *
 * The backward returns the gradients of sum(dy * y) with respect to every input (README,
 * "Gradient Flow" / "Gradient Formulas"; the velocity adjoint also receives the hidden-state
 * adjoint because v_t enters h_t directly).  dB, dC sum over channels, dA over batch and time.
 *
 * Conventions for every entry point
 *   - All array pointers are DEVICE pointers to contiguous row-major buffers owned by the
 *     caller.  The library allocates no memory and keeps no mutable global state.
 *   - Shapes: x, delta, y, dy, dx, ddelta: (Bt, L, D).  A, dA: (D, N) fp32.
 *             B, C, dB, dC: (Bt, L, N).  Dskip, dDskip: (D,) fp32.  last_h, last_v: (Bt, D, N) fp32.
 *   - io selects the element type of x, delta, B, C, y, dy, dx, ddelta, dB, dC:
 *     MSM_F32 (IEEE binary32) or MSM_BF16 (bfloat16, outputs rounded to nearest even).
 *     A, Dskip, dA, dDskip, last_h, last_v are always fp32.  All arithmetic and every state
 *     is fp32 inside the kernels.  A is in natural-log units (the kernels rescale it to base 2).
 *   - stream is a hipStream_t (NULL = the null stream).  Work is enqueued asynchronously; the
 *     function returns once it is enqueued.
 *   - workspace is caller-owned device scratch of at least the size returned by the matching
 *     *_workspace_bytes query for the same shape and io (may be NULL when that size is 0).
 *     Its contents on entry do not matter and are undefined on exit.  Two calls in flight at
 *     the same time must not share a workspace.
 *   - Argument errors are detected before anything is enqueued and reported as a status; no
 *     exception crosses the ABI and nothing is printed.  A launch failure reported by the HIP
 *     runtime is returned as MSM_ERR_LAUNCH.  Non-finite inputs are not checked: NaN/Inf
 *     propagate to the outputs.
 */
#ifndef MSM_H_
#define MSM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MSM_OK = 0,
  MSM_ERR_INVALID_ARG = 1, /* null required pointer, bad size, beta outside [0,1), alpha not
                              finite or negative, an output overlapping an input */
  MSM_ERR_UNSUPPORTED = 2, /* valid by the method but outside this build (N > 64, io value) */
  MSM_ERR_WORKSPACE = 3,   /* workspace smaller than the query result */
  MSM_ERR_LAUNCH = 4       /* the HIP runtime rejected a kernel launch */
} msm_status;

typedef enum { MSM_F32 = 0, MSM_BF16 = 1 } msm_dtype;

/* Optional launch plan.  0 in a field means "choose automatically".
 *   states_per_wave : 1, 2, 4, 8 or 16 -- how many of the N states one lane keeps in registers.
 *                     N pads to 4, 16, 32 or 64 states.  Forward: a 64-lane wavefront serves
 *                     64 channels and a workgroup holds padded-N / states_per_wave wavefronts
 *                     (allowed: 1, 2, 4 at 4 states; 1-16 at 16; 4, 8 at 32; 4, 8, 16 at 64).
 *                     Backward: each 32-lane half of a wavefront holds states_per_wave states of
 *                     32 channels (allowed: 1, 2 at 4 states; 1, 2, 4 at 16; 2 at 32); at 64
 *                     states 2 runs two launches of 32 states and 4 the 64-channel kernel.
 *                     Other values return MSM_ERR_UNSUPPORTED.
 *   chunks          : number of time chunks the sequence is cut into (1..64, forward only);
 *                     chunks > 1 adds a pass that summarises each chunk as an affine map of its
 *                     start state.
 * A plan never changes results beyond fp32 rounding order. */
typedef struct {
  int32_t states_per_wave;
  int32_t chunks;
} msm_plan;

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int32_t msm_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char* msm_status_string(msm_status s);

/* Workspace sizes in bytes.  Valid for every plan the library may choose (automatic or
 * explicit).  Return 0 for invalid sizes. */
size_t msm_scan_fwd_workspace_bytes(int64_t Bt, int64_t L, int64_t D, int64_t N, msm_dtype io);
size_t msm_scan_bwd_workspace_bytes(int64_t Bt, int64_t L, int64_t D, int64_t N, msm_dtype io);

/* The plan msm_scan_fwd / msm_scan_bwd would use for this shape (written to *plan).  The fused
 * backward (msm_selective_scan_bwd with any extra) takes two states per wavefront half at 5-16
 * states instead.  At 64 states with D >= 2^23 the backward takes the 64-channel kernel (4). */
msm_status msm_scan_fwd_plan(int64_t Bt, int64_t L, int64_t D, int64_t N, msm_dtype io,
                             float beta, msm_plan* plan);
msm_status msm_scan_bwd_plan(int64_t Bt, int64_t L, int64_t D, int64_t N, msm_dtype io,
                             float beta, msm_plan* plan);

/* Forward scan.  y is overwritten.  last_h / last_v (the states after the final step) are
 * written when non-NULL.  Dskip may be NULL.  Requirements: Bt, L, D >= 1; 1 <= N <= 64;
 * 0 <= beta < 1; alpha finite and >= 0.  Outputs must not overlap any input. */
msm_status msm_scan_fwd(const void* x, const void* delta, const float* A, const void* B,
                        const void* C, const float* Dskip, void* y, float* last_h,
                        float* last_v, int64_t Bt, int64_t L, int64_t D, int64_t N, float beta,
                        float alpha, msm_dtype io, void* workspace, size_t workspace_bytes,
                        void* stream);

/* Forward scan with an explicit plan (NULL plan = automatic, identical to msm_scan_fwd). */
msm_status msm_scan_fwd_with_plan(const void* x, const void* delta, const float* A,
                                  const void* B, const void* C, const float* Dskip, void* y,
                                  float* last_h, float* last_v, int64_t Bt, int64_t L, int64_t D,
                                  int64_t N, float beta, float alpha, msm_dtype io,
                                  void* workspace, size_t workspace_bytes, void* stream,
                                  const msm_plan* plan);

/* Forward scan started at a given state: h0, v0 are (Bt, D, N) fp32, NULL meaning zero.  This
 * continues a sequence from the last_h / last_v a previous call returned for its first part
 * (the README's last_state outputs; chunked prefill and streaming).  The result equals one call
 * over the whole sequence up to rounding.  h0 and v0 must not overlap any output (continue
 * with a second pair of state buffers rather than in place).  plan may be NULL (automatic).
 * Everything else as msm_scan_fwd_with_plan, which is this call with h0 = v0 = NULL. */
msm_status msm_scan_fwd_state(const void* x, const void* delta, const float* A, const void* B,
                              const void* C, const float* Dskip, const float* h0,
                              const float* v0, void* y, float* last_h, float* last_v, int64_t Bt,
                              int64_t L, int64_t D, int64_t N, float beta, float alpha,
                              msm_dtype io, void* workspace, size_t workspace_bytes, void* stream,
                              const msm_plan* plan);

/* Allocation-free forward scan, for callers that cannot allocate device memory: code under HIP
 * graph capture, tight serving loops, harnesses that forbid hipMalloc.  Same arguments, checks
 * and results as msm_scan_fwd, without the workspace: the chunk summaries of a chunked plan
 * live in a static device array owned by the library, MSM_NOALLOC_SCRATCH_BYTES (32 MiB) per
 * GPU, held until the process ends.  The call allocates nothing (no hipMalloc, no library
 * allocation); the first call on a device looks up that device's copy of the array.  A shape
 * whose summaries exceed the array returns MSM_ERR_WORKSPACE before anything is enqueued (use
 * msm_scan_fwd with a workspace for it).  Every call on one GPU shares that GPU's array: two
 * calls in flight on one GPU at the same time (different streams, or host threads) race and
 * must be ordered by the caller.  Nothing in the array needs to start at zero: every summary is
 * written before it is read within the call. */
#define MSM_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
msm_status msm_scan_fwd_noalloc(const void* x, const void* delta, const float* A, const void* B,
                                const void* C, const float* Dskip, void* y, float* last_h,
                                float* last_v, int64_t Bt, int64_t L, int64_t D, int64_t N,
                                float beta, float alpha, msm_dtype io, void* stream);

/* Backward scan: gradients of sum(dy * y).  dx, ddelta, dB, dC, dA are overwritten (not
 * accumulated).  dDskip is required exactly when Dskip is non-NULL.  The forward is recomputed
 * inside; no saved activations are needed.  Same requirements as msm_scan_fwd, and L < 2^30
 * (a longer sequence returns MSM_ERR_UNSUPPORTED: split it with msm_scan_bwd_state) and
 * 64 * D * (element size) < 2^31 (D < 2^23 channels with fp32 I/O). */
msm_status msm_scan_bwd(const void* x, const void* delta, const float* A, const void* B,
                        const void* C, const float* Dskip, const void* dy, void* dx,
                        void* ddelta, float* dA, void* dB, void* dC, float* dDskip, int64_t Bt,
                        int64_t L, int64_t D, int64_t N, float beta, float alpha, msm_dtype io,
                        void* workspace, size_t workspace_bytes, void* stream);

msm_status msm_scan_bwd_with_plan(const void* x, const void* delta, const float* A,
                                  const void* B, const void* C, const float* Dskip,
                                  const void* dy, void* dx, void* ddelta, float* dA, void* dB,
                                  void* dC, float* dDskip, int64_t Bt, int64_t L, int64_t D,
                                  int64_t N, float beta, float alpha, msm_dtype io,
                                  void* workspace, size_t workspace_bytes, void* stream,
                                  const msm_plan* plan);

/* Backward of a scan started at (h0, v0) (NULL: zero), for the loss
 *   sum(dy * y) + <dlast_h, last_h> + <dlast_v, last_v>
 * (dlast_h, dlast_v: (Bt, D, N) fp32 adjoints of the final state, NULL meaning zero).  Besides
 * the gradients of msm_scan_bwd it writes the adjoints of the initial state, dh0 = a_0 gh_0 and
 * dv0 = beta gv_0 ((Bt, D, N) fp32), when dh0 / dv0 are non-NULL.  A sequence split in two is
 * differentiated by running the second part first and passing its dh0 / dv0 as the first
 * part's dlast_h / dlast_v (Momentum Mamba README, "Gradient Flow", read with the terminal
 * terms of a split sequence).  msm_scan_bwd_with_plan is this call with every state pointer
 * NULL. */
msm_status msm_scan_bwd_state(const void* x, const void* delta, const float* A, const void* B,
                              const void* C, const float* Dskip, const void* dy, const float* h0,
                              const float* v0, const float* dlast_h, const float* dlast_v,
                              void* dx, void* ddelta, float* dA, void* dB, void* dC,
                              float* dDskip, float* dh0, float* dv0, int64_t Bt, int64_t L,
                              int64_t D, int64_t N, float beta, float alpha, msm_dtype io,
                              void* workspace, size_t workspace_bytes, void* stream,
                              const msm_plan* plan);

/* The full selective-scan operation: the function of the Momentum Mamba README ("Low-Level
 * Functions": u, delta, A, B, C, D, z, delta_bias, delta_softplus, beta, alpha, with last
 * states) plus the initial state of msm_scan_fwd_state.  Read as in the Mamba block of
 * "Where the state computation sits in a Mamba block":
 *     delta_eff[b,t,d] = softplus(delta[b,t,d] + delta_bias[d])   when delta_softplus == 1
 *                      = delta[b,t,d] + delta_bias[d]             when delta_softplus == 0
 *     (softplus(u) = log(1 + e^u); a NULL delta_bias is zero),
 *     the scan of msm_scan_fwd_state runs on delta_eff, giving y_raw (skip term included),
 *     y = y_raw * silu(z)  with silu(z) = z / (1 + e^-z), when z (Bt, L, D, io dtype) is given.
 * delta_bias is (D,) fp32.  delta_softplus must be 0 or 1.
 * zero_order_hold (0 or 1) selects the write coefficient: 0 keeps the first-order delta of the
 * README's "Discretization Note"; 1 uses the zero-order hold Bbar = (exp(delta_eff A) - 1) A^{-1} B
 * of the glossary and complextorch pages ("The diagonal SSM"), i.e.
 *     v_t = beta v_{t-1} + alpha ((exp(delta_eff A) - 1) / A) B_t x_t   (delta_eff at A = 0).
 * With z, delta_bias NULL and delta_softplus = zero_order_hold = 0 this is msm_scan_fwd_state.
 * The bias, softplus and gate are applied inside the scan kernels (no extra pass over memory).  Everything else as msm_scan_fwd_state; z and
 * delta_bias are inputs and must not overlap an output. */
msm_status msm_selective_scan_fwd(const void* x, const void* delta, const float* A,
                                  const void* B, const void* C, const float* Dskip, const void* z,
                                  const float* delta_bias, int32_t delta_softplus,
                                  int32_t zero_order_hold, const float* h0, const float* v0,
                                  void* y, float* last_h,
                                  float* last_v, int64_t Bt, int64_t L, int64_t D, int64_t N,
                                  float beta, float alpha, msm_dtype io, void* workspace,
                                  size_t workspace_bytes, void* stream, const msm_plan* plan);

/* Backward of msm_selective_scan_fwd for the loss of msm_scan_bwd_state.  ddelta is the
 * gradient of the raw delta (through the bias and softplus); dz (Bt, L, D, io dtype) is
 * required exactly when z is given and ddelta_bias ((D,) fp32, summed over batch and time)
 * exactly when delta_bias is given.  The output before the gate, which dz needs, is recomputed
 * inside: nothing from the forward is saved.  zero_order_hold as in msm_selective_scan_fwd.
 * With z, delta_bias NULL and delta_softplus = zero_order_hold = 0 this is msm_scan_bwd_state. */
msm_status msm_selective_scan_bwd(const void* x, const void* delta, const float* A,
                                  const void* B, const void* C, const float* Dskip, const void* z,
                                  const float* delta_bias, int32_t delta_softplus,
                                  int32_t zero_order_hold, const void* dy,
                                  const float* h0, const float* v0, const float* dlast_h,
                                  const float* dlast_v, void* dx, void* ddelta, float* dA,
                                  void* dB, void* dC, float* dDskip, void* dz,
                                  float* ddelta_bias, float* dh0, float* dv0, int64_t Bt,
                                  int64_t L, int64_t D, int64_t N, float beta, float alpha,
                                  msm_dtype io, void* workspace, size_t workspace_bytes,
                                  void* stream, const msm_plan* plan);

/* Single-token decode step (the README's Mamba `step`: hidden_states of one position plus the
 * ssm_state and velocity_state caches, "Low-Level Functions" / `allocate_inference_cache`),
 * for the scan part of the block.  x, delta, z, y: (Bt, D) io dtype -- the token's input, raw
 * step size, gate and output; B, C: (Bt, N) io; A (D, N), Dskip (D,), delta_bias (D,) fp32;
 * h, v: (Bt, D, N) fp32 ssm and velocity states, read and overwritten IN PLACE with the states
 * after this token.  Computes, per (b, d, n), with delta_eff as in msm_selective_scan_fwd:
 *     v <- beta v + alpha delta_eff B x,  h <- exp(delta_eff A) h + v,
 *     y  = (sum_n C h + Dskip x) * silu(z)        (gate only when z is non-NULL)
 * which is msm_selective_scan_fwd over a sequence of length one started at (h, v), up to fp32
 * rounding.  Zero-initialised h, v start a new sequence; the last_h / last_v of a prefill call
 * continue one.  z, Dskip and delta_bias may be NULL; delta_softplus and zero_order_hold
 * (as in msm_selective_scan_fwd) are 0 or 1.  h and v must
 * not overlap each other, an input or y.  Needs no workspace.  Same requirements on Bt, D, N,
 * beta, alpha and io as msm_scan_fwd. */
msm_status msm_scan_step(const void* x, const void* delta, const float* A, const void* B,
                         const void* C, const float* Dskip, const void* z,
                         const float* delta_bias, int32_t delta_softplus,
                         int32_t zero_order_hold, float* h, float* v, void* y, int64_t Bt,
                         int64_t D, int64_t N, float beta, float alpha, msm_dtype io,
                         void* stream);

/* Complex-valued scan (Momentum Mamba README, "Complex Number Support": the same recurrence
 * with A, B and C complex; complextorch, "The diagonal SSM", for the complex diagonal state).
 * x, delta, y, dy, dx, ddelta are real (Bt, L, D) io arrays as above; for every (b, d, n):
 *     a_t = exp(delta[b,t,d] * A[d,n])                 (complex exponential)
 *     v_t = beta * v_{t-1} + alpha * delta[b,t,d] * x[b,t,d] * B[b,t,n]
 *     h_t = a_t * h_{t-1} + v_t
 *     y[b,t,d] = Re(sum_n C[b,t,n] * h_t)  (+ Dskip[d] * x[b,t,d])
 * Complex arrays are interleaved (re, im) pairs, i.e. an extra trailing dimension of 2:
 *   A, dA: (D, N, 2) fp32; B, C, dB, dC: (Bt, L, N, 2) in the io dtype (for MSM_F32 the memory
 *   of a complex64 array); h0, v0, last_h, last_v, dlast_h, dlast_v, dh0, dv0: (Bt, D, N, 2) fp32.
 * The real part of C h is the readout (a conjugate-pair convention, C h + conj(C h), would be
 * twice this).  h0, v0 (NULL = zero) start the scan; last_h, last_v (may be NULL) receive the
 * final state.  Requirements as msm_scan_fwd, L < 2^30 (else MSM_ERR_UNSUPPORTED), and
 * 17 * N * D * 8 < 2^31 (the kernels address 17 rows of the state history with 32-bit
 * offsets); B and C must be aligned to a whole complex
 * element (8 bytes for MSM_F32, 4 for MSM_BF16), else MSM_ERR_INVALID_ARG.
 * Needs no workspace. */
msm_status msm_scan_complex_fwd(const void* x, const void* delta, const float* A, const void* B,
                                const void* C, const float* Dskip, const float* h0,
                                const float* v0, void* y, float* last_h, float* last_v,
                                int64_t Bt, int64_t L, int64_t D, int64_t N, float beta,
                                float alpha, msm_dtype io, void* stream);

/* Workspace of msm_scan_complex_bwd: the state history Bt * (L + 1) * N * D * 8 bytes plus the
 * per-block partial sums.  Returns 0 for invalid sizes. */
size_t msm_scan_complex_bwd_workspace_bytes(int64_t Bt, int64_t L, int64_t D, int64_t N,
                                            msm_dtype io);

/* Backward of msm_scan_complex_fwd for the real loss
 *     sum(dy * y) + <dlast_h, last_h> + <dlast_v, last_v>,   <u, w> = Re sum conj(u) w
 * (dlast_h, dlast_v NULL = zero).  The gradient of a complex input is written as
 * dL/dRe + i dL/dIm (the convention of PyTorch's complex autograd for a real loss): dA (summed
 * over batch and time), dB, dC (summed over channels), and dh0, dv0 when non-NULL.  dx, ddelta
 * are real; dDskip is required exactly when Dskip is given.  A forward pass that records every
 * state into the workspace runs first; nothing from an earlier forward call is needed.  The
 * workspace must be 16-byte aligned (MSM_ERR_INVALID_ARG otherwise).
 * Everything else as msm_scan_complex_fwd. */
msm_status msm_scan_complex_bwd(const void* x, const void* delta, const float* A, const void* B,
                                const void* C, const float* Dskip, const float* h0,
                                const float* v0, const void* dy, const float* dlast_h,
                                const float* dlast_v, void* dx, void* ddelta, float* dA,
                                void* dB, void* dC, float* dDskip, float* dh0, float* dv0,
                                int64_t Bt, int64_t L, int64_t D, int64_t N, float beta,
                                float alpha, msm_dtype io, void* workspace,
                                size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------------------------
 * Operators of the block around the scan: the gated delta rule (a recurrence with a matrix
 * state, beside the scan's diagonal one), layer norm, and the norm and clipping of gradients.
 * The conventions above hold for them; parameters, gates, states and statistics are fp32, and
 * workspaces are 16-byte aligned (MSM_ERR_INVALID_ARG otherwise).
 * ------------------------------------------------------------------------------------------- */

/* Gated delta rule.  For every sequence and value head h, with a state S of K x V and the
 * query / key head h / (H / Hk):
 *     e_t = v_t - exp(g_t) S_{t-1}^T k_t          (what the decayed state gets wrong at k_t)
 *     S_t = exp(g_t) S_{t-1} + beta_t k_t e_t^T
 *     o_t = scale S_t^T q_t
 * q, k: (Bt, L, Hk, K), v, o: (Bt, L, H, V) in the io dtype; g (log decay, normally <= 0) and
 * beta: (Bt, L, H) fp32; S0, last_S: (Bt, H, K, V) fp32, S0 NULL meaning zero, last_S written
 * when non-NULL.
 * Packed sequences: with seq_offsets (device memory, Bt + 1 int32 values, not decreasing,
 * from 0 to L) the token arrays hold L rows in all, (L, Hk, K) and so on, and sequence b is
 * rows seq_offsets[b] ... seq_offsets[b+1] - 1; it may be empty, and then last_S = S0.
 * The offsets are read on the device: rows outside the arrays are never touched, whatever they
 * hold, but a token that no sequence covers leaves its output unwritten.
 * Requirements: Bt, L, Hk, H, K, V >= 1, H a multiple of Hk, K <= 256 and 64 rows of q or v (of
 * all heads) below 2^31 bytes (else MSM_ERR_UNSUPPORTED), V <= 2^20, H <= 65535, fewer than 2^31
 * tokens, scale finite; Bt H and the number of chunks (below) under 2^24, else MSM_ERR_UNSUPPORTED
 * (one token at a time has no such bound).  Outputs must not overlap an input.  All sums are
 * fp32; the products run on bf16 matrix cores over values cut into parts that keep 24 bits,
 * whatever the io type.
 * g of minus infinity forgets the state.  Tokens are taken in chunks of 64 (32 for fp32 with
 * K > 128) from a sequence's start: a NaN or an infinity in a token may reach earlier outputs of
 * its own chunk, and no other sequence. */
size_t msm_delta_rule_fwd_workspace_bytes(int64_t Bt, int64_t L, int64_t Hk, int64_t H, int64_t K,
                                          int64_t V, int32_t packed, msm_dtype io);
msm_status msm_delta_rule_fwd(const void* q, const void* k, const void* v, const float* g,
                              const float* beta, const int32_t* seq_offsets, const float* S0,
                              void* o, float* last_S, int64_t Bt, int64_t L, int64_t Hk, int64_t H,
                              int64_t K, int64_t V, float scale, msm_dtype io, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Gradients of sum(do o) + <dlast_S, last_S> (dlast_S NULL: zero): dq, dk, dv in the io dtype
 * (dq and dk summed over the value heads that share a key head), dg, dbeta fp32, dS0 fp32 when
 * non-NULL.  The forward is recomputed inside; nothing of it is saved.  The workspace holds two
 * states per chunk of 64 tokens.  Everything else as msm_delta_rule_fwd. */
size_t msm_delta_rule_bwd_workspace_bytes(int64_t Bt, int64_t L, int64_t Hk, int64_t H, int64_t K,
                                          int64_t V, int32_t packed, msm_dtype io);
msm_status msm_delta_rule_bwd(const void* q, const void* k, const void* v, const float* g,
                              const float* beta, const int32_t* seq_offsets, const float* S0,
                              const void* do_, const float* dlast_S, void* dq, void* dk, void* dv,
                              float* dg, float* dbeta, float* dS0, int64_t Bt, int64_t L,
                              int64_t Hk, int64_t H, int64_t K, int64_t V, float scale,
                              msm_dtype io, void* workspace, size_t workspace_bytes,
                              void* stream);

/* One token of the gated delta rule for Bt sequences: q, k (Bt, Hk, K), v, o (Bt, H, V) io;
 * g, beta (Bt, H) fp32; S (Bt, H, K, V) fp32, read and overwritten IN PLACE.  Needs no
 * workspace.  S must not overlap anything else. */
msm_status msm_delta_rule_step(const void* q, const void* k, const void* v, const float* g,
                               const float* beta, float* S, void* o, int64_t Bt, int64_t Hk,
                               int64_t H, int64_t K, int64_t V, float scale, msm_dtype io,
                               void* stream);

/* Layer norm over the last dimension of x (rows, D):
 *     y = (x - mean) rstd weight + bias,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
 * x, y io dtype; weight, bias (D,) fp32, NULL meaning ones and zeros; mean, rstd (rows,) fp32,
 * written when non-NULL.  1 <= rows < 2^31, 1 <= D <= 2^30, eps >= 0 and finite.  y must not
 * overlap x. */
msm_status msm_layer_norm_fwd(const void* x, const float* weight, const float* bias, void* y,
                              float* mean, float* rstd, int64_t rows, int64_t D, float eps,
                              msm_dtype io, void* stream);

/* Gradients of sum(dy y) from the forward's mean and rstd: dx (rows, D) io; dweight, dbias (D,)
 * fp32, each written when non-NULL (the workspace may be NULL when both are). */
size_t msm_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t D, msm_dtype io);
msm_status msm_layer_norm_bwd(const void* x, const float* weight, const void* dy,
                              const float* mean, const float* rstd, void* dx, float* dweight,
                              float* dbias, int64_t rows, int64_t D, msm_dtype io,
                              void* workspace, size_t workspace_bytes, void* stream);

/* Global 2-norm over count tensors: grads[i] points to numel[i] contiguous elements of dtype
 * dtypes[i] (MSM_F32 or MSM_BF16, mixed freely; numel[i] may be 0).  The three arrays are HOST
 * memory, read during the call only.  norm: one fp32 value on the device.  count may be 0.
 * Neither norm nor the workspace may overlap a tensor or each other (MSM_ERR_INVALID_ARG; gradients
 * may share memory here). */
size_t msm_grad_norm_workspace_bytes(int64_t count);
msm_status msm_grad_norm(const void* const* grads, const int64_t* numel, const int32_t* dtypes,
                         int64_t count, float* norm, void* workspace, size_t workspace_bytes,
                         void* stream);

/* Clipping by the global norm: out[i] = grads[i] * min(1, max_norm / (norm + eps)); norm
 * receives the norm before clipping.  out NULL, or out[i] == grads[i], scales in place (and
 * writes nothing when the factor is 1).  What is written (an out[i], a gradient scaled in place,
 * norm, the workspace) must not overlap anything else of the call, so a gradient is not scaled in
 * place twice (MSM_ERR_INVALID_ARG; MSM_ERR_WORKSPACE if the host has no memory for the check of a
 * long list).  A norm that is NaN makes every gradient NaN; an infinite norm scales by 0.
 * max_norm >= 0, eps >= 0.
 * Workspace as msm_grad_norm. */
msm_status msm_grad_clip(const void* const* grads, void* const* out, const int64_t* numel,
                         const int32_t* dtypes, int64_t count, float max_norm, float eps,
                         float* norm, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------------------------
 * Operators at a language model's ends and between its blocks: token embedding, the norms around
 * a block with its gate and residual scale, cross entropy over a vocabulary.  The conventions
 * above hold for them; arrays may begin at any address that is a multiple of their element's size.
 * ------------------------------------------------------------------------------------------- */

/* Token embedding: y[t] = scale * table[ids[t]], ids (tokens,) int64, table (V, D) in table_io,
 * y (tokens, D) in io (any combination of the two types).  An id outside [0, V) gives a row of
 * zeros.  1 <= tokens < 2^31, 1 <= V < 2^31 - 1, 1 <= D <= 2^24, tokens D and V D <= 2^48, scale
 * finite. */
msm_status msm_embed_fwd(const int64_t* ids, const void* table, void* y, int64_t tokens, int64_t V,
                         int64_t D, float scale, msm_dtype table_io, msm_dtype io, void* stream);

/* Gradient of the table: dtable[v] = scale * sum of dy[t] over {t: ids[t] = v}, every row written
 * (zeros for a row without a token).  Ids outside [0, V) take no part.  Tokens are sorted by id and
 * added in the order of the batch: no atomics, the same result every time.  Sizes as above. */
size_t msm_embed_bwd_workspace_bytes(int64_t tokens, int64_t V, int64_t D);
msm_status msm_embed_bwd(const int64_t* ids, const void* dy, void* dtable, int64_t tokens,
                         int64_t V, int64_t D, float scale, msm_dtype table_io, msm_dtype io,
                         void* workspace, size_t workspace_bytes, void* stream);

/* The norms after a block and before the next one, with the block's gate and residual scale, on
 * rows of D elements; RMS(x) = x / sqrt(mean(x^2) + eps):
 *     r_out = r + scale * post_weight * RMS(o) * silu(z)     (rounded to the io type)
 *     y     = weight * RMS(r_out)
 * r (the residual stream), o (the block's output), z (its gate), r_out, y: (rows, D) io; weight,
 * post_weight: (D,) fp32, NULL meaning ones; rstd, post_rstd: (rows,) fp32, the reciprocal roots of
 * the two norms, written when non-NULL.  z NULL: no gate.  o NULL: y = weight * RMS(r) alone, and
 * post_weight, z, r_out and post_rstd are NULL.  r_out may be r itself (the stream is updated in
 * place); no other overlap.  The sum of a row's squares, of o and of r_out, has to stay below 2^128, and
 * with eps = 0 above 2^-126.  1 <= rows < 2^31, 1 <= D <= 2^30, rows D <= 2^50, scale finite, eps >= 0
 * and finite. */
msm_status msm_block_norm_fwd(const void* r, const float* weight, const void* o,
                              const float* post_weight, const void* z, void* r_out, void* y,
                              float* rstd, float* post_rstd, int64_t rows, int64_t D, float scale,
                              float eps, msm_dtype io, void* stream);

/* Gradients of sum(dy * y) + sum(dr_out * r_out) (dr_out NULL: zero) from the forward's r_out and
 * statistics: dr (also r_out's own) and, with o, do in the io type; dz in it exactly when z is given;
 * dweight and dpost_weight (D,) fp32, each written when non-NULL.  Without o: r_out is r, and do, dz,
 * dpost_weight and the block's inputs are NULL.  Sizes as above. */
size_t msm_block_norm_bwd_workspace_bytes(int64_t rows, int64_t D, msm_dtype io);
msm_status msm_block_norm_bwd(const void* r_out, const void* dy, const float* rstd,
                              const float* weight, const void* o, const float* post_rstd,
                              const float* post_weight, const void* z, const void* dr_out, void* dr,
                              void* do_, void* dz, float* dweight, float* dpost_weight,
                              int64_t rows, int64_t D, float scale, msm_dtype io, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Cross entropy of a linear layer over a vocabulary, without its logits in memory:
 *     l[t][v] = scale * x[t] . weight[v],  lse[t] = log sum_v exp(l[t][v]),
 *     loss[t] = lse[t] - l[t][targets[t]]
 * x (T, D), weight (V, D) io; targets (T,) int64; loss, lse (T,) fp32, lse may be NULL.  A row whose
 * target lies outside [0, V) is left out: its loss and lse are 0, whatever it holds (the other rows'
 * results do not depend on it).  Logits, sums and statistics are fp32; fp32 inputs are multiplied in
 * three bf16 parts that keep 24 bits (an infinite one gives NaN).  A logit of plus infinity makes lse
 * infinite, and the loss too, or NaN if it is the target's.
 * Requirements: T, V, D >= 1; T and V <= 2^22, T V <= 2^37, D <= 2^16 (else MSM_ERR_UNSUPPORTED);
 * scale finite.
 * bf16 weights with D a multiple of 8 that begin at a multiple of 16 bytes are read where they are;
 * others are copied a piece at a time into the workspace. */
size_t msm_linear_cross_entropy_fwd_workspace_bytes(int64_t T, int64_t V, int64_t D, msm_dtype io);
msm_status msm_linear_cross_entropy_fwd(const void* x, const void* weight, const int64_t* targets,
                                        float* loss, float* lse, int64_t T, int64_t V, int64_t D,
                                        float scale, msm_dtype io, void* workspace,
                                        size_t workspace_bytes, void* stream);

/* Gradients of sum(dloss * loss) + sum(dlse * lse) (dlse NULL: zero) from the forward's lse:
 *     g[t][v] = scale * ((dloss[t] + dlse[t]) exp(l[t][v] - lse[t]) - dloss[t] [v = targets[t]])
 *     dx = g weight,  dweight = g^T x
 * dx (T, D), dweight (V, D) io; dweight may be NULL.  A row that is left out has dx = 0 and adds
 * nothing to dweight.  The vocabulary is taken in pieces, whose g (in bf16 for bf16 inputs, where what
 * the target's entry loses by that is made up for in both gradients; 24 bits for fp32 ones) is in the
 * workspace; sums are fp32. */
size_t msm_linear_cross_entropy_bwd_workspace_bytes(int64_t T, int64_t V, int64_t D, msm_dtype io);
msm_status msm_linear_cross_entropy_bwd(const void* x, const void* weight, const int64_t* targets,
                                        const float* lse, const float* dloss, const float* dlse,
                                        void* dx, void* dweight, int64_t T, int64_t V, int64_t D,
                                        float scale, msm_dtype io, void* workspace,
                                        size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MSM_H_ */
