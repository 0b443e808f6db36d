/*
 * bcjr.h -- C ABI of the B200 (sm_100a) BCJR forward-backward library.
 *
 * The operations follow "BCJR-QAT: A Differentiable Relaxation of
 * Trellis-Coded Weight Quantization":
 *   - Abstract: the hard Viterbi argmax of trellis-coded quantisation is
 *     replaced by the BCJR forward-backward sum-product at temperature T; the
 *     result is a soft codeword equal to the Boltzmann expectation over trellis
 *     paths, exactly differentiable, and equal to the hard code as T -> 0; the
 *     computation is the transfer-matrix computation of a 1D Ising-like chain.
 *   - Technical Summary, "Core Mechanism": the soft codeword
 *       w_hat_t(T) = sum_s c(s) p_T(s_t = s | w),
 *     differentiable in the weights and in the trellis parameters (codebook).
 *   - Technical Summary, "Key Technical Innovations": exact gradients through
 *     the forward-backward recursion; a fused kernel of gather, log-sum-exp and
 *     addition.
 *
 * Trellis and energy (the pages leave them open; these are the readings used):
 *   states s in [0, 2^L); D = k*V bits enter per step at the bottom:
 *   succ(p, b) = ((p << D) & (2^L - 1)) | b, b in [0, 2^D);
 *   step t (0 <= t < n, n = len / V) reads weights w[t*V .. t*V+V-1];
 *   E_t(s) = sum_v (w[t*V+v] - c[s][v])^2; a path has weight exp(-sum_t E_t/T);
 *   free start (every state has weight 1 at t = 0) and free end.
 *
 * Conventions for every entry point:
 *   - All array arguments are DEVICE pointers (cudaMalloc'd or managed memory)
 *     to contiguous row-major fp32 / int32 data, 4-byte aligned.  The caller
 *     owns every buffer; the library never frees or retains them.
 *   - `len` counts weights per sequence and must be a positive multiple of V.
 *   - `codebook` is [2^L][V] fp32.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default
 *     stream).  Calls are asynchronous: they validate their arguments, enqueue
 *     the work on `stream` and return.  Argument errors are returned at once and
 *     enqueue nothing.  The library allocates its own scratch space, stream-
 *     ordered on `stream`, from a library-private memory pool of the current
 *     device and frees it on `stream` before returning; freed scratch stays
 *     mapped in that pool for reuse by later calls (up to the largest call's
 *     size, several GB for L=16, until the process exits).  No data is kept
 *     between calls.
 *   - Supported: 1 <= D = k*V <= L <= 16, D <= 6, V in {1, 2, 4},
 *     len <= 8192; T finite and > 0.  n_seq == 0 is a no-op returning BCJR_OK.
 *   - Errors: null or non-device pointers, len not a positive multiple of V,
 *     k < 1, V < 1, D > L, T not finite or <= 0  -> BCJR_ERR_INVALID_ARG;
 *     L > 16, D > 6, V not in {1,2,4}, len > 8192 -> BCJR_ERR_UNSUPPORTED;
 *     a failed CUDA call (allocation, launch)   -> BCJR_ERR_CUDA.
 *   - NaN or infinite weights make that sequence's outputs NaN; other
 *     sequences are unaffected.  The soft-codeword and VJP kernels also check
 *     that the posterior of every step sums to 1 within 1e-2 and, if not (NaN
 *     or infinite inputs, or a numerical breakdown), record BCJR_ERR_NUMERIC
 *     for bcjr_get_device_error.
 */
#ifndef BCJR_H_
#define BCJR_H_

#include <stdint.h>

#if defined(__GNUC__)
#define BCJR_API __attribute__((visibility("default")))
#else
#define BCJR_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  BCJR_OK = 0,
  BCJR_ERR_INVALID_ARG = 1,
  BCJR_ERR_UNSUPPORTED = 2,
  BCJR_ERR_CUDA = 3,
  BCJR_ERR_TIMEOUT = 4,  /* recorded on the device: a bounded wait ran out */
  BCJR_ERR_NUMERIC = 5   /* recorded on the device: a step's posterior mass was off */
} bcjr_status;

/*
 * Soft codeword and log-partition function (Abstract; "Core Mechanism").
 *   w         [n_seq][len]  weights (input)
 *   codebook  [2^L][V]      codewords c(s) (input)
 *   T                       temperature
 *   out_soft  [n_seq][len]  w_hat: out_soft[q][t*V+v] = sum_s c(s)[v] p_t(s)
 *   out_logZ  [n_seq]       natural log of Z = sum over paths of exp(-E/T);
 *                           may be NULL
 */
BCJR_API int bcjr_soft_codeword(const float* w, int64_t n_seq, int64_t len, int L, int k, int V,
                       const float* codebook, float T, float* out_soft, float* out_logZ, void* stream);

/*
 * Vector-Jacobian product of  l = sum_{q,t,v} grad_soft[q][t*V+v] * w_hat[q][t*V+v]
 *                               + sum_q grad_logZ[q] * logZ[q]
 * with respect to the weights and the codebook ("Core Mechanism": exactly
 * differentiable with respect to the weight pre-image and the trellis
 * parameters; "Key Technical Innovations": exact gradients).
 *   grad_soft     [n_seq][len]  upstream gradient on out_soft (input)
 *   grad_logZ     [n_seq]       upstream gradient on out_logZ, or NULL (= 0)
 *   grad_w        [n_seq][len]  dl/dw (output, overwritten)
 *   grad_codebook [2^L][V]      dl/dc summed over all sequences and steps
 *                               (output, overwritten, not accumulated)
 */
BCJR_API int bcjr_vjp(const float* w, int64_t n_seq, int64_t len, int L, int k, int V, const float* codebook,
             float T, const float* grad_soft, const float* grad_logZ, float* grad_w,
             float* grad_codebook, void* stream);

/*
 * Viterbi decode, the T -> 0 limit of the soft codeword (Abstract: "recovering
 * the hard QTIP code as T -> 0").  Min-sum over paths in fp32 with this exact
 * operation order (no fused multiply-add):
 *   q_t(s) = sum over v, in order, of fl(fl(w - c(s)[v])^2);
 *   delta_0(s) = q_0(s);  delta_t(s) = fl(min_{p -> s} delta_{t-1}(p) + q_t(s)).
 * Ties go to the lowest predecessor and, for the final state, the lowest index.
 *   out_states [n_seq][n] int32   decoded state s_t of every step
 *   out_cost   [n_seq] fp32       delta_{n-1}(s_{n-1}), or NULL
 * T plays no part.
 */
BCJR_API int viterbi_decode(const float* w, int64_t n_seq, int64_t len, int L, int k, int V, const float* codebook,
                   int32_t* out_states, float* out_cost, void* stream);

/*
 * Per-step argmax of the posterior p_T(s_t = s | w) ("Core Mechanism"), ties to
 * the lowest state (compared in fp32).
 *   out_argmax [n_seq][n] int32
 */
BCJR_API int bcjr_posterior_argmax(const float* w, int64_t n_seq, int64_t len, int L, int k, int V,
                          const float* codebook, float T, int32_t* out_argmax, void* stream);

/*
 * bcjr_soft_codeword_noalloc -- bcjr_soft_codeword without any allocation.
 * The paper has no counterpart to this entry point; it is an interface
 * variant for callers that must not allocate device memory: for example a
 * plugin inside an application or framework that owns every device
 * allocation, a service whose device-memory budget is fixed at start-up, or a
 * latency-critical path where an allocation could block or fail under memory
 * pressure.
 *
 * Arguments, layouts and errors are those of bcjr_soft_codeword, and so are
 * the results up to rounding: this entry point always runs the general sweep
 * kernel, also where bcjr_soft_codeword runs a specialised one (L = 16 with
 * k*V = 2 or 4), so the two agree within the soft-codeword and logZ
 * tolerances (1e-5 of max|c| and of max(|logZ|, (L + D(n-1)) ln 2)), not bit
 * for bit.
 * The call makes no cudaMalloc, cudaMallocAsync or cudaFree call and uses no
 * allocating library routine.  Its scratch space is one fixed array of
 * BCJR_NOALLOC_SCRATCH_BYTES (64 MiB) in this library's device memory; every
 * GPU that loads the library reserves it until the process exits.
 *
 * Limit: the array must hold the scaled codebook (2^L * V floats) plus the
 * history of one sequence ((len/V) * 2^(L-D) floats and (len/V) doubles, plus
 * 4 * 2^(L-D) floats when the per-sequence state does not fit in shared
 * memory).  Larger problems return BCJR_ERR_UNSUPPORTED and enqueue nothing.
 * When the array holds fewer histories than the GPU can run at once, fewer
 * sequences run concurrently: slower, same results.
 *
 * Set-up: the first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current) and keeps it for the rest
 * of the process; make that first call before any stream capture on the
 * device.  A cudaDeviceReset (or any other way of unloading the library's
 * module from the device) makes the kept address stale: do not call this entry
 * point on a device after resetting it.
 *
 * Sharing: all calls on a device use the same array, which keeps whatever the
 * last call left in it (nothing in it needs to start at zero).  Calls whose
 * GPU work overlaps -- issued on different streams, or from several host
 * threads without ordering -- race on the array and corrupt each other's
 * results; order them, e.g. on one stream.
 */
#define BCJR_NOALLOC_SCRATCH_BYTES (64u << 20)
BCJR_API int bcjr_soft_codeword_noalloc(const float* w, int64_t n_seq, int64_t len, int L, int k, int V,
                                        const float* codebook, float T, float* out_soft, float* out_logZ,
                                        void* stream);

/*
 * One step of quantisation-aware training by self-reconstruction (BCJR-QAT,
 * Technical Summary "Core Mechanism": the soft codeword of the latent weights
 * stands in for the quantised weights, and T is annealed from T0 towards a
 * near-zero T_end over the steps, one call per step with its own T).  With
 * w_hat the soft codeword of w at temperature T,
 *   loss[q] = sum_{t,v} (w_hat[q][t*V+v] - w_target[q][t*V+v])^2,
 * the call computes w_hat and the loss, the VJP of sum_q loss[q] (upstream
 * gradient 2 (w_hat - w_target), no gradient on logZ), and then updates in place
 *   w        <- w        - lr_w * dl/dw
 *   codebook <- codebook - lr_c * dl/dc      (only when lr_c != 0)
 *   w             [n_seq][len]  latent weights (input; updated in place)
 *   w_target      [n_seq][len]  target weights (input)
 *   codebook      [2^L][V]      codewords (input; updated in place when lr_c != 0)
 *   out_soft      [n_seq][len]  w_hat before the update (output)
 *   out_loss      [n_seq]       loss per sequence before the update (output, may be NULL)
 *   grad_w        [n_seq][len]  dl/dw (output)
 *   grad_codebook [2^L][V]      dl/dc (output)
 * All device pointers; w, w_target, out_soft and grad_w must not overlap.
 * lr_w and lr_c must be finite (BCJR_ERR_INVALID_ARG otherwise).  Every step
 * runs in the library's kernels on `stream`; the upstream gradient lives in
 * library scratch.
 */
BCJR_API int bcjr_qat_step(float* w, const float* w_target, int64_t n_seq, int64_t len, int L, int k, int V,
                           float* codebook, float T, float lr_w, float lr_c, float* out_soft, float* out_loss,
                           float* grad_w, float* grad_codebook, void* stream);

/*
 * Layer-wise quantisation-aware training.
 *
 * The loss of a layer is the change of its outputs, ||X (W_hat - W*)^T||^2 for
 * activations X ("Experimental Results": per-layer reconstruction MSE).  Its
 * products run on 8-bit operands (bcjr_fp8_quantise, bcjr_fp8_matmul), its
 * gradient goes through bcjr_vjp to the latent weights, and bcjr_muon_step
 * updates them as matrices (bcjr_orthogonalise is its orthogonalisation alone).
 *
 * Matrices are row-major with a row stride `ld` in elements, at least the
 * number of columns; what lies behind a row's columns is neither read nor
 * written.  Every pointer must belong to the current device (or be managed)
 * and be aligned to its element type, 8-bit codes to 16 bytes with a row stride
 * that is a multiple of 16; otherwise BCJR_ERR_INVALID_ARG.  Outputs must not
 * overlap inputs or one another, except that a weight, momentum or gradient
 * updated in place is itself.  Calls may be captured into a CUDA graph.
 */
typedef enum {
  BCJR_F32 = 0,
  BCJR_F16 = 1,
  BCJR_BF16 = 2,
  BCJR_E4M3 = 3,   /* 8-bit: 4 exponent bits, largest value 448, no infinities */
  BCJR_E5M2 = 4    /* 8-bit: 5 exponent bits, largest value 57344 */
} bcjr_dtype;

/*
 * 8-bit codes with one power-of-two scale for each block of 128 values of a
 * row (block_rows = 1) or of 128 rows x 128 columns (block_rows = 128).  With
 * v = x, or x - minus in fp32, and FMAX = 448 or 57344,
 *   scale = 2^e, e the least integer >= -127 with max |v| <= FMAX 2^e over the
 *           block (e = 0 for a block of zeros),
 *   q     = v / scale rounded to the nearest 8-bit value, ties to even,
 * so that q * scale stands for v.  The scale is stored as the byte e + 127 (the
 * E8M0 type).  A block that holds a NaN or an infinity gets the scale NaN (255)
 * and NaN codes.  The codes of v^T (blocks of 128 values of its rows, i.e. down
 * the columns of x) come from the same pass over x.
 *   x       [rows][cols]  fp32, fp16 or bf16 (input)
 *   minus   [rows][cols]  fp32, or NULL (input)
 *   q       [rows][cols], scale   [ceil(rows / block_rows)][ceil(cols / 128)]
 *   qt      [cols][rows], scale_t [ceil(cols / block_rows)][ceil(rows / 128)]
 * q and scale, or qt and scale_t, may be NULL (not both pairs).  rows or cols
 * of 0 is a no-op.
 */
BCJR_API int bcjr_fp8_quantise(const void* x, int x_type, int64_t rows, int64_t cols, int64_t ld_x,
                               const float* minus, int64_t ld_minus, int q_type, int block_rows, void* q,
                               int64_t ld_q, void* scale, int64_t ld_scale, void* qt, int64_t ld_qt,
                               void* scale_t, int64_t ld_scale_t, void* stream);

/*
 * Product of two matrices of 8-bit codes with block scales, summed in fp32:
 *   out[m][n] = alpha sum_k (a[m][k] scale_a[m / a_block_rows][k / 128])
 *                         * (b[n][k] scale_b[n / b_block_rows][k / 128]).
 * With the codes of activations X and weights W that is X W^T; with those of W
 * transposed it is the gradient dY W, with those of dY and X transposed the
 * gradient dY^T X.
 *   a    [M][K], b [N][K]  e4m3 or e5m2, each of its own type (input)
 *   out  [M][N]            fp32, fp16 or bf16 (output), rounded once
 * M or N of 0 is a no-op, K of 0 gives zeros.  A NaN code or scale makes the
 * entries of out that it enters NaN.  Results are the same bits run to run.
 */
BCJR_API int bcjr_fp8_matmul(const void* a, int a_type, int64_t ld_a, const void* scale_a, int64_t ld_scale_a,
                             int a_block_rows, const void* b, int b_type, int64_t ld_b, const void* scale_b,
                             int64_t ld_scale_b, int b_block_rows, int64_t M, int64_t N, int64_t K, float alpha,
                             void* out, int out_type, int64_t ld_out, void* stream);

/*
 * Orthogonalisation of an update by Newton-Schulz products (as in Muon): with
 * X_0 = G / (||G||_F + eps) and, for each of `steps` steps and its coefficients
 * (a, b, c), X <- a X + (b A + c A^2) X where A = X X^T (X^T X from the right
 * when rows > cols), out is the last X: G with its singular values moved
 * towards 1.  Products sum in fp32.  Their operands, the iterates and Gram
 * matrices, are fp16 scaled by 2^12 (11 bits) and, where it counts, what that
 * rounding left as a second such value (22 bits).  For a bf16 out these are the
 * iterates that are multiplied (but the last, which 11 bits hold well enough) and
 * the diagonals, which keeps out within about 1e-3 of the exact iteration in the
 * 2-norm (2e-3 at most in Muon's five steps), less than its own rounding, whatever
 * the singular values of G (fewer than 32 rows or columns: 22 bits throughout); for
 * an fp16 out all of them (three times the products), which leaves 1e-4
 * before it is rounded, or where few directions carry G what the fp32 sums leave
 * in the others and the steps amplify: 2e-4 (512 x 512) to 1.1e-3 (2048 x 2048).
 *   g       [batch][rows][cols]  fp32, fp16 or bf16 (input)
 *   coeffs  [steps][3]           HOST pointer, read during the call, or NULL
 *                                for Muon's (3.4445, -4.7750, 2.0315)
 *   out     [batch][rows][cols]  fp16 or bf16 (output)
 * batch <= 32767, rows, cols <= 65536, 1 <= steps <= 64, eps >= 0.  Coefficients that drive a
 * singular value of [0, 1] above 2 are BCJR_ERR_INVALID_ARG.  A matrix of zeros
 * gives zeros (eps > 0); NaN or infinities make that matrix NaN.  Entries of X_0
 * below 2^-36 vanish (so does a G whose norm is that far below eps).  Steps amplify
 * the directions whose singular values are small against ||G||_F (Muon's default:
 * 3.4 times each, five of them 485 times), and with them what is there of roundings:
 * of G itself, if it is bf16, and of 22 bits, so that with more than about ten
 * such steps the directions that G does not have are no longer small.
 */
BCJR_API int bcjr_orthogonalise(const void* g, int g_type, int64_t batch, int64_t rows, int64_t cols, int64_t ld_g,
                                int64_t batch_stride_g, int steps, const float* coeffs, float eps, void* out,
                                int out_type, int64_t ld_out, int64_t batch_stride_out, void* stream);

/*
 * One Muon step on a matrix of latent weights, all in place:
 *   momentum <- mu momentum + grad
 *   u         = grad + mu momentum (nesterov != 0), or momentum
 *   w        <- (1 - lr weight_decay) w - lr scale orthogonalise(u)
 *   w, momentum  [rows][cols] fp32 (updated), grad [rows][cols] fp32, fp16 or bf16
 * steps, coeffs and eps as in bcjr_orthogonalise, operands as for its bf16
 * output (the orthogonalised update is as near as that before it is rounded); lr, mu,
 * weight_decay and scale finite.
 */
BCJR_API int bcjr_muon_step(float* w, int64_t ld_w, const void* grad, int grad_type, int64_t ld_grad,
                            float* momentum, int64_t ld_momentum, int64_t rows, int64_t cols, float lr, float mu,
                            int nesterov, float weight_decay, float scale, int steps, const float* coeffs,
                            float eps, void* stream);

/*
 * Synchronises `stream` and returns BCJR_OK, or BCJR_ERR_CUDA if the stream
 * holds a CUDA error, or the first device-side error recorded by a kernel of
 * this library since the last call (BCJR_ERR_NUMERIC: a step's posterior mass
 * left 1 +- 1e-2 or was not finite; BCJR_ERR_TIMEOUT: a wait of the L=16 V=1
 * VJP for a bulk copy into its shared-memory codeword ring did not end within
 * 1 s, after which that CTA computes on without the ring and its sequences'
 * outputs are not usable; or a wait of a matrix product for its copies or sums,
 * after which that tile, and those that its blocks would have taken next, are not
 * written: incomplete sums never are).  The flag is one per device and process, shared by
 * all streams; reading it clears it.
 */
BCJR_API int bcjr_get_device_error(void* stream);

/* Number of kernels this library has launched in this process, on all devices
 * and streams (launches issued, counted on the host; a call that fails before
 * launching adds nothing).  For accounting, e.g. the launches of a timed region. */
BCJR_API uint64_t bcjr_launch_count(void);

/* Static string for a status code. */
BCJR_API const char* bcjr_strerror(int status);

/* Library version, e.g. "0.1.0". */
BCJR_API const char* bcjr_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BCJR_H_ */
