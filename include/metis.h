/*
 * metis.h -- C ABI of the MI355X (gfx950) Metis spectral-split NVFP4 GEMM.
 *
 * The method is described on the web page "Metis: Training LLMs with FP4
 * Quantization" (ICLR 2026 reading notes):
 *   - section 关键设计 1: every GEMM operand M (weight W, activation X, output
 *     gradient D) is split as M = U_k S_k V_k^T + M_R; the factors and the
 *     residual are quantised, the singular values stay in high precision, and
 *     the forward GEMM is
 *       Y = (Q(A_k) L_k Q(B_k^T) + Q(X_R)) (Q(U_k) S_k Q(V_k^T) + Q(W_R));
 *   - section 关键设计 2: the dominant subspace is estimated from a sparse
 *     random row sample and a Gaussian random projection (randomized SVD);
 *   - section 关键设计 3: the factors are reused across steps (refresh every 8);
 *   - section 研究背景与动机: NVFP4 = E2M1 values in blocks of 16 with one FP8
 *     (here E4M3) scale per block; section 损失函数/训练策略: W4A4G4 with
 *     stochastic rounding, rank 1.5%.
 *
 * Conventions shared by every entry point
 *   Memory.  Every pointer argument except the metis_* descriptor structs and
 *     the host-only self-test helpers is DEVICE memory owned by the caller.
 *     The library allocates no device memory in these calls; scratch space is
 *     the caller's workspace (size from the *_workspace functions, 256-byte
 *     aligned).  Buffers must stay valid until the enqueued work completes.
 *   Streams.  `stream` is a hipStream_t passed as void* (NULL = the null
 *     stream).  Calls only enqueue work and return; they are safe to call from
 *     several threads on distinct streams with distinct workspaces.
 *   Layouts.  Matrices are row-major with a leading dimension `ld` (elements).
 *     A quantised orientation (metis_q4) stores codes[n_outer][k_len/2] with the
 *     even K index in the low nibble, scales[n_outer][k_len/16] as E4M3 bytes,
 *     and one binary32 tensor scale.  "K axis" is the reduction axis of the GEMM
 *     the orientation feeds.
 *   Errors.  Argument errors are reported synchronously with METIS_E_INVALID
 *     (nothing is enqueued) and a message from metis_last_error().  Numeric
 *     failure inside a kernel (non-finite input, a Cholesky breakdown that the
 *     shift cannot repair) sets a per-device flag that metis_status_sync()
 *     returns as METIS_E_NUMERIC; outputs are then unspecified.
 *   Determinism.  Identical inputs, seed, tag and step give bit-identical
 *     outputs: reductions that feed quantisation use max, never sums in
 *     varying order.
 */
#ifndef METIS_H
#define METIS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define METIS_ABI_VERSION 1

typedef enum {
  METIS_OK = 0,
  METIS_E_INVALID = -1,     /* bad argument or shape; nothing was enqueued */
  METIS_E_UNSUPPORTED = -2, /* valid but not implemented (e.g. k + s > 96) */
  METIS_E_HIP = -3,         /* a HIP runtime call failed */
  METIS_E_NUMERIC = -4,     /* device-side numeric failure (status_sync only) */
  METIS_E_WORKSPACE = -5    /* workspace too small */
} metis_status;

typedef enum { METIS_BF16 = 0, METIS_F32 = 1 } metis_dtype;
typedef enum { METIS_RNE = 0, METIS_SR = 1 } metis_rounding;

/* Operand roles used in the Philox tag: tag = layer << 16 | operand << 12.
 * The library fills bits 8..11 (the draw's role) itself. */
enum { METIS_OPERAND_W = 1, METIS_OPERAND_X = 2, METIS_OPERAND_D = 3 };

/* Hyper-parameters (Metis notes page, 关键设计 2/3 and 损失函数/训练策略). */
typedef struct {
  int32_t k;        /* rank kept in high precision (1..96) */
  int32_t s;        /* sketch oversampling; the sketch has k + s columns */
  int64_t l_k;      /* sampled rows for operands with sample_rows != 0 */
  int32_t refresh;  /* factor-cache period in steps (>= 1) */
  int32_t rounding; /* metis_rounding */
  uint64_t seed;    /* Philox4x32-10 key */
} metis_config;

/* Factors of one operand (rows x cols).  U: rows x k, S: k (descending),
 * V: cols x k, all binary32 row-major device buffers owned by the caller.
 * V doubles as the factor cache: it holds the basis between calls.
 * refreshed_at is host state: -1 means "no basis yet". */
typedef struct {
  float *U;
  float *S;
  float *V;
  int64_t rows, cols;
  int32_t k;
  int64_t refreshed_at;
} metis_factors;

/* One quantised orientation (device buffers owned by the caller). */
typedef struct {
  uint8_t *codes;       /* n_outer * k_len / 2 bytes */
  uint8_t *scales;      /* n_outer * k_len / 16 bytes */
  float *tensor_scale;  /* 1 binary32 */
  int64_t n_outer;
  int64_t k_len;        /* multiple of 16 */
} metis_q4;

/* A quantised operand M (rows x cols): Q(U) (blocked along rows of U, so
 * n_outer = k, k_len = rows), S (binary32, not quantised), Q(V) (n_outer = k,
 * k_len = cols), and the residual along K = rows (R_ax0: n_outer = cols,
 * k_len = rows) and/or K = cols (R_ax1: n_outer = rows, k_len = cols).
 * k == 0 is direct NVFP4 (U, V, S unused).
 * S: k binary32 values in device memory.  metis_quantize and
 * metis_prepare_operand copy the factors' S into it when it is non-NULL on
 * entry, so the operand keeps the singular values its codes were made with
 * while later calls update the same factors; when it is NULL they set it to
 * f->S, the live factor buffer, which the next decomposition of those factors
 * overwrites. */
typedef struct {
  int64_t rows, cols;
  int32_t k;
  float *S;
  metis_q4 U, V, R_ax0, R_ax1;
} metis_qoperand;

enum { METIS_AXIS0 = 1, METIS_AXIS1 = 2 }; /* bitmask for metis_quantize */

int32_t metis_abi_version(void);
const char *metis_last_error(void);

/* metis_init_device -- set up the library on the current device: its copy of
 * the Gaussian quantile table that Omega is drawn from, the numeric status
 * word that metis_status_sync reads, and the address of the static scratch
 * array of metis_quantize_static.  Every other call does this itself on its
 * first use of a device; it copies to device symbols synchronously, so a
 * caller that captures library calls into a HIP graph calls this first, on
 * each device, outside the capture.  Repeated calls return METIS_OK at once.
 * Errors: METIS_E_HIP (no device, or a failed copy), METIS_E_UNSUPPORTED
 * (device index >= 64). */
metis_status metis_init_device(void);

/* Workspace sizes in bytes (0 never means "no workspace needed"; always
 * pass at least the returned size). */
size_t metis_decompose_workspace(int64_t rows, int64_t cols, const metis_config *cfg,
                                 int32_t sample_rows);
size_t metis_quantize_workspace(int64_t rows, int64_t cols, int32_t k);
size_t metis_gemm_fwd_workspace(const metis_qoperand *X, const metis_qoperand *W);
size_t metis_gemm_bwd_workspace(const metis_qoperand *D, const metis_qoperand *W,
                                const metis_qoperand *X);
size_t metis_prepare_operand_workspace(int64_t rows, int64_t cols, const metis_config *cfg,
                                       int32_t sample_rows);

/* metis_decompose -- spectral split of one operand (关键设计 1-3).
 * M: rows x cols (dtype metis_dtype, leading dimension ld >= cols).
 * If f->refreshed_at < 0 or step - f->refreshed_at >= cfg->refresh, a new
 * basis is sketched: sample l_k rows (sample_rows != 0; weights use all rows),
 * Y = M_s Omega (Omega: cols x (k+s) quantile-exact bf16 Gaussian), shifted
 * CholeskyQR3 of Y, B = Q^T M_s, Jacobi on B B^T, V = B^T Z Theta^-1/2.
 * f->refreshed_at is then set to step (host side, before the call returns).
 * Every call then projects P = M V, rediagonalises P^T P by Jacobi and writes
 * U = P R Lambda^-1/2, S = Lambda^1/2, V <- V R, so U S V^T = M V_old V_old^T.
 * Requires 1 <= k, k + s <= 96 and k + s <= min(l_k (or rows), cols); with
 * sample_rows != 0, rows <= 2^27 (METIS_E_UNSUPPORTED otherwise: the row
 * sampler resolves the boundary of its key histogram among at most 4096 rows).
 * tag: layer << 16 | operand << 12 (Omega and the row sample take roles 4, 5). */
metis_status metis_decompose(const void *M, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                             const metis_config *cfg, int32_t sample_rows, uint32_t tag,
                             int64_t step, metis_factors *f, void *ws, size_t ws_bytes,
                             void *stream);

/* metis_quantize -- NVFP4 fake quantisation of an operand (关键设计 1).
 * With f == NULL the tensor M itself is quantised (direct NVFP4); otherwise
 * the factors are quantised (U and V blocked along their rows) and the
 * residual M_R = M - U diag(S) V^T is formed on the fly (never stored) and
 * quantised along each requested axis (axes: METIS_AXIS0 | METIS_AXIS1).
 * Quantiser: tensor amax A_T, s_g = A_T/2688, block scale = E4M3(RNE, satfinite)
 * of a_b/(6 s_g), y = |x| * (1/(s_b s_g)), E2M1 by RNE or Philox stochastic
 * rounding (16-bit uniform per element).  out->S is set to f->S.
 * residual_out: optional rows x cols binary32 (ld = cols) copy of the exact
 * binary32 residual the quantiser consumed (for verification; NULL normally).
 * Requires K (rows for AXIS0, cols for AXIS1) to be a multiple of 16.
 * out->S: see metis_qoperand (snapshot copy when non-NULL). */
metis_status metis_quantize(const void *M, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                            const metis_factors *f, const metis_config *cfg, uint32_t tag,
                            int64_t step, int32_t axes, metis_qoperand *out, float *residual_out,
                            void *ws, size_t ws_bytes, void *stream);

/* metis_quantize_static -- metis_quantize without a workspace argument, for
 * callers that cannot allocate device memory: code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc.  Arguments, outputs
 * and errors are those of metis_quantize.  The call allocates nothing: its
 * scratch (the tensor amax words and the fp16 operands of the rank-k
 * product) lives in one static device array of the library per GPU,
 * metis_quantize_static_capacity() bytes (16 MiB), held until the process
 * ends.  An operand whose scratch exceeds it (with factors about
 * (rows + cols) * 6 * round_up(k, 16) bytes) returns METIS_E_UNSUPPORTED with
 * nothing enqueued.  Every call on one GPU uses that GPU's array: calls that
 * overlap in time on one GPU (other streams or threads) race, so the caller
 * orders them; the array keeps the last call's contents and each call clears
 * what it needs zeroed. */
size_t metis_quantize_static_capacity(void);
metis_status metis_quantize_static(const void *M, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                                   const metis_factors *f, const metis_config *cfg, uint32_t tag,
                                   int64_t step, int32_t axes, metis_qoperand *out, float *residual_out,
                                   void *stream);

/* metis_prepare_operand -- metis_decompose followed by metis_quantize with
 * the new factors (关键设计 1-3), as one call.  After the projection
 * P = M V_old the residual M_R = M - P V_old^T is quantised on `stream` while
 * the rediagonalisation (Jacobi, V <- V R, U, S) runs on `side_stream`; the
 * two are equal in exact arithmetic because the rotation R is orthogonal
 * (U diag(S) V^T = P R R^T V_old^T), and in binary32 they differ by rounding
 * only.  The factors are then quantised on `stream`, which on return has
 * everything ordered after it.  side_stream may be NULL or equal to stream
 * (then everything runs on stream).  Arguments, requirements and outputs are
 * those of metis_decompose and metis_quantize (f non-NULL; out->k == cfg->k);
 * ws holds at least metis_prepare_operand_workspace(rows, cols, cfg,
 * sample_rows) bytes. */
metis_status metis_prepare_operand(const void *M, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                                   const metis_config *cfg, int32_t sample_rows, uint32_t tag,
                                   int64_t step, metis_factors *f, int32_t axes, metis_qoperand *out,
                                   float *residual_out, void *ws, size_t ws_bytes, void *stream,
                                   void *side_stream);

/* metis_gemm_fwd -- Y = X-hat W-hat (关键设计 1, the split forward GEMM).
 * X: l x m with R_ax1 (K = m); W: m x n with R_ax0 (K = m).  Y: l x n
 * binary32, leading dimension ldy.  Evaluated as
 *   Y = Q(X_R) Q(W_R) + P' Q(V_W)^T + Q(U_X) G,
 *   P' = Q(X_R) Q(U_W) S_W,  G = S_X (Q(V_X)^T Q(W_R) + (Q(V_X)^T Q(U_W)) S_W Q(V_W)^T),
 * which equals the product of the dense dequantised operands. */
metis_status metis_gemm_fwd(const metis_qoperand *X, const metis_qoperand *W, float *Y, int64_t ldy,
                            void *ws, size_t ws_bytes, void *stream);

/* metis_gemm_bwd -- dX = D-hat W-hat^T (K = n: D needs R_ax1, W needs R_ax1)
 * and dW = X-hat^T D-hat (K = l: X needs R_ax0, D needs R_ax0), the same
 * split embedded in the backward GEMMs (W4A4G4, 整体框架).  dX: l x m,
 * dW: m x n, binary32.  Either output pointer may be NULL to skip that
 * product.  The dW product uses the part of ws after the dX product's
 * region, so ws holds metis_gemm_bwd_workspace(D, W, X) bytes even when only
 * dW is asked for. */
metis_status metis_gemm_bwd(const metis_qoperand *D, const metis_qoperand *W, const metis_qoperand *X,
                            float *dX, int64_t lddx, float *dW, int64_t lddw, void *ws,
                            size_t ws_bytes, void *stream);

/* Two-phase form of the split GEMMs.  The low-rank terms of a split product
 * (P' and G of the forward equation of 关键设计 1, and their counterparts in
 * dX and dW) ride along K as bf16 hi/lo operands; building them needs only
 * the quantised operands.  *_prepare builds them into ws on `stream` and
 * *_prepared runs the main GEMM, reading them from the same ws, so a caller
 * can build one product's terms on another stream while an earlier GEMM
 * runs.  Arguments are those of metis_gemm_fwd / metis_gemm_bwd; `which`
 * selects the backward products (METIS_GRAD_DX | METIS_GRAD_DW).  Contract:
 * the prepared call names the same operands, ws and ws_bytes as the prepare
 * call, is ordered after it (same stream or an event), and neither ws nor the
 * operands change in between; the results then equal those of
 * metis_gemm_fwd / metis_gemm_bwd bit for bit.  Argument errors return
 * synchronously as in the one-call form. */
enum { METIS_GRAD_DX = 1, METIS_GRAD_DW = 2 };
metis_status metis_gemm_fwd_prepare(const metis_qoperand *X, const metis_qoperand *W, void *ws,
                                    size_t ws_bytes, void *stream);
metis_status metis_gemm_fwd_prepared(const metis_qoperand *X, const metis_qoperand *W, float *Y, int64_t ldy,
                                     void *ws, size_t ws_bytes, void *stream);
metis_status metis_gemm_bwd_prepare(const metis_qoperand *D, const metis_qoperand *W, const metis_qoperand *X,
                                    int32_t which, void *ws, size_t ws_bytes, void *stream);
metis_status metis_gemm_bwd_prepared(const metis_qoperand *D, const metis_qoperand *W, const metis_qoperand *X,
                                     float *dX, int64_t lddx, float *dW, int64_t lddw, void *ws,
                                     size_t ws_bytes, void *stream);

/* Waits for `stream`, then returns and clears the current device's numeric
 * failure flag (METIS_OK or METIS_E_NUMERIC). */
metis_status metis_status_sync(void *stream);

/* ------------------------------------------------------------------ MXFP4
 * A separate FP4 format, for comparison with NVFP4 on the same hardware: the
 * pages name MXFP4 only as a format their NVFP4 recipes are not claimed for
 * ("Full-Stack FP4: Stable LLM Pretraining with Quantized Projections,
 * Optimizers, and Attention", 局限性).  Its definition is the OCP Microscaling
 * (MX) one: 32 consecutive elements along K share a power-of-two scale
 * X = 2^(floor(log2 amax) - 2), stored as an E8M0 byte (exponent + 127,
 * clamped to [-127, 127]; an all-zero block stores 0); each element is x / X
 * rounded to the nearest E2M1 value, ties to even mantissa, saturating at 6
 * (rounding METIS_RNE), or stochastically (METIS_SR) with the Philox draws of
 * seed, tag and step indexed by the element's position outer * K + k in the
 * output layout.  No spectral split on this path.
 *
 * metis_mxfp4_quantize: M is rows x cols, row-major with leading dimension
 * ld, bf16 or fp32 (dtype), finite (a non-finite block sets the numeric flag
 * of metis_status_sync; its codes are then unspecified).  axis names the K
 * axis: 1 along a row, 0 down a column (the output is then the quantised
 * transpose).  With outer = the other dimension and K its length: codes is
 * outer x K/2 bytes (element 2i in the low nibble of byte i), 16-byte
 * aligned; scales is outer x K/32 E8M0 bytes.  K % 32 == 0, rounding is
 * METIS_RNE or METIS_SR and step >= 0 (METIS_E_INVALID otherwise); with
 * axis 0, rows / 32 <= 65535 (METIS_E_UNSUPPORTED otherwise).  Both buffers
 * are caller-owned device memory, written on stream.
 *
 * metis_mxfp4_gemm: C = A B^T in fp32 (row-major, leading dimension ldc >= N)
 * of two MXFP4 operands in that layout, A with M rows and B with N rows of
 * K elements: codes M x K/2 and N x K/2, scales M x K/32 and N x K/32, all four
 * arrays 16-byte aligned, K % 1024 == 0, M % 8 == 0 and N % 8 == 0
 * (METIS_E_UNSUPPORTED otherwise).
 * Products are exact and accumulate in fp32 on the block-scaled FP4 matrix
 * instruction of gfx950.  M or N == 0 returns METIS_OK with nothing enqueued.
 * Argument errors return synchronously; nothing is allocated. */
metis_status metis_mxfp4_quantize(const void *M, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                                  int32_t axis, int32_t rounding, uint64_t seed, uint32_t tag, int64_t step,
                                  uint8_t *codes, uint8_t *scales, void *stream);
metis_status metis_mxfp4_gemm(const uint8_t *a_codes, const uint8_t *a_scales, const uint8_t *b_codes,
                              const uint8_t *b_scales, int64_t M, int64_t N, int64_t K, float *C,
                              int64_t ldc, void *stream);

/* ------------------------------------------------------------------- int8
 * A third operand format for the same linear layer: 8-bit integers with one
 * binary32 scale per line, a line being what one output row or column of the
 * product reduces over (a token's activations, an output channel's weights).
 * For the products that lose too much in 4 bits, and for serving.  With a the
 * largest magnitude of the line, in binary32 (RN: rounded to nearest),
 *   s = max(RN(a / 127), 2^-126),  inv = RN(1 / s),  y = RN(x inv),
 *   code = y rounded to the nearest integer, ties to even (METIS_RNE), or
 *          floor(y) + [u < y - floor(y)] (METIS_SR),
 * clamped to [-127, 127], where u is 2^-16 times the 16-bit Philox draw of
 * (seed, tag with role 0, step) at the element's row-major position
 * i * cols + j in M, the same draw for both orientations.
 *
 * metis_i8: n_outer lines of k_len codes each, at a row pitch of
 * metis_int8_pitch(k_len) bytes (k_len rounded up to 128); the bytes behind
 * k_len in a row are zero (the quantiser writes them so).  codes is 16-byte
 * aligned.  Device buffers owned by the caller.
 *
 * metis_int8_quantize: M is rows x cols, row-major with leading dimension ld,
 * bf16 or fp32.  axes: METIS_AXIS1 fills ax1 (K along a row: rows lines of
 * cols codes), METIS_AXIS0 fills ax0 (K down a column: cols lines of rows
 * codes, the quantised transpose); an orientation not asked for may be NULL.
 * A non-finite element sets the numeric flag of metis_status_sync and leaves
 * unspecified codes.  ws holds metis_int8_quantize_workspace(rows, cols,
 * axes) bytes, 16-byte aligned.  rows == 0 or cols == 0 returns METIS_OK with
 * nothing enqueued.  rows and cols are below 2^31 and, with METIS_AXIS0,
 * ceil(rows / 128) * ceil(cols / 128) below 2^24 (METIS_E_UNSUPPORTED above).
 *
 * metis_int8_quantize_counted: the same with the step read from the int64 at
 * step_count in device memory when the kernels run, unless that is negative
 * (for graphs, whose replays would otherwise all take the draws of `step`).
 *
 * metis_int8_gemm: C = diag(s_A) (A B^T) diag(s_B), row-major with leading
 * dimension ldc >= B->n_outer, binary32 or bf16 (c_dtype).  A and B have the
 * same k_len, at most 131071 (METIS_E_UNSUPPORTED above): sums are exact in
 * int32 for codes of any value, and an output is RN(RN(RN(sum) s_A) s_B), rounded once more for
 * bf16.  n_outer == 0 on either side is a no-op, k_len == 0 invalid.  ws
 * holds metis_int8_gemm_workspace(A->n_outer, B->n_outer, k_len) bytes (0:
 * may be NULL), 16-byte aligned: a product with few outputs is cut along K.
 *
 * metis_int8_linear: Y = X-hat W-hat for serving: X (tokens x k_len, bf16 or
 * fp32) is quantised to nearest with one scale per token and multiplied with
 * W, the K-down-the-columns orientation of a weight (n_outer output channels
 * of k_len codes).  Equal to metis_int8_quantize along METIS_AXIS1 followed
 * by metis_int8_gemm, bit for bit.  ws holds
 * metis_int8_linear_workspace(tokens, W->n_outer, k_len) bytes (0: may be
 * NULL), 256-byte aligned.
 *
 * Argument errors return synchronously; nothing is allocated. */
typedef struct {
  int8_t *codes;
  float *scales;   /* n_outer binary32 */
  int64_t n_outer;
  int64_t k_len;
} metis_i8;

int64_t metis_int8_pitch(int64_t k_len);
size_t metis_int8_quantize_workspace(int64_t rows, int64_t cols, int32_t axes);
metis_status metis_int8_quantize(const void *M, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                                 int32_t axes, int32_t rounding, uint64_t seed, uint32_t tag, int64_t step,
                                 const metis_i8 *ax0, const metis_i8 *ax1, void *ws, size_t ws_bytes,
                                 void *stream);
metis_status metis_int8_quantize_counted(const void *M, int32_t dtype, int64_t rows, int64_t cols, int64_t ld,
                                         int32_t axes, int32_t rounding, uint64_t seed, uint32_t tag,
                                         int64_t step, const int64_t *step_count, const metis_i8 *ax0, const metis_i8 *ax1,
                                         void *ws, size_t ws_bytes, void *stream);
size_t metis_int8_gemm_workspace(int64_t M, int64_t N, int64_t k_len);
metis_status metis_int8_gemm(const metis_i8 *A, const metis_i8 *B, void *C, int32_t c_dtype, int64_t ldc,
                             void *ws, size_t ws_bytes, void *stream);
size_t metis_int8_linear_workspace(int64_t tokens, int64_t n_outer, int64_t k_len);
metis_status metis_int8_linear(const void *X, int32_t dtype, int64_t tokens, int64_t ldx, const metis_i8 *W,
                               void *Y, int32_t y_dtype, int64_t ldy, void *ws, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------ AdamW
 * The update of the master weights from the layers' gradients, many tensors
 * at once.  Per element, each operation rounded to binary32, g the gradient
 * (times *clip where clip is not NULL):
 *   m' = b1 m + (1 - b1) g,  v' = b2 v + ((1 - b2) g) g,  r' = sqrt(v'),
 *   p' = p (1 - lr wd) - lr / (1 - b1^t) * m' / (r' / sqrt(1 - b2^t) + eps).
 * An element for which m', v' or p' is not finite keeps p, m and v and sets
 * the numeric flag of metis_status_sync.  8-bit moments are kept as values and
 * encoded again with their block's new scale (a larger neighbour coarsens them;
 * a kept r above zero stays above zero).  A stored 8-bit moment that is itself
 * not finite stays NaN; the other elements of its block go on.
 *
 * metis_adamw_tensor: n elements, contiguous; param binary32 (METIS_F32) or
 * bf16, grad binary32 or bf16.  state_bits 32: m and v are binary32 arrays
 * (v the second moment), the scales unused.  state_bits 8: m and v are arrays
 * of E4M3 bytes (v holds r = sqrt(second moment)) in blocks of 256
 * consecutive elements with one binary32 scale each (m_scale, v_scale:
 * ceil(n / 256) values): value = E4M3(code) * scale.  The scale is
 * 2^(floor(log2 amax) - 7), at least 2^-126; a positive r never rounds to
 * zero.  All-zero codes and scales are the initial state.  The update uses
 * the new moments before they are rounded.
 * rounding: METIS_RNE, or METIS_SR for 8-bit states and bf16 parameters:
 * element e takes word e & 3 of the Philox block of counter (e >> 2, tag with
 * role 6, t), the low half for m and the high half for r; a bf16 parameter
 * takes the low half of role 7's word.
 * t: the step, counted from 1: `step`, or where step_count is not NULL the
 * int64 that it points to in device memory when the kernel runs (for graphs;
 * every other value is fixed at the call).
 * No array that is written may appear twice in a call or overlap another one,
 * a gradient included; gradients may overlap each other.
 * A tensor has at most 4096 * (2^24 - 1) elements (METIS_E_UNSUPPORTED above),
 * here and in metis_grad_norm.  Small tensors share launches; the tensor list is
 * read before the call returns.
 *
 * metis_grad_norm: out[0] = the square root of the sum of squares over all
 * tensors' gradients (only grad, grad_dtype and n are read), summed in
 * binary64 in an order fixed by the sizes; out[1] = min(1, max_norm / (norm +
 * 1e-6)), NaN if the norm is.  out: two binary32 in device memory; out + 1
 * serves as metis_adamw_config.clip.  ws holds
 * metis_grad_norm_workspace(tensors, count) bytes, 8-byte aligned. */
typedef struct {
  void *param;
  const void *grad;
  void *m;
  void *v;
  float *m_scale;
  float *v_scale;
  int64_t n;
  int32_t param_dtype; /* metis_dtype */
  int32_t grad_dtype;  /* metis_dtype */
  int32_t state_bits;  /* 32 or 8 */
  uint32_t tag;        /* layer << 16 | operand << 12 */
} metis_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;              /* >= 1 (ignored with step_count) */
  const int64_t *step_count; /* device, or NULL */
  const float *clip;         /* device, or NULL */
  uint64_t seed;
  int32_t rounding;          /* metis_rounding */
} metis_adamw_config;

metis_status metis_adamw_step(const metis_adamw_tensor *tensors, int64_t count, const metis_adamw_config *cfg,
                              void *stream);
size_t metis_grad_norm_workspace(const metis_adamw_tensor *tensors, int64_t count);
metis_status metis_grad_norm(const metis_adamw_tensor *tensors, int64_t count, double max_norm, float *out,
                             void *ws, size_t ws_bytes, void *stream);

/* -------------------------------------------- around the linear layers
 * What a language model has between its linear layers, before and behind them:
 * layer norm, dropout, the embedding and the loss over the vocabulary, each
 * with its gradients.  dtypes are metis_dtype; rows are row-major with a
 * leading dimension of at least their length; sums are binary32 (binary64
 * for the total loss), in an order fixed by the sizes, and each output is
 * rounded once to its type.  Pointers are aligned to their values (rows that
 * are 16-byte aligned run faster); an output may not overlap an input
 * unless it is said below.  Zero rows or tokens are no error.  Argument errors
 * return synchronously; nothing is allocated.
 *
 * metis_layernorm_fwd: y = (x - mean) rstd * weight + bias for each row of
 * cols values, rstd = 1 / sqrt(variance + eps), the variance that of all cols
 * values.  weight and bias (w_dtype) may be NULL: 1 and 0.  y has y_dtype.
 * mean and rstd (rows binary32 each, both or neither NULL) are kept for the
 * backward pass.  Y may be X where the types are equal.
 * metis_layernorm_bwd: from dY (y_dtype), X and the forward pass's mean, rstd:
 * dX (x's type), dweight and dbias (w_dtype); each of them may be NULL.  dX may
 * be dY where the types are equal.  ws holds metis_layernorm_bwd_workspace(rows, cols)
 * bytes, 256-byte aligned, where dweight or dbias is wanted.  1 <= cols < 2^31.
 *
 * metis_dropout: element e = i * cols + j takes the 16-bit Philox draw h(e) of
 * (seed, tag with role 8, step), as in stochastic rounding; with t = 65536 p
 * rounded to the nearest integer, ties to even,
 *   y = (h < t ? 0 : x * s) + residual,  s = 65536 / (65536 - t) in binary32
 * (s = 0 for t = 65536), residual may be NULL (then nothing is added).  A
 * dropped x counts as zero whatever it holds.  The same call on dY, without a
 * residual, gives dX.  X, residual and Y have one type; Y may be X or the
 * residual.  step_count: NULL, or the int64 in device memory that holds the
 * step when the kernel runs, unless it is negative (for graphs).
 * 0 <= p <= 1, rows * cols < 2^63.
 *
 * metis_embedding_fwd: row i of Y is scale times row ids[i] of W (vocab x cols;
 * id_bits 32 or 64: int32 or int64 ids), the product in binary32.  A number
 * outside [0, vocab) sets the numeric flag and gives a row of zeros.
 * metis_embedding_bwd: row v of dW is scale times the sum of the rows of dY
 * whose id is v, over ascending rows in binary32 (in pieces of 16 of the sorted
 * tokens); rows of dW that no token points to, and row padding (negative:
 * none), are zero.  All of dW is written.  ws holds
 * metis_embedding_bwd_workspace(tokens, cols) bytes, 256-byte aligned.
 * vocab < 2^31, tokens < 2^31 (backward: 2^28 - 2^18), METIS_E_UNSUPPORTED
 * above; cols < 2^31.
 *
 * metis_cross_entropy_fwd: the logits of token i are l_v = x_i . w_v (x: tokens
 * x cols; w: vocab x cols), never stored; lse[i] = log sum_v exp l_v and
 * losses[i] = lse[i] - l_target.  A target equal to ignore_index, or outside
 * [0, vocab) (which sets the numeric flag), leaves the token out: its loss is
 * 0 and its gradients are 0, whatever its row of x holds.  losses may be NULL.
 * total: NULL, or two binary32: total[0] the sum of the losses (mean = 0) or
 * their mean over the tokens that are not left out (mean = 1; 0 if all are),
 * total[1] the number of those tokens.
 * metis_cross_entropy_bwd: the gradients of x and w (their types; dX and dW may
 * each be NULL) given lse and the gradient of each loss, grad[i] (grad_each =
 * 1) or grad[0] for all (grad_each = 0), divided by *count where count is not
 * NULL (total + 1 of the forward pass, for the mean).  Logits are formed again
 * in pieces of the vocabulary, so the workspace does not grow with it: a piece
 * has at most 2^28 probabilities (or 4096 words, where that is more) and 2^29
 * values of w (or 256 words).
 * The forward product takes two bf16 operands as they are.  Every other
 * operand becomes binary16 under a common power of two that brings its largest
 * finite value (of the tokens that have a target) into [2^14, 2^15): one value
 * for bf16, two for binary32 where a loss or a binary32 gradient needs both;
 * so do the gradients of the logits, two values where a gradient is binary32,
 * and, where each loss has a gradient (grad_each = 1), each token's under a power
 * of two of its own, which dX's row is free of again; dW's x carries the inverse.
 * One value is off by 2^-11 of itself at most (a bf16 operand by nothing), two
 * by 2^-22, and either by 2^-40 of its operand's largest value.
 * lse of a token that is left out is any value.
 * ws holds metis_cross_entropy_workspace(l, backward) bytes, 256-byte aligned.
 * tokens, cols <= 2^22, vocab < 2^31 (METIS_E_UNSUPPORTED above). */
metis_status metis_layernorm_fwd(const void *X, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                                 const void *weight, const void *bias, int32_t w_dtype, double eps, void *Y,
                                 int32_t y_dtype, int64_t ldy, float *mean, float *rstd, void *stream);
size_t metis_layernorm_bwd_workspace(int64_t rows, int64_t cols);
metis_status metis_layernorm_bwd(const void *dY, int32_t y_dtype, int64_t lddy, const void *X, int32_t x_dtype,
                                 int64_t rows, int64_t cols, int64_t ldx, const void *weight, int32_t w_dtype,
                                 const float *mean, const float *rstd, void *dX, int64_t lddx, void *dweight,
                                 void *dbias, void *ws, size_t ws_bytes, void *stream);
metis_status metis_dropout(const void *X, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx, const void *residual,
                           int64_t ldr, double p, uint64_t seed, uint32_t tag, int64_t step, const int64_t *step_count,
                           void *Y, int64_t ldy, void *stream);
metis_status metis_embedding_fwd(const void *W, int32_t w_dtype, int64_t vocab, int64_t cols, int64_t ldw,
                                 const void *ids, int32_t id_bits, int64_t tokens, double scale, void *Y,
                                 int32_t y_dtype, int64_t ldy, void *stream);
size_t metis_embedding_bwd_workspace(int64_t tokens, int64_t cols);
metis_status metis_embedding_bwd(const void *dY, int32_t y_dtype, int64_t tokens, int64_t cols, int64_t lddy,
                                 const void *ids, int32_t id_bits, int64_t vocab, int64_t padding, double scale,
                                 void *dW, int32_t w_dtype, int64_t lddw, void *ws, size_t ws_bytes, void *stream);

typedef struct {
  const void *x, *w, *targets;
  int64_t tokens, vocab, cols;
  int64_t ldx, ldw;
  int64_t ignore_index;
  int32_t x_dtype, w_dtype;
  int32_t target_bits; /* 32 or 64 */
} metis_loss;

size_t metis_cross_entropy_workspace(const metis_loss *l, int32_t backward);
metis_status metis_cross_entropy_fwd(const metis_loss *l, float *losses, float *lse, int32_t mean, float *total, void *ws,
                                     size_t ws_bytes, void *stream);
metis_status metis_cross_entropy_bwd(const metis_loss *l, const float *lse, const float *grad, int32_t grad_each,
                                     const float *count, void *dX, int64_t lddx, void *dW, int64_t lddw, void *ws,
                                     size_t ws_bytes, void *stream);

/* Kernel timing for benchmarks.  metis_timing_enable(capacity) creates
 * capacity pairs of HIP events (0 disables timing and releases them); while
 * enabled, each main split-GEMM kernel (kind 0; d = M, N, K, K-extension) and
 * each quantiser sweep (kind 1: amax pass, kind 2: quantise pass; d = rows,
 * cols, axes, K of the rank-k product), each MXFP4 GEMM kernel (kind 3;
 * d = M, N, K, 0), the sketch of a refresh step, from the row sample to V
 * (kind 4; d = rows, cols, k + s, l_k), and metis_decompose's projection
 * and rediagonalisation (kind 5; d = rows, cols, k, 1 on a refresh step)
 * is bracketed by events recorded on the launching stream,
 * until the capacity is used up.  metis_timing_read waits
 * for the recorded events, writes up to max_records durations (ms) and
 * 5-tuples (kind, d0, d1, d2, d3), resets the record list and returns the
 * number written. */
metis_status metis_timing_enable(int32_t capacity);
int32_t metis_timing_read(float *ms, int64_t *shape, int32_t max_records);
/* Restricts the recorded kinds to the bits of mask (bit k: kind k; all kinds
 * by default).  Each record adds two event packets to the stream, so a caller
 * timing a whole step records only the kinds it needs. */
metis_status metis_timing_kinds(int32_t mask);

/* Host-only helpers (no GPU needed) exposing the library's own definitions
 * of its random draws, for verification against an independent model.
 * metis_omega_table: the 65536 bf16 bit patterns of the Gaussian quantile
 * table, T[t] = bf16(Phi^-1((t + 0.5) / 65536)).
 * metis_philox4x32_10: one Philox4x32-10 block (Salmon et al., SC'11). */
void metis_omega_table(uint16_t *out65536);
void metis_philox4x32_10(const uint32_t ctr[4], const uint32_t key[2], uint32_t out[4]);

#ifdef __cplusplus
}
#endif
#endif /* METIS_H */
