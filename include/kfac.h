/*
 * kfac.h -- C ABI of the per-GPU K-FAC hot path for AMD Instinct MI355X
 * (gfx950).  One K-FAC step on one GPU is
 *
 *     kfac_factors      A and G Kronecker factors with their running average
 *     kfac_pack_sym     upper triangles of the factors <-> one fused buffer
 *     kfac_damped_inverse  (X + gamma I)^-1 of every factor, batched
 *     kfac_precondition (G + gamma I)^-1 . gradW . (A + gamma I)^-1 per layer
 *
 * and, to feed real layers, kfac_im2col / kfac_grad_rows (factor inputs from
 * a layer's input and output gradient) and kfac_grad_matrix (a layer's
 * weight and bias gradients as one matrix and back).  To train an encoder
 * layer: kfac_attention_forward / _backward (attention with a learned
 * relative position bias), kfac_checkpoint_* (layer inputs kept in 8 bits,
 * with their factor and gradient), kfac_layer_norm_*, kfac_gated_* (the gated
 * feed-forward block), kfac_grad_norm and kfac_grad_clip (the gradients'
 * common norm, and clipping to one).  The method follows "Accelerating
 * Distributed K-FAC with Smart Parallelism of Computing and Communication
 * Tasks" (cited per entry point below).
 *
 * Common rules
 *   - Matrices are row-major.  "Upper" means the entries (i, j) with j >= i.
 *   - Arrays of per-layer pointers (x, m, xinv, grad, ...) and the size
 *     arrays (rows, d, ...) are HOST arrays, read during the call only.  The
 *     pointers they hold are DEVICE pointers, at least 4-byte aligned.
 *   - `workspace` is a device buffer of at least the size returned by the
 *     matching *_workspace_size() call, 256-byte aligned, owned by the
 *     caller, and must stay untouched until the enqueued work has finished.
 *     The library allocates no device memory and keeps no state between
 *     calls; calls on different streams with different workspaces may run
 *     concurrently.
 *   - Every call validates its arguments on the host first.  On an error it
 *     returns a non-zero status and enqueues nothing.  On success the work is
 *     enqueued on `stream` (0 = the null stream) and the call returns
 *     without waiting for it.
 *   - Inputs containing NaN or Inf are not screened; they propagate
 *     (the inverse reports them through `info`).
 */
#ifndef KFAC_H
#define KFAC_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KFAC_OK = 0,
    KFAC_ERR_INVALID_VALUE = 1, /* bad count, size, pointer, alignment, gamma or eps */
    KFAC_ERR_WORKSPACE = 2,     /* workspace missing, misaligned or too small */
    KFAC_ERR_UNSUPPORTED = 3,   /* valid request this build cannot serve */
    KFAC_ERR_HIP = 4            /* a HIP runtime call or kernel launch failed */
} kfac_status_t;

typedef enum { KFAC_F32 = 0, KFAC_BF16 = 1 } kfac_dtype_t;
typedef enum { KFAC_PACK = 0, KFAC_UNPACK = 1 } kfac_pack_dir_t;

/* Largest factor dimension and largest number of layers / matrices per call. */
#define KFAC_MAX_DIM 16384
#define KFAC_MAX_COUNT 4096

/* ABI version of this header (bumped on any incompatible change). */
int kfac_abi_version(void);

/* Static, human-readable name of a status code. */
const char* kfac_status_string(kfac_status_t status);

/* ---------------------------------------------------------------- factors --
 * Kronecker factors with running average.  The page builds, per layer l, the
 * factor A from the layer's input a and the factor G from the gradient with
 * respect to the layer's output g, both symmetric (paragraph introducing the
 * Kronecker factors; the pipelining paragraph computes them in the forward
 * pre-hook and the backward hook, "Eq. (7)" and "Eq. (8)").  For each of the
 * n matrices:
 *
 *     F_i = (1 / rows_i) * X_i^T X_i
 *     M_i <- F_i                                 if first_step != 0
 *     M_i <- eps * M_i + (1 - eps) * F_i         otherwise
 *
 * x[i]   : [rows[i], d[i]] row-major, float32 (in_dtype KFAC_F32) or bfloat16
 *          (KFAC_BF16, accumulated in float32).  float32 products are formed
 *          on the bf16 matrix cores as six bf16 products of exact three-way
 *          splits of each value and carry float32 rounding.  A layer with a bias carries
 *          a trailing column of ones.
 * m[i]   : [d[i], d[i]] float32.  Only the upper triangle is read (when
 *          first_step == 0) and written; the strict lower triangle is left
 *          as it was.
 * eps    : in [0, 1].  1 <= rows[i] <= 2^31 - 1, 1 <= d[i] <= KFAC_MAX_DIM.
 * The x[i] must not overlap any m[j].  Results are deterministic: the same
 * inputs give the same bits on every run.
 */
size_t kfac_factors_workspace_size(int n, const int64_t* rows, const int64_t* d, kfac_dtype_t in_dtype);
kfac_status_t kfac_factors(int n, const void* const* x, const int64_t* rows, const int64_t* d,
                           kfac_dtype_t in_dtype, float* const* m, float eps, int first_step,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------- pack --
 * Tensor fusion of the symmetric factors: only the upper triangle including
 * the diagonal is kept, d(d+1)/2 elements per factor (tensor-fusion
 * paragraph on communicated elements; paragraph on sending only the upper
 * triangles), and consecutive factors are merged into one contiguous buffer
 * (paragraph on dynamic tensor fusion).
 *
 *     packed[off_l + i*d_l - i*(i-1)/2 + (j - i)] = M_l[i][j],  0 <= i <= j < d_l
 *     off_l = sum_{k<l} d_k (d_k + 1) / 2
 *
 * KFAC_PACK reads the upper triangles of m[l] and writes `packed`
 * (kfac_packed_size() float32 elements).  KFAC_UNPACK reads `packed` and
 * writes every element of m[l]: entry (i, j) and its mirror (j, i).  Values
 * are copied bit for bit.  The m[l] must not overlap each other or `packed`.
 * The host passes only the pointers and orders; the offsets off_l are
 * formed on the device, as a prefix sum across a wavefront.  The workspace
 * (kfac_pack_workspace_size() bytes) holds that layer table.
 */
int64_t kfac_packed_size(int n, const int64_t* d);
size_t kfac_pack_workspace_size(int n, const int64_t* d);
kfac_status_t kfac_pack_sym(int n, float* const* m, const int64_t* d, float* packed, kfac_pack_dir_t dir,
                            void* workspace, size_t workspace_bytes, hipStream_t stream);

/* kfac_pack_sym without a workspace, for callers that cannot allocate device
 * memory (code under stream capture, tight serving loops, harnesses that
 * forbid allocation).  Same arguments, results and errors as kfac_pack_sym;
 * the layer table lives in a device array of the library instead (64 KiB per
 * GPU, held until the process ends).  It allocates nothing: no hipMalloc, no
 * hipFree, no allocating library call.  At most KFAC_STATIC_MAX_FACTORS
 * factors per call, else KFAC_ERR_UNSUPPORTED (nothing enqueued).  Every call
 * on one GPU shares that array, and the last call's table stays in it: calls
 * that may overlap on one GPU (different streams, or different host threads
 * without ordering) race and must not be made.
 */
#define KFAC_STATIC_MAX_FACTORS 1024
kfac_status_t kfac_pack_sym_static(int n, float* const* m, const int64_t* d, float* packed, kfac_pack_dir_t dir,
                                   hipStream_t stream);

/* Plain device-to-device copy of `bytes` bytes (16-byte loads and stores,
 * one per lane).  It computes nothing of the method: it is the measured
 * streaming rate that the HBM-bound figures of pack and unpack are set
 * against, beside the published peak.  src and dst are device pointers,
 * 16-byte aligned, not overlapping; bytes is a multiple of 16 (0 is a no-op),
 * else KFAC_ERR_INVALID_VALUE.
 */
kfac_status_t kfac_stream_copy(const void* src, void* dst, size_t bytes, hipStream_t stream);

/* Matrix-core rate reference.  `blocks` workgroups of four waves each run
 * `iters` rounds of four independent matrix-core products on register
 * operands, with no memory traffic besides one float per wave written to
 * `sink` (device, 4 * blocks floats, 4-byte aligned), which keeps the products
 * from being removed.  The products are v_mfma_f32_32x32x16_bf16
 * (KFAC_RATE_BF16, 32768 flops each), v_mfma_f64_16x16x4f64 (KFAC_RATE_F64,
 * 2048) or v_mfma_f32_32x32x2f32 (KFAC_RATE_F32, 4096).  It computes nothing
 * of the method: timed by the caller, it is the rate the matrix cores
 * sustain on this part under its own clock and power limits, the measured
 * reference for the matrix-core-bound stages beside the published peaks.
 * *flops (host, may be NULL) receives the flops of the call.
 * KFAC_ERR_INVALID_VALUE for an unknown kind, iters outside [1, 2^24],
 * blocks outside [1, 65536] or a null sink.
 */
typedef enum { KFAC_RATE_BF16 = 0, KFAC_RATE_F64 = 1, KFAC_RATE_F32 = 2 } kfac_rate_kind_t;
kfac_status_t kfac_matrix_rate(kfac_rate_kind_t kind, int64_t iters, int blocks, float* sink, double* flops,
                               hipStream_t stream);

/* ---------------------------------------------------------------- inverse --
 * Tikhonov-damped inverse of each factor (paragraph on damping before
 * inverting; the inverses of different layers are independent, paragraph on
 * MPD-KFAC; the inverse goes through a Cholesky decomposition, paragraph on
 * the inverse performance model).  For each of the n matrices:
 *
 *     Y_i = X_i + gamma I   (X_i read from the upper triangle of x[i])
 *     Y_i = U^T U  (Cholesky),  V = U^-1,  xinv[i] = V V^T = Y_i^-1
 *
 * The factorisation and V are computed in float64 on the GPU, where errors
 * grow with the condition number; the last product V V^T, whose error
 * relative to ||xinv||_F does not, with float32-accurate products (each
 * float32 product as six bf16 products of exact splits).  xinv[i] is written
 * as float32, both triangles, exactly symmetric.  info[i] (device int32 array of n entries) receives 0 on
 * success, or k > 0 when the leading minor of order k of Y_i is not positive
 * definite or not finite (LAPACK xPOTRF convention); xinv[i] is then
 * unspecified.  gamma must be finite and >= 0.  x[i] and xinv[j] must not
 * overlap.
 */
size_t kfac_inverse_workspace_size(int n, const int64_t* d);
kfac_status_t kfac_damped_inverse(int n, const float* const* x, const int64_t* d, float gamma,
                                  float* const* xinv, int32_t* info,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ----------------------------------------------------------- precondition --
 * Preconditioned gradient of each layer (the damped update rule that follows
 * the Kronecker inverse property (A (x) G)^-1 = A^-1 (x) G^-1):
 *
 *     out[l] = ginv[l] . grad[l] . ainv[l]
 *
 * ginv[l] : [d_g[l], d_g[l]] float32, (G + gamma I)^-1, symmetric;
 * grad[l] : [d_g[l], d_a[l]] float32 weight gradient (bias gradient in the
 *           last column for layers with a bias);
 * ainv[l] : [d_a[l], d_a[l]] float32, (A + gamma I)^-1, symmetric;
 * out[l]  : [d_g[l], d_a[l]] float32.
 * ginv and ainv must be exactly symmetric (as kfac_damped_inverse writes
 * them): the kernels read them in whichever orientation coalesces.  The two
 * products run on the bf16 matrix cores as six bf16 products of exact
 * splits per float32 product, with float32 rounding.  out[l]
 * must not overlap any input.
 */
size_t kfac_precondition_workspace_size(int n, const int64_t* d_g, const int64_t* d_a);
kfac_status_t kfac_precondition(int n, const float* const* ginv, const float* const* grad,
                                const float* const* ainv, const int64_t* d_g, const int64_t* d_a,
                                float* const* out, void* workspace, size_t workspace_bytes,
                                hipStream_t stream);

/* ----------------------------------------------------------------- layers --
 * Factor inputs of real layers.  The page computes A_{l-1} from the layer's
 * input in the forward pre-hook and G_l from the gradient with respect to the
 * layer's output in the backward hook (pipelining paragraph; the optimizer
 * paragraph that registers both hooks on every layer).  For a convolution the
 * rows of a factor input are its patches, one row per sample and output
 * position, so that A = (1/rows) a^T a with rows = batch * H_out * W_out.
 * A fully connected layer is the 1 x 1 case: h = w = kh = kw = 1.
 */
typedef struct {
    int64_t n, c, h, w; /* input [n, c, h, w] row-major; n, c, h, w >= 1 */
    int32_t kh, kw;     /* kernel size >= 1 */
    int32_t sh, sw;     /* stride >= 1 */
    int32_t ph, pw;     /* zero padding >= 0 */
    int32_t dh, dw;     /* dilation >= 1 */
    int32_t ones;       /* 1: a trailing column of ones (the layer has a bias), else 0 */
    int32_t reserved;   /* 0 */
} kfac_conv_t;

/* Patches of each layer input as the rows of its A-factor input:
 *
 *     oh = (h + 2 ph - dh (kh - 1) - 1) / sh + 1,  ow likewise (both >= 1)
 *     a[l][(ni oh + y) ow + x][(ci kh + i) kw + j] = x[l][ni][ci][y sh - ph + i dh][x sw - pw + j dw]
 *
 * zero where the index falls outside the input, and 1 in the last column
 * when ones = 1.  a[l] is [n oh ow, c kh kw + ones] row-major, in `dtype`
 * like x[l]; values are copied bit for bit.  The column order matches a
 * weight [c_out, c, kh, kw] read as [c_out, c kh kw].  a[l] must not
 * overlap any x[j]; at most 2^31 - 1 elements per a[l] and per sample of
 * x[l] (c h w), else KFAC_ERR_INVALID_VALUE.
 */
size_t kfac_im2col_workspace_size(int n);
kfac_status_t kfac_im2col(int n, const void* const* x, const kfac_conv_t* shape, kfac_dtype_t dtype,
                          void* const* a, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Output gradients as the rows of each G-factor input:
 *
 *     g[l][b hw + p][ci] = scale * gy[l][b][ci][p]
 *
 * gy[l] : [batch[l], c[l], hw[l]] (an output gradient [b, c, H, W] with the
 *         positions flattened; a fully connected layer: hw = 1);
 * g[l]  : [batch[l] hw[l], c[l]], the product formed in float32 and stored
 *         in `dtype` like gy[l] (rounded to nearest even for bfloat16).
 * `scale` multiplies every gradient (for a loss averaged over the batch,
 * scale = batch gives per-sample gradients).  g[l] must not overlap gy[j].
 */
size_t kfac_grad_rows_workspace_size(int n);
kfac_status_t kfac_grad_rows(int n, const void* const* gy, const int64_t* batch, const int64_t* c,
                             const int64_t* hw, kfac_dtype_t dtype, float scale, void* const* g,
                             void* workspace, size_t workspace_bytes, hipStream_t stream);

/* A layer's weight and bias gradients as one [d_out, d_in + has_bias] matrix
 * (the gradW of kfac_precondition, bias in the last column) and back:
 *
 *     KFAC_PACK    mat[l][r][k] = wgrad[l][r][k] (k < d_in), mat[l][r][d_in] = bgrad[l][r]
 *     KFAC_UNPACK  the reverse
 *
 * wgrad[l] : [d_out, d_in] float32 (a convolution weight [c_out, c, kh, kw]
 *            with d_in = c kh kw);  bgrad[l] : [d_out] float32 or NULL (no
 *            bias, has_bias = 0).  Values are copied bit for bit; mat[l]
 *            must not overlap wgrad[j] or bgrad[j].
 */
size_t kfac_grad_matrix_workspace_size(int n);
kfac_status_t kfac_grad_matrix(int n, float* const* wgrad, float* const* bgrad, const int64_t* d_out,
                               const int64_t* d_in, float* const* mat, kfac_pack_dir_t dir,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);

/* -------------------------------------------------------------- attention --
 * Softmax attention of an encoder layer with a learned relative position
 * bias by buckets, forward and backward.  Query i stands at position
 * p_i = i + len_k - len_q; it sees key j when j < lens[b] (lens may be NULL)
 * and, with `causal`, j <= p_i.  With dist = |j - p_i| (one-sided:
 * max(p_i - j, 0)) a pair's bucket is the number of borders <= dist, plus
 * n_borders + 1 when two_sided and j > p_i:
 *
 *     s_ij  = scale q_i . k_j + bias[bucket][h]
 *     lse_i = log sum_j exp s_ij,  out_i = sum_j exp(s_ij - lse_i) v_j
 *
 * and the backward pass, which forms the probabilities again from lse:
 *
 *     P_ij = exp(s_ij - lse_i),  dS_ij = P_ij (dout_i . v_j - dout_i . out_i)
 *     dq = scale dS k,  dk = scale dS^T q,  dv = P^T dout (dk and dv summed
 *     over the query heads that share them), dbias[n][h] = the sum of dS
 *     over the batch and the pairs of bucket n
 *
 * q, out, dout, dq : [batch, len_q, heads, dim];  k, v, dk, dv : [batch,
 *   len_k, kv_heads, dim], all of `dtype`, dim contiguous, data 16-byte
 *   aligned and strides (in elements, >= 0) multiples of 16 bytes; a
 *   stride_row of at most 2^30 / 128 bytes.
 * lse  : [batch, heads, len_q] float32, contiguous.
 * bias, dbias : [buckets, heads] float32, buckets = (n_borders + 1) times 2
 *   when two_sided, at most 128; bias NULL for none (then dbias is NULL and
 *   the borders are not read), else dbias must be given.
 * borders : HOST array, ascending, the first >= 1.
 * 8 <= dim <= 128, a multiple of 8; heads a multiple of kv_heads; scale > 0;
 * batch and lengths may be 0.  The outputs must not overlap anything else.
 *
 * Scores, statistics and all sums are float32; P and dS enter their products
 * in `dtype` (float32 products run on the float32 matrix cores); dbias sums
 * the float32 dS.  In bfloat16, the scores that dk and dv are formed from are
 * summed from -lse_i on, so they round at lse_i's size.  A query that sees no key gets out = 0, lse = -infinity
 * and gradients 0.  Keys at and past lens[b] are not read, and their dk and dv are 0.
 * A NaN or infinity in a key or value may also reach queries from which only
 * `causal` hides it.  Results are deterministic.
 */
#define KFAC_MAX_LENGTH (1 << 24)
typedef struct {
    int64_t batch, len_q, len_k;
    int32_t heads, kv_heads, dim;
    int32_t causal;
    float scale;
    int32_t n_borders, two_sided;
    const int32_t* borders; /* host */
    const int32_t* lens;    /* device [batch] or NULL */
    const float* bias;      /* device or NULL */
} kfac_attention_t;

typedef struct {
    void* data;
    int64_t stride_batch, stride_row, stride_head;
} kfac_tensor4_t;

/* Bytes of workspace of a forward (backward = 0) or backward call; 0 when it
 * needs none (workspace may then be NULL), SIZE_MAX when the form is refused. */
size_t kfac_attention_workspace_size(const kfac_attention_t* form, kfac_dtype_t dtype, int backward);
kfac_status_t kfac_attention_forward(const kfac_attention_t* form, kfac_dtype_t dtype, const kfac_tensor4_t* q,
                                     const kfac_tensor4_t* k, const kfac_tensor4_t* v, const kfac_tensor4_t* out,
                                     float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream);
kfac_status_t kfac_attention_backward(const kfac_attention_t* form, kfac_dtype_t dtype, const kfac_tensor4_t* q,
                                      const kfac_tensor4_t* k, const kfac_tensor4_t* v, const kfac_tensor4_t* out,
                                      const float* lse, const kfac_tensor4_t* dout, const kfac_tensor4_t* dq,
                                      const kfac_tensor4_t* dk, const kfac_tensor4_t* dv, float* dbias, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------ checkpoints --
 * A layer's input kept in 8 bits from the forward to the backward pass, for
 * the two products that need it there: the factor A and the gradient
 * [dW | db] (the page computes A from the layer's input in the forward
 * pre-hook; pipelining paragraph).  Both sum over rows, so 32 consecutive
 * rows of a column share a power of two:
 *
 *     e = the least integer >= -117 with |x| <= 448 2^e over the block
 *     code = x 2^-e as e4m3, to nearest even;  x^ = code 2^e
 *
 * codes[l]  : [ceil(rows / 32), d_a, 32] bytes, 16-byte aligned, element r of
 *             block b holding row 32 b + r (rows past the end are 0);
 * scales[l] : [ceil(rows / 32), d_a] bytes, e + 127.
 * NaN and infinities become NaN codes and do not count for e.  x^ is exactly
 * a bfloat16 number (but for magnitudes that round past the largest one,
 * which become infinite).
 *
 * store   : x[l] [rows, d] in `dtype` -> codes, scales with d_a = d + ones;
 *           ones = 1 adds a column of ones (the layer has a bias).
 * load    : y[l] [rows, cols] in `dtype` = the first cols <= d columns of x^.
 * factors : M <- F (first_step) or eps M + (1 - eps) F, F = x^^T x^ / rows,
 *           upper triangle of m[l] [d, d] as in kfac_factors.
 * grad    : mat[l] [d_out, d] float32 = g[l]^T x^, g[l] [rows, d_out] in
 *           `dtype`; with a column of ones the last column is the bias
 *           gradient, as kfac_precondition takes it.  float32 gradients enter
 *           as three bf16 parts, which add up to them from 2^-103 in magnitude
 *           on; below, up to 2^-125 of a gradient may be lost.
 * The workspace sizes of factors and grad are 0 where the call needs none
 * (workspace may then be NULL) and SIZE_MAX where the sizes are refused.
 * In load, factors and grad, d counts the checkpoint's columns.  The products
 * (of a gradient's parts) are exact and summed in float32.  Results are
 * deterministic; outputs must not overlap inputs.
 */
kfac_status_t kfac_checkpoint_store(int n, const void* const* x, const int64_t* rows, const int64_t* d, int ones,
                                    kfac_dtype_t dtype, uint8_t* const* codes, uint8_t* const* scales,
                                    hipStream_t stream);
kfac_status_t kfac_checkpoint_load(int n, const uint8_t* const* codes, const uint8_t* const* scales, const int64_t* rows,
                                   const int64_t* d, const int64_t* cols, kfac_dtype_t dtype, void* const* y,
                                   hipStream_t stream);
size_t kfac_checkpoint_factors_workspace_size(int n, const int64_t* rows, const int64_t* d);
kfac_status_t kfac_checkpoint_factors(int n, const uint8_t* const* codes, const uint8_t* const* scales,
                                      const int64_t* rows, const int64_t* d, float* const* m, float eps, int first_step,
                                      void* workspace, size_t workspace_bytes, hipStream_t stream);
size_t kfac_checkpoint_grad_workspace_size(int n, const int64_t* rows, const int64_t* d_out, const int64_t* d);
kfac_status_t kfac_checkpoint_grad(int n, const void* const* g, const uint8_t* const* codes,
                                   const uint8_t* const* scales, const int64_t* rows, const int64_t* d_out,
                                   const int64_t* d, kfac_dtype_t dtype, float* const* mat, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream);

/* -------------------------------------------------------------- layer norm --
 * Layer norm over the rows of a matrix, and its backward pass:
 *
 *     mean = sum x / d,  rstd = 1 / sqrt(sum (x - mean)^2 / d + eps)
 *     xh = (x - mean) rstd,  y = weight xh + bias
 *     a = weight dy,  dx = rstd (a - mean(a) - xh mean(a xh))
 *     dweight = sum over rows of dy xh,  dbias = sum over rows of dy
 *
 * x, y, dy, dx : [rows, d] in `dtype`, the elements of a row contiguous, rows
 *   x_stride (y_stride, ...) >= d elements apart.
 * mean, rstd   : [rows] float32; forward they may be NULL.
 * weight, bias, dweight, dbias : [d] in `weight_dtype`, KFAC_F32 or `dtype`;
 *   weight NULL: 1, bias NULL: 0.  An output (dx, dweight, dbias) that is NULL
 *   is not formed.
 * 0 <= rows <= 2^31 - 1, 1 <= d <= KFAC_MAX_DIM, eps >= 0 and finite.  The
 * backward pass needs its workspace for dweight and dbias only; they are 0
 * where there are no rows.  Statistics and sums are float32, the variance
 * summed around the mean.  Pointers need the alignment of their type only.
 * Results are deterministic.  Outputs must not overlap inputs or each other.
 */
kfac_status_t kfac_layer_norm_forward(int64_t rows, int64_t d, kfac_dtype_t dtype, const void* x, int64_t x_stride, void* y,
                                      int64_t y_stride, float* mean, float* rstd, const void* weight, const void* bias,
                                      kfac_dtype_t weight_dtype, float eps, hipStream_t stream);
size_t kfac_layer_norm_workspace_size(int64_t rows, int64_t d);
kfac_status_t kfac_layer_norm_backward(int64_t rows, int64_t d, kfac_dtype_t dtype, const void* dy, int64_t dy_stride,
                                       const void* x, int64_t x_stride, const float* mean, const float* rstd,
                                       const void* weight, void* dx, int64_t dx_stride, void* dweight, void* dbias,
                                       kfac_dtype_t weight_dtype, void* workspace, size_t workspace_bytes,
                                       hipStream_t stream);

/* ------------------------------------------------------------------ gated --
 * The gated feed-forward block: both projections of its input, the
 * activation of the one and its product with the other, and the backward pass:
 *
 *     [g | u] = x weight^T + bias,  h = act(g) u
 *     dpre = [dh u act'(g) | dh act(g)]
 *     dx = dpre weight,  dweight = dpre^T x,  dbias = sum over rows of dpre
 *
 * x, dx     : [rows, d] in `dtype`;  h, dh : [rows, width] in `dtype`
 * pre, dpre : [rows, 2 width] in `dtype`, g (gate) in front of u (up).  pre,
 *             as rounded, is what the backward pass goes by; forward it may be
 *             NULL.  dpre, always written, is the output gradient of the joint
 *             layer [gate; up], the rows of its factor G.
 * weight    : [2 width, d] in `dtype`, the gate's rows first
 * dweight   : [2 width, d] in `dweight_dtype`, KFAC_F32 or `dtype`
 * bias, dbias : [2 width] float32; bias NULL: 0
 * An output (dx, dweight, dbias) that is NULL is not formed; x is read for
 * dweight only, weight for dx only.  0 <= rows <= 2^31 - 1, 1 <= d, width <=
 * KFAC_MAX_DIM (KFAC_ERR_UNSUPPORTED where a product would need 2^32 threads,
 * which begins at 2^30 rows).  All contiguous; x, weight and dpre 4-byte
 * aligned.
 *
 * bfloat16 products are exact and summed in float32.  dpre enters dx and
 * dweight as it is given out, and how it is given out is the caller's choice:
 * kfac_gated_backward rounds that of bfloat16 rows to bfloat16, at one product
 * each (half a step of bfloat16 for each term, which leaves the gradients some
 * 1.4 times as far off as their own rounding does); kfac_gated_backward_f32
 * gives it out and multiplies it in float32, as three exact parts, at three.
 * dbias is summed before dpre is rounded.  float32 operands enter as three
 * bfloat16 parts that add up to them (parts under 2^-126 may be lost) and six
 * products of these, with float32 rounding, or, forward with few rows, as they
 * are; an infinity makes a sum that it enters infinite or NaN.  Activations:
 * SILU g / (1 + exp(-g)), GELU g Phi(g) with the normal distribution's Phi,
 * GELU_TANH its approximation g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2,
 * RELU max(g, 0) with slope 0 at 0, SIGMOID 1 / (1 + exp(-g)).  Results are
 * deterministic.  Outputs must not overlap inputs or each other.
 */
typedef enum {
    KFAC_ACT_SILU = 0,
    KFAC_ACT_GELU = 1,
    KFAC_ACT_GELU_TANH = 2,
    KFAC_ACT_RELU = 3,
    KFAC_ACT_SIGMOID = 4
} kfac_act_t;

/* Bytes of workspace of kfac_gated_forward (backward = 0), kfac_gated_backward
 * (1) or kfac_gated_backward_f32 (2; of KFAC_BF16 rows); SIZE_MAX where the
 * sizes are refused, 0 where it needs none. */
size_t kfac_gated_workspace_size(int64_t rows, int64_t d, int64_t width, kfac_dtype_t dtype, int backward);
kfac_status_t kfac_gated_forward(int64_t rows, int64_t d, int64_t width, kfac_dtype_t dtype, kfac_act_t act, const void* x,
                                 const void* weight, const float* bias, void* h, void* pre, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream);
kfac_status_t kfac_gated_backward(int64_t rows, int64_t d, int64_t width, kfac_dtype_t dtype, kfac_act_t act, const void* dh,
                                  const void* x, const void* weight, const void* pre, void* dpre, void* dx, void* dweight,
                                  kfac_dtype_t dweight_dtype, float* dbias, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream);
/* dtype KFAC_BF16, with dpre [rows, 2 width] in float32. */
kfac_status_t kfac_gated_backward_f32(int64_t rows, int64_t d, int64_t width, kfac_act_t act, const void* dh, const void* x,
                                      const void* weight, const void* pre, float* dpre, void* dx, void* dweight,
                                      kfac_dtype_t dweight_dtype, float* dbias, void* workspace, size_t workspace_bytes,
                                      hipStream_t stream);

/* ----------------------------------------------------------- gradient norm --
 * The norm of many gradients taken together, and clipping to a largest norm:
 *
 *     norm   = sqrt(sum over all tensors of g[i]^2)
 *     out[i] = c g[i],  c = min(1, max_norm / (norm + 1e-6))
 *
 * g[i], out[i] : count[i] >= 0 contiguous elements of dtype[i] (HOST arrays;
 *   a tensor without elements may be NULL); out[i] may be g[i] itself.  Apart
 *   from that no two of the tensors may overlap, g[i] twice included
 *   (KFAC_ERR_INVALID_VALUE).
 * norm : DEVICE float32, one element, apart from the tensors (kfac_grad_clip
 *   refuses one that is not).
 * max_norm >= 0, infinity included.  1 <= n <= KFAC_MAX_COUNT, count[i] <=
 * 2^37.  Squares are summed in float64, so that they neither overflow nor
 * vanish, in a fixed order: results are deterministic.  A norm that is not a
 * finite number scales as the formula says: infinity by 0 (infinities then
 * become NaN), NaN by NaN.
 */
size_t kfac_grad_norm_workspace_size(int n);
kfac_status_t kfac_grad_norm(int n, const void* const* g, const int64_t* count, const kfac_dtype_t* dtype, float* norm,
                             void* workspace, size_t workspace_bytes, hipStream_t stream);
kfac_status_t kfac_grad_clip(int n, const void* const* g, void* const* out, const int64_t* count, const kfac_dtype_t* dtype,
                             float max_norm, float* norm, void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KFAC_H */
