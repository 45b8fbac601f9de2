/*
 * miconv.h -- C ABI of libmiconv, the 2-D convolution forward pass (FPROP)
 * its data and filter gradients, pooling, and the feed-forward operators
 * (norm, linear and gated layers with their gradients), for AMD Instinct
 * MI355X (gfx950).
 *
 * The operation (direct convolution, cross-correlation form, zero padding):
 *
 *   y[n,k,p,q] = alpha * sum_{c,r,s} X(n, c, p*u + r - pad_top, q*v + s - pad_left) * F[k,c,r,s]
 *              + beta  * y[n,k,p,q]
 *
 *   X(n,c,h,w) = x[n*sn + c*sc + h*sh + w*sw] inside 0 <= h < H, 0 <= w < W, else 0
 *   P = floor((H + pad_top + pad_bottom - R) / u) + 1
 *   Q = floor((W + pad_left + pad_right - S) / v) + 1
 *
 * Sources: cuDNN page (Chetlur et al., "cuDNN: Efficient Primitives for Deep
 * Learning"), "Proposed Method": a C API over opaque tensor and filter
 * descriptors with arbitrary strides and layouts, single and double
 * precision, user-owned GPU memory and no auxiliary buffers, non-square
 * inputs and asymmetric padding.  maxDNN page (Lavin), "Proposed Method":
 * each output coordinate is the product of the input receptive field with
 * the filter weights.  Zero-memory direct-convolution page (Zhang, Franchetti
 * et al.), Abstract and "Proposed Method": computed directly, without packing
 * or copying, with no memory beyond the operands.
 *
 * Conventions for every call:
 *   - Every call returns a mic_status; nothing is thrown across the ABI.
 *   - Descriptors and handles are host objects owned by the caller (create /
 *     destroy).  They hold no device memory.
 *   - Data pointers are device pointers owned by the caller.  The library
 *     never allocates, frees or keeps device memory: there is no workspace
 *     (the feed-forward operators take the caller's).
 *   - Strides are counted in elements, not bytes, and must be >= 1.
 *   - Not thread-safe per handle: one handle, one host thread at a time.
 */
#ifndef MICONV_H
#define MICONV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MICONV_VERSION_MAJOR 0
#define MICONV_VERSION_MINOR 1
#define MICONV_VERSION_PATCH 0

typedef enum {
    MIC_STATUS_SUCCESS = 0,
    MIC_STATUS_BAD_PARAM = 1,       /* null pointer, bad dimension/stride, shape mismatch */
    MIC_STATUS_NOT_SUPPORTED = 2,   /* valid request this library does not implement */
    MIC_STATUS_LAUNCH_FAILED = 3,   /* the HIP runtime refused a kernel launch */
    MIC_STATUS_INTERNAL_ERROR = 4,  /* HIP runtime error outside a launch (device query) */
    MIC_STATUS_ALLOC_FAILED = 5     /* host allocation of a handle or descriptor failed */
} mic_status;

/* Element types.  Allowed (x, w, y) combinations: (F32, F32, F32),
 * (F64, F64, F64) and (BF16, BF16, F32) (bf16 inputs, fp32 accumulation and
 * output).  Anything else is MIC_STATUS_NOT_SUPPORTED. */
typedef enum {
    MIC_DTYPE_F32 = 0,
    MIC_DTYPE_F64 = 1,
    MIC_DTYPE_BF16 = 2,
    MIC_DTYPE_F8_E4M3 = 3           /* e4m3 without infinities, the feed-forward operators only */
} mic_dtype;

/* Packed layouts for mic_tensor_desc_set_packed.  Any other layout is given
 * through explicit strides with mic_tensor_desc_set. */
typedef enum {
    MIC_LAYOUT_NCHW = 0,
    MIC_LAYOUT_NHWC = 1
} mic_layout;

typedef struct mic_handle_st* mic_handle;
typedef struct mic_tensor_desc_st* mic_tensor_desc;
typedef struct mic_filter_desc_st* mic_filter_desc;
typedef struct mic_conv_desc_st* mic_conv_desc;

/* Static, never-NULL text for a status (unknown values give "unknown status"). */
const char* mic_status_string(mic_status status);

/* Library version; any pointer may be NULL. */
mic_status mic_get_version(int* major, int* minor, int* patch);

/* ---------------------------------------------------------------- handle */

/* Binds the calling thread's current HIP device and the null stream.
 * Queries the device (compute-unit count, architecture); fails with
 * MIC_STATUS_INTERNAL_ERROR when no HIP device is usable and with
 * MIC_STATUS_NOT_SUPPORTED on a device other than gfx950.  No device memory
 * is allocated. */
mic_status mic_create(mic_handle* handle);
mic_status mic_destroy(mic_handle handle);

/* stream is a hipStream_t (NULL = the null stream).  Later calls on this
 * handle enqueue their kernels on it.  The caller keeps the stream alive. */
mic_status mic_set_stream(mic_handle handle, void* stream);
mic_status mic_get_stream(mic_handle handle, void** stream);

/* ---------------------------------------------------------------- tensor descriptor */

mic_status mic_tensor_desc_create(mic_tensor_desc* desc);
mic_status mic_tensor_desc_destroy(mic_tensor_desc desc);

/* Logical N, C, H, W with element strides sn, sc, sh, sw (any order, any
 * gaps: NCHW, NHWC, padded rows and sub-tensor views all fit).  Dimensions
 * and strides must be >= 1, else MIC_STATUS_BAD_PARAM. */
mic_status mic_tensor_desc_set(mic_tensor_desc desc, mic_dtype dtype,
                               int n, int c, int h, int w,
                               int64_t sn, int64_t sc, int64_t sh, int64_t sw);

/* Same, with the strides of a packed NCHW or NHWC tensor. */
mic_status mic_tensor_desc_set_packed(mic_tensor_desc desc, mic_dtype dtype, mic_layout layout,
                                      int n, int c, int h, int w);

/* Read back; any output pointer may be NULL.  strides receives 4 values
 * (sn, sc, sh, sw).  MIC_STATUS_BAD_PARAM if the descriptor was never set. */
mic_status mic_tensor_desc_get(mic_tensor_desc desc, mic_dtype* dtype,
                               int* n, int* c, int* h, int* w, int64_t* strides);

/* Channel-blocked tensor (zero-memory direct-convolution page, "Proposed
 * Method": input and output feature maps in a blocked layout that takes
 * exactly the memory of standard storage): packed [N][C/cb][H][W][cb], so
 * element (n, c, h, w) sits at
 *   n*C*H*W + (c / cb)*H*W*cb + h*W*cb + w*cb + (c % cb).
 * c must be a multiple of cb (no padding channels), cb >= 1, else
 * MIC_STATUS_BAD_PARAM.  Accepted by mic_conv_forward for x and y, any cb:
 * the tap-batched kernels read blocked x when cb is a multiple of their
 * channel chunk (2 or 4 channels fp32/fp64, 16 bf16), the row-streamed
 * kernel (11-wide filter rows) when it is a multiple of 4 and x is 16-byte
 * aligned, the gather kernel's tap order when it is a multiple of 16 (32
 * bf16); other blockings run the gather kernel's flat order or the direct
 * kernel.  The other operations
 * return MIC_STATUS_NOT_SUPPORTED for blocked descriptors.
 * mic_tensor_desc_set / _set_packed reset a descriptor to unblocked. */
mic_status mic_tensor_desc_set_blocked(mic_tensor_desc desc, mic_dtype dtype, int n, int c, int h, int w,
                                       int cb);

/* Channel block cb (0 for an unblocked descriptor) and the element stride
 * between channel blocks; either pointer may be null.  MIC_STATUS_BAD_PARAM
 * if the descriptor was never set. */
mic_status mic_tensor_desc_get_block(mic_tensor_desc desc, int* cb, int64_t* block_stride);

/* ---------------------------------------------------------------- filter descriptor */

mic_status mic_filter_desc_create(mic_filter_desc* desc);
mic_status mic_filter_desc_destroy(mic_filter_desc desc);

/* K filters of C channels and R x S taps, packed K,C,R,S (S fastest).
 * Dimensions must be >= 1. */
mic_status mic_filter_desc_set(mic_filter_desc desc, mic_dtype dtype, int k, int c, int r, int s);
mic_status mic_filter_desc_get(mic_filter_desc desc, mic_dtype* dtype, int* k, int* c, int* r, int* s);

/* Blocked filters (zero-memory direct-convolution page, "Proposed Method":
 * kernel weights in a blocked layout of the same size as standard storage):
 * [K/kb][C/cb][R][S][cb][kb], so F[k, c, r, s] sits at
 *   ((k/kb)*(C/cb) + c/cb)*R*S*cb*kb + ((r*S + s)*cb + c%cb)*kb + k%kb.
 * k must be a multiple of kb and c of cb (kb, cb >= 1), else
 * MIC_STATUS_BAD_PARAM.  Forward pass only, as for blocked tensors: the
 * tap-batched kernels read them when cb is a multiple of their channel
 * chunk and kb of 4 (fp32), 2 (fp64) or 8 (bf16, cb a multiple of 16) with
 * w 16-byte aligned, the row-streamed kernel tap by tap, the gather kernel
 * when cb is a multiple of 16 (32 bf16), else the direct kernel runs.
 * mic_filter_desc_set resets a descriptor to packed KCRS. */
mic_status mic_filter_desc_set_blocked(mic_filter_desc desc, mic_dtype dtype, int k, int c, int r, int s,
                                       int kb, int cb);

/* Filter blocks kb, cb (0, 0 for packed KCRS); either pointer may be null.
 * MIC_STATUS_BAD_PARAM if the descriptor was never set. */
mic_status mic_filter_desc_get_block(mic_filter_desc desc, int* kb, int* cb);

/* ---------------------------------------------------------------- convolution descriptor */

mic_status mic_conv_desc_create(mic_conv_desc* desc);
mic_status mic_conv_desc_destroy(mic_conv_desc desc);

/* Per-side zero padding (>= 0) and stride u along H, v along W (>= 1).
 * No dilation, no groups, no filter flip. */
mic_status mic_conv_desc_set(mic_conv_desc desc, int pad_top, int pad_bottom,
                             int pad_left, int pad_right, int stride_h, int stride_w);
mic_status mic_conv_desc_get(mic_conv_desc desc, int* pad_top, int* pad_bottom,
                             int* pad_left, int* pad_right, int* stride_h, int* stride_w);

/* ---------------------------------------------------------------- forward */

/* Output dimensions (N, K, P, Q).  Host only, no device needed.
 * MIC_STATUS_BAD_PARAM if a descriptor is unset, the channel counts differ,
 * or the output would be empty (P < 1 or Q < 1). */
mic_status mic_conv_forward_output_dim(mic_conv_desc conv, mic_tensor_desc x_desc,
                                       mic_filter_desc w_desc, int* n, int* k, int* p, int* q);

/* y <- alpha * conv(x, w) + beta * y, on the handle's stream, asynchronously.
 *
 * x: device memory described by x_desc; w: packed K,C,R,S device memory;
 * y: device memory described by y_desc, whose dims must equal the output
 * dims.  alpha and beta are rounded to the accumulation type (fp32 for F32
 * and BF16 inputs, fp64 for F64).  With beta == 0, y is only written (its
 * old contents, NaN included, never reach the result).
 *
 * No workspace: nothing is allocated.  The return value covers validation
 * and the launch only; execution errors surface at the next synchronisation.
 * y must not overlap x or w, and y's strides must not map two outputs to one
 * address (neither is checked).  Tensors whose highest element offset
 * reaches 2^31 are MIC_STATUS_NOT_SUPPORTED.
 *
 * Errors: MIC_STATUS_BAD_PARAM (null handle/descriptor/pointer, unset
 * descriptor, shape mismatch), MIC_STATUS_NOT_SUPPORTED (dtype combination,
 * size limit), MIC_STATUS_LAUNCH_FAILED. */
mic_status mic_conv_forward(mic_handle handle, double alpha,
                            mic_tensor_desc x_desc, const void* x,
                            mic_filter_desc w_desc, const void* w,
                            mic_conv_desc conv, double beta,
                            mic_tensor_desc y_desc, void* y);

/* Name of the kernel variant mic_conv_forward would launch for these
 * descriptors (host only; for profiling and reports).  Writes a NUL-
 * terminated string of at most buflen bytes; MIC_STATUS_BAD_PARAM if the
 * descriptors are invalid or buflen is too small. */
mic_status mic_conv_forward_kernel_name(mic_handle handle, mic_tensor_desc x_desc,
                                        mic_filter_desc w_desc, mic_conv_desc conv,
                                        mic_tensor_desc y_desc, char* buf, size_t buflen);

/* ---------------------------------------------------------------- data gradient */

/* dx <- alpha * dgrad(dy, w) + beta * dx: the backward pass with respect to
 * the input, i.e. the adjoint of the forward sum in x,
 *
 *   dx[n,c,h,w] = alpha * sum_{k,r,s} dY(n, k, p, q) * F[k,c,r,s]
 *                 over p*u = h + pad_top - r (0 <= p < P),
 *                      q*v = w + pad_left - s (0 <= q < Q)
 *               + beta * dx[n,c,h,w]
 *
 * on the handle's stream, asynchronously.  The cuDNN page ("Proposed
 * Method") names forward and backward routines and the maxDNN page
 * (Abstract, RQ4) the backward pass, without a formula; this is the plain
 * reading.
 *
 * The geometry is the forward problem's: dx_desc plays x (N, C, H, W),
 * w_desc the packed K,C,R,S filter, conv its padding and strides, and
 * dy_desc must have the forward output dims (N, K, P, Q).  Element types
 * (dy, w, dx): (F32, F32, F32), (F64, F64, F64), (BF16, BF16, F32).  dy and
 * dx are device memory with any element strides; alpha, beta, beta == 0,
 * ownership, overlap and size rules as for mic_conv_forward.  No workspace.
 *
 * Errors: MIC_STATUS_BAD_PARAM (null handle/descriptor/pointer, unset
 * descriptor, dy dims not the forward output dims), MIC_STATUS_NOT_SUPPORTED
 * (dtype combination, size limit), MIC_STATUS_LAUNCH_FAILED. */
mic_status mic_conv_backward_data(mic_handle handle, double alpha,
                                  mic_filter_desc w_desc, const void* w,
                                  mic_tensor_desc dy_desc, const void* dy,
                                  mic_conv_desc conv, double beta,
                                  mic_tensor_desc dx_desc, void* dx);

/* Name of the kernel variant mic_conv_backward_data would launch (host
 * only), as mic_conv_forward_kernel_name. */
mic_status mic_conv_backward_data_kernel_name(mic_handle handle, mic_filter_desc w_desc,
                                              mic_tensor_desc dy_desc, mic_conv_desc conv,
                                              mic_tensor_desc dx_desc, char* buf, size_t buflen);

/* ---------------------------------------------------------------- filter gradient */

/* dw <- alpha * wgrad(x, dy) + beta * dw: the backward pass with respect to
 * the filter, i.e. the adjoint of the forward sum in F,
 *
 *   dw[k,c,r,s] = alpha * sum_{n,p,q} dY(n, k, p, q) * X(n, c, p*u + r - pad_top, q*v + s - pad_left)
 *               + beta * dw[k,c,r,s]
 *
 * on the handle's stream, asynchronously (same reading of the pages as
 * mic_conv_backward_data).  The geometry is the forward problem's: x_desc
 * the input, dw_desc the packed K,C,R,S filter (its dtype is the output's),
 * conv the padding and strides; dy_desc must have the forward output dims
 * (N, K, P, Q).  Element types (x, dy, dw): (F32, F32, F32), (F64, F64,
 * F64), (BF16, BF16, F32).  x and dy with any element strides; dw packed.
 * alpha, beta, ownership and size rules as for mic_conv_forward.  No
 * workspace: the reduction over N*P*Q positions is split across at most two
 * workgroups.  With beta == 0 and dw tiles too few to fill the GPU, the call
 * first zeroes dw, then two workgroups per tile add alpha times their
 * partial sums into it with atomic adds; two terms added onto zero give the
 * same bits in either order, so the result is still deterministic (reruns
 * and any workgroup order bit-identical).  dw's prior contents are not read
 * when beta == 0.
 *
 * Errors: MIC_STATUS_BAD_PARAM (null handle/descriptor/pointer, unset
 * descriptor, dy dims not the forward output dims), MIC_STATUS_NOT_SUPPORTED
 * (dtype combination, size limit), MIC_STATUS_LAUNCH_FAILED. */
mic_status mic_conv_backward_filter(mic_handle handle, double alpha,
                                    mic_tensor_desc x_desc, const void* x,
                                    mic_tensor_desc dy_desc, const void* dy,
                                    mic_conv_desc conv, double beta,
                                    mic_filter_desc dw_desc, void* dw);

/* Name of the kernel variant mic_conv_backward_filter would launch (host
 * only), as mic_conv_forward_kernel_name. */
mic_status mic_conv_backward_filter_kernel_name(mic_handle handle, mic_tensor_desc x_desc,
                                                mic_tensor_desc dy_desc, mic_conv_desc conv,
                                                mic_filter_desc dw_desc, char* buf, size_t buflen);

/* ---------------------------------------------------------------- pooling */

/* Pooling forward pass (cuDNN page, "Proposed Method": pooling among the
 * library's routines; no formula printed, so the plain reading):
 *
 *   MIC_POOL_MAX:             max of X over the window positions inside the
 *                             H x W plane (padding never wins; 0 if none)
 *   MIC_POOL_AVG_INCLUDE_PAD: (sum of X over the positions inside) / (R*S)
 *   MIC_POOL_AVG_EXCLUDE_PAD: (sum over the positions inside) / (their
 *                             number; 0 if none)
 *   y[n,c,p,q] = alpha * that + beta * y[n,c,p,q]
 *
 * The window geometry is the convolution's: R x S window at (p*u - pad_top,
 * q*v - pad_left), output size by the same floor rule.  Channels are pooled
 * independently. */
typedef enum {
    MIC_POOL_MAX = 0,
    MIC_POOL_AVG_INCLUDE_PAD = 1,
    MIC_POOL_AVG_EXCLUDE_PAD = 2
} mic_pool_mode;

typedef struct mic_pool_desc_st* mic_pool_desc;

mic_status mic_pool_desc_create(mic_pool_desc* desc);
mic_status mic_pool_desc_destroy(mic_pool_desc desc);

/* Mode, window (>= 1), per-side padding (>= 0), strides (>= 1); else
 * MIC_STATUS_BAD_PARAM. */
mic_status mic_pool_desc_set(mic_pool_desc desc, mic_pool_mode mode, int window_h, int window_w,
                             int pad_top, int pad_bottom, int pad_left, int pad_right,
                             int stride_h, int stride_w);
mic_status mic_pool_desc_get(mic_pool_desc desc, mic_pool_mode* mode, int* window_h, int* window_w,
                             int* pad_top, int* pad_bottom, int* pad_left, int* pad_right,
                             int* stride_h, int* stride_w);

/* Output dims (N, C, P, Q), host only; MIC_STATUS_BAD_PARAM if a descriptor
 * is unset or the window exceeds the padded input. */
mic_status mic_pool_forward_output_dim(mic_pool_desc pool, mic_tensor_desc x_desc,
                                       int* n, int* c, int* p, int* q);

/* y <- alpha * pool(x) + beta * y on the handle's stream, asynchronously.
 * Element types (x, y): (F32, F32), (F64, F64), (BF16, F32).  x and y with
 * any element strides; y's dims must equal the output dims.  Ownership,
 * alpha/beta, beta == 0 and size rules as for mic_conv_forward.  No
 * workspace.  Errors: MIC_STATUS_BAD_PARAM (null handle/descriptor/pointer,
 * unset descriptor, shape mismatch), MIC_STATUS_NOT_SUPPORTED (dtype
 * combination, size limit), MIC_STATUS_LAUNCH_FAILED. */
mic_status mic_pool_forward(mic_handle handle, double alpha, mic_pool_desc pool,
                            mic_tensor_desc x_desc, const void* x, double beta,
                            mic_tensor_desc y_desc, void* y);

/* ------------------------------------------------------------------ batch-reduce GEMM
 *
 * Single-building-block page (Georganas et al.), "Proposed Method": the
 * batch-reduce GEMM multiplies a batch of A blocks by a batch of B blocks
 * and reduces all products into one C block:
 *
 *   C[i_m, i_n] <- alpha * sum_{i < batch} sum_{i_k < k} A_i[i_m, i_k] * B_i[i_k, i_n]
 *                  + beta * C[i_m, i_n]
 *
 * with A_i[i_m, i_k] = a[i*a_stride_batch + i_m*a_stride_m + i_k*a_stride_k],
 * B_i[i_k, i_n] = b[i*b_stride_batch + i_k*b_stride_k + i_n*b_stride_n] and
 * C[i_m, i_n] = c[i_m*c_stride_m + i_n*c_stride_n], strides in elements.
 * A fully-connected layer is one block product (batch 1, k = input
 * features) or its input features cut into batch blocks.
 *
 * Element types: dtype MIC_DTYPE_F32 (A, B, C fp32), MIC_DTYPE_F64 (all
 * fp64), MIC_DTYPE_BF16 (A, B bf16, C fp32, fp32 accumulation).  a, b, c are
 * device pointers owned by the caller, aligned to their element size; the
 * call is asynchronous on the handle's stream and keeps no reference.
 * beta == 0 writes C without reading it (NaN-safe).  m == 0 or n == 0 is a
 * no-op; k == 0 or batch == 0 gives C <- beta * C (a, b may then be null).
 * C must not overlap A or B; distinct (i_m, i_n) must have distinct C
 * offsets.  No workspace.  Errors: MIC_STATUS_BAD_PARAM (null handle or
 * needed pointer, negative size or stride, misaligned pointer, aliased C
 * elements), MIC_STATUS_NOT_SUPPORTED (unknown dtype, an operand's highest
 * element offset or batch*k reaching 2^30), MIC_STATUS_LAUNCH_FAILED. */
mic_status mic_brgemm(mic_handle handle, mic_dtype dtype, int m, int n, int k, int batch, double alpha,
                      const void* a, int64_t a_stride_batch, int64_t a_stride_m, int64_t a_stride_k,
                      const void* b, int64_t b_stride_batch, int64_t b_stride_k, int64_t b_stride_n,
                      double beta, void* c, int64_t c_stride_m, int64_t c_stride_n);

/* Name of the kernel variant mic_brgemm would launch for these sizes and
 * strides (pointers taken as 16-byte aligned), host only, NUL-terminated
 * into buf of buflen bytes; errors as mic_brgemm's size and stride checks,
 * MIC_STATUS_BAD_PARAM if the name does not fit. */
mic_status mic_brgemm_kernel_name(mic_handle handle, mic_dtype dtype, int m, int n, int k, int batch,
                                  int64_t a_stride_batch, int64_t a_stride_m, int64_t a_stride_k,
                                  int64_t b_stride_batch, int64_t b_stride_k, int64_t b_stride_n,
                                  int64_t c_stride_m, int64_t c_stride_n, char* buf, size_t buflen);

/* ------------------------------------------------------------------ feed-forward operators
 *
 * A feed-forward sublayer, as it is trained and served: the root-mean-square
 * norm with the residual's addition, linear layers with bias, activation and
 * residual in the product's epilogue, gated layers, and their gradients.
 *
 * All matrices are row-major with a row pitch in elements (ld... >= the row's
 * length) and consecutive elements within a row; vectors and scales are
 * packed.  Pointers need their element's alignment and no more; 16-byte
 * aligned rows run faster.  Offsets are 64 bits wide.  Sums, statistics and
 * activations are fp32; a result is rounded once, to its tensor's type, to
 * nearest even.  Zero rows are a no-op, a zero reduction length gives sums of
 * zero.  Outputs must not overlap inputs or each other (not checked).
 *
 * Workspaces are the caller's device memory, 16-byte aligned, of at least the
 * bytes the matching ..._workspace call (host only) returns for the same sizes
 * and handle, or without a handle, which answers for an MI355X whole or in any
 * of its partitions; their contents need no preparation and nothing in them
 * survives a call.  Those bytes are enough for rows at any alignment, which may
 * have to be copied; ..._workspace_aligned returns what a call needs, often
 * nothing, whose operands' pointers and pitches are all multiples of 16 bytes
 * with pitches below 4 MB (and w_gate's that of w_up).  Calls are asynchronous on the handle's stream and may be captured
 * into graphs.  Results do not depend on workgroup order: no atomics.
 *
 * Errors: MIC_STATUS_BAD_PARAM (null handle or needed pointer, negative size,
 * pitch below the row's length, misaligned pointer, workspace too small),
 * MIC_STATUS_NOT_SUPPORTED (element type or activation, a size reaching 2^30,
 * a row pitch of 2^23 bytes or more, more outputs than a launch of 128 x 128
 * tiles reaches, about 2^38), MIC_STATUS_LAUNCH_FAILED. */
typedef enum {
    MIC_ACT_NONE = 0,
    MIC_ACT_RELU = 1,
    MIC_ACT_GELU = 2,        /* z Phi(z), Phi the normal distribution function */
    MIC_ACT_GELU_TANH = 3,   /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
    MIC_ACT_SILU = 4         /* z / (1 + e^-z) */
} mic_activation;

/* s = x + residual (x alone when residual is null), rstd = 1/sqrt(mean(s^2) + eps),
 * y = s * rstd * weight.
 *
 * dtype (F32 or BF16) is x's, residual's, weight's and sum's.  y has dtype, or
 * F8_E4M3 with scale[row] = max|y| / 448 (1 for a row of zeros) and y / scale
 * stored.  sum receives s (null: not stored), rstd the row's factor (fp32, may
 * be null); both are what the gradient needs. */
mic_status mic_rms_norm(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, int rows, int cols, double eps,
                        const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                        void* y, int64_t ldy, void* sum, int64_t lds, float* rstd, float* scale);

/* With g = dy * weight:  dx = rstd * (g - s * rstd^2 * mean(g * s)) + dsum,
 * dweight = sum over rows of dy * s * rstd.  dx is the gradient of x and of
 * residual alike; dsum (may be null) is the gradient that reaches s past the
 * norm.  dweight may be null. */
mic_status mic_rms_norm_backward_workspace(mic_handle handle, int rows, int cols, size_t* bytes);
mic_status mic_rms_norm_backward(mic_handle handle, mic_dtype dtype, int rows, int cols, const void* dy, int64_t lddy,
                                 const void* sum, int64_t lds, const void* weight, const float* rstd,
                                 const void* dsum, int64_t ldd, void* dx, int64_t lddx, void* dweight,
                                 void* workspace, size_t workspace_bytes);

/* y[m,n] = act(x_scale[m] w_scale[n] sum_k x[m,k] w[n,k] + bias[n]) + residual[m,n].
 *
 * Types: F32 or BF16 throughout, or x and w F8_E4M3 with both scales (fp32)
 * and bias, residual, preact and y of out_dtype, F32 or BF16.  bias, residual
 * and preact may be null; preact receives the value before the activation,
 * which the gradient needs.
 *
 * fast_sums concerns e4m3 operands only.  0: their products are added in fp32.
 * Not 0: by the e4m3 matrix instruction, at up to twice the rate, which keeps
 * about 13 bits of each product below the largest of the 64 it adds (off by up
 * to 2^-11 of that one): far below a bf16 output's rounding unless the sum
 * nearly cancels. */
mic_status mic_linear_forward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes);
mic_status mic_linear_forward_workspace_aligned(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes);
mic_status mic_linear_forward(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, mic_activation act,
                              int fast_sums, int m, int n, int k, const void* x, int64_t ldx, const void* w, int64_t ldw,
                              const float* x_scale, const float* w_scale, const void* bias, const void* residual,
                              int64_t ldr, void* y, int64_t ldy, void* preact, int64_t ldp, void* workspace,
                              size_t workspace_bytes);

/* With z = preact and dz = dy * act'(z) (MIC_ACT_NONE: dz = dy, preact unused):
 *   dx[m,k] = sum_n dz[m,n] w[n,k]    dw[n,k] = sum_m dz[m,n] x[m,k]    dbias[n] = sum_m dz[m,n]
 * F32 or BF16.  dx, dw and dbias may each be null: that gradient is not
 * computed (w is needed for dx only, x for dw only).  The residual's gradient
 * is dy itself.  dz enters the products in the tensors' type. */
mic_status mic_linear_backward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes);
mic_status mic_linear_backward_workspace_aligned(mic_handle handle, mic_dtype dtype, mic_activation act, int m, int n, int k,
                                                 size_t* bytes);
mic_status mic_linear_backward(mic_handle handle, mic_dtype dtype, mic_activation act, int m, int n, int k,
                               const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w, int64_t ldw,
                               const void* preact, int64_t ldp, void* dx, int64_t lddx, void* dw, int64_t lddw,
                               void* dbias, void* workspace, size_t workspace_bytes);

/* gate = x w_gate^T, up = x w_up^T (with scales as in mic_linear_forward),
 * y[m,n] = act(gate[m,n]) * up[m,n].  gate and up (both or neither null)
 * receive the two products, which the gradient needs. */
mic_status mic_gated_linear_forward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k, size_t* bytes);
mic_status mic_gated_linear_forward_workspace_aligned(mic_handle handle, mic_dtype dtype, int m, int n, int k,
                                                      size_t* bytes);
mic_status mic_gated_linear_forward(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, mic_activation act,
                                    int fast_sums, int m, int n, int k, const void* x, int64_t ldx, const void* w_gate,
                                    int64_t ldg, const void* w_up, int64_t ldu, const float* x_scale,
                                    const float* w_gate_scale, const float* w_up_scale, void* y, int64_t ldy,
                                    void* gate, int64_t ldgate, void* up, int64_t ldup, void* workspace,
                                    size_t workspace_bytes);

/* dgate = dy * up * act'(gate), dup = dy * act(gate):
 *   dx = dgate w_gate + dup w_up    dw_gate = dgate^T x    dw_up = dup^T x
 * F32 or BF16.  dx may be null, and dw_gate and dw_up together. */
mic_status mic_gated_linear_backward_workspace(mic_handle handle, mic_dtype dtype, int m, int n, int k,
                                               size_t* bytes);
mic_status mic_gated_linear_backward_workspace_aligned(mic_handle handle, mic_dtype dtype, int m, int n, int k,
                                                       size_t* bytes);
mic_status mic_gated_linear_backward(mic_handle handle, mic_dtype dtype, mic_activation act, int m, int n, int k,
                                     const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w_gate,
                                     int64_t ldg, const void* w_up, int64_t ldu, const void* gate, int64_t ldgate,
                                     const void* up, int64_t ldup, void* dx, int64_t lddx, void* dw_gate,
                                     int64_t lddg, void* dw_up, int64_t lddu, void* workspace,
                                     size_t workspace_bytes);

/* How a call runs its products, host only, NUL-terminated into buf of buflen
 * bytes (MIC_STATUS_BAD_PARAM if it does not fit; 128 do): "few" rows, large
 * tiles ("fast 256x192") or small ones through registers ("any 64x64"), in how
 * many parts the reduction is split and which operands are packed first; a
 * gradient's as "dx: ..., dw: ...".  aligned: as ..._workspace_aligned's operands.
 * Without a handle the answer is that of a whole MI355X.  Errors as the
 * call's own checks of sizes and types. */
mic_status mic_linear_forward_kernel_name(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, int fast_sums, int m,
                                          int n, int k, int aligned, char* buf, size_t buflen);
mic_status mic_gated_linear_forward_kernel_name(mic_handle handle, mic_dtype dtype, mic_dtype out_dtype, int fast_sums,
                                                int m, int n, int k, int aligned, char* buf, size_t buflen);
mic_status mic_linear_backward_kernel_name(mic_handle handle, mic_dtype dtype, mic_activation act, int m, int n, int k,
                                           int aligned, char* buf, size_t buflen);
mic_status mic_gated_linear_backward_kernel_name(mic_handle handle, mic_dtype dtype, int m, int n, int k, int aligned,
                                                 char* buf, size_t buflen);

#ifdef __cplusplus
}
#endif

#endif /* MICONV_H */
