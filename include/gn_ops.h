/*
 * gn_ops.h -- C ABI of libgn.so, second part: the root-mean-square norm over rows with the
 * residual's addition (forward, backward, and an output in 8 bits with scales), and the
 * global norm of many gradient tensors with clipping, on MI355X (gfx950).
 *
 * Ownership, ordering and errors are those of gn.h: the caller owns every buffer and the
 * workspace, the library never allocates device memory, never synchronizes and copies
 * nothing to the host; work is enqueued on `stream` in stream order; every check runs
 * before anything is enqueued, and on any error other than GN_ERR_LAUNCH no output is
 * touched. Every pointer argument must be device memory of one device, the one that owns
 * the first tensor, whatever device is current. A workspace needs no initialization and
 * carries nothing from one call to the next; calls that may overlap in time need one each.
 * No call uses atomics: repeated calls give the same bits.
 *
 * Statuses are gn_status codes (gn.h) and the gn_ops_status codes below;
 * gn_ops_status_string describes both. Data types are gn_dtype codes.
 */
#ifndef GN_OPS_H
#define GN_OPS_H

#include <stddef.h>
#include <stdint.h>

#include "gn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gn_ops_status {
    GN_ERR_ROWS = 32,    /* T < 0, H < 1, H > GN_RMS_MAX_COLUMNS, a row stride below H, or a
                            negative element count */
    GN_ERR_OVERLAP = 33, /* an output overlaps another argument other than as allowed */
    GN_ERR_BLOCK = 34,   /* block is not 0, 32, 64 or 128 */
    GN_ERR_NORM = 35     /* unknown norm type, or max_norm negative or NaN */
} gn_ops_status;

/* Static English description of a gn_status or gn_ops_status code (never NULL). */
const char* gn_ops_status_string(int status);

/* ------------------------------------------------------------------ row norm
 *
 * T rows of H columns. x holds element (t, i) at t * x_stride + i (x_stride >= H); every
 * other tensor is contiguous. Pointers are aligned to their element; whole 16-byte
 * alignment is not needed, nor a multiple of anything in H.
 *
 *   h    = x + residual, in fp32, rounded once to residual's dtype and stored (without a
 *          residual h is x, and nothing is stored)
 *   rstd = 1 / sqrt(mean_i(h^2) + eps), of h as stored, in fp32
 *   y    = h * rstd * weight, in fp32, rounded once
 *
 * x: any gn_dtype; residual: x's dtype or GN_F32; weight: x's dtype or GN_F32 (NULL: all
 * ones); y: x's dtype or GN_F32. A row's results depend on that row, H and the dtypes
 * alone: not on T, nor on the row's place. T == 0 is a call that does nothing.
 * A NaN in a row gives a NaN row; an infinity gives rstd == 0, y NaN there and 0 elsewhere.
 * The mean of squares is taken in fp32: H * mean(h^2) must stay below its maximum.
 */
#define GN_RMS_MAX_COLUMNS 32768

/*
 * Forward. h may be residual itself (the residual stream updated in place), and y may be x
 * itself (same dtype, x_stride == H); no other overlap with an output. rstd [T] may be NULL.
 * One kernel.
 */
int gn_rms_forward(const void* x, int x_dtype, int64_t x_stride, const void* residual, int r_dtype,
                   const void* weight, int w_dtype, int64_t T, int64_t H, float eps,
                   void* y, int y_dtype, void* h, float* rstd, void* stream);

/* The 8-bit formats of gn_rms_forward_q8. */
typedef enum gn_q8 {
    GN_Q_INT8 = 0, /* signed integers, -127 to 127 */
    GN_Q_E4M3 = 1  /* 8-bit floating point, 4 exponent and 3 mantissa bits, finite up to 448 */
} gn_q8;

/*
 * Forward with the output in 8 bits: y as above, kept in fp32, and for each row (block == 0)
 * or each run of `block` columns (32, 64 or 128; a row's last may be shorter)
 *   scale = max(max|y| / qmax, 2^-126),  q = y / scale rounded to nearest, ties to even,
 * with qmax = 127 or 448. The scale is the correctly rounded fp32 quotient; y / scale is taken
 * in fp32 to (1/2 + 2^-20) ulp. scale is [T][ceil(H / block)] fp32 ([T] for block == 0). Where a
 * run holds a NaN or an infinity its scale is NaN and its q are 0 (so q * scale is NaN).
 * q [T][H]; h, rstd and the allowed overlaps as gn_rms_forward's (q overlaps nothing).
 * One kernel.
 */
int gn_rms_forward_q8(const void* x, int x_dtype, int64_t x_stride, const void* residual, int r_dtype,
                      const void* weight, int w_dtype, int64_t T, int64_t H, float eps, int64_t block,
                      void* q, int q_dtype, float* scale, void* h, float* rstd, void* stream);

/* out = q * scale, in fp32, rounded once to out_dtype: the values that q stands for. */
int gn_q8_dequantize(const void* q, int q_dtype, const float* scale, int64_t T, int64_t H, int64_t block,
                     void* out, int out_dtype, void* stream);

/*
 * Backward, from h (x itself where there was no residual; h_stride as x_stride above) and
 * the rstd that the forward wrote. With g = dy * weight and xhat = h * rstd,
 *   d = rstd * (g - xhat * mean_i(g * xhat)) + dh,   dweight = sum over rows of dy * xhat,
 * where dh (h's dtype, NULL for none) is the gradient that reaches h by the residual
 * stream. d is the gradient of x and of the residual alike: it is written to dx in x_dtype
 * and to dres in h's dtype (either may be NULL; where the two dtypes are one, one of them
 * serves both). dweight [H] has weight's dtype (NULL: not computed; NULL weight: fp32) and
 * is written, not accumulated. dy has x_dtype or GN_F32; x_dtype is h's dtype, or any where
 * h is GN_F32. dx or dres may be dy, dh or h itself where dtype and layout agree; no other
 * overlap. All sums are fp32 in a fixed order. One kernel, and one more with dweight.
 */
size_t gn_rms_workspace_bytes(int64_t T, int64_t H);

int gn_rms_backward(const void* dy, int dy_dtype, const void* h, int h_dtype, int64_t h_stride,
                    const float* rstd, const void* weight, int w_dtype, const void* dh,
                    int64_t T, int64_t H, void* dx, int x_dtype, void* dres, void* dweight,
                    void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ gradients
 *
 * One gradient tensor: numel elements of dtype at data (numel 0 is allowed, data is then
 * ignored), and for gn_grad_clip the output: out may be data itself (out_dtype == dtype),
 * or a separate tensor of numel elements, in dtype or GN_F32. Pointers are aligned to their
 * element. The order of a tensor's elements does not matter, so any dense layout serves.
 */
typedef struct gn_grad_tensor {
    const void* data;
    void* out;
    int64_t numel;
    int32_t dtype;
    int32_t out_dtype;
} gn_grad_tensor;

typedef enum gn_norm {
    GN_NORM_2 = 0,  /* square root of the sum of squares */
    GN_NORM_INF = 1 /* largest magnitude */
} gn_norm;

/* Workspace for a list of n tensors; 0 for a list that the calls below would reject. */
size_t gn_grad_workspace_bytes(const gn_grad_tensor* tensors, int64_t n);

/*
 * norm[0] (fp32) = the norm of all elements of the n tensors together. Squares are summed
 * in fp64, in an order fixed by the sizes, so no fp32 gradient's square overflows or is
 * lost. A NaN or infinity anywhere gives a NaN or infinite norm. A tensor listed twice
 * counts twice. The list itself (host memory) is read before the call returns.
 */
int gn_grad_norm(const gn_grad_tensor* tensors, int64_t n, int norm_type, float* norm,
                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * The same norm (norm may not be NULL), and for every tensor
 *   out = data * coef,  coef = min(1, max_norm / (norm + 1e-6)),
 * coef taken in fp64 and rounded to fp32, the product rounded once to out_dtype. coef is
 * decided on the device: nothing waits for the norm. A NaN norm makes every output NaN; an
 * infinite one makes coef 0, unless max_norm is infinite too: that clips nothing, coef is 1.
 * In place with coef == 1 the tensors are left as they are.
 * Outputs may not overlap one another or another tensor's data (a tensor listed twice).
 */
int gn_grad_clip(const gn_grad_tensor* tensors, int64_t n, int norm_type, double max_norm, float* norm,
                 void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GN_OPS_H */
