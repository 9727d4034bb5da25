// gn_ops_internal.hpp -- what the torch binding calls of libgn.so beside the C ABI: the same
// calls with one argument more, the device that the caller has seen every tensor and the
// stream to belong to. The library then need not ask the runtime about each pointer (about
// 0.1 us of host time for each: 1 us of a row norm's 5, half of a list of 150 gradients). With
// device -1 they are the C ABI's calls.
#pragma once

#include "gn_ops.h"

namespace gn {

int rms_forward(const void* x, int x_dtype, int64_t x_stride, const void* residual, int r_dtype, const void* weight,
                int w_dtype, int64_t T, int64_t H, float eps, void* y, int y_dtype, void* h, float* rstd,
                void* stream, int device);
int rms_forward_q8(const void* x, int x_dtype, int64_t x_stride, const void* residual, int r_dtype,
                   const void* weight, int w_dtype, int64_t T, int64_t H, float eps, int64_t block, void* q,
                   int q_dtype, float* scale, void* h, float* rstd, void* stream, int device);
int q8_dequantize(const void* q, int q_dtype, const float* scale, int64_t T, int64_t H, int64_t block, void* out,
                  int out_dtype, void* stream, int device);
int rms_backward(const void* dy, int dy_dtype, const void* h, int h_dtype, int64_t h_stride, const float* rstd,
                 const void* weight, int w_dtype, const void* dh, int64_t T, int64_t H, void* dx, int x_dtype,
                 void* dres, void* dweight, void* workspace, size_t workspace_bytes, void* stream, int device);

// gn_grad_norm (clip false) and gn_grad_clip.
int grads(const gn_grad_tensor* t, int64_t n, int norm_type, bool clip, double max_norm, float* norm, void* ws,
          size_t ws_bytes, void* stream, int device);

}  // namespace gn
