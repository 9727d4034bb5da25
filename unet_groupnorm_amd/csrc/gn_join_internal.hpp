// gn_join_internal.hpp -- what the torch binding calls of libgn.so beside gn_join.h: the same calls
// with one argument more, the device that the caller has seen every tensor and the stream to
// belong to (-1: not known, the C ABI's calls).
#pragma once

#include "gn_join.h"

namespace gn {

struct JoinForwardPtrs {
    const void *x, *residual, *weight, *post_weight, *gate, *scale;
    void *y, *h;
    float *rstd, *post_rstd;
    void* h_q;
    float* h_scale;
    void* x_q;
    float* x_scale;
};
int join_forward(const gn_join* j, const JoinForwardPtrs& p, void* stream, int device);

struct JoinBackwardPtrs {
    const void *dy, *dh, *h;
    const float* h_scale;
    const void* x;
    const float *x_scale, *rstd, *post_rstd;
    const void *weight, *post_weight, *gate, *scale;
    void *dx, *dres, *dweight, *dpost_weight, *dgate, *dscale;
    void* workspace;
    size_t workspace_bytes;
};
int join_backward(const gn_join* j, const JoinBackwardPtrs& p, void* stream, int device);

int q8_quantize(const void* x, int x_dtype, int64_t x_stride, int64_t T, int64_t H, int64_t block, void* q,
                int q_dtype, float* scale, void* stream, int device);

}  // namespace gn
