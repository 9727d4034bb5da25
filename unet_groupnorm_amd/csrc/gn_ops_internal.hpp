// gn_ops_internal.hpp -- what the torch binding calls of libgn.so beside the C ABI.
#pragma once

#include "gn_ops.h"

namespace gn {

// gn_grad_norm (clip false) and gn_grad_clip. devices_known: the caller has seen that every
// tensor of the list lives on norm's device, so that the library need not ask the runtime
// for each pointer (about 0.1 us of host time for each of them).
int grads(const gn_grad_tensor* t, int64_t n, int norm_type, bool clip, double max_norm, float* norm, void* ws,
          size_t ws_bytes, void* stream, bool devices_known);

}  // namespace gn
