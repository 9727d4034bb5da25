// gn_tensors.hpp -- how the compiled bindings of gn_ops.h and gn_join.h check and allocate torch
// tensors. Every function lives in an unnamed namespace.
#pragma once

#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPStream.h>
#include <torch/extension.h>

#include <cstdint>
#include <initializer_list>
#include <string>
#include <vector>

#include "gn_ops.h"

namespace {

namespace py = pybind11;
using OptTensor = c10::optional<at::Tensor>;

int code_of(const at::Tensor& t, const char* name)
{
    switch (t.scalar_type()) {
        case at::kFloat: return GN_F32;
        case at::kBFloat16: return GN_BF16;
        case at::kHalf: return GN_F16;
        default:
            throw py::type_error(std::string(name) + ": unsupported dtype " +
                                 std::string(c10::toString(t.scalar_type())) + " (float32, bfloat16 or float16)");
    }
}

at::ScalarType type_of_code(int code)
{
    return code == GN_F32 ? at::kFloat : code == GN_BF16 ? at::kBFloat16 : at::kHalf;
}

int q_code_of(const at::Tensor& t)
{
    if (t.scalar_type() == at::kChar) return GN_Q_INT8;
    if (t.scalar_type() == at::kFloat8_e4m3fn) return GN_Q_E4M3;
    throw py::type_error("q: unsupported dtype " + std::string(c10::toString(t.scalar_type())) +
                         " (int8 or float8_e4m3fn)");
}

void* stream_of(int didx)
{
    return didx < 0 ? nullptr : static_cast<void*>(c10::hip::getCurrentHIPStream(didx).stream());
}

struct Rows {
    int64_t T, H, stride;
};

// The distance between t's rows if they are whole and evenly spaced over the leading
// dimensions, else -1.
int64_t row_stride(const at::Tensor& t)
{
    const int64_t d = t.dim(), H = t.size(d - 1);
    if (t.numel() == 0 || t.is_contiguous()) return H;
    if (H != 1 && t.stride(d - 1) != 1) return -1;
    int64_t stride = H, expect = -1;
    for (int64_t i = d - 2; i >= 0; --i) {
        if (t.size(i) == 1) continue;
        if (expect < 0) stride = t.stride(i);
        else if (t.stride(i) != expect) return -1;
        expect = t.stride(i) * t.size(i);
    }
    return stride < H ? -1 : stride;
}

Rows rows_of(const at::Tensor& t, const char* name)
{
    if (t.dim() < 1 || t.size(-1) < 1) throw py::value_error(std::string(name) + " needs rows of at least one element");
    const Rows r{t.numel() / t.size(-1), t.size(-1), row_stride(t)};
    if (r.stride < 0) throw py::value_error(std::string(name) + "'s rows must be contiguous and evenly spaced");
    return r;
}

// A contiguous tensor of x's shape on x's device.
void* like(const char* name, const at::Tensor& t, const at::Tensor& x)
{
    if (t.sizes() != x.sizes() || !t.is_contiguous())
        throw py::value_error(std::string(name) + " must be contiguous and have x's shape");
    if (t.get_device() != x.get_device()) throw py::value_error(std::string(name) + " must be on x's device");
    return t.data_ptr();
}

void* vec(const char* name, const at::Tensor& t, int64_t n, int didx)
{
    if (t.numel() != n || t.get_device() != didx || !t.is_contiguous())
        throw py::value_error(std::string(name) + " must be a contiguous tensor of " + std::to_string(n) +
                              " elements on x's device");
    return t.data_ptr();
}

float* f32(const char* name, const at::Tensor& t, int64_t n, int didx)
{
    if (t.scalar_type() != at::kFloat || t.numel() != n || t.get_device() != didx || !t.is_contiguous())
        throw py::value_error(std::string(name) + " must be a contiguous Float tensor of " + std::to_string(n) +
                              " elements on x's device");
    return static_cast<float*>(t.data_ptr());
}

// A new contiguous tensor on x's device. On a GPU this goes to the allocator without torch's
// dispatcher, which small calls would feel (three outputs: 3.1 us against 1.9).
at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& x)
{
    if (x.is_cuda()) return at::Tensor(at::detail::empty_cuda(sizes, type, x.device(), c10::nullopt));
    return at::empty(sizes, x.options().dtype(type));
}

// Tells autograd that a call wrote into tensors of the caller's: a graph that has saved one of
// them refuses its backward pass instead of using the new values.
void mark_written(const at::Tensor& t)
{
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void mark_written(int status, std::initializer_list<const OptTensor*> given)
{
    if (status != GN_OK) return;
    for (const OptTensor* t : given)
        if (t->has_value()) mark_written(**t);
}

py::object or_none(const at::Tensor& t) { return t.defined() ? py::cast(t) : py::none(); }

// The sizes of x without its last dimension, and with n in its place where n >= 0.
std::vector<int64_t> lead(const at::Tensor& x, int64_t n = -1)
{
    std::vector<int64_t> s(x.sizes().begin(), x.sizes().end() - 1);
    if (n >= 0) s.push_back(n);
    return s;
}

int64_t scales_of(int64_t H, int64_t block) { return block > 0 ? (H + block - 1) / block : 1; }

at::Tensor rstd_of(const at::Tensor& x, const OptTensor& rstd, bool need)
{
    if (rstd.has_value()) return *rstd;
    return need ? fresh(lead(x), at::kFloat, x) : at::Tensor();
}

// The dtype asked for (negative: none) and that of the output given.
void agree(const char* name, int asked, int given)
{
    if (asked >= 0 && asked != given) throw py::type_error(std::string(name) + " is not the dtype of the given output");
}

// An output that the caller gives and at the same time does not want.
void wanted(const OptTensor& given, bool need, const std::string& name)
{
    if (given.has_value() && !need) throw py::value_error(name + " is given, but need_" + name + " declines it");
}

}  // namespace
