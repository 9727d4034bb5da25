// gn_ops_binding.cpp -- the compiled binding (Python module _gnbind) of include/gn_ops.h for
// torch tensors: the row norm, its 8-bit form, and the gradient list.
//
// Argument marshalling only: every tensor is checked (device, dtype, sizes, layout), outputs
// not given are allocated on the first tensor's device, that device's current HIP stream is
// taken from torch, and the library is called; its status is returned with the outputs.
#include <c10/hip/HIPStream.h>
#include <hip/hip_runtime.h>
#include <torch/csrc/autograd/variable.h>
#include <torch/extension.h>

#include <cstdint>
#include <initializer_list>
#include <string>
#include <vector>

#include "gn_ops.h"
#include "gn_ops_internal.hpp"
#include "gn_tensors.hpp"

namespace {

struct Inputs {
    Rows r;
    int didx, xc, rc, wc;
    void *res, *w;
};

Inputs inputs_of(const at::Tensor& x, const OptTensor& weight, const OptTensor& residual)
{
    Inputs in{rows_of(x, "x"), x.get_device(), code_of(x, "x"), GN_F32, GN_F32, nullptr, nullptr};
    if (residual.has_value()) {
        in.rc = code_of(*residual, "residual");
        in.res = like("residual", *residual, x);
    }
    if (weight.has_value()) {
        in.wc = code_of(*weight, "weight");
        in.w = vec("weight", *weight, in.r.H, in.didx);
    }
    return in;
}

// h, stored beside a residual (in its dtype); without one h is x and nothing is written.
at::Tensor h_of(const at::Tensor& x, const OptTensor& residual, const OptTensor& h)
{
    if (!residual.has_value()) {
        if (h.has_value()) throw py::value_error("h is an output of a call with a residual");
        return x;
    }
    if (!h.has_value()) return fresh(residual->sizes(), residual->scalar_type(), *residual);
    like("h", *h, x);
    if (h->scalar_type() != residual->scalar_type()) throw py::type_error("h must have residual's dtype");
    return *h;
}

py::tuple rms_forward(const at::Tensor& x, const OptTensor& weight, double eps, const OptTensor& residual,
                      int out_code, bool need_rstd, const OptTensor& out, const OptTensor& h_out,
                      const OptTensor& rstd_out)
{
    const Inputs in = inputs_of(x, weight, residual);
    const at::Tensor y = out.has_value() ? *out : fresh(x.sizes(), out_code < 0 ? x.scalar_type() : type_of_code(out_code), x);
    void* yp = like("out", y, x);
    const int yc = code_of(y, "out");
    agree("out_dtype", out_code, yc);
    const at::Tensor h = h_of(x, residual, h_out), rstd = rstd_of(x, rstd_out, need_rstd);
    float* rp = rstd.defined() ? f32("rstd", rstd, in.r.T, in.didx) : nullptr;
    const int status = gn::rms_forward(x.data_ptr(), in.xc, in.r.stride, in.res, in.rc, in.w, in.wc, in.r.T, in.r.H,
                                      float(eps), yp, yc, residual.has_value() ? h.data_ptr() : nullptr, rp,
                                      stream_of(in.didx), in.didx);
    mark_written(status, {&out, &h_out, &rstd_out});
    return py::make_tuple(y, h, or_none(rstd), status);
}

py::tuple rms_forward_q8(const at::Tensor& x, const OptTensor& weight, double eps, const OptTensor& residual,
                         int q_dtype, int64_t block, bool need_rstd, const OptTensor& out, const OptTensor& scale_out,
                         const OptTensor& h_out, const OptTensor& rstd_out)
{
    const Inputs in = inputs_of(x, weight, residual);
    const at::Tensor q = out.has_value()
                             ? *out
                             : fresh(x.sizes(), q_dtype == GN_Q_E4M3 ? at::kFloat8_e4m3fn : at::kChar, x);
    void* qp = like("out", q, x);
    const int qc = q_code_of(q);
    agree("q_dtype", q_dtype, qc);
    const int64_t n = scales_of(in.r.H, block);
    const at::Tensor scale = scale_out.has_value() ? *scale_out : fresh(lead(x, n), at::kFloat, x);
    float* sp = f32("scale", scale, in.r.T * n, in.didx);
    const at::Tensor h = h_of(x, residual, h_out), rstd = rstd_of(x, rstd_out, need_rstd);
    float* rp = rstd.defined() ? f32("rstd", rstd, in.r.T, in.didx) : nullptr;
    const int status = gn::rms_forward_q8(x.data_ptr(), in.xc, in.r.stride, in.res, in.rc, in.w, in.wc, in.r.T, in.r.H,
                                         float(eps), block, qp, qc, sp, residual.has_value() ? h.data_ptr() : nullptr,
                                         rp, stream_of(in.didx), in.didx);
    mark_written(status, {&out, &scale_out, &h_out, &rstd_out});
    return py::make_tuple(q, scale, h, or_none(rstd), status);
}

py::tuple q8_dequantize(const at::Tensor& q, const at::Tensor& scale, int out_code, int64_t block,
                        const OptTensor& out)
{
    const Rows r = rows_of(q, "q");
    if (!q.is_contiguous()) throw py::value_error("q must be contiguous");
    const int qc = q_code_of(q), didx = q.get_device();
    const at::Tensor o =
        out.has_value() ? *out : fresh(q.sizes(), type_of_code(out_code < 0 ? GN_F32 : out_code), q);
    void* op = like("out", o, q);
    const int oc = code_of(o, "out");
    agree("out_dtype", out_code, oc);
    const int status = gn::q8_dequantize(q.data_ptr(), qc, f32("scale", scale, r.T * scales_of(r.H, block), didx), r.T,
                                        r.H, block, op, oc, stream_of(didx), didx);
    mark_written(status, {&out});
    return py::make_tuple(o, status);
}

py::tuple rms_backward(const at::Tensor& dy, const at::Tensor& h, const at::Tensor& rstd, const OptTensor& weight,
                       const OptTensor& dh, int x_code, bool need_dx, bool need_dres, bool need_dweight,
                       const OptTensor& workspace, const OptTensor& dx_out, const OptTensor& dres_out,
                       const OptTensor& dweight_out)
{
    const Rows r = rows_of(h, "h");
    const int didx = h.get_device(), hc = code_of(h, "h"), dyc = code_of(dy, "dy");
    const int xc = x_code < 0 ? hc : x_code;
    void* dyp = like("dy", dy, h);
    float* rp = f32("rstd", rstd, r.T, didx);
    void *wp = nullptr, *dhp = nullptr;
    int wc = GN_F32;
    if (weight.has_value()) {
        wc = code_of(*weight, "weight");
        wp = vec("weight", *weight, r.H, didx);
    }
    if (dh.has_value()) {
        dhp = like("dh", *dh, h);
        if (dh->scalar_type() != h.scalar_type()) throw py::type_error("dh must have h's dtype");
    }
    wanted(dx_out, need_dx, "dx");
    wanted(dres_out, need_dres, "dres");
    wanted(dweight_out, need_dweight, "dweight");
    at::Tensor dx, dres, dw;
    if (need_dx) {
        dx = dx_out.has_value() ? *dx_out : fresh(h.sizes(), type_of_code(xc), h);
        like("dx", dx, h);
        if (code_of(dx, "dx") != xc) throw py::type_error("dx must have x's dtype");
    }
    if (need_dres) {
        // one tensor is both gradients where the dtypes agree
        if (dres_out.has_value()) dres = *dres_out;
        else dres = need_dx && xc == hc ? dx : fresh(h.sizes(), h.scalar_type(), h);
        like("dres", dres, h);
        if (dres.scalar_type() != h.scalar_type()) throw py::type_error("dres must have h's dtype");
    }
    if (need_dweight) {
        if (dweight_out.has_value()) dw = *dweight_out;
        else dw = weight.has_value() ? fresh(weight->sizes(), type_of_code(wc), h) : fresh({r.H}, type_of_code(wc), h);
        vec("dweight", dw, r.H, didx);
        if (code_of(dw, "dweight") != wc) throw py::type_error("dweight must have weight's dtype");
    }
    at::Tensor ws;
    void* wsp = nullptr;
    size_t wsb = 0;
    if (need_dweight) {
        ws = workspace.has_value() ? *workspace
                                   : fresh({int64_t(gn_rms_workspace_bytes(r.T, r.H))}, at::kByte, h);
        if (ws.get_device() != didx || !ws.is_contiguous())
            throw py::value_error("workspace must be a contiguous tensor on h's device");
        wsp = ws.data_ptr();
        wsb = size_t(ws.numel()) * ws.element_size();
    }
    const bool apart = dres.defined() && !(dx.defined() && dres.is_same(dx));
    const int status =
        gn::rms_backward(dyp, dyc, h.data_ptr(), hc, r.stride, rp, wp, wc, dhp, r.T, r.H,
                        dx.defined() ? dx.data_ptr() : nullptr, xc, apart ? dres.data_ptr() : nullptr,
                        dw.defined() ? dw.data_ptr() : nullptr, wsp, wsb, stream_of(didx), didx);
    mark_written(status, {&dx_out, &dres_out, &dweight_out});
    return py::make_tuple(or_none(dx), or_none(dw), or_none(dres), status);
}

// ------------------------------------------------------------------ gradient list

// A tensor whose elements fill its memory, in whatever order.
void dense(const at::Tensor& t, const char* name, int didx)
{
    if (t.layout() != at::kStrided || !t.is_non_overlapping_and_dense())
        throw py::value_error(std::string(name) + " must be dense tensors (every element of their memory once)");
    if (t.get_device() != didx) throw py::value_error(std::string(name) + " must be on one device");
}

// Whether tensors of one shape hold their elements in one order: the strides of dimensions of
// one element do not count, nor any of an empty tensor.
bool same_order(const at::Tensor& a, const at::Tensor& b)
{
    if (a.numel() == 0 || a.strides() == b.strides()) return true;
    for (int64_t i = 0; i < a.dim(); ++i)
        if (a.size(i) != 1 && a.stride(i) != b.stride(i)) return false;
    return true;
}

// The list of `grads` (each with its output where `out` is given; in place where clip is
// set without one), the norm and, where asked for, the scaled tensors.
py::tuple grads(const std::vector<at::Tensor>& g, const c10::optional<std::vector<at::Tensor>>& out, bool clip,
                double max_norm, int norm_type, const OptTensor& norm_out, const OptTensor& workspace)
{
    if (g.empty()) throw py::value_error("at least one gradient is needed");
    if (out.has_value() && out->size() != g.size()) throw py::value_error("out must have one tensor for each gradient");
    const int didx = g[0].get_device();
    std::vector<gn_grad_tensor> t(g.size());
    for (size_t i = 0; i < g.size(); ++i) {
        dense(g[i], "gradients", didx);
        t[i].data = g[i].data_ptr();
        t[i].numel = g[i].numel();
        t[i].dtype = t[i].out_dtype = code_of(g[i], "gradient");
        t[i].out = clip ? g[i].data_ptr() : nullptr;
        if (out.has_value()) {
            const at::Tensor& o = (*out)[i];
            dense(o, "out", didx);
            if (o.sizes() != g[i].sizes() || !same_order(o, g[i]))
                throw py::value_error("out must have the gradients' shapes and layouts");
            t[i].out = o.data_ptr();
            t[i].out_dtype = code_of(o, "out");
        }
    }
    const at::Tensor norm = norm_out.has_value() ? *norm_out : fresh({}, at::kFloat, g[0]);
    float* np = f32("norm", norm, 1, didx);
    const int64_t n = int64_t(t.size());
    const at::Tensor ws = workspace.has_value() ? *workspace
                                                : fresh({int64_t(gn_grad_workspace_bytes(t.data(), n))}, at::kByte, g[0]);
    if (ws.get_device() != didx || !ws.is_contiguous())
        throw py::value_error("workspace must be a contiguous tensor on the gradients' device");
    const size_t wsb = size_t(ws.numel()) * ws.element_size();
    const int status = gn::grads(t.data(), n, norm_type, clip, max_norm, np, ws.data_ptr(), wsb, stream_of(didx), didx);
    if (clip && status == GN_OK)
        for (const at::Tensor& w : out.has_value() ? *out : g)
            mark_written(w);
    mark_written(status, {&norm_out});
    return py::make_tuple(norm, status);
}

int64_t grad_workspace_bytes(const std::vector<at::Tensor>& g)
{
    std::vector<gn_grad_tensor> t(g.size());
    for (size_t i = 0; i < g.size(); ++i) t[i] = {g[i].data_ptr(), nullptr, g[i].numel(), code_of(g[i], "gradient"), GN_F32};
    return int64_t(gn_grad_workspace_bytes(t.data(), int64_t(t.size())));
}

// Throws where a graph is being captured on the current stream of a leaf's device while a
// live eager graph holds the leaf's gradient accumulation on another stream: the captured
// backward pass would run into that stream, which ends the capture and the process.
void capture_check(const std::vector<OptTensor>& leaves)
{
    for (const OptTensor& t : leaves) {
        if (!t.has_value() || !t->is_cuda() || !t->requires_grad() || !t->is_leaf()) continue;
        const auto cur = c10::hip::getCurrentHIPStream(t->get_device());
        hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
        if (hipStreamIsCapturing(cur.stream(), &st) != hipSuccess) (void)hipGetLastError();
        if (st == hipStreamCaptureStatusNone) continue;
        const auto acc = torch::autograd::impl::try_get_grad_accumulator(*t);
        if (!acc) continue;
        const auto s = acc->stream();  // its device type is torch's name for HIP, not HIP's own: compare ids
        if (s.has_value() && s->id() != cur.id())
            throw std::runtime_error(
                "an eager graph of the same leaf tensor is alive while this one is captured: drop its outputs "
                "before the capture");
    }
}

}  // namespace

void bind_ops(py::module_& m)
{
    m.def("rms_forward", &rms_forward, "gn_rms_forward: (y, h, rstd, status)", py::arg("x"), py::arg("weight"),
          py::arg("eps"), py::arg("residual"), py::arg("out_code"), py::arg("need_rstd"), py::arg("out"), py::arg("h"),
          py::arg("rstd"));
    m.def("rms_forward_q8", &rms_forward_q8, "gn_rms_forward_q8: (q, scale, h, rstd, status)", py::arg("x"),
          py::arg("weight"), py::arg("eps"), py::arg("residual"), py::arg("q_dtype"), py::arg("block"),
          py::arg("need_rstd"), py::arg("out"), py::arg("scale"), py::arg("h"), py::arg("rstd"));
    m.def("q8_dequantize", &q8_dequantize, "gn_q8_dequantize: (values, status)", py::arg("q"), py::arg("scale"),
          py::arg("out_code"), py::arg("block"), py::arg("out"));
    m.def("rms_backward", &rms_backward, "gn_rms_backward: (dx, dweight, dres, status)", py::arg("dy"), py::arg("h"),
          py::arg("rstd"), py::arg("weight"), py::arg("dh"), py::arg("x_code"), py::arg("need_dx"),
          py::arg("need_dres"), py::arg("need_dweight"), py::arg("workspace"), py::arg("dx"), py::arg("dres"),
          py::arg("dweight"));
    m.def("grads", &grads, "gn_grad_norm or gn_grad_clip: (norm, status)", py::arg("grads"), py::arg("out"),
          py::arg("clip"), py::arg("max_norm"), py::arg("norm_type"), py::arg("norm"), py::arg("workspace"));
    m.def("grad_workspace_bytes", &grad_workspace_bytes, py::arg("grads"));
    m.def("even_rows", [](const at::Tensor& t) { return t.dim() < 1 || row_stride(t) >= 0; }, py::arg("t"));
    m.def("capture_check", &capture_check, py::arg("leaves"));
}
