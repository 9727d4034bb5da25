// gn_ops_api.cpp -- the C ABI declared in include/gn_ops.h: validation and launches.
//
// Every check runs before anything is enqueued. The library allocates nothing on the device,
// never synchronizes, never reads device memory from the host and keeps no state.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <new>
#include <vector>

#include "gn_ops.h"
#include "gn_ops.hpp"
#include "gn_ops_internal.hpp"

namespace {

bool dtype_ok(int d) { return d == GN_F32 || d == GN_BF16 || d == GN_F16; }
int64_t size_of(int d) { return d == GN_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t a) { return (reinterpret_cast<uintptr_t>(p) & uintptr_t(a - 1)) == 0; }
int launch_status(hipError_t e) { return e == hipSuccess ? GN_OK : GN_ERR_LAUNCH; }

// The device that owns p, or -1 if p is not device memory.
int device_of(const void* p)
{
    hipPointerAttribute_t attr;
    if (hipPointerGetAttributes(&attr, p) != hipSuccess) {
        (void)hipGetLastError();
        return -1;
    }
    if (attr.type != hipMemoryTypeDevice && attr.type != hipMemoryTypeManaged) return -1;
    return attr.device;
}

// Makes the device that owns p current for the duration of a call; a stream or another
// pointer argument of another device is refused.
class OnDeviceOf {
  public:
    // known: the device that the caller has seen every pointer and the stream to belong to, or
    // -1 (they are looked at here).
    explicit OnDeviceOf(int known = -1) : known_(known) {}
    int enter(const void* p, void* stream)
    {
        const int dev = known_ >= 0 ? known_ : device_of(p);
        int cur = -1;
        if (dev < 0 || hipGetDevice(&cur) != hipSuccess) return GN_ERR_DEVICE;
        if (stream && known_ < 0) {
            hipDevice_t sdev = -1;
            if (hipStreamGetDevice(static_cast<hipStream_t>(stream), &sdev) != hipSuccess) {
                (void)hipGetLastError();
                return GN_ERR_DEVICE;
            }
            if (sdev != dev) return GN_ERR_DEVICE;
        }
        if (cur != dev) {
            if (hipSetDevice(dev) != hipSuccess) return GN_ERR_DEVICE;
            prev_ = cur;
        }
        dev_ = dev;
        return GN_OK;
    }
    int holds(std::initializer_list<const void*> ptrs) const
    {
        if (known_ >= 0) return GN_OK;
        for (const void* p : ptrs)
            if (p && device_of(p) != dev_) return GN_ERR_DEVICE;
        return GN_OK;
    }
    ~OnDeviceOf()
    {
        if (prev_ >= 0) (void)hipSetDevice(prev_);
    }

  private:
    int known_, prev_ = -1, dev_ = -1;
};

// ------------------------------------------------------------------ row norm

// The bytes that an argument covers.
struct Span {
    uintptr_t b = 0, e = 0;
    Span() = default;
    Span(const void* p, int64_t bytes)
        : b(reinterpret_cast<uintptr_t>(p)), e(p ? reinterpret_cast<uintptr_t>(p) + uintptr_t(bytes) : 0)
    {
    }
    bool meets(const Span& o) const { return b < o.e && o.b < e; }
    bool is(const Span& o) const { return b == o.b && e == o.e; }
};

bool meets_any(const Span& s, std::initializer_list<Span> all)
{
    for (const Span& o : all)
        if (s.meets(o)) return true;
    return false;
}

// Rows of the largest launch, in workgroups (the threads of a launch stay below 2^32).
constexpr int64_t kMaxGroups = int64_t(1) << 21;

int rows_check(int64_t T, int64_t H, int64_t stride)
{
    if (T < 0 || H < 1 || H > GN_RMS_MAX_COLUMNS || stride < H) return GN_ERR_ROWS;
    // Offsets stay within 62 bits of bytes.
    if (T > 0 && (T > (int64_t(1) << 44) || stride > (int64_t(1) << 58) / T)) return GN_ERR_ROWS;
    return GN_OK;
}

// The bytes of T rows of H elements, `stride` apart.
int64_t rows_bytes(int64_t T, int64_t H, int64_t stride, int dt)
{
    return T > 0 ? ((T - 1) * stride + H) * size_of(dt) : 0;
}

const void* at(const void* p, int64_t bytes) { return p ? static_cast<const char*>(p) + bytes : nullptr; }
void* at(void* p, int64_t bytes) { return p ? static_cast<char*>(p) + bytes : nullptr; }

// The forward of both outputs: y is the 8-bit tensor where q_dtype >= 0.
int forward(const void* x, int x_dtype, int64_t x_stride, const void* res, int r_dtype, const void* w, int w_dtype,
            int64_t T, int64_t H, float eps, void* y, int y_dtype, int q_dtype, int64_t block, float* scale, void* h,
            float* rstd, void* stream, int device)
{
    const bool q8 = q_dtype >= 0;
    int rc = rows_check(T, H, x_stride);
    if (rc) return rc;
    if (!dtype_ok(x_dtype) || (res && !(r_dtype == x_dtype || r_dtype == GN_F32)) ||
        (w && !(w_dtype == x_dtype || w_dtype == GN_F32)))
        return GN_ERR_DTYPE;
    if (q8 ? q_dtype != GN_Q_INT8 && q_dtype != GN_Q_E4M3 : !(y_dtype == x_dtype || y_dtype == GN_F32))
        return GN_ERR_DTYPE;
    if (q8 && block != 0 && block != 32 && block != 64 && block != 128) return GN_ERR_BLOCK;
    if (!std::isfinite(eps) || eps < 0.0f) return GN_ERR_EPS;
    if (T == 0) return GN_OK;
    if (!x || !y || (res != nullptr) != (h != nullptr) || (q8 && !scale)) return GN_ERR_NULL;
    const int64_t ys = q8 ? 1 : size_of(y_dtype), scales = q8 && block ? (H + block - 1) / block : 1;
    if (!aligned(x, size_of(x_dtype)) || !aligned(y, ys) || (w && !aligned(w, size_of(w_dtype))) ||
        (res && (!aligned(res, size_of(r_dtype)) || !aligned(h, size_of(r_dtype)))) || !aligned(rstd, 4) ||
        !aligned(scale, 4))
        return GN_ERR_ALIGN;
    const Span sx(x, rows_bytes(T, H, x_stride, x_dtype)), sr(res, res ? T * H * size_of(r_dtype) : 0),
        sw(w, w ? H * size_of(w_dtype) : 0), sy(y, T * H * ys), sh(h, res ? T * H * size_of(r_dtype) : 0),
        ss(rstd, T * 4), sc(q8 ? scale : nullptr, T * scales * 4);
    const bool y_is_x = !q8 && y == x && y_dtype == x_dtype && x_stride == H;
    if ((sy.meets(sx) && !y_is_x) || meets_any(sy, {sr, sw, sh, ss, sc}) || (sh.meets(sr) && !sh.is(sr)) ||
        meets_any(sh, {sx, sw, ss, sc}) || meets_any(ss, {sx, sr, sw, sc}) || meets_any(sc, {sx, sr, sw}))
        return GN_ERR_OVERLAP;
    OnDeviceOf dev(device);
    if ((rc = dev.enter(x, stream)) || (rc = dev.holds({res, w, y, h, rstd, scale}))) return rc;
    const gn::RowPlan p =
        gn::row_plan(H, x_dtype == GN_F32 || (res && r_dtype == GN_F32) || (!q8 && y_dtype == GN_F32));
    gn::RmsArgs a{};
    a.w = w;
    a.H = H;
    a.x_stride = x_stride;
    a.eps = eps;
    a.inv_H = 1.0f / float(H);
    a.w_dtype = w_dtype;
    a.y_f32 = y_dtype == GN_F32;
    a.lanes = p.lanes;
    a.rows = p.rows;
    a.q_dtype = q_dtype;
    a.block = int32_t(block);
    a.scales = scales;
    a.nt = T * H * (size_of(x_dtype) + ys + (res ? 2 * size_of(r_dtype) : 0)) > gn::kRowStreamBytes;
    for (int64_t t = 0; t < T; t += kMaxGroups * p.rows) {
        a.T = std::min(T - t, kMaxGroups * p.rows);
        a.x = at(x, t * x_stride * size_of(x_dtype));
        a.res = at(res, t * H * size_of(r_dtype));
        a.h = at(h, t * H * size_of(r_dtype));
        a.y = at(y, t * H * ys);
        a.rstd = rstd ? rstd + t : nullptr;
        a.scale = scale ? scale + t * scales : nullptr;
        if (hipError_t e = gn::launch_rms_fwd(a, x_dtype, r_dtype, q8, p, static_cast<hipStream_t>(stream)))
            return launch_status(e);
    }
    return GN_OK;
}

// ------------------------------------------------------------------ gradient list

int tensors_check(const gn_grad_tensor* t, int64_t n, bool clip)
{
    if (!t) return GN_ERR_NULL;
    if (n < 1) return GN_ERR_ROWS;
    for (int64_t i = 0; i < n; ++i) {
        if (t[i].numel < 0 || t[i].numel > (int64_t(1) << 48)) return GN_ERR_ROWS;
        if (!dtype_ok(t[i].dtype)) return GN_ERR_DTYPE;
        if (clip && !(t[i].out_dtype == t[i].dtype || t[i].out_dtype == GN_F32)) return GN_ERR_DTYPE;
        if (t[i].numel == 0) continue;
        if (!t[i].data || (clip && !t[i].out)) return GN_ERR_NULL;
        if (!aligned(t[i].data, size_of(t[i].dtype)) || (clip && !aligned(t[i].out, size_of(t[i].out_dtype))))
            return GN_ERR_ALIGN;
    }
    return GN_OK;
}

// Whether every output is apart from every other output and from every other tensor's data.
// Both lists are often ascending already (a model's gradients in one buffer).
bool outputs_apart(const gn_grad_tensor* t, int64_t n)
try {
    std::vector<Span> outs, ins;
    outs.reserve(size_t(n));
    ins.reserve(size_t(n));
    for (int64_t i = 0; i < n; ++i) {
        if (t[i].numel == 0) continue;
        const Span d(t[i].data, t[i].numel * size_of(t[i].dtype)), o(t[i].out, t[i].numel * size_of(t[i].out_dtype));
        outs.push_back(o);
        if (!(d.is(o) && t[i].dtype == t[i].out_dtype)) ins.push_back(d);
    }
    const auto before = [](const Span& a, const Span& b) { return a.b < b.b; };
    for (std::vector<Span>* v : {&outs, &ins})
        if (!std::is_sorted(v->begin(), v->end(), before)) std::sort(v->begin(), v->end(), before);
    for (size_t i = 1; i < outs.size(); ++i)
        if (outs[i].b < outs[i - 1].e) return false;
    // Inputs may overlap one another: walk the outputs past those that end before each input.
    size_t k = 0;
    for (const Span& d : ins) {
        while (k < outs.size() && outs[k].e <= d.b) ++k;
        if (k < outs.size() && outs[k].b < d.e) return false;
    }
    return true;
} catch (const std::bad_alloc&) {  // nothing is thrown across the ABI: out of host memory, the call is refused
    return false;
}

// The list cut into tables: entries of at most kGradMaxElems elements, empty tensors left
// out. Calls f(table) for each; every list has at least one (perhaps empty) table.
template <typename F>
int for_tables(const gn_grad_tensor* t, int64_t n, F&& f)
{
    gn::GradTable tab;
    tab.n = 0;
    tab.tiles = 0;
    bool any = false;
    const auto flush = [&]() {
        any = true;
        const int rc = f(tab);
        tab.n = 0;
        tab.tiles = 0;
        return rc;
    };
    for (int64_t i = 0; i < n; ++i)
        for (int64_t k = 0; k < t[i].numel; k += gn::kGradMaxElems) {
            const int64_t m = std::min(t[i].numel - k, gn::kGradMaxElems);
            if (tab.n == gn::kGradEntries)
                if (const int rc = flush()) return rc;
            gn::GradEntry& e = tab.e[tab.n++];
            e.data = at(t[i].data, k * size_of(t[i].dtype));
            e.out = at(t[i].out, k * size_of(t[i].out_dtype));
            e.numel = uint32_t(m);
            e.dtype = uint32_t(t[i].dtype) & 3u;
            e.out_dtype = uint32_t(t[i].out_dtype) & 3u;
            e.tile0 = tab.tiles;
            tab.tiles += uint32_t((m + gn::kGradTile - 1) / gn::kGradTile);
        }
    return tab.n || !any ? flush() : GN_OK;
}

// Tiles of the whole list.
int64_t tiles_of(const gn_grad_tensor* t, int64_t n)
{
    int64_t tiles = 0;
    for (int64_t i = 0; i < n; ++i)  // an entry's last tile may be short, whole ones divide kGradMaxElems
        tiles += (t[i].numel + gn::kGradTile - 1) / gn::kGradTile;
    return tiles;
}
static_assert(gn::kGradMaxElems % gn::kGradTile == 0, "tiles of a long tensor");

// A table's workgroups: its share of `grid` by tiles, with no more than a step's work for
// each, and one at least.
int64_t grid_of_table(const gn::GradTable& t, int64_t tiles, int64_t grid)
{
    const int64_t steps = (int64_t(t.tiles) + gn::kGradStep - 1) / gn::kGradStep;
    return std::max<int64_t>(1, std::min(steps, int64_t(t.tiles) * grid / std::max<int64_t>(tiles, 1)));
}

// Partials of the whole list (a count from the sizes alone); the workspace holds one word
// more, the factor.
int64_t partials_of(const gn_grad_tensor* t, int64_t n)
{
    const int64_t tiles = tiles_of(t, n);
    int64_t parts = 0;
    (void)for_tables(t, n, [&](const gn::GradTable& tab) {
        parts += grid_of_table(tab, tiles, gn::kGradGrid);
        return GN_OK;
    });
    return parts;
}

}  // namespace

int gn::grads(const gn_grad_tensor* t, int64_t n, int norm_type, bool clip, double max_norm, float* norm, void* ws,
              size_t ws_bytes, void* stream, int device)
{
    int rc = tensors_check(t, n, clip);
    if (rc) return rc;
    if ((norm_type != GN_NORM_2 && norm_type != GN_NORM_INF) || (clip && !(max_norm >= 0.0))) return GN_ERR_NORM;
    if (!norm || !ws) return GN_ERR_NULL;
    if (!aligned(norm, 4) || !aligned(ws, 16)) return GN_ERR_ALIGN;
    const int64_t parts = partials_of(t, n), tiles = tiles_of(t, n);
    if (ws_bytes < size_t(parts + 1) * sizeof(double)) return GN_ERR_WORKSPACE;
    const Span sn(norm, 4), sws(ws, (parts + 1) * int64_t(sizeof(double)));
    if (sn.meets(sws) || (clip && !outputs_apart(t, n))) return GN_ERR_OVERLAP;
    for (int64_t i = 0; i < n; ++i) {
        const Span d(t[i].data, t[i].numel * size_of(t[i].dtype)),
            o(clip ? t[i].out : nullptr, t[i].numel * size_of(t[i].out_dtype));
        if (t[i].numel && (meets_any(sws, {d, o}) || meets_any(sn, {d, o}))) return GN_ERR_OVERLAP;
    }
    OnDeviceOf dev(device);
    if ((rc = dev.enter(norm, stream)) || (rc = dev.holds({ws}))) return rc;
    for (int64_t i = 0; i < n && device < 0; ++i)
        if (t[i].numel && ((rc = dev.holds({t[i].data})) || (clip && t[i].out != t[i].data && (rc = dev.holds({t[i].out})))))
            return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const bool inf = norm_type == GN_NORM_INF;
    double* part = static_cast<double*>(ws);
    int64_t done = 0;
    rc = for_tables(t, n, [&](const gn::GradTable& tab) {
        const int64_t g = grid_of_table(tab, tiles, gn::kGradGrid);
        const int s = launch_status(gn::launch_grad_partials(tab, inf, part + done, g, st));
        done += g;
        return s;
    });
    if (rc) return rc;
    const bool fold = clip && tiles <= gn::kGradFoldTiles;
    float* coef = reinterpret_cast<float*>(part + parts);
    if (!fold) {
        rc = launch_status(gn::launch_grad_norm(part, parts, inf, max_norm, norm, clip ? coef : nullptr, st));
        if (rc || !clip) return rc;
    }
    float* out = fold ? norm : nullptr;
    return for_tables(t, n, [&](const gn::GradTable& tab) {
        const int64_t g = grid_of_table(tab, tiles, fold ? gn::kGradGrid : kMaxGroups);
        const int s = launch_status(gn::launch_grad_scale(tab, part, parts, inf, max_norm, out, fold ? nullptr : coef, g, st));
        out = nullptr;  // written once
        return s;
    });
}

int gn::rms_forward(const void* x, int x_dtype, int64_t x_stride, const void* residual, int r_dtype,
                    const void* weight, int w_dtype, int64_t T, int64_t H, float eps,
                    void* y, int y_dtype, void* h, float* rstd, void* stream, int device)
{
    return forward(x, x_dtype, x_stride, residual, r_dtype, weight, w_dtype, T, H, eps, y, y_dtype, -1, 0, nullptr, h,
                   rstd, stream, device);
}

int gn::rms_forward_q8(const void* x, int x_dtype, int64_t x_stride, const void* residual, int r_dtype,
                       const void* weight, int w_dtype, int64_t T, int64_t H, float eps, int64_t block,
                       void* q, int q_dtype, float* scale, void* h, float* rstd, void* stream, int device)
{
    if (q_dtype < 0) return GN_ERR_DTYPE;
    return forward(x, x_dtype, x_stride, residual, r_dtype, weight, w_dtype, T, H, eps, q, GN_F32, q_dtype, block,
                   scale, h, rstd, stream, device);
}

int gn::q8_dequantize(const void* q, int q_dtype, const float* scale, int64_t T, int64_t H, int64_t block,
                      void* out, int out_dtype, void* stream, int device)
{
    int rc = rows_check(T, H, H);
    if (rc) return rc;
    if ((q_dtype != GN_Q_INT8 && q_dtype != GN_Q_E4M3) || !dtype_ok(out_dtype)) return GN_ERR_DTYPE;
    if (block != 0 && block != 32 && block != 64 && block != 128) return GN_ERR_BLOCK;
    if (T == 0) return GN_OK;
    if (!q || !scale || !out) return GN_ERR_NULL;
    if (!aligned(scale, 4) || !aligned(out, size_of(out_dtype))) return GN_ERR_ALIGN;
    const int64_t scales = block ? (H + block - 1) / block : 1;
    if (meets_any(Span(out, T * H * size_of(out_dtype)), {Span(q, T * H), Span(scale, T * scales * 4)}))
        return GN_ERR_OVERLAP;
    OnDeviceOf dev(device);
    if ((rc = dev.enter(q, stream)) || (rc = dev.holds({scale, out}))) return rc;
    return launch_status(gn::launch_q8_dequantize(q, q_dtype, scale, T, H, block, out, out_dtype,
                                                  static_cast<hipStream_t>(stream)));
}

int gn::rms_backward(const void* dy, int dy_dtype, const void* h, int h_dtype, int64_t h_stride,
                     const float* rstd, const void* weight, int w_dtype, const void* dh,
                     int64_t T, int64_t H, void* dx, int x_dtype, void* dres, void* dweight,
                     void* workspace, size_t workspace_bytes, void* stream, int device)
{
    int rc = rows_check(T, H, h_stride);
    if (rc) return rc;
    if (!dtype_ok(h_dtype) || !dtype_ok(x_dtype) || !(x_dtype == h_dtype || h_dtype == GN_F32) ||
        !(dy_dtype == x_dtype || dy_dtype == GN_F32) ||
        !(w_dtype == GN_F32 || ((weight || dweight) && w_dtype == x_dtype)))
        return GN_ERR_DTYPE;
    if (!weight && w_dtype != GN_F32) return GN_ERR_DTYPE;
    if (T > 0 && !dx && !dres && !dweight) return GN_ERR_NULL;
    if (dweight && (!workspace || !aligned(workspace, 16) || !aligned(dweight, size_of(w_dtype))))
        return workspace ? GN_ERR_ALIGN : GN_ERR_NULL;
    if (dweight && workspace_bytes < gn_rms_workspace_bytes(T, H)) return GN_ERR_WORKSPACE;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (T == 0) {  // no row: the weight's gradient is zero
        if (!dweight) return GN_OK;
        OnDeviceOf dev(device);
        if ((rc = dev.enter(dweight, stream)) || (rc = dev.holds({workspace}))) return rc;
        return launch_status(gn::launch_rms_dweight(static_cast<float*>(workspace), 0, H, dweight, w_dtype, st));
    }
    if (!dy || !h || !rstd) return GN_ERR_NULL;
    if (!aligned(dy, size_of(dy_dtype)) || !aligned(h, size_of(h_dtype)) || !aligned(rstd, 4) ||
        !aligned(weight, size_of(w_dtype)) || !aligned(dh, size_of(h_dtype)) || !aligned(dx, size_of(x_dtype)) ||
        !aligned(dres, size_of(h_dtype)))
        return GN_ERR_ALIGN;
    const gn::BwdPlan p = gn::bwd_plan(T, H, dy_dtype == GN_F32 || h_dtype == GN_F32);
    const int64_t parts = p.parts;
    const Span sy(dy, T * H * size_of(dy_dtype)), sh(h, rows_bytes(T, H, h_stride, h_dtype)), ss(rstd, T * 4),
        sw(weight, H * size_of(w_dtype)), sd(dh, T * H * size_of(h_dtype)), ox(dx, T * H * size_of(x_dtype)),
        orr(dres, T * H * size_of(h_dtype)), ow(dweight, H * size_of(w_dtype)),
        sws(dweight ? workspace : nullptr, parts * H * 4);
    // An output may take the place of an input with the same element for element layout.
    const auto clear = [&](const Span& o, int dt) {
        return !(o.meets(sy) && !(o.is(sy) && dt == dy_dtype)) &&
               !(o.meets(sh) && !(o.b == sh.b && h_stride == H && dt == h_dtype)) &&
               !(o.meets(sd) && !(o.is(sd) && dt == h_dtype)) && !meets_any(o, {ss, sw, ow, sws});
    };
    if (!clear(ox, x_dtype) || !clear(orr, h_dtype) || ox.meets(orr) || meets_any(ow, {sy, sh, ss, sw, sd, sws}) ||
        meets_any(sws, {sy, sh, ss, sw, sd}))
        return GN_ERR_OVERLAP;
    OnDeviceOf dev(device);
    if ((rc = dev.enter(dy, stream)) ||
        (rc = dev.holds({h, rstd, weight, dh, dx, dres, dweight, dweight ? workspace : nullptr})))
        return rc;
    gn::RmsBwdArgs a{};
    a.dy = dy;
    a.h = h;
    a.w = weight;
    a.dh = dh;
    a.rstd = rstd;
    // one output in h's type, and a second where the types differ or both are asked for
    a.d = dres ? dres : x_dtype == h_dtype ? dx : nullptr;
    a.dx = a.d == dx ? nullptr : dx;
    a.part = dweight ? static_cast<float*>(workspace) : nullptr;
    a.T = T;
    a.H = H;
    a.h_stride = h_stride;
    a.parts = parts;
    a.w_dtype = w_dtype;
    a.x_dtype = x_dtype;
    a.lanes = p.lanes;
    a.rows = p.rows;
    a.inv_H = 1.0f / float(H);
    a.nt = T * H * (size_of(dy_dtype) + size_of(h_dtype) * (dh ? 2 : 1) + (dx ? size_of(x_dtype) : 0) +
                    (dres ? size_of(h_dtype) : 0)) > gn::kRowStreamBytes;
    if (hipError_t e = gn::launch_rms_bwd(a, dy_dtype, h_dtype, p, st)) return launch_status(e);
    return dweight ? launch_status(gn::launch_rms_dweight(a.part, parts, H, dweight, w_dtype, st)) : GN_OK;
}

extern "C" {

const char* gn_ops_status_string(int status)
{
    switch (status) {
        case GN_ERR_ROWS: return "invalid sizes (T >= 0, 1 <= H <= GN_RMS_MAX_COLUMNS, row stride >= H; a list of at least one tensor, sizes >= 0)";
        case GN_ERR_OVERLAP: return "an output overlaps another argument";
        case GN_ERR_BLOCK: return "block must be 0, 32, 64 or 128";
        case GN_ERR_NORM: return "norm type must be GN_NORM_2 or GN_NORM_INF, and max_norm >= 0";
        case GN_ERR_WORKSPACE: return "workspace smaller than the call's workspace query says";
        case GN_ERR_ALIGN: return "misaligned pointer (tensors to their element, workspace to 16 bytes)";
        case GN_ERR_DEVICE: return "a pointer argument is not device memory of the call's device, or the stream belongs to another device";
        default: return gn_status_string(status);
    }
}

int gn_rms_forward(const void* x, int x_dtype, int64_t x_stride, const void* residual, int r_dtype,
                   const void* weight, int w_dtype, int64_t T, int64_t H, float eps,
                   void* y, int y_dtype, void* h, float* rstd, void* stream)
{
    return gn::rms_forward(x, x_dtype, x_stride, residual, r_dtype, weight, w_dtype, T, H, eps, y, y_dtype, h,
                           rstd, stream, -1);
}

int gn_rms_forward_q8(const void* x, int x_dtype, int64_t x_stride, const void* residual, int r_dtype,
                      const void* weight, int w_dtype, int64_t T, int64_t H, float eps, int64_t block,
                      void* q, int q_dtype, float* scale, void* h, float* rstd, void* stream)
{
    return gn::rms_forward_q8(x, x_dtype, x_stride, residual, r_dtype, weight, w_dtype, T, H, eps, block, q,
                              q_dtype, scale, h, rstd, stream, -1);
}

int gn_q8_dequantize(const void* q, int q_dtype, const float* scale, int64_t T, int64_t H, int64_t block,
                     void* out, int out_dtype, void* stream)
{
    return gn::q8_dequantize(q, q_dtype, scale, T, H, block, out, out_dtype, stream, -1);
}

size_t gn_rms_workspace_bytes(int64_t T, int64_t H)
{
    if (rows_check(T, H, H)) return 0;
    // whichever the types will be
    const int64_t parts = std::max(gn::bwd_plan(T, H, false).parts, gn::bwd_plan(T, H, true).parts);
    return size_t(std::max<int64_t>(parts, 1)) * size_t(H) * sizeof(float);
}

int gn_rms_backward(const void* dy, int dy_dtype, const void* h, int h_dtype, int64_t h_stride,
                    const float* rstd, const void* weight, int w_dtype, const void* dh,
                    int64_t T, int64_t H, void* dx, int x_dtype, void* dres, void* dweight,
                    void* workspace, size_t workspace_bytes, void* stream)
{
    return gn::rms_backward(dy, dy_dtype, h, h_dtype, h_stride, rstd, weight, w_dtype, dh, T, H, dx, x_dtype, dres,
                            dweight, workspace, workspace_bytes, stream, -1);
}

size_t gn_grad_workspace_bytes(const gn_grad_tensor* tensors, int64_t n)
{
    return tensors_check(tensors, n, false) ? 0 : size_t(partials_of(tensors, n) + 1) * sizeof(double);
}

int gn_grad_norm(const gn_grad_tensor* tensors, int64_t n, int norm_type, float* norm,
                 void* workspace, size_t workspace_bytes, void* stream)
{
    return gn::grads(tensors, n, norm_type, false, 0.0, norm, workspace, workspace_bytes, stream, -1);
}

int gn_grad_clip(const gn_grad_tensor* tensors, int64_t n, int norm_type, double max_norm, float* norm,
                 void* workspace, size_t workspace_bytes, void* stream)
{
    return gn::grads(tensors, n, norm_type, true, max_norm, norm, workspace, workspace_bytes, stream, -1);
}

}  // extern "C"
