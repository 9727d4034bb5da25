// gn_rms_bwd.hip -- backward of the root-mean-square norm over rows.
//
//   d = rstd * (dy * weight - h * rstd * c) + dh,  c = mean(dy * weight * h * rstd)
//   dweight = sum over rows of dy * h * rstd
//
// Bound by the bytes it moves (12 operations for 8 bytes): a row of each tensor is read once
// into registers and its gradient written once. Measured, bf16, 8192 x 4096 with dh: 47.8 us,
// 5.6 TB/s, 44 of them here (6.1 TB/s) and 4 in the second kernel; 131072 x 128 without dh: 20.5
// us, 17 and 4. One persistent workgroup of 512 threads for each CU: with two the partial sums
// double and the call takes 53 us, and workgroups of 1024 threads, 128 registers a lane, 85.
#include "gn_rows.hpp"

namespace gn {

namespace {

// One piece of a row: h becomes xhat, dy becomes dy * weight, dw takes dy * xhat; returns the
// piece's sum of dy * weight * xhat.
template <int W>
__device__ __forceinline__ float take_sums(float (&dy)[W], float (&h)[W], const float (&w)[W], float rstd,
                                           float (&dw)[W])
{
#pragma unroll
    for (int e = 0; e < W; ++e) {
        h[e] = h[e] * rstd;
        dw[e] = fmaf(dy[e], h[e], dw[e]);
        dy[e] = dy[e] * w[e];
    }
    return tree_sumprod(dy, h);
}

// The gradient of piece i of the row whose first element is `at`, stored: rstd * g + dh - xhat
// * c, with g = dy * weight and c the mean of g * xhat times rstd.
template <typename HT, bool DH, int W, int END>
__device__ __forceinline__ void store_gradient(const RmsBwdArgs& a, const Row<W>& r, int64_t at, int32_t i,
                                               const float (&g)[W], const float (&xhat)[W], const float (&dh)[W],
                                               float rstd, float c)
{
    float d[W];
#pragma unroll
    for (int e = 0; e < W; ++e) d[e] = DH ? fmaf(g[e], rstd, fmaf(-xhat[e], c, dh[e])) : fmaf(g[e], rstd, -xhat[e] * c);
    if (a.d) store_values<HT, W, END>(out<HT>(a.d) + at, r, i, d);
    if (!a.dx) return;
    if (sizeof(HT) == 2)  // x's type is h's, unless that is fp32
        store_values<HT, W, END>(out<HT>(a.dx) + at, r, i, d);
    else if (a.x_dtype == GN_F32)
        store_values<float, W, END>(out<float>(a.dx) + at, r, i, d);
    else if (a.x_dtype == GN_BF16)
        store_values<uint16_t, W, END>(out<uint16_t>(a.dx) + at, r, i, d);
    else
        store_values<_Float16, W, END>(out<_Float16>(a.dx) + at, r, i, d);
}

// Workgroup b takes the row groups b, b + parts, ... (a.rows rows at once, a.lanes lanes
// each; MANY: more than 64). DEPTH groups' loads are in flight behind the one in use, refilled
// as soon as a group is widened. With 8 columns a lane two, so that no wait for loads is also
// one for the stores just issued (43690 x 768 bf16: 54 us with one, 50 with two); with 16 one
// (8192 x 4096 bf16: 48 us with one, 49 with two); fewer where registers end. Every lane keeps its columns' sums of
// dy * xhat in registers over all groups; at the end the workgroup adds its rows' sums in LDS
// and leaves one partial sum for each column in the workspace.
// NT: nontemporal loads, a variant of its own, since a choice in the loop is a branch that
// loads in flight are waited for at (8192 x 4096 bf16: 50 -> 58 us).
template <typename DT, typename HT, bool DH, int W, int V, bool MANY, int END, int DEPTH, bool NT>
__global__ void __launch_bounds__(kBwdBlock)
rms_bwd_kernel(RmsBwdArgs a)
{
    __shared__ uint32_t s_sum[2][kBwdBlock / 64];
    __shared__ __align__(16) float s_dw[kBwdBlock * W];
    const int32_t sub = int32_t(threadIdx.x) / a.lanes;
    const Row<W> r = row_of<W>(a.H, a.lanes, int32_t(threadIdx.x) - sub * a.lanes);
    float w[V][W], dw[V][W];
#pragma unroll
    for (int u = 0; u < V; ++u) {
        load_weight<W, END>(a.w, a.w_dtype, r, r.piece(u), w[u]);
#pragma unroll
        for (int e = 0; e < W; ++e) dw[u][e] = 0.0f;
    }
    struct Loaded {
        Piece<DT, W> dy[V];
        Piece<HT, W> h[V];
        Piece<HT, W> dh[DH ? V : 1];
        float rstd;
    };
    // The row in use and the row loaded next, with their first elements' places.
    const int64_t step = a.parts * a.rows;
    int64_t t = int64_t(blockIdx.x) * a.rows + sub, at = t * a.H;
    int64_t load_t = t, load_at = at, load_h = t * a.h_stride;
    const auto load = [&](Loaded& l) {
        const bool past = load_t >= a.T;  // past the last row: the last row again, unused
        const int64_t k = past ? (a.T - 1) * a.H : load_at, kh = past ? (a.T - 1) * a.h_stride : load_h;
        load_row_as<DT, W, V, END, NT>(in<DT>(a.dy) + k, r, l.dy);
        load_row_as<HT, W, V, END, NT>(in<HT>(a.h) + kh, r, l.h);
        if constexpr (DH) load_row_as<HT, W, V, END, NT>(in<HT>(a.dh) + k, r, l.dh);
        l.rstd = a.rstd[past ? a.T - 1 : load_t];
        load_t += step;
        load_at += step * a.H;
        load_h += step * a.h_stride;
    };
    int phase = 0;
    const auto group = [&](Loaded& l) {
        if constexpr (DEPTH == 0) load(l);
        float dy[V][W], h[V][W], d[DH ? V : 1][W];
        const float rstd = l.rstd;
#pragma unroll
        for (int u = 0; u < V; ++u) {
            widen_piece<DT, W, END>(l.dy[u], r, r.piece(u), dy[u]);
            widen_piece<HT, W, END>(l.h[u], r, r.piece(u), h[u]);
            if constexpr (DH) l.dh[u].widen(d[u]);
        }
        if constexpr (DEPTH > 0) load(l);
        float c = 0.0f;
        if (t < a.T) {
#pragma unroll
            for (int u = 0; u < V; ++u) c = c + take_sums<W>(dy[u], h[u], w[u], rstd, dw[u]);
        }
        if (a.d || a.dx) {
            c = row_sum<MANY>(c, r, s_sum[phase] + sub * (r.lanes >> 6)) * a.inv_H;
            phase ^= 1;
            if (t < a.T) {  // after the row's barrier
#pragma unroll
                for (int u = 0; u < V; ++u)
                    store_gradient<HT, DH, W, END>(a, r, at, r.piece(u), dy[u], h[u], d[DH ? u : 0], rstd, c * rstd);
            }
        }
        t += step;
        at += step * a.H;
    };
    const int64_t groups = (a.T + a.rows - 1) / a.rows;
    Loaded l[DEPTH > 1 ? DEPTH : 1];
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) load(l[k]);
    for (int64_t g = blockIdx.x; g < groups;) {
#pragma unroll
        for (int k = 0; k < (DEPTH > 1 ? DEPTH : 1); ++k) {
            if (k && g >= groups) break;
            group(l[k]);
            g += a.parts;
        }
    }
    if (!a.part) return;
    float* part = a.part + int64_t(blockIdx.x) * a.H;
    if (a.rows == 1) {
#pragma unroll
        for (int u = 0; u < V; ++u) store_values<float, W, END>(part, r, r.piece(u), dw[u]);
        return;
    }
#pragma unroll
    for (int u = 0; u < V; ++u) {
        if (u) __syncthreads();
#pragma unroll
        for (int e = 0; e < W; ++e) s_dw[threadIdx.x * W + e] = dw[u][e];
        __syncthreads();
        const int32_t first = u * a.lanes * W, n = a.lanes * W;
        for (int32_t k = threadIdx.x; k < n; k += blockDim.x) {
            const int32_t i = first / W + k / W, e = k % W;
            if (END == kTiny ? first + k >= r.H : e < r.skip(i)) continue;
            float s = s_dw[k];
            for (int32_t j = 1; j < a.rows; ++j) s = s + s_dw[j * n + k];
            part[r.column(i) + e] = s;
        }
    }
}

// Rows of more than 512 lanes, which leave 128 registers a lane: a row is read twice, for its
// sums and, from the caches, for its gradient, 16 columns a lane at a time, and the sums of
// dy * xhat are kept in LDS, whose traffic is a twelfth of the row's time in memory. One row
// in a workgroup.
template <typename DT, typename HT, bool DH, int W, int V, int END>
__global__ void __launch_bounds__(kRowMaxBlock)
rms_bwd_wide_kernel(RmsBwdArgs a)
{
    constexpr int kAtOnce = 16 / W, kFours = W / 4;
    static_assert(V % kAtOnce == 0, "whole turns");
    __shared__ uint32_t s_sum[2][kRowMaxBlock / 64];
    __shared__ f32x4 s_dw[V * kFours * kRowMaxBlock];
    const Row<W> r = row_of<W>(a.H, a.lanes, int32_t(threadIdx.x));
    const auto dw_of = [&](int u, int k) -> f32x4& { return s_dw[(u * kFours + k) * kRowMaxBlock + int(threadIdx.x)]; };
#pragma unroll 1
    for (int u = 0; u < V; ++u)
#pragma unroll
        for (int k = 0; k < kFours; ++k) dw_of(u, k) = f32x4{0.0f, 0.0f, 0.0f, 0.0f};  // a lane's own
    int phase = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += a.parts, phase ^= 1) {
        const int64_t at = t * a.H;
        const DT* dy_row = in<DT>(a.dy) + at;
        const HT* h_row = in<HT>(a.h) + t * a.h_stride;
        const float rstd = a.rstd[t];
        float c = 0.0f;
#pragma unroll 1
        for (int u0 = 0; u0 < V; u0 += kAtOnce) {
            Piece<DT, W> rdy[kAtOnce];
            Piece<HT, W> rh[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                load_piece<DT, W, END, false>(dy_row, r, r.piece(u0 + u), rdy[u]);
                load_piece<HT, W, END, false>(h_row, r, r.piece(u0 + u), rh[u]);
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int32_t i = r.piece(u0 + u);
                float dy[W], h[W], w[W], dw[W];
                load_weight<W, END>(a.w, a.w_dtype, r, i, w);
                widen_piece<DT, W, END>(rdy[u], r, i, dy);
                widen_piece<HT, W, END>(rh[u], r, i, h);
#pragma unroll
                for (int e = 0; e < W; ++e) dw[e] = dw_of(u0 + u, e / 4)[e & 3];
                c = c + take_sums<W>(dy, h, w, rstd, dw);
#pragma unroll
                for (int k = 0; k < kFours; ++k)
                    dw_of(u0 + u, k) = f32x4{dw[4 * k], dw[4 * k + 1], dw[4 * k + 2], dw[4 * k + 3]};
            }
        }
        if (!a.d && !a.dx) continue;
        c = row_sum<true>(c, r, s_sum[phase]) * a.inv_H * rstd;
#pragma unroll 1
        for (int u0 = 0; u0 < V; u0 += kAtOnce) {
            Piece<DT, W> rdy[kAtOnce];
            Piece<HT, W> rh[kAtOnce], rdh[DH ? kAtOnce : 1];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                load_piece<DT, W, END, false>(dy_row, r, r.piece(u0 + u), rdy[u]);
                load_piece<HT, W, END, false>(h_row, r, r.piece(u0 + u), rh[u]);
                if constexpr (DH) load_piece<HT, W, END, false>(in<HT>(a.dh) + at, r, r.piece(u0 + u), rdh[u]);
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int32_t i = r.piece(u0 + u);
                float dy[W], h[W], d[W], w[W];
                load_weight<W, END>(a.w, a.w_dtype, r, i, w);
                widen_piece<DT, W, END>(rdy[u], r, i, dy);
                widen_piece<HT, W, END>(rh[u], r, i, h);
                if constexpr (DH) rdh[u].widen(d);
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    h[e] = h[e] * rstd;
                    dy[e] = dy[e] * w[e];
                }
                store_gradient<HT, DH, W, END>(a, r, at, i, dy, h, d, rstd, c);
            }
        }
    }
    if (!a.part) return;
#pragma unroll 1
    for (int u = 0; u < V; ++u) {
        float dw[W];
#pragma unroll
        for (int e = 0; e < W; ++e) dw[e] = dw_of(u, e / 4)[e & 3];
        store_values<float, W, END>(a.part + int64_t(blockIdx.x) * a.H, r, r.piece(u), dw);
    }
}

// A workgroup adds 32 columns of all parts: thread (slice, quad) takes 4 columns of the parts
// slice, slice + 128, ... in order; the 8 slices of a wave are added by lane exchanges, the
// waves in order. Bound by one trip to memory, not by bytes: a thread's few loads are in
// flight together. Workgroups of 256 threads, backward of 8192 x 4096 bf16 47.7 us against 47.8
// with these, of 131072 x 128 20.2 against 20.5, but of 509 x 1001 fp32 9.35 against 9.1.
constexpr int kDwBlock = 1024, kDwCols = 32, kDwSlices = kDwBlock / (kDwCols / 4);

__global__ void __launch_bounds__(kDwBlock)
rms_dweight_kernel(const float* part, int64_t parts, int64_t H, void* dw, int w_dtype)
{
    __shared__ float s[kDwBlock / 64][kDwCols];
    const int quad = threadIdx.x & 7, slice = threadIdx.x >> 3;
    const int64_t c = int64_t(blockIdx.x) * kDwCols + quad * 4;
    const int n = H - c >= 4 ? 4 : H > c ? int(H - c) : 0;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n == 4) {
#pragma unroll 8
        for (int64_t p = slice; p < parts; p += kDwSlices) {
            Piece<float, 4> q;
            q.load<false>(part + p * H + c);
            float x[4];
            q.widen(x);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = v[e] + x[e];
        }
    } else {
        for (int64_t p = slice; p < parts; p += kDwSlices)
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < n) v[e] = v[e] + part[p * H + c + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // lanes 8, 16 and 32 apart
        uint32_t b = __float_as_uint(v[e]);
        b = AddOp::f(b, dpp<0x128>(b));
        const auto x = __builtin_amdgcn_permlane16_swap(b, b, false, false);
        b = AddOp::f(x[0], x[1]);
        const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
        v[e] = __uint_as_float(AddOp::f(y[0], y[1]));
    }
    if ((threadIdx.x & 63) < 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[threadIdx.x >> 6][quad * 4 + e] = v[e];
    __syncthreads();
    const int64_t col = int64_t(blockIdx.x) * kDwCols + threadIdx.x;
    if (threadIdx.x < kDwCols && col < H) {
        float x = s[0][threadIdx.x];
#pragma unroll
        for (int k = 1; k < kDwBlock / 64; ++k) x = x + s[k][threadIdx.x];
        if (w_dtype == GN_F32)
            Io<float>::store1(out<float>(dw) + col, x);
        else if (w_dtype == GN_BF16)
            Io<uint16_t>::store1(out<uint16_t>(dw) + col, x);
        else
            Io<_Float16>::store1(out<_Float16>(dw) + col, x);
    }
}

template <typename DT, typename HT>
hipError_t bwd(const RmsBwdArgs& a, const BwdPlan& p, hipStream_t st)
{
    constexpr int W = sizeof(DT) == 4 || sizeof(HT) == 4 ? 4 : 8;
    return with_row<W>(p, a.H, [&](auto v, auto end) {
        constexpr int V = decltype(v)::value;
        constexpr int E = decltype(end)::value;
        constexpr int kDepth = V * W <= 8 ? 2 : V * W <= 16 || W == 8 ? 1 : 0;
        const dim3 grid = dim3(unsigned(a.parts)), block = dim3(p.block);
        const auto go = [&](auto many, auto nt) {
            constexpr bool kMany = decltype(many)::value, kNt = decltype(nt)::value;
            return a.dh ? launch(rms_bwd_kernel<DT, HT, true, W, V, kMany, E, kDepth, kNt>, grid, block, st, a)
                        : launch(rms_bwd_kernel<DT, HT, false, W, V, kMany, E, kDepth, kNt>, grid, block, st, a);
        };
        const std::true_type yes;
        const std::false_type no;
        if constexpr (V * W == 32)
            if (p.block > kBwdBlock)
                return a.dh ? launch(rms_bwd_wide_kernel<DT, HT, true, W, V, E>, grid, block, st, a)
                            : launch(rms_bwd_wide_kernel<DT, HT, false, W, V, E>, grid, block, st, a);
        if constexpr (V == 1)
            if (p.lanes <= 64) {
                if constexpr (E == kExact)
                    if (a.nt) return go(no, yes);
                return go(no, no);
            }
        if constexpr (E == kExact)
            if (a.nt) return go(yes, yes);
        if constexpr (E == kTiny)
            return hipErrorInvalidValue;  // one lane, above
        else
            return go(yes, no);
    });
}

}  // namespace

hipError_t launch_rms_bwd(const RmsBwdArgs& a, int dy_dtype, int h_dtype, const BwdPlan& p, hipStream_t st)
{
    if (h_dtype == GN_BF16)
        return dy_dtype == GN_F32 ? bwd<float, uint16_t>(a, p, st) : bwd<uint16_t, uint16_t>(a, p, st);
    if (h_dtype == GN_F16)
        return dy_dtype == GN_F32 ? bwd<float, _Float16>(a, p, st) : bwd<_Float16, _Float16>(a, p, st);
    if (dy_dtype == GN_BF16) return bwd<uint16_t, float>(a, p, st);
    if (dy_dtype == GN_F16) return bwd<_Float16, float>(a, p, st);
    return bwd<float, float>(a, p, st);
}

hipError_t launch_rms_dweight(const float* part, int64_t parts, int64_t H, void* dw, int w_dtype, hipStream_t st)
{
    return launch(rms_dweight_kernel, dim3(unsigned((H + kDwCols - 1) / kDwCols)), dim3(kDwBlock), st, part, parts, H,
                  dw, w_dtype);
}

}  // namespace gn
