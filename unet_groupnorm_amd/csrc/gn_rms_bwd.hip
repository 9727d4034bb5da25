// gn_rms_bwd.hip -- backward of the root-mean-square norm over rows.
//
//   d = rstd * (dy * weight - h * rstd * c) + dh,  c = mean(dy * weight * h * rstd)
//   dweight = sum over rows of dy * h * rstd
//
// Bound by the bytes it moves (12 operations for 8 bytes): a row of each tensor is read once
// into registers and its gradient written once.
#include "gn_rows.hpp"

namespace gn {

namespace {

// Workgroup b takes the row groups b, b + parts, ... (a.rows rows at once, a.lanes lanes
// each); the next group's vectors are loaded before this group's are used. Every lane keeps
// its columns' sums of dy * xhat in registers over all of them; at the end the workgroup adds
// its rows' sums in LDS and leaves one partial sum for each column in the workspace.
template <typename DT, typename HT, bool DH, int W, int V, bool EXACT, int BLOCK>
__global__ void __launch_bounds__(BLOCK)
rms_bwd_kernel(RmsBwdArgs a)
{
    __shared__ uint32_t s_sum[2][BLOCK / 64];
    __shared__ __align__(16) float s_dw[BLOCK * W];
    const int32_t sub = int32_t(threadIdx.x) / a.lanes;
    const Row<W> r = row_of<W>(a.H, a.lanes, int32_t(threadIdx.x) - sub * a.lanes);
    float w[V][W], dw[V][W];
    load_weight<W, V, EXACT>(a.w, a.w_dtype, r, w);
#pragma unroll
    for (int u = 0; u < V; ++u)
#pragma unroll
        for (int e = 0; e < W; ++e) dw[u][e] = 0.0f;
    Piece<DT, W> next_dy[V];
    Piece<HT, W> next_h[V], next_dh[V];
    float next_rstd;
    const auto load = [&](int64_t t) {  // past the last row: the last row again, unused
        t = t < a.T ? t : a.T - 1;
        load_row<DT, W, V, EXACT>(in<DT>(a.dy) + t * a.H, r, a.nt, next_dy);
        load_row<HT, W, V, EXACT>(in<HT>(a.h) + t * a.h_stride, r, a.nt, next_h);
        if constexpr (DH) load_row<HT, W, V, EXACT>(in<HT>(a.dh) + t * a.H, r, a.nt, next_dh);
        next_rstd = a.rstd[t];
    };
    const int64_t groups = (a.T + a.rows - 1) / a.rows;
    int phase = 0;
    load(int64_t(blockIdx.x) * a.rows + sub);
    for (int64_t g = blockIdx.x; g < groups; g += a.parts, phase ^= 1) {
        const int64_t t = g * a.rows + sub;
        float dy[V][W], h[V][W], d[V][W];
        widen_row<DT, W, V>(next_dy, dy);
        widen_row<HT, W, V>(next_h, h);
        if constexpr (DH) widen_row<HT, W, V>(next_dh, d);
        const float rstd = next_rstd;
        if (g + a.parts < groups) load(t + a.parts * a.rows);
        const bool row = t < a.T;
        float c = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u) {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                h[u][e] = h[u][e] * rstd;
                if (row) dw[u][e] = fmaf(dy[u][e], h[u][e], dw[u][e]);
                dy[u][e] = dy[u][e] * w[u][e];
            }
            c = c + tree_sumprod(dy[u], h[u]);
        }
        if (!a.dx && !a.dres) continue;
        c = row_sum(c, r, s_sum[phase] + sub * (r.lanes >> 6)) / float(a.H);
        if (!row) continue;  // after the row's barrier
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int e = 0; e < W; ++e) {
                const float v = rstd * fmaf(-h[u][e], c, dy[u][e]);
                dy[u][e] = DH ? v + d[u][e] : v;
            }
        if (a.dres) store_row<HT, W, V, EXACT>(out<HT>(a.dres) + t * a.H, r, dy);
        if (a.dx) {
            if (sizeof(HT) == 2)
                store_row<HT, W, V, EXACT>(out<HT>(a.dx) + t * a.H, r, dy);
            else if (a.x_dtype == GN_F32)
                store_f32<W, V, EXACT>(out<float>(a.dx) + t * a.H, r, dy);
            else if (a.x_dtype == GN_BF16)
                store_row<uint16_t, W, V, EXACT>(out<uint16_t>(a.dx) + t * a.H, r, dy);
            else
                store_row<_Float16, W, V, EXACT>(out<_Float16>(a.dx) + t * a.H, r, dy);
        }
    }
    if (!a.part) return;
    float* part = a.part + int64_t(blockIdx.x) * a.H;
    if (a.rows == 1) {
        store_f32<W, V, EXACT>(part, r, dw);
        return;
    }
#pragma unroll
    for (int u = 0; u < V; ++u) {
        if (u) __syncthreads();
#pragma unroll
        for (int e = 0; e < W; ++e) s_dw[threadIdx.x * W + e] = dw[u][e];
        __syncthreads();
        const int32_t first = u * a.lanes * W, n = a.lanes * W;
        for (int32_t c = threadIdx.x; c < n && first + c < a.H; c += blockDim.x) {
            float s = s_dw[c];
            for (int32_t k = 1; k < a.rows; ++k) s = s + s_dw[k * n + c];
            part[first + c] = s;
        }
    }
}

// A workgroup adds 32 columns of all parts: thread (slice, quad) takes 4 columns of the parts
// slice, slice + 128, ... in order; the 8 slices of a wave are added by lane exchanges, the
// waves in order. Bound by one trip to memory, not by bytes: a thread's few loads are in
// flight together.
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
    return with_row<W>(p, [&](auto v, auto exact) {
        constexpr int V = decltype(v)::value;
        constexpr bool E = decltype(exact)::value;
        const dim3 grid = dim3(unsigned(a.parts)), block = dim3(p.block);
        // only the widest rows take more than 512 lanes, with the most pieces a lane
        if (V * W < 32 || p.block <= kBwdBlock)
            return a.dh ? launch(rms_bwd_kernel<DT, HT, true, W, V, E, kBwdBlock>, grid, block, st, a)
                        : launch(rms_bwd_kernel<DT, HT, false, W, V, E, kBwdBlock>, grid, block, st, a);
        if constexpr (V * W == 32)
            return a.dh ? launch(rms_bwd_kernel<DT, HT, true, W, V, E, kRowMaxBlock>, grid, block, st, a)
                        : launch(rms_bwd_kernel<DT, HT, false, W, V, E, kRowMaxBlock>, grid, block, st, a);
        return hipErrorInvalidValue;
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
