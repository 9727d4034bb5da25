// gn_join.hip -- the join of a block's output into the residual stream, forward, with the norms on
// both sides of it and 8-bit checkpoints of what its backward pass reads; and the checkpoint of
// an activation by itself.
//
//   u = x * post_rstd * post_weight;  h = round(residual_scale * residual + branch_scale * gate * u)
//   y = h * rstd * weight * (1 + scale)
//
// A row is read once into registers, reduced there twice (x for the norm after the block, h for
// the norm before the next one, which is of the rounded sum and so cannot be had from the same
// pass), and written once.
#include "gn_join_vec.hpp"

namespace gn {

namespace {

constexpr int kRowMaxWaves = kRowMaxBlock / 64;

// A row's sum and its largest magnitude (bits), over all its lanes with one barrier.
template <int W>
__device__ __forceinline__ void row_sum_max(float& sum, uint32_t& top, bool many, const Row<W>& r, uint32_t* s)
{
    uint32_t a = __float_as_uint(sum);
    if (!many) {
        sum = __uint_as_float(lanes_all<AddOp>(a, r.lanes));
        top = lanes_all<MaxBitsOp>(top, r.lanes);
        return;
    }
    a = lanes_all<AddOp>(a, 64);
    top = lanes_all<MaxBitsOp>(top, 64);
    if ((r.lane & 63) == 0) {
        s[r.lane >> 6] = a;
        s[kRowMaxWaves + (r.lane >> 6)] = top;
    }
    __syncthreads();
    const int nw = r.lanes >> 6, k = r.lane & 15;
    a = s[k < nw ? k : 0];
    top = s[kRowMaxWaves + (k < nw ? k : 0)];
    sum = __uint_as_float(lanes_all<AddOp>(k < nw ? a : 0u, 16));
    top = lanes_all<MaxBitsOp>(k < nw ? top : 0u, 16);
}

// A lane's pieces v of a row to 8 bits at q, with its scales at scale; top: the bits of the row's
// largest magnitude, for block == 0.
template <int W, int V, int END>
__device__ __forceinline__ void store_checkpoint(uint8_t* q, float* scale, int32_t block, int q_dtype, const Row<W>& r,
                                                 uint32_t top, const float (&v)[V][W])
{
    const int32_t share = lanes_of_scale(block, r);
#pragma unroll
    for (int u = 0; u < V; ++u) {
        float t[W];
#pragma unroll
        for (int e = 0; e < W; ++e) t[e] = v[u][e];
        const uint32_t m = block ? lanes_all<MaxBitsOp>(piece_amax(t), share) : top;
        store_q8<W, END>(q, scale, block, r, r.piece(u), share, scale_of(m, q_dtype), q_dtype, t);
    }
}

template <int W, int V>
__device__ __forceinline__ uint32_t lane_amax(const float (&v)[V][W])
{
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < V; ++u) m = MaxBitsOp::f(m, piece_amax(v[u]));
    return m;
}

// ------------------------------------------------------------------ join

// h and y are written after the second reduction's barrier: they may take an input's place, and
// lanes at the row's end read columns of others. CK: checkpoints may be asked for.
template <typename XT, typename HT, int W, int V, int END, bool CK>
__global__ void __launch_bounds__(kRowMaxBlock)
join_fwd_kernel(JoinArgs a)
{
    __shared__ uint32_t s_x[2 * kRowMaxWaves], s_h[2 * kRowMaxWaves];
    const int32_t sub = a.lanes > 64 ? 0 : int32_t(threadIdx.x) / a.lanes;
    const Row<W> r = row_of<W>(a.H, a.lanes, int32_t(threadIdx.x) - sub * a.lanes);
    const int64_t t = int64_t(blockIdx.x) * a.rows + sub;
    if (t >= a.T) return;  // whole rows leave, and with more than 64 lanes whole workgroups
    const bool many = V > 1 || a.lanes > 64;
    float x[V][W], h[V][W];
    Piece<XT, W> rx[V];
    Piece<HT, W> rr[V];
    load_row<XT, W, V, END>(in<XT>(a.x) + t * a.x_stride, r, a.nt, rx);
    load_row<HT, W, V, END>(in<HT>(a.res) + t * a.H, r, a.nt, rr);
    const int64_t n = a.one ? 0 : sequence_of(a.first + t, a.len);
    RawVecs<W> rv[V];
#pragma unroll
    for (int u = 0; u < V; ++u) rv[u].template load<END>(a.v, n, r, r.piece(u));
    float ss = 0.0f;
    uint32_t top = 0;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        widen_piece<XT, W, END>(rx[u], r, r.piece(u), x[u]);
        ss = ss + tree_sumsq(x[u]);
    }
    const bool row_scale = CK && a.block == 0;
    float post_rstd = 1.0f;
    if (a.post || (row_scale && a.x_q)) {
        if (row_scale) top = lane_amax(x);
        row_sum_max(ss, top, many, r, s_x);
        if (a.post) {
            post_rstd = inverse_rms(ss, a.H, a.inv_H, a.eps);
            if (a.post_rstd && r.lane == 0) a.post_rstd[t] = post_rstd;
        }
    }
    if constexpr (CK)
        if (a.x_q) store_checkpoint<W, V, END>(a.x_q + t * a.H, a.x_scale + t * a.scales, a.block, a.q_dtype, r, top, x);
    ss = 0.0f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        float c[W];
        rv[u].template branch<END>(a.v, r, r.piece(u), c);
        widen_piece<HT, W, END>(rr[u], r, r.piece(u), h[u]);
#pragma unroll
        for (int e = 0; e < W; ++e) h[u][e] = fmaf(x[u][e] * post_rstd, c[e], a.residual_scale * h[u][e]);
        rr[u].narrow(h[u]);  // taken as stored
        rr[u].widen(h[u]);
        if (END == kEnds && r.piece(u) >= r.full) {  // columns that are not its own: 0 * inf is NaN
            const int32_t skip = r.skip(r.piece(u));
#pragma unroll
            for (int e = 0; e < W; ++e) h[u][e] = e < skip ? 0.0f : h[u][e];
        }
        ss = ss + tree_sumsq(h[u]);
    }
    top = row_scale ? lane_amax(h) : 0u;
    row_sum_max(ss, top, many, r, s_h);
#pragma unroll
    for (int u = 0; u < V; ++u) store_values<HT, W, END>(out<HT>(a.h) + t * a.H, r, r.piece(u), h[u]);
    if constexpr (CK)
        if (a.h_q) store_checkpoint<W, V, END>(a.h_q + t * a.H, a.h_scale + t * a.scales, a.block, a.q_dtype, r, top, h);
    if (!a.y) return;
    const float rstd = inverse_rms(ss, a.H, a.inv_H, a.eps);
    if (a.rstd && r.lane == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        float m[W];
        rv[u].template multiplier<END>(a.v, r, r.piece(u), m);
#pragma unroll
        for (int e = 0; e < W; ++e) h[u][e] = h[u][e] * rstd * m[e];
        store_values<XT, W, END>(out<XT>(a.y) + t * a.H, r, r.piece(u), h[u]);
    }
}

template <typename XT, typename HT, int W>
hipError_t fwd(const JoinArgs& a, const RowPlan& p, hipStream_t st)
{
    const dim3 grid = dim3(unsigned((a.T + p.rows - 1) / p.rows));
    return with_row<W>(p, a.H, [&](auto v, auto end) {
        constexpr int V = decltype(v)::value;
        constexpr int E = decltype(end)::value;
        return a.h_q || a.x_q ? launch(join_fwd_kernel<XT, HT, W, V, E, true>, grid, dim3(p.block), st, a)
                              : launch(join_fwd_kernel<XT, HT, W, V, E, false>, grid, dim3(p.block), st, a);
    });
}

// ------------------------------------------------------------------ a checkpoint by itself

template <typename XT, int W, int V, int END>
__global__ void __launch_bounds__(kRowMaxBlock)
quantize_kernel(QuantArgs a)
{
    __shared__ uint32_t s_top[2 * kRowMaxWaves];
    const int32_t sub = a.lanes > 64 ? 0 : int32_t(threadIdx.x) / a.lanes;
    const Row<W> r = row_of<W>(a.H, a.lanes, int32_t(threadIdx.x) - sub * a.lanes);
    const int64_t t = int64_t(blockIdx.x) * a.rows + sub;
    if (t >= a.T) return;
    float x[V][W];
    Piece<XT, W> rx[V];
    load_row<XT, W, V, END>(in<XT>(a.x) + t * a.x_stride, r, a.nt, rx);
#pragma unroll
    for (int u = 0; u < V; ++u) widen_piece<XT, W, END>(rx[u], r, r.piece(u), x[u]);
    uint32_t top = 0;
    if (a.block == 0) {
        float unused = 0.0f;
        top = lane_amax(x);
        row_sum_max(unused, top, V > 1 || a.lanes > 64, r, s_top);
    }
    store_checkpoint<W, V, END>(a.q + t * a.H, a.scale + t * a.scales, a.block, a.q_dtype, r, top, x);
}

}  // namespace

hipError_t launch_join_fwd(const JoinArgs& a, int x_dtype, int r_dtype, const RowPlan& p, hipStream_t st)
{
    if (x_dtype == GN_F32) return fwd<float, float, 4>(a, p, st);
    if (r_dtype == GN_F32)
        return x_dtype == GN_BF16 ? fwd<uint16_t, float, 4>(a, p, st) : fwd<_Float16, float, 4>(a, p, st);
    return x_dtype == GN_BF16 ? fwd<uint16_t, uint16_t, 8>(a, p, st) : fwd<_Float16, _Float16, 8>(a, p, st);
}

hipError_t launch_q8_quantize(const QuantArgs& a, int x_dtype, const RowPlan& p, hipStream_t st)
{
    return with_type(x_dtype, [&](auto t) {
        using XT = decltype(t);
        constexpr int W = sizeof(XT) == 4 ? 4 : 8;
        return with_row<W>(p, a.H, [&](auto v, auto end) {
            return launch(quantize_kernel<XT, W, decltype(v)::value, decltype(end)::value>,
                          dim3(unsigned((a.T + p.rows - 1) / p.rows)), dim3(p.block), st, a);
        });
    });
}

}  // namespace gn
