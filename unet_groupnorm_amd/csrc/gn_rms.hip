// gn_rms.hip -- the root-mean-square norm over rows, forward, with the residual's addition
// (output in x's dtype, fp32 or 8 bits with scales), and the 8-bit form's values.
//
//   h = round(x + residual);  rstd = 1 / sqrt(mean(h^2) + eps);  y = h * rstd * weight
//
// Bound by the bytes it moves (5 operations for 7 to 8 bytes): a row is read once into
// registers, reduced there, and written once.
#include <algorithm>

#include "gn_rows.hpp"

namespace gn {

namespace {

constexpr int kRowMaxWaves = kRowMaxBlock / 64;

// ------------------------------------------------------------------ 8 bits

constexpr float kQMin = 0x1p-126f;  // smallest scale, the smallest normal fp32

// 4 quotients, |v| <= qmax, to 4 bytes: nearest, ties to even.
__device__ __forceinline__ uint32_t quantize4(float a, float b, float c, float d, int q_dtype)
{
    if (q_dtype == GN_Q_INT8)
        return (uint32_t(int32_t(rintf(a))) & 0xffu) | ((uint32_t(int32_t(rintf(b))) & 0xffu) << 8) |
               ((uint32_t(int32_t(rintf(c))) & 0xffu) << 16) | (uint32_t(int32_t(rintf(d))) << 24);
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true));
}

// W (4 or 8) quotients to n of their W bytes.
template <int W>
__device__ __forceinline__ void store_q(uint8_t* p, int n, const float (&v)[W], int q_dtype)
{
    uint32_t q[W / 4];
#pragma unroll
    for (int k = 0; k < W / 4; ++k) q[k] = quantize4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3], q_dtype);
    if (n >= W) {
        typedef uint32_t WordsAny __attribute__((ext_vector_type(W / 4), aligned(1)));
        WordsAny t;
#pragma unroll
        for (int k = 0; k < W / 4; ++k) t[k] = q[k];
        *reinterpret_cast<WordsAny*>(p) = t;
    } else {
#pragma unroll
        for (int e = 0; e < W - 1; ++e)
            if (e < n) p[e] = uint8_t((q[e / 4] >> (8 * (e & 3))) & 0xffu);
    }
}

struct Scaled {
    float scale, inv;
};

// The scale of a run whose largest magnitude has the bits `amax`.
__device__ __forceinline__ Scaled scale_of(uint32_t amax, float qmax)
{
    if (amax >= 0x7f800000u) return Scaled{__uint_as_float(0x7fc00000u), 0.0f};
    const float s = fmaxf(__uint_as_float(amax) / qmax, kQMin);
    return Scaled{s, 1.0f / s};
}

// ------------------------------------------------------------------ forward

template <typename XT, typename RT, int W, int V, bool EXACT, bool Q8>
__global__ void __launch_bounds__(kRowMaxBlock)
rms_fwd_kernel(RmsArgs a)
{
    constexpr bool kRes = !std::is_void<RT>::value;
    using HT = typename std::conditional<kRes, RT, XT>::type;
    __shared__ uint32_t s_sum[kRowMaxWaves], s_max[kRowMaxWaves];
    const int32_t sub = a.lanes > 64 ? 0 : int32_t(threadIdx.x) / a.lanes;
    const Row<W> r = row_of<W>(a.H, a.lanes, int32_t(threadIdx.x) - sub * a.lanes);
    const int64_t t = int64_t(blockIdx.x) * a.rows + sub;
    if (t >= a.T) return;  // whole rows leave, and with more than 64 lanes whole workgroups
    float h[V][W], w[V][W];
    Piece<XT, W> rx[V];
    load_row<XT, W, V, EXACT>(in<XT>(a.x) + t * a.x_stride, r, a.nt, rx);
    if constexpr (kRes) {
        float d[V][W];
        Piece<HT, W> rd[V];
        load_row<HT, W, V, EXACT>(in<HT>(a.res) + t * a.H, r, a.nt, rd);
        load_weight<W, V, EXACT>(a.w, a.w_dtype, r, w);
        widen_row<XT, W, V>(rx, h);
        widen_row<HT, W, V>(rd, d);
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int e = 0; e < W; ++e) h[u][e] = round_to<HT>(h[u][e] + d[u][e]);
        store_row<HT, W, V, EXACT>(out<HT>(a.h) + t * a.H, r, h);
    } else {
        load_weight<W, V, EXACT>(a.w, a.w_dtype, r, w);
        widen_row<XT, W, V>(rx, h);
    }
    float ss = tree_sumsq(h[0]);
#pragma unroll
    for (int u = 1; u < V; ++u) ss = ss + tree_sumsq(h[u]);
    ss = row_sum(ss, r, s_sum);
    const float rstd = 1.0f / sqrtf(ss / float(a.H) + a.eps);
    if (a.rstd && r.lane == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int u = 0; u < V; ++u)
#pragma unroll
        for (int e = 0; e < W; ++e) h[u][e] = h[u][e] * rstd * w[u][e];
    if constexpr (!Q8) {
        if (W == 4 && a.y_f32)
            store_f32<W, V, EXACT>(out<float>(a.y) + t * a.H, r, h);
        else
            store_row<XT, W, V, EXACT>(out<XT>(a.y) + t * a.H, r, h);
    } else {
        const float qmax = a.q_dtype == GN_Q_INT8 ? 127.0f : 448.0f;
        uint32_t m[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            m[u] = 0;
#pragma unroll
            for (int e = 0; e < W; ++e) m[u] = MaxBitsOp::f(m[u], __float_as_uint(h[u][e]) & 0x7fffffffu);
        }
        // Lanes that share a scale: the row's, or block / W neighbours (a row of fewer lanes
        // than that is one run).
        const int32_t share = a.block == 0 ? r.lanes : a.block / W < r.lanes ? a.block / W : r.lanes;
        if (a.block == 0) {
#pragma unroll
            for (int u = 1; u < V; ++u) m[0] = MaxBitsOp::f(m[0], m[u]);
            m[0] = row_all<MaxBitsOp>(m[0], r, s_max);
        }
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int32_t i = r.piece(u);
            const uint32_t amax = a.block == 0 ? m[0] : lanes_all<MaxBitsOp>(m[u], share);
            const Scaled sc = scale_of(amax, qmax);
            const bool bad = amax >= 0x7f800000u;
            float q[W];
#pragma unroll
            for (int e = 0; e < W; ++e) q[e] = bad ? 0.0f : h[u][e] * sc.inv;
            const int n = EXACT || i < r.full ? W : i == r.full ? r.tail : 0;
            if (n) {
                store_q<W>(out<uint8_t>(a.y) + t * a.H + i * W, n, q, a.q_dtype);
                if (a.block == 0 ? u == 0 && r.lane == 0 : i % share == 0)
                    a.scale[t * a.scales + (a.block == 0 ? 0 : i / share)] = sc.scale;
            }
        }
    }
}

// ------------------------------------------------------------------ values of the 8-bit form

// A workgroup takes whole rows' pieces of W columns in turn (4 for an fp32 output, so that
// its stores are 16 bytes a lane; 8 otherwise).
template <typename OT, int W>
__global__ void __launch_bounds__(256)
q8_dequantize_kernel(const uint8_t* q, int q_dtype, const float* scale, int64_t H, int64_t block, int64_t scales,
                     OT* values, uint32_t pieces, uint64_t total)
{
    const uint64_t step = uint64_t(gridDim.x) * 256;
    for (uint64_t j = uint64_t(blockIdx.x) * 256 + threadIdx.x; j < total; j += step) {
        const uint64_t t = total >> 32 ? j / pieces : uint64_t(uint32_t(j) / pieces);
        const int64_t c = int64_t(j - t * pieces) * W, at = int64_t(t) * H + c;
        const int n = H - c < W ? int(H - c) : W;
        const float s = scale[int64_t(t) * scales + (block ? uint32_t(c) / uint32_t(block) : 0u)];
        uint32_t b[W / 4];
        if (n == W) {
            typedef uint32_t WordsAny __attribute__((ext_vector_type(W / 4), aligned(1)));
            const WordsAny x = *reinterpret_cast<const WordsAny*>(q + at);
#pragma unroll
            for (int k = 0; k < W / 4; ++k) b[k] = x[k];
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e) {
                if ((e & 3) == 0) b[e / 4] = 0;
                if (e < n) b[e / 4] |= uint32_t(q[at + e]) << (8 * (e & 3));
            }
        }
        float v[W];
#pragma unroll
        for (int k = 0; k < W / 4; ++k) {
            if (q_dtype == GN_Q_INT8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * k + e] = float(int8_t(b[k] >> (8 * e)));
            } else {
                v[4 * k] = __builtin_amdgcn_cvt_f32_fp8(int(b[k]), 0);
                v[4 * k + 1] = __builtin_amdgcn_cvt_f32_fp8(int(b[k]), 1);
                v[4 * k + 2] = __builtin_amdgcn_cvt_f32_fp8(int(b[k]), 2);
                v[4 * k + 3] = __builtin_amdgcn_cvt_f32_fp8(int(b[k]), 3);
            }
        }
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = v[e] * s;
        Piece<OT, W> o;
        o.narrow(v);
        if (n == W)
            o.template store<false>(values + at);
        else
            o.store_part(values + at, n);
    }
}

template <typename XT, typename RT, int W>
hipError_t fwd(const RmsArgs& a, bool q8, const RowPlan& p, hipStream_t st)
{
    const dim3 grid = dim3(unsigned((a.T + p.rows - 1) / p.rows));
    return with_row<W>(p, [&](auto v, auto exact) {
        constexpr int V = decltype(v)::value;
        constexpr bool E = decltype(exact)::value;
        return q8 ? launch(rms_fwd_kernel<XT, RT, W, V, E, true>, grid, dim3(p.block), st, a)
                  : launch(rms_fwd_kernel<XT, RT, W, V, E, false>, grid, dim3(p.block), st, a);
    });
}

template <typename XT>
hipError_t fwd16(const RmsArgs& a, int r_dtype, bool q8, const RowPlan& p, hipStream_t st)
{
    if (a.res && r_dtype == GN_F32) return fwd<XT, float, 4>(a, q8, p, st);
    if (p.width == 4) return a.res ? fwd<XT, XT, 4>(a, q8, p, st) : fwd<XT, void, 4>(a, q8, p, st);
    return a.res ? fwd<XT, XT, 8>(a, q8, p, st) : fwd<XT, void, 8>(a, q8, p, st);
}

}  // namespace

hipError_t launch_rms_fwd(const RmsArgs& a, int x_dtype, int r_dtype, bool q8, const RowPlan& p, hipStream_t st)
{
    if (x_dtype == GN_F32) return a.res ? fwd<float, float, 4>(a, q8, p, st) : fwd<float, void, 4>(a, q8, p, st);
    return x_dtype == GN_BF16 ? fwd16<uint16_t>(a, r_dtype, q8, p, st) : fwd16<_Float16>(a, r_dtype, q8, p, st);
}

hipError_t launch_q8_dequantize(const void* q, int q_dtype, const float* scale, int64_t T, int64_t H, int64_t block,
                                void* values, int out_dtype, hipStream_t st)
{
    return with_type(out_dtype, [&](auto t) {
        using OT = decltype(t);
        constexpr int W = sizeof(OT) == 4 ? 4 : 8;
        const int64_t pieces = (H + W - 1) / W, total = T * pieces, scales = block ? (H + block - 1) / block : 1;
        const int64_t grid = std::min<int64_t>((total + 255) / 256, int64_t(1) << 22);
        return launch(q8_dequantize_kernel<OT, W>, dim3(unsigned(grid)), dim3(256), st, cp<uint8_t>(q), q_dtype, scale,
                      H, block, scales, mp<OT>(values), uint32_t(pieces), uint64_t(total));
    });
}

}  // namespace gn
