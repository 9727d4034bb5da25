// gn_rms.hip -- the root-mean-square norm over rows, forward, with the residual's addition
// (output in x's dtype, fp32 or 8 bits with scales), and the 8-bit form's values.
//
//   h = round(x + residual);  rstd = 1 / sqrt(mean(h^2) + eps);  y = h * rstd * weight
//
// Bound by the bytes it moves (5 operations for 7 to 8 bytes): a row is read once into
// registers, reduced there, and written once. Measured, bf16 with the residual, 8192 x 4096:
// 41.7 us, 6.44 TB/s (a copy: 6.3; counted HBM bytes equal these); 4096 x 8192 to int8: 39.7 us,
// 5.9 TB/s. One workgroup for each row of more than 512 columns, and no persistent ones: the
// loads in flight are those of the other workgroups on the CU. Rows of 128 columns (131072 of
// them, 13.0 us, 5.2 TB/s) are bound by their instructions; 4 rows a lane with one load of the
// weight gained 8% there and lost as much at 65536 rows, and was not kept. One token (1 x 4096)
// takes 2.0 us on the GPU, an empty launch's time, and 5 us of the host.
#include <algorithm>

#include "gn_rows.hpp"

namespace gn {

namespace {

constexpr int kRowMaxWaves = kRowMaxBlock / 64;

// ------------------------------------------------------------------ 8 bits

constexpr float kQMin = 0x1p-126f;  // smallest scale, the smallest normal fp32

struct Scaled {
    float scale, inv;  // inv: 1 / scale, within an ulp
};

// The scale of a run whose largest magnitude has the bits `amax`: a NaN where that is a NaN or
// an infinity, else the quotient amax / qmax as a division rounds it. A product with 1 / qmax
// and one correction by its remainder give that for every significand (both qmax checked over
// all of them); the remainder is exact down to the floor's quotients.
__device__ __forceinline__ Scaled scale_of(uint32_t amax, int q_dtype)
{
    if (amax >= 0x7f800000u) return Scaled{__uint_as_float(0x7fc00000u), 0.0f};
    const float a = __uint_as_float(amax), d = q_dtype == GN_Q_INT8 ? 127.0f : 448.0f,
                c = q_dtype == GN_Q_INT8 ? 1.0f / 127.0f : 1.0f / 448.0f, q = a * c;
    const float s = fmaxf(fmaf(fmaf(-q, d, a), c, q), kQMin);
    return Scaled{s, __builtin_amdgcn_rcpf(s)};  // s is a normal number
}

// v[e] = v[e] / scale. The product with the run's reciprocal is off by 2.5 ulp at most; its
// remainder, exact but for 2^-25 of itself, corrects that to (1/2 + 2^-20) ulp of the quotient,
// which is a division's result unless the quotient lies 2^-20 ulp from halfway between two
// numbers. The remainder has to stay clear of fp32's smallest numbers: for scales from 2^-80 it
// does wherever the quotient is not far below the formats' smallest steps. Smaller scales, and
// a NaN, take the division itself (for all elements: 65536 x 512 bf16 to e4m3 by 32 28.0 us a
// call against 22.5, 4096 x 8192 bf16 to int8 41.4 against 39.7).
constexpr float kQDirect = 0x1p-80f;

template <int W>
__device__ __forceinline__ void divide(float (&v)[W], Scaled sc)
{
    if (sc.scale >= kQDirect) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const float q = v[e] * sc.inv;
            v[e] = fmaf(fmaf(-q, sc.scale, v[e]), sc.inv, q);
        }
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = v[e] / sc.scale;
    }
}

// Bits of the largest magnitude of a piece. The comparison is that of integers, which orders
// a NaN above all numbers.
template <int W>
__device__ __forceinline__ uint32_t piece_amax(const float (&v)[W])
{
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < W; ++e) m = MaxBitsOp::f(m, __float_as_uint(v[e]) & 0x7fffffffu);
    return m;
}

// 4 quotients, at most an ulp above qmax in magnitude, to 4 bytes: nearest, ties to even. For
// int8 1.5 * 2^23 is added, which leaves the integer in the sum's low bits. `zero` (a run that
// holds a NaN or an infinity) makes them 0.
__device__ __forceinline__ uint32_t quantize4(const float* v, bool zero, int q_dtype)
{
    uint32_t q;
    if (q_dtype == GN_Q_INT8) {
        uint32_t b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) b[e] = __float_as_uint(v[e] + 0x1.8p23f);
        // byte 0 of each, first value lowest
        q = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u),
                                  __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u), 0x05040100u);
    } else {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
        q = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true));
    }
    return zero ? 0u : q;
}

// W (4 or 8) values over the scale to their bytes lo to hi - 1.
template <int W>
__device__ __forceinline__ void store_q(uint8_t* p, int lo, int hi, float (&v)[W], Scaled sc, int q_dtype)
{
    uint32_t q[W / 4];
    divide(v, sc);
#pragma unroll
    for (int k = 0; k < W / 4; ++k) q[k] = quantize4(v + 4 * k, sc.scale != sc.scale, q_dtype);
    if (lo == 0 && hi == W) {
        typedef uint32_t WordsAny __attribute__((ext_vector_type(W / 4), aligned(1)));
        WordsAny t;
#pragma unroll
        for (int k = 0; k < W / 4; ++k) t[k] = q[k];
        *reinterpret_cast<WordsAny*>(p) = t;
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e)
            if (e >= lo && e < hi) p[e] = uint8_t((q[e / 4] >> (8 * (e & 3))) & 0xffu);
    }
}

// ------------------------------------------------------------------ forward

// 1 / sqrt(ss / H + eps) from an estimate r and v, the mean (a product with the rounded 1 / H,
// corrected by its remainder) plus eps, each rounded once: p + lo = v * r exactly, so e = 1 - v
// * r^2 is known to its last bits, and r + r * e / 2 is off by 3/8 e^2 of it before its one
// rounding. An estimate of zero or infinity has no correction.
__device__ __forceinline__ float inverse_rms(float ss, const RmsArgs& a)
{
    const float r = rsqrtf(fmaf(ss, a.inv_H, a.eps)), m = ss * a.inv_H;
    const float v = fmaf(fmaf(-m, float(a.H), ss), a.inv_H, m) + a.eps;
    const float p = v * r, lo = fmaf(v, r, -p), e = fmaf(-lo, r, fmaf(-p, r, 1.0f));
    return r > 0.0f && r < __builtin_huge_valf() ? fmaf(0.5f * r, e, r) : r;
}

// One piece's output in 8 bits; `share` lanes share the scale, and the first of them stores it.
template <int W, int END>
__device__ __forceinline__ void store_q8(const RmsArgs& a, const Row<W>& r, int64_t t, int32_t i, int32_t share,
                                         Scaled sc, float (&v)[W])
{
    if (END != kExact && (i > r.full || (i == r.full && !r.tail))) return;
    const bool whole = END == kExact || i < r.full;
    store_q<W>(out<uint8_t>(a.y) + t * a.H + (whole ? i * W : r.column(i)), whole || END == kTiny ? 0 : W - r.tail,
               whole || END == kEnds ? W : r.H, v, sc, a.q_dtype);
    if (a.block == 0 ? i == 0 : i % share == 0) a.scale[t * a.scales + (a.block == 0 ? 0 : i / share)] = sc.scale;
}

// Lanes that share a scale: the row's, or block / W neighbours (a row of fewer lanes than that
// is one run).
template <int W>
__device__ __forceinline__ int32_t lanes_of_scale(const RmsArgs& a, const Row<W>& r)
{
    return a.block == 0 || a.block / W >= r.lanes ? r.lanes : a.block / W;
}

// Outputs are written after the sum's barrier: an output may take an input's place, and lanes
// at the row's end read columns of others.
template <typename XT, typename RT, int W, int V, int END, bool Q8>
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
    Piece<HT, W> rd[kRes ? V : 1];
    Piece<XT, W> rx[V];
    load_row<XT, W, V, END>(in<XT>(a.x) + t * a.x_stride, r, a.nt, rx);
    if constexpr (kRes) load_row<HT, W, V, END>(in<HT>(a.res) + t * a.H, r, a.nt, rd);
#pragma unroll
    for (int u = 0; u < V; ++u) load_weight<W, END>(a.w, a.w_dtype, r, r.piece(u), w[u]);
    float ss = 0.0f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
        widen_piece<XT, W, END>(rx[u], r, r.piece(u), h[u]);
        if constexpr (kRes) {  // the sum rounded to the residual's type, and taken as stored
            float d[W];
            widen_piece<HT, W, END>(rd[u], r, r.piece(u), d);
#pragma unroll
            for (int e = 0; e < W; ++e) d[e] = h[u][e] + d[e];
            rd[u].narrow(d);
            rd[u].widen(h[u]);
        }
        ss = ss + tree_sumsq(h[u]);
    }
    ss = V > 1 || r.lanes > 64 ? row_sum<true>(ss, r, s_sum) : row_sum<false>(ss, r, s_sum);
    if constexpr (kRes) {
#pragma unroll
        for (int u = 0; u < V; ++u) store_values<HT, W, END>(out<HT>(a.h) + t * a.H, r, r.piece(u), h[u]);
    }
    const float rstd = inverse_rms(ss, a);
    if (a.rstd && r.lane == 0) a.rstd[t] = rstd;
#pragma unroll
    for (int u = 0; u < V; ++u)
#pragma unroll
        for (int e = 0; e < W; ++e) h[u][e] = h[u][e] * rstd * w[u][e];
    if constexpr (!Q8) {
        if (W == 4 && a.y_f32) {
#pragma unroll
            for (int u = 0; u < V; ++u) store_values<float, W, END>(out<float>(a.y) + t * a.H, r, r.piece(u), h[u]);
        } else {
#pragma unroll
            for (int u = 0; u < V; ++u) store_values<XT, W, END>(out<XT>(a.y) + t * a.H, r, r.piece(u), h[u]);
        }
    } else {
        const int32_t share = lanes_of_scale(a, r);
        uint32_t m[V];
#pragma unroll
        for (int u = 0; u < V; ++u) m[u] = piece_amax(h[u]);
        if (a.block == 0) {
#pragma unroll
            for (int u = 1; u < V; ++u) m[0] = MaxBitsOp::f(m[0], m[u]);
            m[0] = V > 1 || r.lanes > 64 ? row_all<MaxBitsOp, true>(m[0], r, s_max) : row_all<MaxBitsOp, false>(m[0], r, s_max);
            const Scaled sc = scale_of(m[0], a.q_dtype);
#pragma unroll
            for (int u = 0; u < V; ++u) store_q8<W, END>(a, r, t, r.piece(u), share, sc, h[u]);
        } else {
#pragma unroll
            for (int u = 0; u < V; ++u)
                store_q8<W, END>(a, r, t, r.piece(u), share, scale_of(lanes_all<MaxBitsOp>(m[u], share), a.q_dtype), h[u]);
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
    // 16-bit inputs in pieces of 4 have an fp32 output, or an fp32 residual
    constexpr bool kQ8 = W == 8 || sizeof(XT) == 4 || std::is_same<RT, float>::value;
    const dim3 grid = dim3(unsigned((a.T + p.rows - 1) / p.rows));
    return with_row<W>(p, a.H, [&](auto v, auto end) {
        constexpr int V = decltype(v)::value;
        constexpr int E = decltype(end)::value;
        if constexpr (kQ8)
            if (q8) return launch(rms_fwd_kernel<XT, RT, W, V, E, true>, grid, dim3(p.block), st, a);
        return q8 ? hipErrorInvalidValue : launch(rms_fwd_kernel<XT, RT, W, V, E, false>, grid, dim3(p.block), st, a);
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
