// gn_q8.hpp -- 8 bits with scales, shared by the kernel files that write or read them: the scale of a
// run, quotients rounded to the format, and the values that 8-bit pieces stand for. Every
// function lives in an unnamed namespace.
#pragma once

#include "gn_rows.hpp"

namespace gn {

namespace {

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

// The same of a whole 16-bit piece as loaded: two elements' magnitude bits to an instruction.
template <typename T, int W>
__device__ __forceinline__ uint32_t piece_amax16(const Piece<T, W>& raw)
{
    typedef uint16_t Pair __attribute__((ext_vector_type(2)));
    Pair m = {0, 0};
#pragma unroll
    for (int k = 0; k < W / 2; ++k) m = __builtin_elementwise_max(m, __builtin_bit_cast(Pair, raw.w[k] & 0x7fff7fffu));
    const uint32_t top = m[0] > m[1] ? m[0] : m[1];
    if constexpr (std::is_same<T, uint16_t>::value)
        return top << 16;
    else
        return __float_as_uint(Io<_Float16>::lo(top));
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

// One piece of the row of 8-bit values at q, whose scales are at scale; `share` lanes share one, and
// the first of them stores it.
template <int W, int END>
__device__ __forceinline__ void store_q8(uint8_t* q, float* scale, int32_t block, const Row<W>& r, int32_t i,
                                         int32_t share, Scaled sc, int q_dtype, float (&v)[W])
{
    if (END != kExact && (i > r.full || (i == r.full && !r.tail))) return;
    const bool whole = END == kExact || i < r.full;
    store_q<W>(q + (whole ? i * W : r.column(i)), whole || END == kTiny ? 0 : W - r.tail,
               whole || END == kEnds ? W : r.H, v, sc, q_dtype);
    // share is a power of two where block is not 0
    if (block == 0 ? i == 0 : (i & (share - 1)) == 0) scale[block == 0 ? 0 : i >> (__ffs(share) - 1)] = sc.scale;
}

// Lanes that share a scale: the row's, or block / W neighbours (a row of fewer lanes than that
// is one run).
template <int W>
__device__ __forceinline__ int32_t lanes_of_scale(int32_t block, const Row<W>& r)
{
    return block == 0 || block / W >= r.lanes ? r.lanes : block / W;
}

// The W (4 or 8) numbers of an 8-bit piece, before its scale.
template <int W>
__device__ __forceinline__ void widen_q8(const uint32_t (&b)[W / 4], int q_dtype, float (&v)[W])
{
#pragma unroll
    for (int k = 0; k < W / 4; ++k) {
        if (q_dtype == GN_Q_INT8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * k + e] = float(int8_t(b[k] >> (8 * e)));
        } else {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(b[k]), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(b[k]), true);
            v[4 * k] = lo[0];
            v[4 * k + 1] = lo[1];
            v[4 * k + 2] = hi[0];
            v[4 * k + 3] = hi[1];
        }
    }
}

}  // namespace

}  // namespace gn
