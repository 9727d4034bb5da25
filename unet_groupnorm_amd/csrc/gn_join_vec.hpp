// gn_join_vec.hpp -- the vectors of a residual join as a lane takes them, and pieces of saved rows,
// shared by the join's kernel files. Every function lives in an unnamed namespace.
#pragma once

#include "gn_join.hpp"
#include "gn_q8.hpp"

namespace gn {

namespace {

// Element c of the row at p by its distance in bytes, 32 bits of it: where p is the same for all lanes,
// an access is then a scalar address and one register, not two registers for each access.
template <typename T>
__device__ __forceinline__ T* element(T* p, int32_t c)
{
    using Byte = typename std::conditional<std::is_const<T>::value, const char, char>::type;
    return reinterpret_cast<T*>(reinterpret_cast<Byte*>(p) + uint32_t(c) * uint32_t(sizeof(T)));
}

// The first column that a lane reads for piece i.
template <int W, int END>
__device__ __forceinline__ int32_t first_column(const Row<W>& r, int32_t i)
{
    return END == kExact ? i * W : r.column(i);
}

template <typename T, int W, int END, bool NT>
__device__ __forceinline__ void load_at(const T* p, const Row<W>& r, int32_t i, Piece<T, W>& raw)
{
    if (END == kTiny)
        raw.load_part(p, i == 0 ? r.H : 0);
    else
        raw.template load<NT>(element(p, first_column<W, END>(r, i)));
}

// v's vector of sequence n.
__device__ __forceinline__ const void* vector_of(const JoinVec& v, int64_t n)
{
    const int64_t e = n * v.stride;
    return !v.p ? nullptr : v.dtype == GN_F32 ? static_cast<const void*>(in<float>(v.p) + e) : in<uint16_t>(v.p) + e;
}

// A piece of a vector as loaded, of whatever type: the load by itself, so that the four vectors' loads
// are in flight together (one after the other each waits for the one before).
template <int W>
struct RawVec {
    uint32_t w[W];  // fp32 in all of them, 16-bit types in the first half
    template <int END>
    __device__ __forceinline__ void load(const void* p, int dtype, const Row<W>& r, int32_t i)
    {
        if (!p) return;
        if (END == kTiny) {  // as fp32
            float v[W];
            load_weight<W, END>(p, dtype, r, i, v);
#pragma unroll
            for (int e = 0; e < W; ++e) w[e] = __float_as_uint(v[e]);
            return;
        }
        const int32_t c = first_column<W, END>(r, i);
        if (dtype == GN_F32) {
#pragma unroll
            for (int k = 0; k < W; k += 4) {
                Piece<float, 4> q;
                q.load<false>(element(in<float>(p), c + k));
#pragma unroll
                for (int e = 0; e < 4; ++e) w[k + e] = q.w[e];
            }
        } else {
            Piece<uint16_t, W> q;
            q.template load<false>(element(in<uint16_t>(p), c));
#pragma unroll
            for (int e = 0; e < W / 2; ++e) w[e] = q.w[e];
        }
    }
    // Its values, `none` where there is no vector, zeros in columns that are not the piece's own.
    template <int END>
    __device__ __forceinline__ void widen(const void* p, int dtype, const Row<W>& r, int32_t i, float none,
                                          float (&v)[W]) const
    {
        if (!p) {
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = none;
            return;
        }
        if (END == kTiny || dtype == GN_F32) {
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = __uint_as_float(w[e]);
        } else {
            Piece<uint16_t, W> q;
#pragma unroll
            for (int e = 0; e < W / 2; ++e) q.w[e] = w[e];
            if (dtype == GN_BF16)
                q.widen(v);
            else
                Piece<_Float16, W>{q.w}.widen(v);
        }
        if (END == kEnds && i >= r.full) {
            const int32_t skip = r.skip(i);
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = e < skip ? 0.0f : v[e];
        }
    }
};

// Piece i of the coefficient c = (branch_scale * gate) * post_weight.
template <int END, int W>
__device__ __forceinline__ void branch_of(const JoinVecs& j, const RawVec<W>& gate, const RawVec<W>& post, const Row<W>& r,
                                          int32_t i, float (&c)[W])
{
    float p[W];
    gate.template widen<END>(j.gate.p, j.gate.dtype, r, i, 1.0f, c);
    post.template widen<END>(j.post.p, j.post.dtype, r, i, 1.0f, p);
#pragma unroll
    for (int e = 0; e < W; ++e) c[e] = j.branch_scale * c[e] * p[e];
}

// Piece i of the multiplier m = weight * (1 + scale).
template <int END, int W>
__device__ __forceinline__ void multiplier_of(const JoinVecs& j, const RawVec<W>& w, const RawVec<W>& scale, const Row<W>& r,
                                              int32_t i, float (&m)[W])
{
    float s[W];
    w.template widen<END>(j.w.p, j.w.dtype, r, i, 1.0f, m);
    scale.template widen<END>(j.scale.p, j.scale.dtype, r, i, 0.0f, s);
#pragma unroll
    for (int e = 0; e < W; ++e) m[e] = m[e] * (1.0f + s[e]);
}

// A piece of the four vectors of sequence n.
template <int W>
struct RawVecs {
    RawVec<W> gate, post, w, scale;
    template <int END>
    __device__ __forceinline__ void load(const JoinVecs& j, int64_t n, const Row<W>& r, int32_t i)
    {
        gate.template load<END>(vector_of(j.gate, n), j.gate.dtype, r, i);
        post.template load<END>(j.post.p, j.post.dtype, r, i);
        w.template load<END>(j.w.p, j.w.dtype, r, i);
        scale.template load<END>(vector_of(j.scale, n), j.scale.dtype, r, i);
    }
    template <int END>
    __device__ __forceinline__ void branch(const JoinVecs& j, const Row<W>& r, int32_t i, float (&c)[W]) const
    {
        branch_of<END>(j, gate, post, r, i, c);
    }
    template <int END>
    __device__ __forceinline__ void multiplier(const JoinVecs& j, const Row<W>& r, int32_t i, float (&m)[W]) const
    {
        multiplier_of<END>(j, w, scale, r, i, m);
    }
};

// The sequence of row t.
__device__ __forceinline__ int64_t sequence_of(int64_t t, int64_t len)
{
    return (t | len) >> 32 ? t / len : int64_t(uint32_t(t) / uint32_t(len));
}

// A piece of a saved row of T as loaded: its elements, or CK, its 8-bit values and their scale.
template <typename T, int W, bool CK>
struct Saved {
    Piece<T, W> raw;
    template <int END, bool NT>
    __device__ __forceinline__ void load(const void* p, int64_t at, const Row<W>& r, int32_t i, const float*, int64_t,
                                         int32_t)
    {
        load_at<T, W, END, NT>(in<T>(p) + at, r, i, raw);
    }
    template <int END>
    __device__ __forceinline__ void widen(const Row<W>& r, int32_t i, int, float (&v)[W]) const
    {
        widen_piece<T, W, END>(raw, r, i, v);
    }
};

template <typename T, int W>
struct Saved<T, W, true> {
    typedef uint32_t Words __attribute__((ext_vector_type(W / 4)));
    typedef uint32_t WordsAny __attribute__((ext_vector_type(W / 4), aligned(1)));
    Words b;
    float s;
    // The row starts at element `at` of p, and its scales at s_at. A piece's own columns lie in one
    // block (blocks are whole pieces, and a row's shorter last piece ends inside its block).
    template <int END, bool NT>
    __device__ __forceinline__ void load(const void* p, int64_t at, const Row<W>& r, int32_t i, const float* scale,
                                         int64_t s_at, int32_t block)
    {
        const uint8_t* q = in<uint8_t>(p) + at;
        if (END == kTiny) {
#pragma unroll
            for (int k = 0; k < W / 4; ++k) {
                b[k] = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (i == 0 && 4 * k + e < r.H) b[k] |= uint32_t(q[4 * k + e]) << (8 * e);
            }
            s = scale[s_at];  // fewer columns than a piece: one scale
            return;
        }
        const WordsAny* w = reinterpret_cast<const WordsAny*>(element(q, first_column<W, END>(r, i)));
        b = NT ? __builtin_nontemporal_load(w) : *w;
        const int32_t last = END == kExact || r.tail ? r.full : r.full - 1;  // the row's last piece
        s = *element(scale + s_at, block ? int32_t(uint32_t((END == kExact || i <= last ? i : last) * W) / uint32_t(block)) : 0);
    }
    template <int END>
    __device__ __forceinline__ void widen(const Row<W>& r, int32_t i, int q_dtype, float (&v)[W]) const
    {
        uint32_t t[W / 4];
#pragma unroll
        for (int k = 0; k < W / 4; ++k) t[k] = b[k];
        widen_q8<W>(t, q_dtype, v);
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = v[e] * s;
        if (END != kExact && i >= (END == kTiny ? 1 : r.full)) {
            const int32_t skip = END == kTiny ? W : r.skip(i);
#pragma unroll
            for (int e = 0; e < W; ++e) v[e] = e < skip ? 0.0f : v[e];
        }
    }
};

}  // namespace

}  // namespace gn
