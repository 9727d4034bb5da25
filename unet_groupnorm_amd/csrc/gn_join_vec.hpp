// gn_join_vec.hpp -- the vectors of a residual join as a lane takes them, and pieces of saved rows,
// shared by the join's kernel files. Every function lives in an unnamed namespace.
#pragma once

#include "gn_join.hpp"
#include "gn_q8.hpp"

namespace gn {

namespace {

// v's vector of sequence n.
__device__ __forceinline__ const void* vector_of(const JoinVec& v, int64_t n)
{
    const int64_t e = n * v.stride;
    return !v.p ? nullptr : v.dtype == GN_F32 ? static_cast<const void*>(in<float>(v.p) + e) : in<uint16_t>(v.p) + e;
}

// Piece i of the coefficient c = (branch_scale * gate) * post_weight of sequence n.
template <int W, int END>
__device__ __forceinline__ void load_branch(const JoinVecs& j, int64_t n, const Row<W>& r, int32_t i, float (&c)[W])
{
    float p[W];
    load_weight<W, END>(vector_of(j.gate, n), j.gate.dtype, r, i, c);
    load_weight<W, END>(j.post.p, j.post.dtype, r, i, p);
#pragma unroll
    for (int e = 0; e < W; ++e) c[e] = j.branch_scale * c[e] * p[e];
}

// Piece i of the multiplier m = weight * (1 + scale) of sequence n.
template <int W, int END>
__device__ __forceinline__ void load_multiplier(const JoinVecs& j, int64_t n, const Row<W>& r, int32_t i, float (&m)[W])
{
    load_weight<W, END>(j.w.p, j.w.dtype, r, i, m);
    if (j.scale.p) {
        float s[W];
        load_weight<W, END>(vector_of(j.scale, n), j.scale.dtype, r, i, s);
#pragma unroll
        for (int e = 0; e < W; ++e) m[e] = m[e] * (1.0f + s[e]);
    }
}

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
        load_piece<T, W, END, NT>(in<T>(p) + at, r, i, raw);
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
        const WordsAny* w = reinterpret_cast<const WordsAny*>(q + (END == kExact ? i * W : r.column(i)));
        b = NT ? __builtin_nontemporal_load(w) : *w;
        const int32_t last = END == kExact || r.tail ? r.full : r.full - 1;  // the row's last piece
        s = scale[s_at + (block ? (END == kExact || i <= last ? i : last) * W / block : 0)];
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
