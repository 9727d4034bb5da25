// gn_any.hpp -- pieces of 4 or 8 elements at any element's address, shared by the kernel files of
// the row norm and of the gradient list. Every function lives in an unnamed namespace.
#pragma once

#include "gn_device.hpp"

namespace gn {

namespace {

template <typename T>
__device__ __forceinline__ const T* in(const void* p)
{
    return static_cast<const T*>(p);
}
template <typename T>
__device__ __forceinline__ T* out(void* p)
{
    return static_cast<T*>(p);
}

// W (4 or 8) elements as one lane loads and stores them: fp32 in fours and 16-bit types in
// eights are 16-byte accesses, 16-bit types in fours 8-byte ones. A wave's accesses cover
// whole lines in each case; eight fp32 values of one lane would be two accesses that each
// touch half of every line (clipping 420M bf16 gradients into fp32: 600 us that way, 566 this).
// They assume no more than the element's own alignment: gfx950 takes unaligned global
// accesses, so these are the same single instructions as aligned ones.
template <typename T, int W>
struct Piece {
    static constexpr int kWords = W * int(sizeof(T)) / 4;
    static_assert(kWords == 2 || kWords == 4, "8- or 16-byte access");
    typedef uint32_t Words __attribute__((ext_vector_type(kWords)));
    typedef uint32_t WordsAny __attribute__((ext_vector_type(kWords), aligned(sizeof(T))));
    Words w;

    template <bool NT>
    __device__ __forceinline__ void load(const T* p)
    {
        const WordsAny* q = reinterpret_cast<const WordsAny*>(p);
        w = NT ? __builtin_nontemporal_load(q) : *q;
    }
    // The first n (below W) elements, zeros behind them.
    __device__ __forceinline__ void load_part(const T* p, int n)
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < W; ++e) w[e] = e < n ? __float_as_uint(p[e]) : 0u;
        } else {
            const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
            for (int e = 0; e < W; e += 2)
                w[e / 2] = (e < n ? uint32_t(q[e]) : 0u) | (e + 1 < n ? uint32_t(q[e + 1]) << 16 : 0u);
        }
    }
    __device__ __forceinline__ void widen(float (&v)[W]) const
    {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            if constexpr (sizeof(T) == 4)
                v[e] = __uint_as_float(w[e]);
            else if constexpr (std::is_same<T, uint16_t>::value)
                v[e] = e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
            else
                v[e] = e & 1 ? Io<_Float16>::hi(w[e / 2]) : Io<_Float16>::lo(w[e / 2]);
        }
    }
    __device__ __forceinline__ void narrow(const float (&v)[W])
    {
#pragma unroll
        for (int e = 0; e < kWords; ++e) {
            if constexpr (sizeof(T) == 4)
                w[e] = __float_as_uint(v[e]);
            else if constexpr (std::is_same<T, uint16_t>::value)
                w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
            else
                w[e] = Io<_Float16>::pack(v[2 * e], v[2 * e + 1]);
        }
    }
    template <bool NT>
    __device__ __forceinline__ void store(T* p) const
    {
        WordsAny* q = reinterpret_cast<WordsAny*>(p);
        const WordsAny t = w;
        if (NT)
            __builtin_nontemporal_store(t, q);
        else
            *q = t;
    }
    __device__ __forceinline__ void store_part(T* p, int n) const { store_some(p, 0, n); }
    // Elements lo to hi - 1.
    __device__ __forceinline__ void store_some(T* p, int lo, int hi) const
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < W; ++e)
                if (e >= lo && e < hi) p[e] = __uint_as_float(w[e]);
        } else {
            uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
            for (int e = 0; e < W; ++e)
                if (e >= lo && e < hi) q[e] = uint16_t(w[e / 2] >> (16 * (e & 1)));
        }
    }
};

}  // namespace

}  // namespace gn
