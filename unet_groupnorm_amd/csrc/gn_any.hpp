// gn_any.hpp -- 8-element vectors at any element's address, shared by the kernel files of
// the row norm and of the gradient list. Every function lives in an unnamed namespace.
#pragma once

#include "gn_device.hpp"

namespace gn {

namespace {

// 16- and 8-byte accesses that assume no more than the element's own alignment: gfx950 takes
// unaligned global accesses, so these are the same single instructions as aligned ones.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

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

template <typename T>
__device__ __forceinline__ typename Io<T>::Raw load_any(const T* p)
{
    typename Io<T>::Raw r;
    if constexpr (sizeof(T) == 4) {
        const f32x4_any* q = reinterpret_cast<const f32x4_any*>(p);
        r.a = q[0];
        r.b = q[1];
    } else {
        r.u = *reinterpret_cast<const u32x4_any*>(p);
    }
    return r;
}

template <typename T>
__device__ __forceinline__ void store_any(T* p, const float (&v)[8])
{
    if constexpr (sizeof(T) == 4) {
        f32x4_any* q = reinterpret_cast<f32x4_any*>(p);
        q[0] = f32x4{v[0], v[1], v[2], v[3]};
        q[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        alignas(16) T t[8];
        Io<T>::template store8<false>(t, v);
        *reinterpret_cast<u32x4_any*>(p) = *reinterpret_cast<const u32x4*>(t);
    }
}

// The first n (1 to 7) elements of a vector, zeros behind them.
template <typename T>
__device__ __forceinline__ void load_part(const T* p, int n, float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? Io<T>::load1(p + e) : 0.0f;
}

template <typename T>
__device__ __forceinline__ void store_part(T* p, int n, const float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < n) Io<T>::store1(p + e, v[e]);
}

}  // namespace

}  // namespace gn
