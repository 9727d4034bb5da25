// gn_grad.hip -- the norm of many gradient tensors together, and clipping by it.
//
//   norm = sqrt(sum g^2) or max |g|;  out = g * min(1, max_norm / (norm + 1e-6))
//
// A launch takes a table of tensors in its arguments. The tensors are cut into tiles, the
// tiles are shared out evenly in list order, and each workgroup leaves one fp64 partial; the
// scaling pass first adds the partials itself (each workgroup, in the same fixed order), so
// that clipping is two kernels for each table. Both passes are bound by the bytes they move.
#include "gn_any.hpp"
#include "gn_ops.hpp"

namespace gn {

namespace {

constexpr int kBlock = 256;
constexpr int kTileVecs = int(kGradTile / (8 * kBlock));  // 8-element vectors of a lane in a tile

// A lane's running result: the sum of squares in fp64 (the square of any fp32 value is
// exact there, and none overflows or vanishes), or the bits of the largest magnitude (which
// order a NaN above everything).
struct Acc {
    double s = 0.0;
    uint32_t m = 0;
    template <bool INF>
    __device__ __forceinline__ void take(float v)
    {
        if constexpr (INF) {
            const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
            m = b > m ? b : m;
        } else {
            s = fma(double(v), double(v), s);
        }
    }
};

template <bool INF>
__device__ __forceinline__ double join(double a, double b)
{
    if constexpr (INF) return a >= b || a != a ? a : b;  // a NaN on either side stays
    return a + b;
}

// The workgroup's result, in thread 0: lane i takes lane i + off for off = 32 ... 1, then the
// waves in order.
template <bool INF>
__device__ __forceinline__ double block_join(double v, double* s)
{
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v = join<INF>(v, __shfl_down(v, off));
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    double r = s[0];
    for (int w = 1; w < kBlock / 64; ++w) r = join<INF>(r, s[w]);
    return r;
}

// The tiles of workgroup b: [b * tiles / grid, (b + 1) * tiles / grid).
__device__ __forceinline__ uint32_t first_tile(uint32_t tiles, uint32_t b, uint32_t grid)
{
    return uint32_t(uint64_t(tiles) * b / grid);
}

// The entry that holds tile k.
__device__ __forceinline__ int entry_of(const GradTable& t, uint32_t k)
{
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.e[mid].tile0 <= k) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Calls f(entry, first element, elements) for each tile of this workgroup.
template <typename F>
__device__ __forceinline__ void for_tiles(const GradTable& t, F&& f)
{
    uint32_t k = first_tile(t.tiles, blockIdx.x, gridDim.x);
    const uint32_t end = first_tile(t.tiles, blockIdx.x + 1, gridDim.x);
    if (k >= end) return;
    int i = entry_of(t, k);
    for (; k < end; ++k) {
        while (i + 1 < t.n && t.e[i + 1].tile0 <= k) ++i;
        const uint32_t at = (k - t.e[i].tile0) * uint32_t(kGradTile);
        const uint32_t left = t.e[i].numel - at;
        f(t.e[i], at, left < kGradTile ? int(left) : int(kGradTile));
    }
}

template <typename T, bool INF>
__device__ __forceinline__ void tile_norm(const T* p, int n, Acc& acc)
{
    const int tid = threadIdx.x;
    if (n == kGradTile) {
        typename Io<T>::Raw raw[kTileVecs];
#pragma unroll
        for (int u = 0; u < kTileVecs; ++u) raw[u] = load_any(p + (u * kBlock + tid) * 8);
#pragma unroll
        for (int u = 0; u < kTileVecs; ++u) {
            float v[8];
            Io<T>::widen(raw[u], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc.take<INF>(v[e]);
        }
        return;
    }
    const int full = n >> 3;
    for (int i = tid; i < full; i += kBlock) {
        float v[8];
        Io<T>::widen(load_any(p + i * 8), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc.take<INF>(v[e]);
    }
    if (tid < (n & 7)) acc.take<INF>(Io<T>::load1(p + full * 8 + tid));
}

template <bool INF>
__global__ void __launch_bounds__(kBlock)
grad_partials_kernel(GradTable t, double* part)
{
    __shared__ double s[kBlock / 64];
    Acc acc;
    for_tiles(t, [&](const GradEntry& e, uint32_t at, int n) {
        if (e.dtype == GN_BF16)
            tile_norm<uint16_t, INF>(in<uint16_t>(e.data) + at, n, acc);
        else if (e.dtype == GN_F16)
            tile_norm<_Float16, INF>(in<_Float16>(e.data) + at, n, acc);
        else
            tile_norm<float, INF>(in<float>(e.data) + at, n, acc);
    });
    const double r = block_join<INF>(INF ? double(__uint_as_float(acc.m)) : acc.s, s);
    if (threadIdx.x == 0) part[blockIdx.x] = r;
}

// The norm from the partials: thread t adds part[t], part[t + 256], ..., then the workgroup.
template <bool INF>
__device__ __forceinline__ double norm_of(const double* part, int64_t parts, double* s)
{
    double v = 0.0;
    for (int64_t p = threadIdx.x; p < parts; p += kBlock) v = join<INF>(v, part[p]);
    v = block_join<INF>(v, s);
    return INF ? v : sqrt(v);
}

template <bool INF>
__global__ void __launch_bounds__(kBlock)
grad_norm_kernel(const double* part, int64_t parts, float* norm)
{
    __shared__ double s[kBlock / 64];
    const double v = norm_of<INF>(part, parts, s);
    if (threadIdx.x == 0) norm[0] = float(v);
}

template <typename T, typename O>
__device__ __forceinline__ void tile_scale(const T* p, O* o, int n, float coef)
{
    const int tid = threadIdx.x;
    if (n == kGradTile) {
        typename Io<T>::Raw raw[kTileVecs];
#pragma unroll
        for (int u = 0; u < kTileVecs; ++u) raw[u] = load_any(p + (u * kBlock + tid) * 8);
#pragma unroll
        for (int u = 0; u < kTileVecs; ++u) {
            float v[8];
            Io<T>::widen(raw[u], v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * coef;
            store_any(o + (u * kBlock + tid) * 8, v);
        }
        return;
    }
    const int full = n >> 3;
    for (int i = tid; i < full; i += kBlock) {
        float v[8];
        Io<T>::widen(load_any(p + i * 8), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * coef;
        store_any(o + i * 8, v);
    }
    if (tid < (n & 7)) {
        const int i = full * 8 + tid;
        Io<O>::store1(o + i, Io<T>::load1(p + i) * coef);
    }
}

template <bool INF>
__global__ void __launch_bounds__(kBlock)
grad_scale_kernel(GradTable t, const double* part, int64_t parts, float max_norm, float* norm)
{
    __shared__ double s[kBlock / 64];
    const double v = norm_of<INF>(part, parts, s);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = float(v);
    const double c = double(max_norm) / (v + 1e-6);
    const float coef = c >= 1.0 ? 1.0f : float(c);  // a NaN stays
    for_tiles(t, [&](const GradEntry& e, uint32_t at, int n) {
        if (coef == 1.0f && e.data == e.out) return;
        if (e.dtype == GN_BF16) {
            const uint16_t* p = in<uint16_t>(e.data) + at;
            if (e.out_dtype == GN_F32) tile_scale(p, out<float>(e.out) + at, n, coef);
            else tile_scale(p, out<uint16_t>(e.out) + at, n, coef);
        } else if (e.dtype == GN_F16) {
            const _Float16* p = in<_Float16>(e.data) + at;
            if (e.out_dtype == GN_F32) tile_scale(p, out<float>(e.out) + at, n, coef);
            else tile_scale(p, out<_Float16>(e.out) + at, n, coef);
        } else {
            tile_scale(in<float>(e.data) + at, out<float>(e.out) + at, n, coef);
        }
    });
}

}  // namespace

hipError_t launch_grad_partials(const GradTable& t, bool inf, double* part, int64_t grid, hipStream_t st)
{
    return inf ? launch(grad_partials_kernel<true>, dim3(unsigned(grid)), dim3(kBlock), st, t, part)
               : launch(grad_partials_kernel<false>, dim3(unsigned(grid)), dim3(kBlock), st, t, part);
}

hipError_t launch_grad_norm(const double* part, int64_t parts, bool inf, float* norm, hipStream_t st)
{
    return inf ? launch(grad_norm_kernel<true>, dim3(1), dim3(kBlock), st, part, parts, norm)
               : launch(grad_norm_kernel<false>, dim3(1), dim3(kBlock), st, part, parts, norm);
}

hipError_t launch_grad_scale(const GradTable& t, const double* part, int64_t parts, bool inf, float max_norm,
                             float* norm, int64_t grid, hipStream_t st)
{
    return inf ? launch(grad_scale_kernel<true>, dim3(unsigned(grid)), dim3(kBlock), st, t, part, parts, max_norm, norm)
               : launch(grad_scale_kernel<false>, dim3(unsigned(grid)), dim3(kBlock), st, t, part, parts, max_norm, norm);
}

}  // namespace gn
