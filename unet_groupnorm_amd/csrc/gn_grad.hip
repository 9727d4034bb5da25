// gn_grad.hip -- the norm of many gradient tensors together, and clipping by it.
//
//   norm = sqrt(sum g^2) or max |g|;  out = g * min(1, max_norm / (norm + 1e-6))
//
// A launch takes a table of tensors in its arguments. The tensors are cut into tiles, which
// the workgroups share out, and each workgroup leaves one fp64 partial. In short lists the
// scaling pass adds the partials itself (each workgroup, in the same fixed order), so that
// clipping is two kernels for each table; in long ones a kernel between the passes does.
// Both passes are bound by the bytes they move: 420M bf16 gradients into fp32 take 565 us, 126
// of them for the norm (6.6 TB/s) and 432 for the scaling (5.8 TB/s; two thirds of its bytes
// are written, and a pure write reaches 5.9); in place 392, 261 of them the scaling.
#include "gn_any.hpp"
#include "gn_ops.hpp"

namespace gn {

namespace {

constexpr int kBlock = 256;
// A lane's vectors of a step are in flight together.
constexpr int kStepTiles = int(kGradStep);
// Loads are nontemporal, in both passes: 613 -> 566 us for 420M bf16 gradients clipped into
// fp32, 55 -> 51 us for 23M fp32 ones.
constexpr bool kNt = true;
// Registers are held to what lets every workgroup of a grid of 8 for each CU be resident.
constexpr int kWavesPerSimd = 8;
static_assert(kGradTile == kBlock * 8, "a vector for each lane in a tile");

// A lane's running result: the sum of squares in fp64 (the square of any fp32 value is exact
// there, and none overflows or vanishes), or the bits of the largest magnitude (which order a
// NaN above everything). The fp64 work is hidden behind the loads: adding a piece's squares in
// fp32 first took the same time (420M bf16 gradients, norm alone: 128 and 129 us, 6.5 TB/s).
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

// The launch's table in LDS. A search through it where it arrives, in the kernel's
// arguments, is a chain of dependent reads of memory that no cache of the chip holds yet:
// here every entry is read at once.
struct Shared {
    GradEntry e[kGradEntries];
    double part[kBlock / 64];
};

__device__ __forceinline__ void stage(const GradTable& t, Shared& s)
{
    static_assert(kGradEntries <= kBlock, "an entry for each lane");
    if (int(threadIdx.x) < t.n) s.e[threadIdx.x] = t.e[threadIdx.x];
}

// An entry with its words in scalar registers (all lanes read the same one).
__device__ __forceinline__ GradEntry uniform_entry(const GradEntry& e)
{
    struct Words {
        uint32_t w[sizeof(GradEntry) / 4];
    };
    Words x = __builtin_bit_cast(Words, e);
#pragma unroll
    for (uint32_t& w : x.w) w = uint32_t(__builtin_amdgcn_readfirstlane(int(w)));
    return __builtin_bit_cast(GradEntry, x);
}

// Calls f(entry, first element, elements) over this workgroup's tiles: of the list's steps of
// kStepTiles tiles it takes steps blockIdx.x, blockIdx.x + gridDim.x, ..., so that the whole
// launch moves over the list together, each step split where an entry ends in it. Every lane
// takes part; the table is staged and the workgroup synchronized before.
template <typename F>
__device__ __forceinline__ void for_tiles(const Shared& s, int n, uint32_t tiles, F&& f)
{
    const auto tile0 = [&](int i) {
        return i < n ? uint32_t(__builtin_amdgcn_readfirstlane(int(s.e[i].tile0))) : tiles;
    };
    const uint32_t steps = (tiles + kStepTiles - 1) / kStepTiles;
    int i = 0;
    for (uint32_t step = blockIdx.x; step < steps; step += gridDim.x) {
        uint32_t k = step * kStepTiles;
        const uint32_t end = k + kStepTiles < tiles ? k + kStepTiles : tiles;
        int hi = n - 1;  // the entry of tile k, behind the last one taken
        while (i < hi) {
            const int mid = (i + hi + 1) >> 1;
            if (tile0(mid) <= k) i = mid;
            else hi = mid - 1;
        }
        for (int j = i; k < end; ++j) {
            const GradEntry e = uniform_entry(s.e[j]);
            const uint32_t last = tile0(j + 1), t1 = end < last ? end : last;
            const uint32_t at = (k - e.tile0) * uint32_t(kGradTile), left = e.numel - at;
            const uint32_t most = (t1 - k) * uint32_t(kGradTile);
            k = t1;
            f(e, at, int(left < most ? left : most));
        }
    }
}

// Calls f(first element, values) for each of the lane's whole pieces of W elements in a step
// of n, whose loads are all issued first, and g(element, value) for an element behind them.
template <typename T, int W, typename F, typename G>
__device__ __forceinline__ void for_pieces(const T* p, int n, F&& f, G&& g)
{
    constexpr int kPieces = int(kStepTiles * kGradTile) / (W * kBlock);
    const int tid = threadIdx.x;
    Piece<T, W> raw[kPieces];
    if (n == kStepTiles * kGradTile) {
#pragma unroll
        for (int u = 0; u < kPieces; ++u) raw[u].template load<kNt>(p + (u * kBlock + tid) * W);
#pragma unroll
        for (int u = 0; u < kPieces; ++u) {
            float v[W];
            raw[u].widen(v);
            f((u * kBlock + tid) * W, v);
        }
        return;
    }
    const int full = n / W, behind = n % W;
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
        if (u * kBlock + tid < full) raw[u].template load<kNt>(p + (u * kBlock + tid) * W);
    float last = 0.0f;
    if (tid < behind) last = Io<T>::load1(p + full * W + tid);
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
        if (u * kBlock + tid < full) {
            float v[W];
            raw[u].widen(v);
            f((u * kBlock + tid) * W, v);
        }
    if (tid < behind) g(full * W + tid, last);
}

template <typename T, bool INF>
__device__ __forceinline__ void step_norm(const T* p, int n, Acc& acc)
{
    constexpr int W = sizeof(T) == 4 ? 4 : 8;
    for_pieces<T, W>(
        p, n,
        [&](int, const float(&v)[W]) {
#pragma unroll
            for (int e = 0; e < W; ++e) acc.take<INF>(v[e]);
        },
        [&](int, float v) { acc.take<INF>(v); });
}

template <bool INF>
__global__ void __launch_bounds__(kBlock, kWavesPerSimd)
grad_partials_kernel(GradTable t, double* part)
{
    __shared__ Shared s;
    stage(t, s);
    __syncthreads();
    Acc acc;
    for_tiles(s, t.n, t.tiles, [&](const GradEntry& e, uint32_t at, int n) {
        if (e.dtype == GN_BF16)
            step_norm<uint16_t, INF>(in<uint16_t>(e.data) + at, n, acc);
        else if (e.dtype == GN_F16)
            step_norm<_Float16, INF>(in<_Float16>(e.data) + at, n, acc);
        else
            step_norm<float, INF>(in<float>(e.data) + at, n, acc);
    });
    const double r = block_join<INF>(INF ? double(__uint_as_float(acc.m)) : acc.s, s.part);
    if (threadIdx.x == 0) part[blockIdx.x] = r;
}

// The norm from the partials: thread t adds part[t], part[t + 256], ..., then the workgroup.
template <bool INF>
__device__ __forceinline__ double norm_of(const double* part, int64_t parts, double* s)
{
    double v = 0.0;
#pragma unroll 8
    for (int64_t p = threadIdx.x; p < parts; p += kBlock) v = join<INF>(v, part[p]);
    v = block_join<INF>(v, s);
    return INF ? v : sqrt(v);
}

template <bool NT, typename T, typename O>
__device__ __forceinline__ void step_scale(const T* p, O* o, int n, float coef)
{
    constexpr int W = sizeof(O) == 4 ? 4 : 8;
    for_pieces<T, W>(
        p, n,
        [&](int i, const float(&v)[W]) {
            float w[W];
#pragma unroll
            for (int e = 0; e < W; ++e) w[e] = v[e] * coef;
            Piece<O, W> q;
            q.narrow(w);
            q.template store<NT>(o + i);
        },
        [&](int i, float v) { Io<O>::store1(o + i, v * coef); });
}

// coef from the norm; a NaN stays. An infinite max_norm clips nothing, an infinite norm neither.
__device__ __forceinline__ float coef_of(double norm, double max_norm)
{
    if (max_norm == __builtin_huge_val() && norm == norm) return 1.0f;
    const double c = max_norm / (norm + 1e-6);
    return c >= 1.0 ? 1.0f : float(c);
}

// norm[0], and the factor where coef is not null.
template <bool INF>
__global__ void __launch_bounds__(kBlock)
grad_norm_kernel(const double* part, int64_t parts, double max_norm, float* norm, float* coef)
{
    __shared__ double s[kBlock / 64];
    const double v = norm_of<INF>(part, parts, s);
    if (threadIdx.x != 0) return;
    norm[0] = float(v);
    if (coef) coef[0] = coef_of(v, max_norm);
}

// FOLD: every workgroup takes the norm from the partials itself (norm is then written too,
// where it is not null); otherwise grad_norm_kernel has left the factor in ready[0]. That
// form, for long lists, stores nontemporally (857 -> 838 us for 420M fp32 gradients); outputs
// that the last-level cache holds are stored plainly (51 -> 49 us for 23M).
template <bool INF, bool FOLD>
__global__ void __launch_bounds__(kBlock, kWavesPerSimd)
grad_scale_kernel(GradTable t, const double* part, int64_t parts, double max_norm, float* norm, const float* ready)
{
    __shared__ Shared s;
    stage(t, s);
    float coef;
    if constexpr (FOLD) {
        const double v = norm_of<INF>(part, parts, s.part);  // synchronizes
        if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = float(v);
        coef = coef_of(v, max_norm);
    } else {
        coef = ready[0];
        __syncthreads();
    }
    for_tiles(s, t.n, t.tiles, [&](const GradEntry& e, uint32_t at, int n) {
        if (coef == 1.0f && e.data == e.out) return;
        if (e.dtype == GN_BF16) {
            const uint16_t* p = in<uint16_t>(e.data) + at;
            if (e.out_dtype == GN_F32) step_scale<!FOLD>(p, out<float>(e.out) + at, n, coef);
            else step_scale<!FOLD>(p, out<uint16_t>(e.out) + at, n, coef);
        } else if (e.dtype == GN_F16) {
            const _Float16* p = in<_Float16>(e.data) + at;
            if (e.out_dtype == GN_F32) step_scale<!FOLD>(p, out<float>(e.out) + at, n, coef);
            else step_scale<!FOLD>(p, out<_Float16>(e.out) + at, n, coef);
        } else {
            step_scale<!FOLD>(in<float>(e.data) + at, out<float>(e.out) + at, n, coef);
        }
    });
}

}  // namespace

hipError_t launch_grad_partials(const GradTable& t, bool inf, double* part, int64_t grid, hipStream_t st)
{
    return inf ? launch(grad_partials_kernel<true>, dim3(unsigned(grid)), dim3(kBlock), st, t, part)
               : launch(grad_partials_kernel<false>, dim3(unsigned(grid)), dim3(kBlock), st, t, part);
}

hipError_t launch_grad_norm(const double* part, int64_t parts, bool inf, double max_norm, float* norm, float* coef,
                            hipStream_t st)
{
    return inf ? launch(grad_norm_kernel<true>, dim3(1), dim3(kBlock), st, part, parts, max_norm, norm, coef)
               : launch(grad_norm_kernel<false>, dim3(1), dim3(kBlock), st, part, parts, max_norm, norm, coef);
}

hipError_t launch_grad_scale(const GradTable& t, const double* part, int64_t parts, bool inf, double max_norm,
                             float* norm, const float* ready, int64_t grid, hipStream_t st)
{
    const dim3 g = dim3(unsigned(grid)), b = dim3(kBlock);
    if (ready) return launch(grad_scale_kernel<false, false>, g, b, st, t, part, parts, max_norm, norm, ready);
    return inf ? launch(grad_scale_kernel<true, true>, g, b, st, t, part, parts, max_norm, norm, ready)
               : launch(grad_scale_kernel<false, true>, g, b, st, t, part, parts, max_norm, norm, ready);
}

}  // namespace gn
