// gn_rms.hip -- the root-mean-square norm over rows: forward with the residual's addition
// (output in x's dtype, fp32 or 8 bits with scales), backward, and the 8-bit form's values.
//
//   h = round(x + residual);  rstd = 1 / sqrt(mean(h^2) + eps);  y = h * rstd * weight
//   d = rstd * (dy * weight - h * rstd * c) + dh,  c = mean(dy * weight * h * rstd)
//
// Every kernel is bound by the bytes it moves (5 to 12 operations for 7 to 8 bytes): a row is
// read once into registers, reduced there, and written once.
#include "gn_any.hpp"
#include "gn_ops.hpp"

namespace gn {

namespace {

// ------------------------------------------------------------------ rows in registers

// A lane's view of a row: vector u of the lane is the row's vector lane + u * lanes.
struct Row {
    int32_t lane, lanes;
    int32_t full;  // whole vectors of the row
    int32_t tail;  // elements of the vector behind them
    __device__ __forceinline__ int32_t vec(int u) const { return lane + u * lanes; }
};

__device__ __forceinline__ Row row_of(int64_t H, int32_t lanes, int32_t lane)
{
    return Row{lane, lanes, int32_t(H >> 3), int32_t(H & 7)};
}

template <typename T, int V>
using RawRow = typename Io<T>::Raw[V];

template <typename T, int V, bool EXACT, bool NT>
__device__ __forceinline__ void load_raw_row(const T* p, const Row& r, RawRow<T, V>& raw)
{
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int32_t i = r.vec(u);
        if (EXACT || i < r.full)
            raw[u] = load_any<T, NT>(p + i * 8);
        else
            raw[u] = load_part(p + i * 8, i == r.full ? r.tail : 0);
    }
}

// A lane's vectors of a row as loaded, zeros behind the row's end; nt (one value for the
// launch): nontemporal.
template <typename T, int V, bool EXACT>
__device__ __forceinline__ void load_raw_row(const T* p, const Row& r, bool nt, RawRow<T, V>& raw)
{
    if (nt)
        load_raw_row<T, V, EXACT, true>(p, r, raw);
    else
        load_raw_row<T, V, EXACT, false>(p, r, raw);
}

template <typename T, int V>
__device__ __forceinline__ void widen_row(const RawRow<T, V>& raw, float (&v)[V][8])
{
#pragma unroll
    for (int u = 0; u < V; ++u) Io<T>::widen(raw[u], v[u]);
}

template <typename T, int V, bool EXACT, bool NT>
__device__ __forceinline__ void store_row_as(T* p, const Row& r, const float (&v)[V][8])
{
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int32_t i = r.vec(u);
        if (EXACT || i < r.full)
            store_any<T, NT>(p + i * 8, v[u]);
        else if (i == r.full && r.tail)
            store_part(p + i * 8, r.tail, v[u]);
    }
}

template <typename T, int V, bool EXACT>
__device__ __forceinline__ void store_row(T* p, const Row& r, bool nt, const float (&v)[V][8])
{
    if (nt)
        store_row_as<T, V, EXACT, true>(p, r, v);
    else
        store_row_as<T, V, EXACT, false>(p, r, v);
}

// weight as fp32 (ones where it is null).
template <typename T, int V, bool EXACT>
__device__ __forceinline__ void load_weight(const void* w, bool f32, const Row& r, float (&v)[V][8])
{
    if (!w) {
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[u][e] = 1.0f;
    } else if (f32) {
        RawRow<float, V> raw;
        load_raw_row<float, V, EXACT, false>(in<float>(w), r, raw);
        widen_row<float, V>(raw, v);
    } else {
        RawRow<T, V> raw;
        load_raw_row<T, V, EXACT, false>(in<T>(w), r, raw);
        widen_row<T, V>(raw, v);
    }
}

// v rounded to T and back.
template <typename T>
__device__ __forceinline__ float round_to(float v)
{
    if constexpr (sizeof(T) == 4) return v;
    T t;
    Io<T>::store1(&t, v);
    return Io<T>::load1(&t);
}

// ------------------------------------------------------------------ sums over a row's lanes

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v)
{
    return uint32_t(__builtin_amdgcn_update_dpp(int(v), int(v), CTRL, 0xF, 0xF, false));
}

struct AddOp {
    static __device__ __forceinline__ uint32_t f(uint32_t a, uint32_t b)
    {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }
};
// Largest of two magnitudes by their bits, which orders NaN above infinity: a NaN stays.
struct MaxBitsOp {
    static __device__ __forceinline__ uint32_t f(uint32_t a, uint32_t b) { return a > b ? a : b; }
};

// Every one of `lanes` (a power of two up to 64) neighbouring lanes gets the result over
// them: exchanges with the lane 1, 2 apart, with the mirrored lane of the half row and of the
// row of 16, and with the neighbouring rows, whose members all hold one value by then; both
// sides of an exchange combine the same two values, so all lanes hold the same bits.
template <typename Op>
__device__ __forceinline__ uint32_t lanes_all(uint32_t v, int32_t lanes)
{
    if (lanes >= 2) v = Op::f(v, dpp<0xB1>(v));
    if (lanes >= 4) v = Op::f(v, dpp<0x4E>(v));
    if (lanes >= 8) v = Op::f(v, dpp<0x141>(v));
    if (lanes >= 16) v = Op::f(v, dpp<0x140>(v));
    if (lanes >= 32) {
        const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = Op::f(s[0], s[1]);
    }
    if (lanes >= 64) {
        const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = Op::f(s[0], s[1]);
    }
    return v;
}

// The result over a whole row for each of its lanes. The waves of a longer row meet in s (a
// word for each wave of the row), in wave order; the whole workgroup takes part, and s is free
// again once every wave has passed another barrier.
template <typename Op>
__device__ __forceinline__ uint32_t row_all(uint32_t v, const Row& r, uint32_t* s)
{
    v = lanes_all<Op>(v, r.lanes < 64 ? r.lanes : 64);
    if (r.lanes > 64) {
        const int nw = r.lanes >> 6;
        if ((r.lane & 63) == 0) s[r.lane >> 6] = v;
        __syncthreads();
        v = s[0];
        for (int w = 1; w < nw; ++w) v = Op::f(v, s[w]);
    }
    return v;
}

__device__ __forceinline__ float row_sum(float v, const Row& r, uint32_t* s)
{
    return __uint_as_float(row_all<AddOp>(__float_as_uint(v), r, s));
}

constexpr int kRowMaxWaves = kRowMaxBlock / 64;

// ------------------------------------------------------------------ 8 bits

constexpr float kQMin = 0x1p-126f;  // smallest scale, the smallest normal fp32

// 8 quotients, |v| <= qmax, to 8 bytes: nearest, ties to even.
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], int q_dtype)
{
    uint2 o;
    if (q_dtype == GN_Q_INT8) {
        uint32_t b[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) b[e] = uint32_t(int32_t(rintf(v[e]))) & 0xffu;
        o.x = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
        o.y = b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24);
    } else {
        int a = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
        a = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], a, true);
        int b = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
        b = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], b, true);
        o.x = uint32_t(a);
        o.y = uint32_t(b);
    }
    return o;
}

__device__ __forceinline__ void store_q(uint8_t* p, int n, uint2 q)
{
    if (n >= 8) {
        u32x2_any t = {q.x, q.y};
        *reinterpret_cast<u32x2_any*>(p) = t;
    } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
            if (e < n) p[e] = uint8_t((e < 4 ? q.x >> (8 * e) : q.y >> (8 * (e - 4))) & 0xffu);
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

template <typename XT, typename RT, int V, bool EXACT, bool Q8>
__global__ void __launch_bounds__(kRowMaxBlock)
rms_fwd_kernel(RmsArgs a)
{
    constexpr bool kRes = !std::is_void<RT>::value;
    using HT = typename std::conditional<kRes, RT, XT>::type;
    __shared__ uint32_t s_sum[kRowMaxWaves], s_max[kRowMaxWaves];
    const int32_t sub = a.lanes > 64 ? 0 : int32_t(threadIdx.x) / a.lanes;
    const Row r = row_of(a.H, a.lanes, int32_t(threadIdx.x) - sub * a.lanes);
    const int64_t t = int64_t(blockIdx.x) * a.rows + sub;
    if (t >= a.T) return;  // whole rows leave, and with more than 64 lanes whole workgroups
    float h[V][8], w[V][8];
    RawRow<XT, V> rx;
    load_raw_row<XT, V, EXACT>(in<XT>(a.x) + t * a.x_stride, r, a.nt, rx);
    if constexpr (kRes) {
        float d[V][8];
        RawRow<HT, V> rd;
        load_raw_row<HT, V, EXACT>(in<HT>(a.res) + t * a.H, r, a.nt, rd);
        load_weight<XT, V, EXACT>(a.w, a.w_f32, r, w);
        widen_row<XT, V>(rx, h);
        widen_row<HT, V>(rd, d);
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[u][e] = round_to<HT>(h[u][e] + d[u][e]);
        store_row<HT, V, EXACT>(out<HT>(a.h) + t * a.H, r, a.nt, h);
    } else {
        load_weight<XT, V, EXACT>(a.w, a.w_f32, r, w);
        widen_row<XT, V>(rx, h);
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
        for (int e = 0; e < 8; ++e) h[u][e] = h[u][e] * rstd * w[u][e];
    if constexpr (!Q8) {
        if (a.y_f32)
            store_row<float, V, EXACT>(out<float>(a.y) + t * a.H, r, a.nt, h);
        else
            store_row<XT, V, EXACT>(out<XT>(a.y) + t * a.H, r, a.nt, h);
    } else {
        const float qmax = a.q_dtype == GN_Q_INT8 ? 127.0f : 448.0f;
        uint32_t m[V];
#pragma unroll
        for (int u = 0; u < V; ++u) {
            m[u] = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) m[u] = MaxBitsOp::f(m[u], __float_as_uint(h[u][e]) & 0x7fffffffu);
        }
        // Lanes that share a scale: the row's, or block / 8 neighbours (a row of fewer lanes
        // than that is one run).
        const int32_t share = a.block == 0 ? r.lanes : a.block / 8 < r.lanes ? a.block / 8 : r.lanes;
        if (a.block == 0) {
#pragma unroll
            for (int u = 1; u < V; ++u) m[0] = MaxBitsOp::f(m[0], m[u]);
            m[0] = row_all<MaxBitsOp>(m[0], r, s_max);
        }
#pragma unroll
        for (int u = 0; u < V; ++u) {
            const int32_t i = r.vec(u);
            const uint32_t amax = a.block == 0 ? m[0] : lanes_all<MaxBitsOp>(m[u], share);
            const Scaled sc = scale_of(amax, qmax);
            const bool bad = amax >= 0x7f800000u;
            float q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) q[e] = bad ? 0.0f : h[u][e] * sc.inv;
            const int n = EXACT || i < r.full ? 8 : i == r.full ? r.tail : 0;
            if (n) {
                store_q(out<uint8_t>(a.y) + t * a.H + i * 8, n, quantize8(q, a.q_dtype));
                if (a.block == 0 ? u == 0 && r.lane == 0 : i % share == 0)
                    a.scale[t * a.scales + (a.block == 0 ? 0 : i / share)] = sc.scale;
            }
        }
    }
}

// ------------------------------------------------------------------ backward

// Workgroup b takes the row groups b, b + parts, ... (a.rows rows at once, a.lanes lanes
// each); the next group's vectors are loaded before this group's are used. Every lane keeps
// its columns' sums of dy * xhat in registers over all of them; at the end the workgroup adds
// its rows' sums in LDS and leaves one partial sum for each column in the workspace.
template <typename DT, typename HT, bool DH, int V, bool EXACT, int BLOCK>
__global__ void __launch_bounds__(BLOCK)
rms_bwd_kernel(RmsBwdArgs a)
{
    __shared__ uint32_t s_sum[2][BLOCK / 64];
    __shared__ __align__(16) float s_dw[BLOCK * 8];
    const int32_t sub = int32_t(threadIdx.x) / a.lanes;
    const Row r = row_of(a.H, a.lanes, int32_t(threadIdx.x) - sub * a.lanes);
    float w[V][8], dw[V][8];
    if (!a.w || a.w_dtype == GN_F32)
        load_weight<float, V, EXACT>(a.w, true, r, w);
    else if (a.w_dtype == GN_BF16)
        load_weight<uint16_t, V, EXACT>(a.w, false, r, w);
    else
        load_weight<_Float16, V, EXACT>(a.w, false, r, w);
#pragma unroll
    for (int u = 0; u < V; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[u][e] = 0.0f;
    RawRow<DT, V> next_dy;
    RawRow<HT, V> next_h, next_dh;
    float next_rstd;
    const auto load = [&](int64_t t) {  // past the last row: the last row again, unused
        t = t < a.T ? t : a.T - 1;
        load_raw_row<DT, V, EXACT>(in<DT>(a.dy) + t * a.H, r, a.nt, next_dy);
        load_raw_row<HT, V, EXACT>(in<HT>(a.h) + t * a.h_stride, r, a.nt, next_h);
        if constexpr (DH) load_raw_row<HT, V, EXACT>(in<HT>(a.dh) + t * a.H, r, a.nt, next_dh);
        next_rstd = a.rstd[t];
    };
    const int64_t groups = (a.T + a.rows - 1) / a.rows;
    int phase = 0;
    load(int64_t(blockIdx.x) * a.rows + sub);
    for (int64_t g = blockIdx.x; g < groups; g += a.parts, phase ^= 1) {
        const int64_t t = g * a.rows + sub;
        float dy[V][8], h[V][8], d[V][8];
        widen_row<DT, V>(next_dy, dy);
        widen_row<HT, V>(next_h, h);
        if constexpr (DH) widen_row<HT, V>(next_dh, d);
        const float rstd = next_rstd;
        if (g + a.parts < groups) load(t + a.parts * a.rows);
        const bool row = t < a.T;
        float c = 0.0f;
#pragma unroll
        for (int u = 0; u < V; ++u) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                h[u][e] = h[u][e] * rstd;
                if (row) dw[u][e] = fmaf(dy[u][e], h[u][e], dw[u][e]);
                dy[u][e] = dy[u][e] * w[u][e];
            }
            c = c + tree_sumprod(dy[u], h[u]);
        }
        if (!a.dx && !a.dres) continue;
        c = row_sum(c, r, s_sum[phase] + sub * (r.lanes >> 6)) / float(a.H);
        if (!row) continue;  // after the row's barrier
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = rstd * fmaf(-h[u][e], c, dy[u][e]);
                dy[u][e] = DH ? v + d[u][e] : v;
            }
        if (a.dres) store_row<HT, V, EXACT>(out<HT>(a.dres) + t * a.H, r, a.nt, dy);
        if (a.dx) {
            if (a.x_dtype == GN_F32)
                store_row<float, V, EXACT>(out<float>(a.dx) + t * a.H, r, a.nt, dy);
            else if (a.x_dtype == GN_BF16)
                store_row<uint16_t, V, EXACT>(out<uint16_t>(a.dx) + t * a.H, r, a.nt, dy);
            else
                store_row<_Float16, V, EXACT>(out<_Float16>(a.dx) + t * a.H, r, a.nt, dy);
        }
    }
    if (!a.part) return;
    float* part = a.part + int64_t(blockIdx.x) * a.H;
    if (a.rows == 1) {
        store_row<float, V, EXACT>(part, r, false, dw);
        return;
    }
#pragma unroll
    for (int u = 0; u < V; ++u) {
        if (u) __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) s_dw[threadIdx.x * 8 + e] = dw[u][e];
        __syncthreads();
        const int32_t first = u * a.lanes * 8, n = a.lanes * 8;
        for (int32_t c = threadIdx.x; c < n && first + c < a.H; c += blockDim.x) {
            float s = s_dw[c];
            for (int32_t k = 1; k < a.rows; ++k) s = s + s_dw[k * n + c];
            part[first + c] = s;
        }
    }
}

// A workgroup adds 32 columns of all parts: thread (slice, quad) takes 4 columns of the parts
// slice, slice + 128, ... in order, and the 128 slices are added in a tree. Bound by one
// trip to memory, not by bytes: every thread's few loads are in flight together.
constexpr int kDwBlock = 1024, kDwCols = 32, kDwSlices = kDwBlock / (kDwCols / 4);

__global__ void __launch_bounds__(kDwBlock)
rms_dweight_kernel(const float* part, int64_t parts, int64_t H, void* dw, int w_dtype)
{
    __shared__ float s[kDwSlices][kDwCols];
    const int quad = threadIdx.x & 7, slice = threadIdx.x >> 3;
    const int64_t c = int64_t(blockIdx.x) * kDwCols + quad * 4;
    const int n = H - c >= 4 ? 4 : H > c ? int(H - c) : 0;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (n == 4) {
#pragma unroll 8
        for (int64_t p = slice; p < parts; p += kDwSlices) {
            const f32x4 q = *reinterpret_cast<const f32x4_any*>(part + p * H + c);
            v[0] = v[0] + q.x; v[1] = v[1] + q.y; v[2] = v[2] + q.z; v[3] = v[3] + q.w;
        }
    } else {
        for (int64_t p = slice; p < parts; p += kDwSlices)
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < n) v[e] = v[e] + part[p * H + c + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) s[slice][quad * 4 + e] = v[e];
    __syncthreads();
    for (int half = kDwSlices / 2; half >= 1; half >>= 1) {
        for (int i = threadIdx.x; i < half * kDwCols; i += kDwBlock) {
            const int k = i / kDwCols, j = i % kDwCols;
            s[k][j] = s[k][j] + s[k + half][j];
        }
        __syncthreads();
    }
    const int64_t col = int64_t(blockIdx.x) * kDwCols + threadIdx.x;
    if (threadIdx.x < kDwCols && col < H) {
        if (w_dtype == GN_F32)
            Io<float>::store1(out<float>(dw) + col, s[0][threadIdx.x]);
        else if (w_dtype == GN_BF16)
            Io<uint16_t>::store1(out<uint16_t>(dw) + col, s[0][threadIdx.x]);
        else
            Io<_Float16>::store1(out<_Float16>(dw) + col, s[0][threadIdx.x]);
    }
}

// ------------------------------------------------------------------ values of the 8-bit form

template <typename OT>
__global__ void __launch_bounds__(256)
q8_dequantize_kernel(const uint8_t* q, int q_dtype, const float* scale, int64_t T, int64_t H, int64_t block,
                     int64_t scales, OT* values, int64_t vecs, int64_t total)
{
    for (int64_t j = int64_t(blockIdx.x) * 256 + threadIdx.x; j < total; j += int64_t(gridDim.x) * 256) {
        const int64_t t = j / vecs, i = j - t * vecs;
        const int64_t c = i * 8, at = t * H + c;
        const int n = H - c < 8 ? int(H - c) : 8;
        const float s = scale[t * scales + (block ? c / block : 0)];
        uint32_t lo = 0, hi = 0;
        if (n == 8) {
            const u32x2_any b = *reinterpret_cast<const u32x2_any*>(q + at);
            lo = b.x;
            hi = b.y;
        } else {
            for (int e = 0; e < n; ++e) {
                const uint32_t b = q[at + e];
                if (e < 4) lo |= b << (8 * e);
                else hi |= b << (8 * (e - 4));
            }
        }
        float v[8];
        if (q_dtype == GN_Q_INT8) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = float(int8_t(lo >> (8 * e)));
                v[4 + e] = float(int8_t(hi >> (8 * e)));
            }
        } else {
            v[0] = __builtin_amdgcn_cvt_f32_fp8(int(lo), 0); v[1] = __builtin_amdgcn_cvt_f32_fp8(int(lo), 1);
            v[2] = __builtin_amdgcn_cvt_f32_fp8(int(lo), 2); v[3] = __builtin_amdgcn_cvt_f32_fp8(int(lo), 3);
            v[4] = __builtin_amdgcn_cvt_f32_fp8(int(hi), 0); v[5] = __builtin_amdgcn_cvt_f32_fp8(int(hi), 1);
            v[6] = __builtin_amdgcn_cvt_f32_fp8(int(hi), 2); v[7] = __builtin_amdgcn_cvt_f32_fp8(int(hi), 3);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * s;
        if (n == 8)
            store_any(values + at, v);
        else
            store_part(values + at, n, v);
    }
}

// Calls f with std::integral_constant<int, V> for a plan's vectors (1, 2 or 4).
template <typename F>
hipError_t with_row(const RowPlan& p, F&& f)
{
    auto go = [&](auto v) { return p.exact ? f(v, std::true_type{}) : f(v, std::false_type{}); };
    if (p.vecs == 1) return go(std::integral_constant<int, 1>{});
    if (p.vecs == 2) return go(std::integral_constant<int, 2>{});
    return go(std::integral_constant<int, 4>{});
}

template <typename XT, typename RT>
hipError_t fwd(const RmsArgs& a, bool q8, const RowPlan& p, hipStream_t st)
{
    const dim3 grid = dim3(unsigned((a.T + p.rows - 1) / p.rows));
    return with_row(p, [&](auto v, auto exact) {
        constexpr int V = decltype(v)::value;
        constexpr bool E = decltype(exact)::value;
        return q8 ? launch(rms_fwd_kernel<XT, RT, V, E, true>, grid, dim3(p.block), st, a)
                  : launch(rms_fwd_kernel<XT, RT, V, E, false>, grid, dim3(p.block), st, a);
    });
}

template <typename DT, typename HT>
hipError_t bwd(const RmsBwdArgs& a, const BwdPlan& p, hipStream_t st)
{
    return with_row(p, [&](auto v, auto exact) {
        constexpr int V = decltype(v)::value;
        constexpr bool E = decltype(exact)::value;
        const dim3 grid = dim3(unsigned(a.parts)), block = dim3(p.block);
        if (p.block <= 512)
            return a.dh ? launch(rms_bwd_kernel<DT, HT, true, V, E, 512>, grid, block, st, a)
                        : launch(rms_bwd_kernel<DT, HT, false, V, E, 512>, grid, block, st, a);
        return a.dh ? launch(rms_bwd_kernel<DT, HT, true, V, E, 1024>, grid, block, st, a)
                    : launch(rms_bwd_kernel<DT, HT, false, V, E, 1024>, grid, block, st, a);
    });
}

}  // namespace

hipError_t launch_rms_fwd(const RmsArgs& a, int x_dtype, int r_dtype, bool q8, const RowPlan& p, hipStream_t st)
{
    if (x_dtype == GN_F32) return a.res ? fwd<float, float>(a, q8, p, st) : fwd<float, void>(a, q8, p, st);
    if (x_dtype == GN_BF16) {
        if (!a.res) return fwd<uint16_t, void>(a, q8, p, st);
        return r_dtype == GN_F32 ? fwd<uint16_t, float>(a, q8, p, st) : fwd<uint16_t, uint16_t>(a, q8, p, st);
    }
    if (!a.res) return fwd<_Float16, void>(a, q8, p, st);
    return r_dtype == GN_F32 ? fwd<_Float16, float>(a, q8, p, st) : fwd<_Float16, _Float16>(a, q8, p, st);
}

hipError_t launch_rms_bwd(const RmsBwdArgs& a, int dy_dtype, int h_dtype, const BwdPlan& p, hipStream_t st)
{
    if (h_dtype == GN_BF16)
        return dy_dtype == GN_F32 ? bwd<float, uint16_t>(a, p, st) : bwd<uint16_t, uint16_t>(a, p, st);
    if (h_dtype == GN_F16)
        return dy_dtype == GN_F32 ? bwd<float, _Float16>(a, p, st) : bwd<_Float16, _Float16>(a, p, st);
    if (dy_dtype == GN_BF16) return bwd<uint16_t, float>(a, p, st);
    if (dy_dtype == GN_F16) return bwd<_Float16, float>(a, p, st);
    return bwd<float, float>(a, p, st);
}

hipError_t launch_rms_dweight(const float* part, int64_t parts, int64_t H, void* dw, int w_dtype, hipStream_t st)
{
    return launch(rms_dweight_kernel, dim3(unsigned((H + kDwCols - 1) / kDwCols)), dim3(kDwBlock), st, part, parts, H, dw, w_dtype);
}

hipError_t launch_q8_dequantize(const void* q, int q_dtype, const float* scale, int64_t T, int64_t H, int64_t block,
                                void* out, int out_dtype, hipStream_t st)
{
    const int64_t vecs = (H + 7) / 8, total = T * vecs, scales = block ? (H + block - 1) / block : 1;
    const int64_t want = (total + 255) / 256;
    const dim3 grid = grid_of(want);
    return with_type(out_dtype, [&](auto t) {
        using OT = decltype(t);
        return launch(q8_dequantize_kernel<OT>, grid, dim3(256), st, cp<uint8_t>(q), q_dtype, scale, T, H, block,
                      scales, mp<OT>(out), vecs, total);
    });
}

}  // namespace gn
