// gn_rows.hpp -- a row in the registers of its lanes: loads, stores and sums shared by the row
// norm's kernel files. Every function lives in an unnamed namespace.
#pragma once

#include "gn_any.hpp"
#include "gn_ops.hpp"

namespace gn {

namespace {

// ------------------------------------------------------------------ rows in registers

// A lane's view of a row: its piece u (of W columns) is the row's piece lane + u * lanes.
template <int W>
struct Row {
    int32_t lane, lanes;
    int32_t full;  // whole pieces of the row
    int32_t tail;  // columns of the piece behind them
    __device__ __forceinline__ int32_t piece(int u) const { return lane + u * lanes; }
};

template <int W>
__device__ __forceinline__ Row<W> row_of(int64_t H, int32_t lanes, int32_t lane)
{
    return Row<W>{lane, lanes, int32_t(H) / W, int32_t(H) % W};
}

// A lane's pieces of a row as loaded, zeros behind the row's end.
template <typename T, int W, int V, bool EXACT, bool NT>
__device__ __forceinline__ void load_row_as(const T* p, const Row<W>& r, Piece<T, W> (&raw)[V])
{
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int32_t i = r.piece(u);
        if (EXACT || i < r.full)
            raw[u].template load<NT>(p + i * W);
        else
            raw[u].load_part(p + i * W, i == r.full ? r.tail : 0);
    }
}

// nt (one value for the launch): nontemporal. The fences keep the compiler from making one
// load of the two kinds, which drops the hint; they cost nothing.
template <typename T, int W, int V, bool EXACT>
__device__ __forceinline__ void load_row(const T* p, const Row<W>& r, bool nt, Piece<T, W> (&raw)[V])
{
    if (nt) {
        asm volatile("" ::: "memory");
        load_row_as<T, W, V, EXACT, true>(p, r, raw);
        asm volatile("" ::: "memory");
    } else {
        load_row_as<T, W, V, EXACT, false>(p, r, raw);
    }
}

template <typename T, int W, int V>
__device__ __forceinline__ void widen_row(const Piece<T, W> (&raw)[V], float (&v)[V][W])
{
#pragma unroll
    for (int u = 0; u < V; ++u) raw[u].widen(v[u]);
}

template <typename T, int W, int V, bool EXACT>
__device__ __forceinline__ void store_row(T* p, const Row<W>& r, const float (&v)[V][W])
{
#pragma unroll
    for (int u = 0; u < V; ++u) {
        const int32_t i = r.piece(u);
        Piece<T, W> q;
        q.narrow(v[u]);
        if (EXACT || i < r.full)
            q.template store<false>(p + i * W);
        else if (i == r.full && r.tail)
            q.store_part(p + i * W, r.tail);
    }
}

// A row of fp32 values, in fours.
template <int W, int V, bool EXACT>
__device__ __forceinline__ void store_f32(float* p, const Row<W>& r, const float (&v)[V][W])
{
#pragma unroll
    for (int u = 0; u < V; ++u)
#pragma unroll
        for (int k = 0; k < W; k += 4) {
            const int32_t i = r.piece(u) * W + k, n = r.full * W + r.tail - i;
            const float x[4] = {v[u][k], v[u][k + 1], v[u][k + 2], v[u][k + 3]};
            Piece<float, 4> q;
            q.narrow(x);
            if (EXACT || n >= 4)
                q.template store<false>(p + i);
            else if (n > 0)
                q.store_part(p + i, n);
        }
}

// weight, of gn_dtype `dtype`, as fp32 (ones where it is null).
template <int W, int V, bool EXACT>
__device__ __forceinline__ void load_weight(const void* w, int dtype, const Row<W>& r, float (&v)[V][W])
{
    if (!w) {
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int e = 0; e < W; ++e) v[u][e] = 1.0f;
    } else if (dtype == GN_F32) {
#pragma unroll
        for (int u = 0; u < V; ++u)
#pragma unroll
            for (int k = 0; k < W; k += 4) {
                const int32_t i = r.piece(u) * W + k, n = r.full * W + r.tail - i;
                Piece<float, 4> raw;
                if (EXACT || n >= 4)
                    raw.load<false>(in<float>(w) + i);
                else
                    raw.load_part(in<float>(w) + i, n);
                float q[4];
                raw.widen(q);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[u][k + e] = q[e];
            }
    } else {
        Piece<uint16_t, W> raw[V];
        load_row_as<uint16_t, W, V, EXACT, false>(in<uint16_t>(w), r, raw);
        if (dtype == GN_BF16) {
            widen_row<uint16_t, W, V>(raw, v);
        } else {
#pragma unroll
            for (int u = 0; u < V; ++u) Piece<_Float16, W>{raw[u].w}.widen(v[u]);
        }
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
template <typename Op, int W>
__device__ __forceinline__ uint32_t row_all(uint32_t v, const Row<W>& r, uint32_t* s)
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

template <int W>
__device__ __forceinline__ float row_sum(float v, const Row<W>& r, uint32_t* s)
{
    return __uint_as_float(row_all<AddOp>(__float_as_uint(v), r, s));
}

// Calls f(pieces of a lane, whether they are whole) with a plan's values as constants.
template <int W, typename F>
hipError_t with_row(const RowPlan& p, F&& f)
{
    auto go = [&](auto v) { return p.exact ? f(v, std::true_type{}) : f(v, std::false_type{}); };
    if (p.vecs == 1) return go(std::integral_constant<int, 1>{});
    if (p.vecs == 2) return go(std::integral_constant<int, 2>{});
    if constexpr (W == 4)
        if (p.vecs == 8) return go(std::integral_constant<int, 8>{});
    return go(std::integral_constant<int, 4>{});
}

}  // namespace

}  // namespace gn
