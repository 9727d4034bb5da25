// gn_rows.hpp -- a row in the registers of its lanes: loads, stores and sums shared by the row
// norm's kernel files. Every function lives in an unnamed namespace.
#pragma once

#include "gn_any.hpp"
#include "gn_ops.hpp"

namespace gn {

namespace {

// ------------------------------------------------------------------ rows in registers

// How rows end: with every lane's pieces whole and inside the row; with lanes that have none,
// or a shorter one; or before a single piece is whole.
constexpr int kExact = 0, kEnds = 1, kTiny = 2;

// A lane's view of a row: its piece u (of W columns) is the row's piece i = lane + u * lanes.
// Rows that are not whole pieces end in a shorter one, whose lane reads the row's last W
// columns and takes the last `tail` of them as its own; lanes past it read those columns too
// and take none. So every load is a whole piece at an address inside the row, without a
// branch that loads in flight would have to wait at. Rows of fewer than W columns are read
// element by element.
template <int W>
struct Row {
    int32_t lane, lanes;
    int32_t H;
    int32_t full;  // whole pieces of the row
    int32_t tail;  // columns of the piece behind them
    __device__ __forceinline__ int32_t piece(int u) const { return lane + u * lanes; }
    // First column read for piece i, and how many of its columns from there are not its own.
    __device__ __forceinline__ int32_t column(int32_t i) const { return i < full ? i * W : H < W ? 0 : H - W; }
    __device__ __forceinline__ int32_t skip(int32_t i) const { return i < full ? 0 : i == full && tail ? W - tail : W; }
};

template <int W>
__device__ __forceinline__ Row<W> row_of(int64_t H, int32_t lanes, int32_t lane)
{
    return Row<W>{lane, lanes, int32_t(H), int32_t(H) / W, int32_t(H) % W};
}

template <typename T, int W, int END, bool NT>
__device__ __forceinline__ void load_piece(const T* p, const Row<W>& r, int32_t i, Piece<T, W>& raw)
{
    if (END == kExact)
        raw.template load<NT>(p + i * W);
    else if (END == kEnds)
        raw.template load<NT>(p + r.column(i));
    else
        raw.load_part(p, i == 0 ? r.H : 0);
}

// A lane's pieces of a row as loaded, the columns that are not its own among them.
template <typename T, int W, int V, int END, bool NT>
__device__ __forceinline__ void load_row_as(const T* p, const Row<W>& r, Piece<T, W> (&raw)[V])
{
#pragma unroll
    for (int u = 0; u < V; ++u) load_piece<T, W, END, NT>(p, r, r.piece(u), raw[u]);
}

// nt (one value for the launch): nontemporal. The fences keep the compiler from making one
// load of the two kinds, which drops the hint; they cost nothing.
template <typename T, int W, int V, int END>
__device__ __forceinline__ void load_row(const T* p, const Row<W>& r, bool nt, Piece<T, W> (&raw)[V])
{
    if (nt) {
        asm volatile("" ::: "memory");
        load_row_as<T, W, V, END, true>(p, r, raw);
        asm volatile("" ::: "memory");
    } else {
        load_row_as<T, W, V, END, false>(p, r, raw);
    }
}

// Piece i's values, zeros for columns that are not its own.
template <typename T, int W, int END>
__device__ __forceinline__ void widen_piece(const Piece<T, W>& raw, const Row<W>& r, int32_t i, float (&v)[W])
{
    raw.widen(v);
    if (END == kEnds && i >= r.full) {
        const int32_t skip = r.skip(i);
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = e < skip ? 0.0f : v[e];
    }
}

template <typename T, int W, int END>
__device__ __forceinline__ void store_piece(T* p, const Row<W>& r, int32_t i, const Piece<T, W>& q)
{
    if (END == kExact || i < r.full)
        q.template store<false>(p + i * W);
    else if (i == r.full && r.tail)
        q.store_some(p + r.column(i), END == kTiny ? 0 : W - r.tail, END == kTiny ? r.H : W);
}

template <typename T, int W, int END>
__device__ __forceinline__ void store_values(T* p, const Row<W>& r, int32_t i, const float (&v)[W])
{
    if constexpr (sizeof(T) == 4 && W == 8) {  // fp32 in fours
        const float a[4] = {v[0], v[1], v[2], v[3]}, b[4] = {v[4], v[5], v[6], v[7]};
        Piece<T, 4> q, s;
        q.narrow(a);
        s.narrow(b);
        if (END == kExact || i < r.full) {
            q.template store<false>(p + i * W);
            s.template store<false>(p + i * W + 4);
        } else if (i == r.full && r.tail) {
            const int32_t c = r.column(i), lo = END == kTiny ? 0 : W - r.tail, hi = END == kTiny ? r.H : W;
            q.store_some(p + c, lo, hi < 4 ? hi : 4);
            s.store_some(p + c + 4, lo > 4 ? lo - 4 : 0, hi - 4);
        }
    } else {
        Piece<T, W> q;
        q.narrow(v);
        store_piece<T, W, END>(p, r, i, q);
    }
}

// Piece i of weight, of gn_dtype `dtype`, as fp32: ones where it is null, zeros for columns
// that are not the piece's own.
template <int W, int END>
__device__ __forceinline__ void load_weight(const void* w, int dtype, const Row<W>& r, int32_t i, float (&v)[W])
{
    if (!w) {
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = 1.0f;
    } else if (END == kTiny) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const bool own = i == 0 && e < r.H;
            v[e] = !own ? 0.0f : dtype == GN_F32 ? in<float>(w)[e] : dtype == GN_BF16 ? Io<uint16_t>::load1(in<uint16_t>(w) + e)
                                                                                    : Io<_Float16>::load1(in<_Float16>(w) + e);
        }
    } else if (dtype == GN_F32) {
        const float* p = in<float>(w) + (END == kExact ? i * W : r.column(i));
#pragma unroll
        for (int k = 0; k < W; k += 4) {
            Piece<float, 4> raw;
            raw.load<false>(p + k);
            float q[4];
            raw.widen(q);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[k + e] = q[e];
        }
    } else {
        Piece<uint16_t, W> raw;
        raw.template load<false>(in<uint16_t>(w) + (END == kExact ? i * W : r.column(i)));
        if (dtype == GN_BF16)
            raw.widen(v);
        else
            Piece<_Float16, W>{raw.w}.widen(v);
    }
    if (END == kEnds && i >= r.full) {
        const int32_t skip = r.skip(i);
#pragma unroll
        for (int e = 0; e < W; ++e) v[e] = e < skip ? 0.0f : v[e];
    }
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

// The result over a whole row for each of its lanes. MANY: the row has more than 64 lanes; its
// waves meet in s (a word for each wave of the row, up to 16), which every wave then reads
// and combines in one tree. The whole workgroup takes part in that, and s is free again once
// every wave has passed another barrier. 0 is the operations' neutral element.
template <typename Op, bool MANY, int W>
__device__ __forceinline__ uint32_t row_all(uint32_t v, const Row<W>& r, uint32_t* s)
{
    if (!MANY) return lanes_all<Op>(v, r.lanes);
    v = lanes_all<Op>(v, 64);
    if ((r.lane & 63) == 0) s[r.lane >> 6] = v;
    __syncthreads();
    const int nw = r.lanes >> 6, k = r.lane & 15;
    v = s[k < nw ? k : 0];
    return lanes_all<Op>(k < nw ? v : 0u, 16);
}

template <bool MANY, int W>
__device__ __forceinline__ float row_sum(float v, const Row<W>& r, uint32_t* s)
{
    return __uint_as_float(row_all<AddOp, MANY>(__float_as_uint(v), r, s));
}

// Calls f(pieces of a lane, how rows end) with a plan's values as constants.
template <int W, typename F>
hipError_t with_row(const RowPlan& p, int64_t H, F&& f)
{
    using Exact = std::integral_constant<int, kExact>;
    using Ends = std::integral_constant<int, kEnds>;
    if (H < W) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, kTiny>{});
    auto go = [&](auto v) { return p.exact ? f(v, Exact{}) : f(v, Ends{}); };
    if (p.vecs == 1) return go(std::integral_constant<int, 1>{});
    if (p.vecs == 2) return go(std::integral_constant<int, 2>{});
    if constexpr (W == 4)
        if (p.vecs == 8) return go(std::integral_constant<int, 8>{});
    return go(std::integral_constant<int, 4>{});
}

}  // namespace

}  // namespace gn
