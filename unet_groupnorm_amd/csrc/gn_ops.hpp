// gn_ops.hpp -- kernel arguments and launchers shared by gn_ops_api.cpp and the kernel files
// of the row norm (gn_rms.hip) and of the gradient list (gn_grad.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gn_ops.h"

namespace gn {

// ------------------------------------------------------------------ row norm

// How a row of H columns is laid over lanes: in pieces of `width` columns, 4 where an fp32
// tensor is streamed (16 bytes a lane) and 8 where all are 16-bit. `lanes` lanes hold one row,
// each `vecs` pieces (piece v belongs to lane v mod lanes); lanes is a power of two up to 64
// with 256 / lanes rows in a workgroup, or a multiple of 64 with one row in a workgroup. A pure
// function of H and the types, so a row's sums are taken in the same order whatever T is.
struct RowPlan {
    int32_t width, lanes, vecs;
    int32_t block, rows;  // threads and rows of a workgroup
    bool exact;           // every lane's pieces are whole and inside the row
};

constexpr int kRowMaxBlock = 1024;
// Threads of a workgroup over rows of up to 64 lanes.
constexpr int kShortBlock = 256;
static_assert(int64_t(kRowMaxBlock) * 4 * 8 == GN_RMS_MAX_COLUMNS, "widest row: 4 pieces of 8, or 8 of 4");

// Pieces of a lane, from the pieces of the row: as few as keep the row to few waves. Measured,
// forward bf16 of 2^25 elements with 1, 2 and 4 pieces: rows of 1024 columns 43.9, 43.1, 60.2
// us; of 4096 42.2, 41.9, 47.6; of 8192 45.3, 43.1, 46.8; of 12288 -, 45.7, 52.2; fp32 of 2^24
// elements with 2, 4 and 8: rows of 4096 42.4, 42.6, 45.6; of 8192 45.6, 43.6, 45.1; of 12288 -,
// 48.3, 49.7. The backward's workgroups hold 512 lanes (many registers each), so it goes to
// more pieces sooner.
inline int32_t row_pieces(int64_t n, bool fp32, bool backward)
{
    if (n <= 256) return 1;
    if (n <= (fp32 || backward ? 1024 : 2048)) return 2;
    return !fp32 || n <= (backward ? 2048 : 4096) ? 4 : 8;
}

inline RowPlan row_plan(int64_t H, bool fp32, bool backward = false)
{
    RowPlan p;
    p.width = fp32 ? 4 : 8;
    const int64_t n = (H + p.width - 1) / p.width;
    if (n <= 64) {
        p.lanes = 1;
        while (p.lanes < n) p.lanes *= 2;
        p.vecs = 1;
        p.block = kShortBlock;
        p.rows = kShortBlock / p.lanes;
    } else {
        p.vecs = row_pieces(n, fp32, backward);
        p.lanes = int32_t(((n + p.vecs - 1) / p.vecs + 63) / 64 * 64);
        p.block = p.lanes;
        p.rows = 1;
    }
    p.exact = int64_t(p.lanes) * p.vecs * p.width == H;
    return p;
}

// The backward's plan: the lanes of a row likewise, as many rows at once as a workgroup of 512
// threads holds (fewer where T rows would not fill the chip with such workgroups), and the
// workgroups, each taking every parts-th group of rows and leaving one partial weight
// gradient.
struct BwdPlan : RowPlan {
    int64_t parts;
};

constexpr int kBwdBlock = 512;
constexpr int64_t kBwdParts = 256;

inline BwdPlan bwd_plan(int64_t T, int64_t H, bool fp32)
{
    BwdPlan p;
    static_cast<RowPlan&>(p) = row_plan(H, fp32, true);
    const int32_t least = p.lanes < 64 ? 64 / p.lanes : 1;  // rows of a whole wave
    int64_t rows = kBwdBlock / p.lanes;
    while (rows > least && (T + rows - 1) / rows < kBwdParts) rows /= 2;
    p.rows = int32_t(rows < least ? least : rows);
    p.block = p.rows * p.lanes;
    const int64_t groups = (T + p.rows - 1) / p.rows;
    p.parts = groups < kBwdParts ? groups : kBwdParts;
    return p;
}

// Calls that move more than this many bytes load their rows nontemporally. Measured, plain
// against nontemporal, on inputs that the last-level cache may still hold in part: forward of
// 2048 x 4096 bf16 (64 MiB) 11.2 and 13.3 us, 8192 x 4096 (256 MiB) 41.8 and 42.1, 16384 x 4096
// (512 MiB) 92.7 and 78.4; backward of 8192 x 4096 bf16 49.4 and 48.2, fp32 (512 MiB) 99 and 86.
constexpr int64_t kRowStreamBytes = int64_t(200) << 20;

struct RmsArgs {
    const void* x;
    const void* res;
    const void* w;
    void* h;
    void* y;       // or q
    float* rstd;
    float* scale;
    int64_t T, H, x_stride;
    float eps, inv_H;
    int32_t w_dtype, y_f32;   // weight's gn_dtype (it may be null); y in fp32, else in x's dtype
    int32_t lanes, rows;
    int32_t q_dtype, block;   // 8-bit output: format, columns of a scale (0: the row)
    int64_t scales;           // scales of a row
    bool nt;                  // nontemporal loads of the rows
};

struct RmsBwdArgs {
    const void* dy;
    const void* h;
    const void* w;
    const void* dh;
    const float* rstd;
    void* d;       // the gradient in h's type (null: none)
    void* dx;      // once more, in x's type (null: none)
    float* part;   // [parts][H], null: no weight gradient
    int64_t T, H, h_stride, parts;
    int32_t w_dtype, x_dtype;  // gn_dtype codes
    int32_t lanes, rows;
    float inv_H;
    bool nt;                   // nontemporal loads of the rows
};

hipError_t launch_rms_fwd(const RmsArgs& a, int x_dtype, int r_dtype, bool q8, const RowPlan& p, hipStream_t st);
hipError_t launch_rms_bwd(const RmsBwdArgs& a, int dy_dtype, int h_dtype, const BwdPlan& p, hipStream_t st);
// dweight[c] = sum over parts of part[p][c].
hipError_t launch_rms_dweight(const float* part, int64_t parts, int64_t H, void* dw, int w_dtype, hipStream_t st);
hipError_t launch_q8_dequantize(const void* q, int q_dtype, const float* scale, int64_t T, int64_t H, int64_t block,
                                void* out, int out_dtype, hipStream_t st);

// ------------------------------------------------------------------ gradient list

// Elements of one tile, the unit in which workgroups share out the list; a tile never
// crosses from one tensor to the next.
constexpr int64_t kGradTile = 2048;
// Tiles that a workgroup takes at once.
constexpr int64_t kGradStep = 4;
// Longest entry of a launch's table (longer tensors take several) and entries of a table,
// which travels in the kernel's arguments (4 KB at most).
constexpr int64_t kGradMaxElems = int64_t(1) << 27;
constexpr int kGradEntries = 160;
// Workgroups of the launches over a list together, hence its partial results (and one more
// for each further table at most).
constexpr int64_t kGradGrid = 2048;
// Lists of more tiles than this are scaled by one workgroup for each step, after a kernel
// that takes the norm and the factor from the partials; in shorter ones each of up to
// kGradGrid workgroups does that itself. Measured, separate against folded: 22.6M fp32
// gradients 51.1 and 48.7 us, 26.2M 62.4 and 64.1 (into fp32 from bf16 47.6 and 49.0), 105M
// 206.9 and 225.1.
constexpr int64_t kGradFoldTiles = 12288;

struct GradEntry {
    const void* data;
    void* out;
    uint32_t numel : 28, dtype : 2, out_dtype : 2;
    uint32_t tile0;  // tiles of the entries before this one
};

struct GradTable {
    GradEntry e[kGradEntries];
    int32_t n;
    uint32_t tiles;
};
static_assert(sizeof(GradTable) + 64 <= 4096, "kernel arguments");

// Partial norms of one table's entries: one fp64 for each of `grid` workgroups.
hipError_t launch_grad_partials(const GradTable& t, bool inf, double* part, int64_t grid, hipStream_t st);
// norm[0] from `parts` partials, and the factor where coef is not null.
hipError_t launch_grad_norm(const double* part, int64_t parts, bool inf, double max_norm, float* norm, float* coef,
                            hipStream_t st);
// out = data * coef for one table. ready null: each workgroup takes the norm from the partials
// and norm[0] is written too where norm is not null; else coef is ready[0].
hipError_t launch_grad_scale(const GradTable& t, const double* part, int64_t parts, bool inf, double max_norm,
                             float* norm, const float* ready, int64_t grid, hipStream_t st);

}  // namespace gn
