// gn_join.hpp -- kernel arguments, plans and launchers shared by gn_join_api.cpp and the kernel
// files of the residual join (gn_join.hip, gn_join_bwd.hip) and of the 8-bit checkpoints
// (gn_join.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gn_join.h"
#include "gn_ops.hpp"

namespace gn {

// A vector of H columns for each sequence (stride elements apart), or one (stride 0).
struct JoinVec {
    const void* p;   // null: ones (scale: zeros)
    int64_t stride;
    int32_t dtype;
};

struct JoinVecs {
    JoinVec w, post, gate, scale;
    float branch_scale;
};

struct JoinArgs {
    const void* x;
    const void* res;
    void* h;
    void* y;          // null: none
    float* rstd;      // either may be null
    float* post_rstd;
    uint8_t* h_q;     // checkpoints, each null or not
    float* h_scale;
    uint8_t* x_q;
    float* x_scale;
    JoinVecs v;
    int64_t T, H, x_stride;
    int64_t first;    // the launch's first row
    int64_t len;      // rows of a sequence
    int64_t scales;   // scales of a row of a checkpoint
    float eps, inv_H, residual_scale;
    int32_t lanes, rows;
    int32_t q_dtype, block;
    bool post, one;   // the norm after the block; one sequence
    bool nt;          // nontemporal loads of the rows
};

struct JoinBwdArgs {
    const void* dy;   // null: none
    const void* dh;   // null: none
    const void* h;    // or its checkpoint
    const void* x;    // or its checkpoint; null: not read
    const float* h_scale;
    const float* x_scale;
    const float* rstd;
    const float* post_rstd;
    void* dx;         // null: none
    void* dres;       // null: none
    JoinVecs v;
    float* part;      // [2][chunks][H]: sums of dy * xhat, then of d * xpost; null: none
    float2* row;      // two-kernel path: c1 * rstd and the mean of d * c * xpost of each row
    int64_t T, H, x_stride;
    int64_t len;      // rows of a sequence
    int64_t chunks;   // of all sequences together, `split` of each
    int64_t split;
    int64_t scales;
    float inv_H, residual_scale;
    int32_t lanes, rows;
    int32_t q_dtype, block;
    bool post;
    bool nt;
};

// How the backward pass shares out the rows: every sequence is cut into `split` chunks, chunk k
// taking the row groups k, k + split, ... of its sequence, and a workgroup takes whole chunks
// and leaves two partial sums for each column of each.
struct JoinSplit {
    int64_t len, split, chunks;
};

// Chunks of all sequences: as many as fill the chip's kBwdParts workgroups in whole turns as well
// as up to eight turns can, and no more than there are rows.
inline JoinSplit join_split(int64_t T, int64_t samples)
{
    JoinSplit s{samples > 0 ? T / samples : 0, 1, samples};
    if (s.len < 2 || samples >= 8 * kBwdParts) return s;
    double best = -1.0;
    for (int64_t turns = 1; turns <= 8; ++turns) {
        int64_t k = turns * kBwdParts / samples;
        if (k < 1) continue;
        k = k < s.len ? k : s.len;
        const int64_t chunks = k * samples, rounds = (chunks + kBwdParts - 1) / kBwdParts;
        const double used = double(chunks) / double(rounds * kBwdParts);
        if (used > best + 0.03) {
            best = used;
            s.split = k;
        }
    }
    s.chunks = s.split * samples;
    return s;
}

hipError_t launch_join_fwd(const JoinArgs& a, int x_dtype, int r_dtype, const RowPlan& p, hipStream_t st);

// The rows' means (a.row) and then the gradients and partial sums, two kernels.
hipError_t launch_join_bwd_rows(const JoinBwdArgs& a, int x_dtype, int r_dtype, hipStream_t st);

// The vectors' gradients from the partial sums.
struct JoinVecGrads {
    const float* part;
    void* dw;
    void* dpost;
    void* dgate;
    void* dscale;
    JoinVecs v;
    int64_t H, chunks, split, samples;
};
hipError_t launch_join_vectors(const JoinVecGrads& a, hipStream_t st);

struct QuantArgs {
    const void* x;
    uint8_t* q;
    float* scale;
    int64_t T, H, x_stride, scales;
    int32_t lanes, rows, q_dtype, block;
    bool nt;
};
hipError_t launch_q8_quantize(const QuantArgs& a, int x_dtype, const RowPlan& p, hipStream_t st);

}  // namespace gn
