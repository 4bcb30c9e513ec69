// launch_norm.h -- internal interface between the host API of the norm
// (api_norm.cpp) and its kernels.  Not installed.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "launch.h"

namespace mxk {

struct NormArgs {
    const uint16_t *x, *res, *w;   // res, w may be null
    int64_t M, K;
    float eps;
    uint16_t *h, *y;               // h iff res; y may be null
    uint8_t *q_row, *s_row;        // null without row-wise outputs
    uint8_t *q_h, *s_h;            // 8-bit copy of h, may be null
    float *rstd;
    int tiled;                     // s_row in the tile layout
};

struct NormBackArgs {
    const uint16_t *dy, *h;        // h null: q_h, s_h
    const uint8_t *q_h, *s_h;
    const float *rstd;
    const uint16_t *w, *dres;      // may be null
    int64_t M, K;
    uint16_t *dh;
    float *partials, *dweight;     // both null: no weight gradient
};

// A row in registers: a lane holds 1 or 2 chunks of 8 elements, chunk c of the
// row in lane c mod threads, in whole waves, 1024 threads at most.
constexpr int64_t kNormMaxRow = 16384;
struct NormShape {
    int chunks, threads;   // chunks per lane; 0: the two-pass kernel
};
inline NormShape norm_shape(int64_t K)
{
    if (K % 8 != 0 || K > kNormMaxRow)
        return NormShape{0, 256};
    const int64_t n = K / 8;
    const int chunks = n <= 64 ? 1 : 2;
    return NormShape{chunks, (int)((n + 64 * chunks - 1) / (64 * chunks)) * 64};
}

// Workgroups of the backward kernel, each of which leaves one row of partial
// weight gradients; of the two-pass kernels: row slices.
inline int64_t norm_back_parts(int64_t M, int64_t K)
{
    const NormShape s = norm_shape(K);
    const int64_t most = s.chunks == 0 ? 64 : 256 * (s.threads <= 512 ? 2 : 1);
    return M < most ? M : most;
}

hipError_t launch_norm(unsigned fmt, const NormArgs &a, hipStream_t s);
hipError_t launch_norm_back(const NormBackArgs &a, hipStream_t s);
// The column-wise casts of the norm's output (OP_NORM), from h and rstd: a as
// for launch_mx_cast with aux the weight (ldg 0) and row_scale; gt null, or for
// transposed rows at any byte the tensor as a stack of one group.
hipError_t launch_mx_cast_norm(unsigned fmt, const MxArgs &a, const GroupTable *gt, hipStream_t s);

}  // namespace mxk
