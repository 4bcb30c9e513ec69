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
    float *cut, *low;              // rstd as two numbers (norm_value, device_math.h), for
                                   // the column-wise cast, or null
    int tiled;                     // s_row in the tile layout
    int stream;                    // too large for the caches: norm_streams
};

struct NormBackArgs {
    const uint16_t *dy, *h;        // h null: q_h, s_h
    const uint8_t *q_h, *s_h;
    const float *rstd;
    const uint16_t *w, *dres;      // may be null
    int64_t M, K;
    uint16_t *dh;
    float *partials, *dweight;     // both null: no weight gradient
    int stream;                    // too large for the caches: norm_streams
};

// Tensors of 32 MiB and more, of which a call's do not stay in the 256 MiB of the
// last cache until they are used again: what is read or written once goes by
// non-temporal accesses (16384 x 7168 with both casts and the checkpoint 251 -> 247
// us, 8192 x 7168 with both casts 125 -> 102 us, 4096 x 8192 row-wise 46 -> 41 us,
// 2048 x 8192 23.6 -> 23.1 us; the backward of 4096 x 7168 50 -> 44 us).  Smaller ones
// may still be there from the kernel that wrote them (backward of 1024 x 8192: 19.3
// and 21.1 us).
inline bool norm_streams(int64_t M, int64_t K) { return 2 * M * K >= int64_t(1) << 25; }

// A row in registers: a lane holds 1 or 2 chunks of 8 elements, chunk c of the
// row in lane c mod threads, in whole waves, 1024 threads at most.  Longer rows are
// read twice.
constexpr int64_t kNormMaxRow = 16384;
struct NormShape {
    int chunks, threads;   // chunks per lane; 0: the two-pass kernels
};
inline NormShape norm_shape(int64_t K)
{
    if (K > kNormMaxRow)
        return NormShape{0, 512};
    const int64_t n = (K + 7) / 8;
    const int chunks = n <= 64 ? 1 : 2;
    return NormShape{chunks, (int)((n + 64 * chunks - 1) / (64 * chunks)) * 64};
}

// The backward kernel's workgroups: as many rows at a time as 512 threads hold (a
// row's elements stay with the same threads, whose weight gradients they are), one
// workgroup a CU, each of which leaves one row of partial sums.  The two-pass kernels: 64
// slices of the rows.
inline int norm_back_rows(const NormShape &s) { return s.threads >= 512 ? 1 : 512 / s.threads; }
inline int64_t norm_back_parts(int64_t M, int64_t K)
{
    const NormShape s = norm_shape(K);
    const int64_t turns = s.chunks == 0 ? M : (M + norm_back_rows(s) - 1) / norm_back_rows(s);
    const int64_t most = s.chunks == 0 ? 64 : 256;
    return turns < most ? turns : most;
}

hipError_t launch_norm(unsigned fmt, const NormArgs &a, hipStream_t s);
hipError_t launch_norm_back(const NormBackArgs &a, hipStream_t s);
// The column-wise casts of the norm's output (OP_NORM), from h and rstd: a as
// for launch_mx_cast with aux the weight (ldg 0), row_scale and row_low; gt null, or for
// transposed rows at any byte the tensor as a stack of one group.
hipError_t launch_mx_cast_norm(unsigned fmt, const MxArgs &a, const GroupTable *gt, hipStream_t s);

}  // namespace mxk
