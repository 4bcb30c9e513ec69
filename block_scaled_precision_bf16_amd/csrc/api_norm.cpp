// api_norm.cpp -- the extern "C" entry points of the root-mean-square norm
// (declared and documented in include/mxcast.h): argument validation on the
// host, then one to two kernel launches on the caller's stream.  As in api.cpp,
// validation runs before any HIP call.

#include "mxcast.h"

#include <float.h>
#include <stdint.h>

#include "launch_norm.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 23;
constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr unsigned kModeBits =
    MX_ROWWISE | MX_COLWISE | MX_ELEM_E5M2 | MX_SCALE_ROUND_UP | MX_SCALE_TILED;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {
    const void *p;
    uint64_t n;   // bytes
};

bool overlap(const Span &a, const Span &b)
{
    if (!a.p || !b.p || a.n == 0 || b.n == 0)
        return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

// Every output must be disjoint from every input and from every other output.
bool any_alias(const Span *in, int nin, const Span *out, int nout)
{
    for (int i = 0; i < nout; i++) {
        for (int j = 0; j < nin; j++)
            if (overlap(out[i], in[j]))
                return true;
        for (int j = i + 1; j < nout; j++)
            if (overlap(out[i], out[j]))
                return true;
    }
    return false;
}

bool all_aligned(const Span *s, int n)
{
    for (int i = 0; i < n; i++)
        if (s[i].p && !aligned(s[i].p, 16))
            return false;
    return true;
}

bool size_ok(int64_t M, int64_t K)
{
    return M > 0 && K > 0 && M <= kMaxDim && K <= kMaxDim && M * K <= kMaxElems;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

uint64_t scale_bytes(int64_t rows, int64_t cols, bool tiled)
{
    const int64_t nb = ceil_div(cols, 32);
    return (uint64_t)(tiled ? ceil_div(rows, 32) * ceil_div(nb, 8) * 256 : rows * nb);
}

mx_status from_hip(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_HIP; }

// The column-wise casts of the norm's output, from h and the rows' scales.
mx_status norm_columns(const void *h, const void *weight, int64_t M, int64_t K, unsigned axis_mask,
                       uint8_t *q_col, uint8_t *s_col, const float *cut, const float *low,
                       hipStream_t stream)
{
    const unsigned fmt = axis_mask & (MX_ELEM_E5M2 | MX_SCALE_ROUND_UP);
    mxk::MxArgs a{};
    a.x = static_cast<const uint16_t *>(h);
    a.aux = static_cast<const uint16_t *>(weight);
    a.row_scale = cut;
    a.row_low = low;
    a.M = M;
    a.K = a.ldx = K;
    a.q_col = q_col;
    a.s_col = s_col;
    a.tiled = (axis_mask & MX_SCALE_TILED) != 0;
    a.qcol_nt = mxk::norm_streams(M, K);
    mxk::GroupTable gt{};
    gt.count = 1;
    gt.row0[1] = M;
    if (K % 8 != 0) {
        gt.len[0] = mxk::any_walk_len(&M, 1, K);
        gt.walk0[1] = (int)ceil_div(ceil_div(M, mxk::kAnyTileM), gt.len[0]);
        a.tiles_k = (int)ceil_div(K, mxk::kAnyTileK);
        a.tiles_m = (int)ceil_div(M, mxk::kAnyTileM);
        a.group = gt.len[0];
        a.groups_m = gt.walk0[1];
        return from_hip(mxk::launch_mx_cast_any(mxk::OP_NORM, MX_COLWISE, fmt, false, a, gt, stream));
    }
    const bool rag = M % 16 != 0;
    a.tiles_k = (int)ceil_div(K, mxk::kTileK);
    a.tiles_m = (int)ceil_div(M, mxk::kTileM);
    // walks as for the other fused casts; the tile layout needs two sub-tiles
    a.group = mxk::pick_group(a.tiles_m, a.tiles_k, mxk::target_workgroups(mxk::OP_NORM, false),
                              rag ? mxk::kMaxRagGroup : mxk::kMaxGroup);
    if (a.tiled && a.group < 2)
        a.group = 2;
    a.groups_m = (int)ceil_div(a.tiles_m, a.group);
    gt.len[0] = a.group;
    gt.walk0[1] = a.groups_m;
    return from_hip(mxk::launch_mx_cast_norm(fmt, a, rag ? &gt : nullptr, stream));
}

}  // namespace

extern "C" {

mx_status mx_rmsnorm(const void *x, const void *residual, const void *weight, int64_t M, int64_t K,
                     float eps, unsigned axis_mask, void *h, void *y, uint8_t *q_row,
                     uint8_t *s_row, uint8_t *q_col, uint8_t *s_col, uint8_t *q_h, uint8_t *s_h,
                     float *rstd, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    const bool row = axis_mask & MX_ROWWISE, col = axis_mask & MX_COLWISE;
    if ((axis_mask & ~kModeBits) || (axis_mask && !row && !col) || !(eps >= 0.0f && eps <= FLT_MAX))
        return MX_ERR_ENUM;
    if (!x || !rstd || (residual && !h) || (row && (!q_row || !s_row)) ||
        (col && (!q_col || !s_col)) || (!q_h != !s_h))
        return MX_ERR_NULL;
    if (!size_ok(M, K))
        return MX_ERR_SHAPE;
    const bool tiled = (axis_mask & MX_SCALE_TILED) != 0;
    const uint64_t n = (uint64_t)(M * K);
    const Span in[3] = {{x, 2 * n}, {residual, 2 * n}, {weight, 2 * (uint64_t)K}};
    const uint64_t need = mx_rmsnorm_workspace_size(M, axis_mask);
    const Span out[10] = {{residual ? h : nullptr, 2 * n},
                         {y, 2 * n},
                         {row ? q_row : nullptr, n},
                         {row ? s_row : nullptr, scale_bytes(M, K, tiled)},
                         {col ? q_col : nullptr, n},
                         {col ? s_col : nullptr, scale_bytes(K, M, tiled)},
                         {q_h, n},
                         {s_h, scale_bytes(M, K, false)},
                         {rstd, 4 * (uint64_t)M},
                         {need ? workspace : nullptr, need}};
    if (!all_aligned(in, 3) || !all_aligned(out, 10))
        return MX_ERR_ALIGN;
    if (need && (!workspace || workspace_bytes < need))
        return MX_ERR_WORKSPACE;
    if (any_alias(in, 3, out, 10))
        return MX_ERR_ALIAS;

    mxk::NormArgs a{};
    a.x = static_cast<const uint16_t *>(x);
    a.res = static_cast<const uint16_t *>(residual);
    a.w = static_cast<const uint16_t *>(weight);
    a.M = M;
    a.K = K;
    a.eps = eps;
    a.h = static_cast<uint16_t *>(residual ? h : nullptr);
    a.y = static_cast<uint16_t *>(y);
    a.q_row = row ? q_row : nullptr;
    a.s_row = row ? s_row : nullptr;
    a.q_h = q_h;
    a.s_h = s_h;
    a.rstd = rstd;
    a.cut = need ? static_cast<float *>(workspace) : nullptr;
    a.low = need ? a.cut + M : nullptr;
    a.tiled = tiled;
    a.stream = mxk::norm_streams(M, K);
    const hipError_t e =
        mxk::launch_norm(axis_mask & (MX_ELEM_E5M2 | MX_SCALE_ROUND_UP), a, stream);
    if (e != hipSuccess || !col)
        return from_hip(e);
    return norm_columns(residual ? h : x, weight, M, K, axis_mask, q_col, s_col, a.cut, a.low, stream);
}

size_t mx_rmsnorm_workspace_size(int64_t M, unsigned axis_mask)
{
    return (axis_mask & MX_COLWISE) && M > 0 && M <= kMaxDim ? (size_t)M * 2 * sizeof(float) : 0;
}

size_t mx_rmsnorm_backward_workspace_size(int64_t M, int64_t K)
{
    return size_ok(M, K) ? (size_t)(mxk::norm_back_parts(M, K) * K) * sizeof(float) : 0;
}

mx_status mx_rmsnorm_backward(const void *dy, const void *h, const uint8_t *q_h, const uint8_t *s_h,
                              const float *rstd, const void *weight, const void *dres, int64_t M,
                              int64_t K, void *dh, float *dweight, void *workspace,
                              size_t workspace_bytes, hipStream_t stream)
{
    if (!dy || !rstd || !dh || (!h == !q_h) || (!q_h != !s_h))
        return MX_ERR_NULL;
    if (!size_ok(M, K))
        return MX_ERR_SHAPE;
    const uint64_t n = (uint64_t)(M * K);
    const uint64_t need = dweight ? mx_rmsnorm_backward_workspace_size(M, K) : 0;
    const Span in[7] = {{dy, 2 * n},   {h, 2 * n},    {q_h, n},
                        {s_h, scale_bytes(M, K, false)}, {rstd, 4 * (uint64_t)M},
                        {weight, 2 * (uint64_t)K},       {dres, 2 * n}};
    const Span out[3] = {{dh, 2 * n}, {dweight, 4 * (uint64_t)K}, {dweight ? workspace : nullptr, need}};
    if (!all_aligned(in, 7) || !all_aligned(out, 3))
        return MX_ERR_ALIGN;
    if (dweight && (!workspace || workspace_bytes < need))
        return MX_ERR_WORKSPACE;
    if (any_alias(in, 7, out, 3))
        return MX_ERR_ALIAS;

    mxk::NormBackArgs a{};
    a.dy = static_cast<const uint16_t *>(dy);
    a.h = static_cast<const uint16_t *>(h);
    a.q_h = q_h;
    a.s_h = s_h;
    a.rstd = rstd;
    a.w = static_cast<const uint16_t *>(weight);
    a.dres = static_cast<const uint16_t *>(dres);
    a.M = M;
    a.K = K;
    a.dh = static_cast<uint16_t *>(dh);
    a.partials = dweight ? static_cast<float *>(workspace) : nullptr;
    a.dweight = dweight;
    a.stream = mxk::norm_streams(M, K);
    return from_hip(mxk::launch_norm_back(a, stream));
}

}  // extern "C"
