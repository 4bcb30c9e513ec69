// api_moe.cpp -- the extern "C" entry points of the router and of the rows' way
// to the experts and back (declared and documented in include/mxcast.h): argument
// validation on the host, then the launches on the caller's stream.  As in
// api.cpp, validation runs before any HIP call.

#include "mxcast.h"

#include <math.h>
#include <stdint.h>

#include "launch_moe.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 23;
constexpr int64_t kMaxElems = int64_t(1) << 40;
constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxExperts = 1024, kMaxTop = 64, kMaxGroups = 64, kMaxAlign = 4096;

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

// Alignment of every operand (16 bytes), and every output disjoint from every
// input and from every other output.
mx_status check_spans(const Span *in, int nin, const Span *out, int nout)
{
    for (int i = 0; i < nin; i++)
        if (!aligned(in[i].p, 16))
            return MX_ERR_ALIGN;
    for (int i = 0; i < nout; i++)
        if (!aligned(out[i].p, 16))
            return MX_ERR_ALIGN;
    for (int i = 0; i < nout; i++) {
        for (int j = 0; j < nin; j++)
            if (overlap(out[i], in[j]))
                return MX_ERR_ALIAS;
        for (int j = i + 1; j < nout; j++)
            if (overlap(out[i], out[j]))
                return MX_ERR_ALIAS;
    }
    return MX_OK;
}

mx_status from_hip(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_HIP; }

bool in(int64_t v, int64_t lo, int64_t hi) { return v >= lo && v <= hi; }

bool route_size(int64_t T, int64_t E, int64_t top)
{
    return in(T, 1, kMaxDim) && in(E, 1, kMaxExperts) && in(top, 1, kMaxTop) && top <= E;
}

bool slots_ok(int64_t T, int64_t top)
{
    return in(T, 1, kMaxDim) && in(top, 1, kMaxTop) && T * top <= kMaxDim;
}

bool sort_size(int64_t T, int64_t top, int64_t E, int64_t align)
{
    return slots_ok(T, top) && in(E, 1, kMaxExperts) && in(align, 1, kMaxAlign);
}

// Experts' rows, tokens and row length of the way back.
bool combine_size(int64_t T, int64_t top, int64_t rows, int64_t K, bool listed)
{
    return slots_ok(T, top) && in(rows, 1, kMaxRows) && in(K, 1, kMaxDim) && T * K <= kMaxElems &&
           rows * K <= kMaxElems && (listed || rows == T * top);
}

constexpr unsigned kRouteBits = MX_ROUTE_SIGMOID | MX_ROUTE_RENORM | MX_ROUTE_GROUP_PAIR | MX_ROUTE_F32;

}  // namespace

extern "C" {

mx_status moe_route(const void *logits, const float *bias, int64_t T, int64_t E, int64_t top,
                    int64_t groups, int64_t top_groups, float scale, unsigned flags,
                    int32_t *experts, float *weights, float *scores, hipStream_t stream)
{
    if ((flags & ~kRouteBits) || !isfinite(scale))
        return MX_ERR_ENUM;
    if (!logits || !experts || !weights)
        return MX_ERR_NULL;
    if (!route_size(T, E, top) || !in(groups, 1, kMaxGroups) || E % groups != 0 ||
        !in(top_groups, 1, groups))
        return MX_ERR_SHAPE;
    const bool f32 = (flags & MX_ROUTE_F32) != 0;
    if (!aligned(bias, 4))
        return MX_ERR_ALIGN;
    const Span ins[1] = {{logits, (uint64_t)(T * E) * (f32 ? 4 : 2)}};
    const Span outs[3] = {{experts, 4 * (uint64_t)(T * top)},
                          {weights, 4 * (uint64_t)(T * top)},
                          {scores, 4 * (uint64_t)(T * E)}};
    const mx_status st = check_spans(ins, 1, outs, 3);
    if (st != MX_OK)
        return st;
    for (const Span &o : outs)
        if (overlap(o, Span{bias, 4 * (uint64_t)E}))
            return MX_ERR_ALIAS;

    mxk::RouteArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.T = T;
    a.E = (int)E;
    a.top = (int)top;
    a.groups = (int)groups;
    a.top_groups = (int)top_groups;
    a.scale = scale;
    a.sigmoid = (flags & MX_ROUTE_SIGMOID) != 0;
    a.renorm = (flags & MX_ROUTE_RENORM) != 0;
    a.pair = (flags & MX_ROUTE_GROUP_PAIR) != 0;
    a.f32 = f32;
    a.experts = experts;
    a.weights = weights;
    a.scores = scores;
    return from_hip(mxk::launch_route(a, stream));
}

mx_status moe_route_backward(const void *logits, const int32_t *experts, const float *dweights,
                             const float *dscores, int64_t T, int64_t E, int64_t top, float scale,
                             unsigned flags, void *dlogits, hipStream_t stream)
{
    if ((flags & ~kRouteBits) || !isfinite(scale))
        return MX_ERR_ENUM;
    if (!logits || !experts || !dweights || !dlogits)
        return MX_ERR_NULL;
    if (!route_size(T, E, top))
        return MX_ERR_SHAPE;
    const bool f32 = (flags & MX_ROUTE_F32) != 0;
    const uint64_t n = (uint64_t)(T * E) * (f32 ? 4 : 2);
    const Span ins[4] = {{logits, n},
                         {experts, 4 * (uint64_t)(T * top)},
                         {dweights, 4 * (uint64_t)(T * top)},
                         {dscores, 4 * (uint64_t)(T * E)}};
    const Span outs[1] = {{dlogits, n}};
    const mx_status st = check_spans(ins, 4, outs, 1);
    if (st != MX_OK)
        return st;

    mxk::RouteBackArgs a{};
    a.logits = logits;
    a.experts = experts;
    a.dweights = dweights;
    a.dscores = dscores;
    a.T = T;
    a.E = (int)E;
    a.top = (int)top;
    a.scale = scale;
    a.sigmoid = (flags & MX_ROUTE_SIGMOID) != 0;
    a.renorm = (flags & MX_ROUTE_RENORM) != 0;
    a.f32 = f32;
    a.dlogits = dlogits;
    return from_hip(mxk::launch_route_back(a, stream));
}

int64_t moe_sort_rows(int64_t T, int64_t top, int64_t E, int64_t align)
{
    if (!sort_size(T, top, E, align))
        return 0;
    const int64_t n = T * top;
    return n + (E < n ? E : n) * (align - 1);
}

size_t moe_sort_workspace_size(int64_t T, int64_t top, int64_t E)
{
    if (!sort_size(T, top, E, 1) || T * top <= mxk::kSortFew)
        return 0;
    const int64_t chunk = mxk::sort_chunk(T * top), blocks = (T * top + chunk - 1) / chunk;
    return (size_t)(blocks * E) * sizeof(int32_t);
}

mx_status moe_sort(const int32_t *experts, int64_t T, int64_t top, int64_t E, int64_t align,
                   int64_t rows, int32_t *counts, int32_t *pos, int32_t *slots, void *workspace,
                   size_t workspace_bytes, hipStream_t stream)
{
    if (!experts || !counts || !pos || !slots)
        return MX_ERR_NULL;
    if (!sort_size(T, top, E, align) || !in(rows, moe_sort_rows(T, top, E, align), kMaxRows))
        return MX_ERR_SHAPE;
    const size_t need = moe_sort_workspace_size(T, top, E);
    const uint64_t n = 4 * (uint64_t)(T * top);
    const Span ins[1] = {{experts, n}};
    const Span outs[4] = {{counts, 4 * (uint64_t)E},
                          {pos, n},
                          {slots, 4 * (uint64_t)rows},
                          {need ? workspace : nullptr, need}};
    const mx_status st = check_spans(ins, 1, outs, 4);
    if (st == MX_ERR_ALIGN)
        return st;
    if (need && (!workspace || workspace_bytes < need))
        return MX_ERR_WORKSPACE;
    if (st != MX_OK)
        return st;

    mxk::SortArgs a{};
    a.experts = experts;
    a.N = T * top;
    a.E = (int)E;
    a.align = (int)align;
    a.rows = rows;
    a.counts = counts;
    a.pos = pos;
    a.slots = slots;
    a.ws = need ? static_cast<int32_t *>(workspace) : nullptr;
    a.chunk = (int)mxk::sort_chunk(a.N);
    a.blocks = (int)((a.N + a.chunk - 1) / a.chunk);
    return from_hip(mxk::launch_sort(a, stream));
}

mx_status moe_gather(const void *x, int64_t T, int64_t top, const int32_t *slots, int64_t rows,
                     int64_t row_bytes, void *out, hipStream_t stream)
{
    if (!x || !slots || !out)
        return MX_ERR_NULL;
    if (!slots_ok(T, top) || !in(rows, 1, kMaxRows) || !in(row_bytes, 1, kMaxRows) ||
        row_bytes * (rows > T ? rows : T) > 2 * kMaxElems)
        return MX_ERR_SHAPE;
    const Span ins[2] = {{x, (uint64_t)(T * row_bytes)}, {slots, 4 * (uint64_t)rows}};
    const Span outs[1] = {{out, (uint64_t)(rows * row_bytes)}};
    const mx_status st = check_spans(ins, 2, outs, 1);
    if (st != MX_OK)
        return st;

    mxk::GatherArgs a{};
    a.x = static_cast<const uint8_t *>(x);
    a.slots = slots;
    a.T = T;
    a.rows = rows;
    a.row_bytes = row_bytes;
    a.top = (int)top;
    a.out = static_cast<uint8_t *>(out);
    return from_hip(mxk::launch_gather(a, stream));
}

mx_status moe_combine(const void *y, int64_t rows, int64_t K, const int32_t *pos,
                      const float *weights, int64_t T, int64_t top, void *out, hipStream_t stream)
{
    if (!y || !out)
        return MX_ERR_NULL;
    if (!combine_size(T, top, rows, K, pos != nullptr))
        return MX_ERR_SHAPE;
    const uint64_t n = 4 * (uint64_t)(T * top);
    const Span ins[3] = {{y, 2 * (uint64_t)(rows * K)}, {pos, n}, {weights, n}};
    const Span outs[1] = {{out, 2 * (uint64_t)(T * K)}};
    const mx_status st = check_spans(ins, 3, outs, 1);
    if (st != MX_OK)
        return st;

    mxk::CombineArgs a{};
    a.y = static_cast<const uint16_t *>(y);
    a.pos = pos;
    a.weights = weights;
    a.T = T;
    a.rows = rows;
    a.K = K;
    a.top = (int)top;
    a.out = static_cast<uint16_t *>(out);
    return from_hip(mxk::launch_combine(a, stream));
}

mx_status moe_combine_backward(const void *dout, const void *y, int64_t rows, int64_t K,
                               const int32_t *pos, const int32_t *slots, const float *weights,
                               int64_t T, int64_t top, void *dy, float *dweights,
                               hipStream_t stream)
{
    if (!dout || !y || !dy || (!pos != !slots))
        return MX_ERR_NULL;
    if (!combine_size(T, top, rows, K, pos != nullptr))
        return MX_ERR_SHAPE;
    const uint64_t n = 4 * (uint64_t)(T * top), ny = 2 * (uint64_t)(rows * K);
    const Span ins[5] = {{dout, 2 * (uint64_t)(T * K)}, {y, ny}, {pos, n},
                         {slots, 4 * (uint64_t)rows}, {weights, n}};
    const Span outs[2] = {{dy, ny}, {dweights, n}};
    const mx_status st = check_spans(ins, 5, outs, 2);
    if (st != MX_OK)
        return st;

    mxk::CombineArgs a{};
    a.y = static_cast<const uint16_t *>(y);
    a.dout = static_cast<const uint16_t *>(dout);
    a.pos = pos;
    a.slots = slots;
    a.weights = weights;
    a.T = T;
    a.rows = rows;
    a.K = K;
    a.top = (int)top;
    a.out = static_cast<uint16_t *>(dy);
    a.dweights = dweights;
    return from_hip(mxk::launch_combine_back(a, stream));
}

}  // extern "C"
