// api_matmul.cpp -- the extern "C" entry points of the products on quantised
// operands (declared and documented in include/mxcast.h): argument validation
// on the host, then one kernel launch on the caller's stream.  As in api.cpp,
// validation runs before any HIP call.

#include "mxcast.h"

#include <stdint.h>

#include "launch_mm.h"

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 23;
constexpr int64_t kMaxElems = int64_t(1) << 40;
// Workgroups of one launch (256 threads each, 2^32 threads in all, and a last
// round in parts).
constexpr int64_t kMaxTiles = (int64_t(1) << 24) - 4096;

constexpr unsigned kMmBits =
    MX_A_E5M2 | MX_B_E5M2 | MX_SCALE_TILED | MX_OUT_F32 | MX_OUT_ACCUMULATE;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb)
{
    if (!a || !b || na == 0 || nb == 0)
        return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

bool size_ok(int64_t a, int64_t b)
{
    return a > 0 && b > 0 && a <= kMaxDim && b <= kMaxDim && a * b <= kMaxElems;
}

mx_status from_hip(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_HIP; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Bytes of the scales of a [rows][cols] operand blocked along cols (0 for an
// operand without elements).
int64_t scale_bytes(int64_t rows, int64_t cols, bool tiled)
{
    const int64_t nb = ceil_div(cols, 32);
    return tiled ? ceil_div(rows, 32) * ceil_div(nb, 8) * 256 : rows * nb;
}

// Bytes of each operand of a launch, as the table lays them out.
struct MmBytes {
    uint64_t qa, sa, qb, sb, y;
};

// Validates the group sizes and fills the table but for tile0.  dim and N as
// in MmArgs.
bool build_table(const int64_t *rows, int G, int64_t dim, int64_t N, bool sum_rows, bool tiled,
                 int out_size, mxk::MmTable &t, MmBytes &n)
{
    if (!rows || G < 1 || G > mxk::kMmMaxGroups || dim <= 0 || N <= 0)
        return false;
    t = mxk::MmTable{};
    t.count = G;
    int64_t M = 0, sa = 0, sb = 0;
    for (int g = 0; g < G; g++) {
        if (rows[g] < 0 || rows[g] > kMaxDim)
            return false;
        M += rows[g];
    }
    if (!size_ok(M, dim) || !size_ok(M, N) || !size_ok(dim, N) || G * (dim * N) > kMaxElems)
        return false;
    // Weight gradients: the longest sums first, so that short ones fill the end.
    int order[mxk::kMmMaxGroups];
    for (int g = 0; g < G; g++) {
        int at = g;
        for (; sum_rows && at > 0 && rows[order[at - 1]] < rows[g]; at--)
            order[at] = order[at - 1];
        order[at] = g;
    }
    int place[mxk::kMmMaxGroups];
    for (int i = 0; i < G; i++)
        place[order[i]] = i;
    int64_t r = 0;
    for (int g = 0; g < G; g++) {
        const int i = place[g];
        t.rows[i] = (int32_t)rows[g];
        t.index[i] = g;
        t.row0[i] = r;
        t.sa_off[i] = sa;
        t.sb_off[i] = sb;
        r += rows[g];
        if (sum_rows) {
            sa += scale_bytes(dim, rows[g], tiled);
            sb += scale_bytes(N, rows[g], tiled);
        } else {
            sa += scale_bytes(rows[g], dim, tiled);
            sb += scale_bytes(N, dim, tiled);
        }
    }
    n.qa = (uint64_t)(M * dim);
    n.qb = (uint64_t)(sum_rows ? M * N : G * dim * N);
    n.sa = (uint64_t)sa;
    n.sb = (uint64_t)sb;
    n.y = (uint64_t)(sum_rows ? G * dim * N : M * N) * (uint64_t)out_size;
    return true;
}

// How a product is computed.
enum MmKind { kAny, kSmall, kTiles };

struct MmPlan {
    MmKind kind;
    int tile_m, tile_n;
    int waves;                 // of a small product's workgroup
    bool square;               // tiles of 128 x 128
    bool pack;                 // rows are copied to 128-byte boundaries first
    int64_t pack_a, pack_b;    // bytes of the copies
};

// In how many parts each of the last of n tiles, too few to fill the CUs, goes:
// 128 x 128 or 256 x 128, if those fill them once at most (2048 x 4096 outputs with
// 4096 k: 53 us in two rounds of 128 x 128, 51 us whole, 40 us in halves).
int last_parts(int64_t n)
{
    const int64_t last = n % mxk::kMmCUs;
    return last == 0 ? 1 : 4 * last <= mxk::kMmCUs ? 4 : 2 * last <= mxk::kMmCUs ? 2 : 1;
}

// The kernel for a launch and, in t, its tiles.  False if there are too many.
bool plan_mm(const mxk::MmArgs &a, mxk::MmTable &t, const MmBytes &n, MmPlan &p)
{
    const int G = t.count;
    int64_t most_m = 0, most_k = 0, big = 0, small32 = 0, small64 = 0, pitches = 0;
    double tile_steps = 0;
    bool rows16 = true;
    for (int g = 0; g < G; g++) {
        const int64_t m = a.sum_rows ? a.dim : t.rows[g], k = a.sum_rows ? t.rows[g] : a.dim;
        rows16 = rows16 && k % 16 == 0;
        most_m = m > most_m ? m : most_m;
        most_k = k > most_k ? k : most_k;
        const int64_t tiles = ceil_div(m, mxk::kMmTileM) * ceil_div(a.N, mxk::kMmTileN);
        big += tiles;
        tile_steps += (double)(tiles * ceil_div(k, 128));
        small32 += ceil_div(m, 32) * ceil_div(a.N, mxk::kMmSmallN);
        small64 += ceil_div(m, 64) * ceil_div(a.N, mxk::kMmSmallN);
        t.packed0[g] = pitches;
        pitches += mxk::mm_pitch(k);
    }
    // Small products: 32 rows at a time where that still does not fill the CUs more
    // than once (64 x 2048 outputs with 2048 k: 5.7 us, 64 rows at a time 7.5 us), or
    // there are no more; otherwise 64 share the loads of B (512 x 2048: 13.4 and 12
    // us).
    const int small_m = small32 <= mxk::kMmCUs || most_m <= 32 ? 32 : 64;
    const int64_t small = small_m == 32 ? small32 : small64;
    double small_bytes = 1, slow_bytes = 1;
    for (int g = 0; g < G; g++) {
        const int64_t m = a.sum_rows ? a.dim : t.rows[g], k = a.sum_rows ? t.rows[g] : a.dim;
        const double b = (double)(ceil_div(m, small_m) * ceil_div(a.N, mxk::kMmSmallN) * (small_m + mxk::kMmSmallN) * k);
        small_bytes += b;
        slow_bytes += b * (k % 16 == 0 ? a.out_f32 ? 1.2 : 1.0 : a.out_f32 ? 2.0 : 1.5);
    }
    p = MmPlan{};
    p.waves = small <= mxk::kMmCUs ? 8 : 4;
    // Microseconds, as measured (graph replays).
    // The small kernel: its waves' share of k, one after the other, and what each
    // workgroup reads for itself, at 14 TB/s from the caches, partly at the same time;
    // for each workgroup that does not start at once 5.4 ns, or 9 with its reads; all
    // that 1.2 times for fp32 outputs, 1.5 (2) times for unaligned rows.
    const double lat = (double)ceil_div(most_k, 128) *
                       (small_m == 32 ? p.waves == 8 ? 0.10 : 0.14 : p.waves == 8 ? 0.19 : 0.22);
    const double read = small_bytes / 14e6, each = 9e-3 - read / (double)small;
    const double more = small > mxk::kMmCUs ? (double)(small - mxk::kMmCUs) : 0;
    const double small_us = 3 + slow_bytes / small_bytes * ((lat > read ? lat + read / 4 : read + lat / 4) +
                                                            (each > 5.4e-3 ? each : 5.4e-3) * more);
    // The tiled one: rounds of tiles, of which the outputs are 8 us (in fp32 14), and the
    // last, partial one, whose steps in parts take longer than their share; in fp32
    // twice the time of a step; at least the longest sum; the copy of unaligned rows.
    const int parts = last_parts(big);
    const int64_t last = big % mxk::kMmCUs;
    auto round = [&](double steps) { return a.out_f32 ? 14 + 3 * steps : 8 + 1.5 * steps; };
    auto partial = [&](double steps) {
        const double f = a.out_f32 ? 2 : 1;
        return parts == 4   ? 1 + (a.out_f32 ? 0.8 : 0.5) * steps + f * (double)last / 32
               : parts == 2 ? 4 * f + 0.95 * f * steps
                            : round(steps);
    };
    const double steps = tile_steps / (double)big, most = (double)ceil_div(most_k, 128);
    const double all = (double)(big / mxk::kMmCUs) * round(steps) + (last ? partial(steps) : 0);
    const double longest = big < mxk::kMmCUs ? partial(most) : round(most);
    const double tile_us = 4 + (all > longest ? all : longest) + (rows16 ? 0 : 7 + (double)(n.qa + n.qb) / 2e6);
    if (n.qa < 16 || n.qb < 16 || n.sa < 8 || n.sb < 8) {
        p.kind = kAny;
        p.tile_m = p.tile_n = mxk::kMmAnyTile;
    } else if (small_us < tile_us && small <= kMaxTiles) {
        p.kind = kSmall;
        p.tile_m = small_m;
        p.tile_n = mxk::kMmSmallN;
    } else {
        p.kind = kTiles;
        p.tile_m = mxk::kMmTileM;
        p.tile_n = mxk::kMmTileN;
        p.pack = !rows16;
        // Tiles of 128 x 128, two workgroups per CU, whose outputs and starts overlap,
        // where the sums are short (4096 x 8192 outputs with 512 k: 31.6 -> 28.7 us) or
        // there are few tiles (2048 x 4096 with 2048 k: 24.3 -> 21.6 us); elsewhere their
        // reads take longer (8192^3: 414 -> 574 us; 2048^2 with 4096 k, where parts
        // have four buffers: 22.8 -> 26.3 us).
        p.square = 4 * big <= kMaxTiles &&
                   (steps <= 4 || (2 * big <= mxk::kMmCUs && steps <= 20));
        if (p.square)
            p.tile_m = p.tile_n = mxk::kMmPart;
    }
    if (p.pack) {
        const int64_t rows_a = a.sum_rows ? 0 : (int64_t)n.qa / a.dim, pitch = mxk::mm_pitch(a.dim);
        p.pack_a = a.sum_rows ? pitches * a.dim : rows_a * pitch;
        p.pack_b = a.sum_rows ? pitches * a.N : (int64_t)n.qb / a.dim * pitch;
    }
    int64_t tiles = 0;
    for (int g = 0; g < G; g++) {
        t.tile0[g] = (int32_t)tiles;
        tiles += ceil_div(a.sum_rows ? a.dim : t.rows[g], p.tile_m) * ceil_div(a.N, p.tile_n);
        if (tiles > kMaxTiles)
            return false;
    }
    t.tile0[G] = (int32_t)tiles;
    t.parts = p.kind == kTiles && !p.square ? parts : 1;
    t.square = p.square;
    t.whole = (int32_t)(t.parts == 1 ? tiles : tiles - tiles % mxk::kMmCUs);
    return true;
}

// Arguments, table and plan of a product, from valid flags; an error otherwise.
mx_status mm_setup(int64_t dim, int64_t N, const int64_t *rows, int G, bool sum_rows, unsigned flags,
                   mxk::MmArgs &a, mxk::MmTable &t, MmBytes &n, MmPlan &p)
{
    const bool tiled = (flags & MX_SCALE_TILED) != 0;
    if (!build_table(rows, G, dim, N, sum_rows, tiled, flags & MX_OUT_F32 ? 4 : 2, t, n))
        return MX_ERR_SHAPE;
    a = mxk::MmArgs{};
    a.dim = dim;
    a.N = N;
    a.sum_rows = sum_rows;
    a.tiled = tiled;
    a.a_e5m2 = (flags & MX_A_E5M2) != 0;
    a.b_e5m2 = (flags & MX_B_E5M2) != 0;
    a.out_f32 = (flags & MX_OUT_F32) != 0;
    a.accumulate = (flags & MX_OUT_ACCUMULATE) != 0;
    a.qa_bytes = (int64_t)n.qa;
    a.qb_bytes = (int64_t)n.qb;
    a.sa_bytes = (int64_t)n.sa;
    a.sb_bytes = (int64_t)n.sb;
    return plan_mm(a, t, n, p) ? MX_OK : MX_ERR_SHAPE;
}

bool mm_flags_ok(unsigned flags)
{
    return !(flags & ~kMmBits) && (!(flags & MX_OUT_ACCUMULATE) || (flags & MX_OUT_F32));
}

size_t mm_workspace(int64_t dim, int64_t N, const int64_t *rows, int G, bool sum_rows, unsigned flags)
{
    mxk::MmArgs a;
    mxk::MmTable t;
    MmBytes n;
    MmPlan p;
    if (!mm_flags_ok(flags) || mm_setup(dim, N, rows, G, sum_rows, flags, a, t, n, p) != MX_OK)
        return 0;
    return (size_t)(p.pack_a + p.pack_b);
}

mx_status mm_impl(const uint8_t *qa, const uint8_t *sa, const uint8_t *qb, const uint8_t *sb,
                  int64_t dim, int64_t N, const int64_t *rows, int G, bool sum_rows, unsigned flags,
                  void *y, void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    if (!mm_flags_ok(flags))
        return MX_ERR_ENUM;
    if (!qa || !sa || !qb || !sb || !y || !rows)
        return MX_ERR_NULL;
    mxk::MmArgs a;
    mxk::MmTable t;
    MmBytes n;
    MmPlan p;
    const mx_status st = mm_setup(dim, N, rows, G, sum_rows, flags, a, t, n, p);
    if (st != MX_OK)
        return st;
    const uint64_t nw = (uint64_t)(p.pack_a + p.pack_b);
    if (!aligned(qa, 16) || !aligned(sa, 16) || !aligned(qb, 16) || !aligned(sb, 16) ||
        !aligned(y, 16) || (nw && !aligned(workspace, 16)))
        return MX_ERR_ALIGN;
    if (nw && (!workspace || workspace_bytes < nw))
        return MX_ERR_WORKSPACE;
    const void *in[4] = {qa, sa, qb, sb};
    const uint64_t in_bytes[4] = {n.qa, n.sa, n.qb, n.sb};
    for (int i = 0; i < 4; i++)
        if (overlap(y, n.y, in[i], in_bytes[i]) || overlap(workspace, nw, in[i], in_bytes[i]))
            return MX_ERR_ALIAS;
    if (overlap(y, n.y, workspace, nw))
        return MX_ERR_ALIAS;

    a.qa = qa;
    a.sa = sa;
    a.qb = qb;
    a.sb = sb;
    a.y = y;
    if (p.kind == kAny)
        return from_hip(mxk::launch_mm_any(a, t, stream));
    if (p.kind == kSmall)
        return from_hip(mxk::launch_mm_small(a, t, p.tile_m, p.waves, stream));
    if (p.pack) {
        uint8_t *const wa = static_cast<uint8_t *>(workspace), *const wb = wa + p.pack_a;
        const hipError_t e = mxk::launch_mm_pack(a, t, wa, wb, stream);
        if (e != hipSuccess)
            return MX_ERR_HIP;
        a.packed = 1;
        a.qa = wa;
        a.qb = wb;
    }
    return from_hip((a.out_f32 ? mxk::launch_mm_tile_f32 : mxk::launch_mm_tile)(a, t, stream));
}

mx_status mv_impl(const void *x, const int32_t *experts, int64_t T, int64_t top, const uint8_t *qw,
                  const uint8_t *sw, const float *sg, int G, int64_t N, int64_t K, unsigned flags,
                  void *y, hipStream_t stream)
{
    if (!size_ok(T, K) || !size_ok(N, K) || top < 1 || top > 64 || !size_ok(T * top, N) || G < 1 ||
        G > 1024 || G * (N * K) > kMaxElems)
        return MX_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(qw, 16) || !aligned(sw, 16) || !aligned(y, 16) ||
        !aligned(sg, 4) || (experts && !aligned(experts, 4)))
        return MX_ERR_ALIGN;
    const uint64_t ny = (uint64_t)(T * top * N) * (flags & MX_OUT_F32 ? 4 : 2);
    if (overlap(y, ny, x, 2 * (uint64_t)(T * K)) ||
        overlap(y, ny, qw, (uint64_t)(G * N * ((K + 1) / 2))) ||
        overlap(y, ny, sw, (uint64_t)(G * N * ((K + 15) / 16))) ||
        overlap(y, ny, sg, 4 * (uint64_t)G) ||
        overlap(y, ny, experts, 4 * (uint64_t)(T * top)))
        return MX_ERR_ALIAS;

    mxk::MvArgs a{};
    a.x = static_cast<const uint16_t *>(x);
    a.experts = experts;
    a.qw = qw;
    a.sw = sw;
    a.sg = sg;
    a.y = y;
    a.T = (int32_t)T;
    a.N = (int32_t)N;
    a.K = (int32_t)K;
    a.top = (int32_t)top;
    a.G = G;
    a.out_f32 = (flags & MX_OUT_F32) != 0;
    return from_hip(mxk::launch_mv(a, stream));
}

}  // namespace

extern "C" {

size_t mx_matmul_workspace_size(int64_t M, int64_t N, int64_t K, unsigned flags)
{
    return mm_workspace(K, N, &M, 1, false, flags);
}

size_t mx_matmul_grouped_workspace_size(int64_t N, int64_t K, const int64_t *group_rows, int G,
                                        unsigned flags)
{
    return mm_workspace(K, N, group_rows, G, false, flags);
}

size_t mx_matmul_wgrad_grouped_workspace_size(int64_t N, int64_t K, const int64_t *group_rows, int G,
                                              unsigned flags)
{
    return mm_workspace(N, K, group_rows, G, true, flags);
}

mx_status mx_matmul(const uint8_t *qa, const uint8_t *sa, const uint8_t *qb, const uint8_t *sb,
                    int64_t M, int64_t N, int64_t K, unsigned flags, void *y, void *workspace,
                    size_t workspace_bytes, hipStream_t stream)
{
    return mm_impl(qa, sa, qb, sb, K, N, &M, 1, false, flags, y, workspace, workspace_bytes, stream);
}

mx_status mx_matmul_grouped(const uint8_t *qa, const uint8_t *sa, const uint8_t *qb,
                            const uint8_t *sb, int64_t N, int64_t K, const int64_t *group_rows,
                            int G, unsigned flags, void *y, void *workspace, size_t workspace_bytes,
                            hipStream_t stream)
{
    return mm_impl(qa, sa, qb, sb, K, N, group_rows, G, false, flags, y, workspace, workspace_bytes,
                   stream);
}

mx_status mx_matmul_wgrad_grouped(const uint8_t *qa, const uint8_t *sa, const uint8_t *qb,
                                  const uint8_t *sb, int64_t N, int64_t K,
                                  const int64_t *group_rows, int G, unsigned flags, void *dw,
                                  void *workspace, size_t workspace_bytes, hipStream_t stream)
{
    return mm_impl(qa, sa, qb, sb, N, K, group_rows, G, true, flags, dw, workspace, workspace_bytes,
                   stream);
}

mx_status nvfp4_matvec(const void *x, int64_t T, const uint8_t *qw, const uint8_t *sw,
                       const float *sg, int64_t N, int64_t K, unsigned flags, void *y,
                       hipStream_t stream)
{
    if (flags & ~MX_OUT_F32)
        return MX_ERR_ENUM;
    if (!x || !qw || !sw || !sg || !y)
        return MX_ERR_NULL;
    return mv_impl(x, nullptr, T, 1, qw, sw, sg, 1, N, K, flags, y, stream);
}

mx_status nvfp4_matvec_experts(const void *x, const int32_t *experts, int64_t T, int64_t top,
                               const uint8_t *qw, const uint8_t *sw, const float *sg, int G,
                               int64_t N, int64_t K, unsigned flags, void *y, hipStream_t stream)
{
    if (flags & ~MX_OUT_F32)
        return MX_ERR_ENUM;
    if (!x || !experts || !qw || !sw || !sg || !y)
        return MX_ERR_NULL;
    return mv_impl(x, experts, T, top, qw, sw, sg, G, N, K, flags, y, stream);
}

}  // extern "C"
