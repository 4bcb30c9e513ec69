// The entry points of the norm, the router and the rows' way to the experts
// (csrc/api_norm.cpp, csrc/api_moe.cpp) on the host, with recording stand-ins for the
// kernel launchers: random sizes up to the limits, each launch plan checked against
// what the kernels assume.  Built under ASan and UBSan by
// tests/test_layer_hostcheck.py.
#include <stdint.h>
#include <stdio.h>

#include <random>

#include "launch_moe.h"
#include "launch_norm.h"
#include "mxcast.h"

using namespace mxk;

static int g_norm, g_cols, g_any, g_back, g_moe;
static NormArgs g_n;
static NormBackArgs g_b;
static MxArgs g_m;
static GroupTable g_t;
static bool g_rag;
static RouteArgs g_route;
static SortArgs g_sort;
static GatherArgs g_gather;
static CombineArgs g_combine;

namespace mxk {
hipError_t launch_norm(unsigned, const NormArgs &a, hipStream_t) { g_norm++, g_n = a; return hipSuccess; }
hipError_t launch_norm_back(const NormBackArgs &a, hipStream_t) { g_back++, g_b = a; return hipSuccess; }
hipError_t launch_mx_cast_norm(unsigned, const MxArgs &a, const GroupTable *t, hipStream_t)
{
    g_cols++, g_m = a, g_rag = t != nullptr;
    if (t)
        g_t = *t;
    return hipSuccess;
}
hipError_t launch_mx_cast_any(int, unsigned, unsigned, bool, const MxArgs &a, const GroupTable &t, hipStream_t)
{
    g_any++, g_m = a, g_t = t;
    return hipSuccess;
}
hipError_t launch_route(const RouteArgs &a, hipStream_t) { g_moe++, g_route = a; return hipSuccess; }
hipError_t launch_route_back(const RouteBackArgs &, hipStream_t) { g_moe++; return hipSuccess; }
hipError_t launch_sort(const SortArgs &a, hipStream_t) { g_moe++, g_sort = a; return hipSuccess; }
hipError_t launch_gather(const GatherArgs &a, hipStream_t) { g_moe++, g_gather = a; return hipSuccess; }
hipError_t launch_combine(const CombineArgs &a, hipStream_t) { g_moe++, g_combine = a; return hipSuccess; }
hipError_t launch_combine_back(const CombineArgs &a, hipStream_t) { g_moe++, g_combine = a; return hipSuccess; }
}  // namespace mxk

static int g_checks, g_failed;
#define CHECK(c)                                                                   \
    do {                                                                           \
        g_checks++;                                                                \
        if (!(c)) {                                                                \
            g_failed++;                                                            \
            printf("line %d: %s\n", __LINE__, #c);                                 \
        }                                                                          \
    } while (0)

static int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
// Addresses far from each other, never read.
static void *at(int i) { return reinterpret_cast<void *>(int64_t(i) << 46); }
template <class T>
static T *as(int i) { return static_cast<T *>(at(i)); }

static std::mt19937_64 rng(7);
static int64_t size(int64_t most)
{
    const int64_t n = int64_t(1) << (rng() % 24);
    const int64_t v = (n + int64_t(rng() % uint64_t(n))) / (rng() % 3 ? 1 : 8) * (rng() % 3 ? 1 : 8);
    return v < 1 ? 1 : v > most ? most : v;
}

static void norm_case(int64_t M, int64_t K, unsigned axis, bool res)
{
    const int before = g_norm + g_cols + g_any;
    const mx_status st = mx_rmsnorm(at(1), res ? at(2) : nullptr, at(3), M, K, 1e-6f, axis, at(4), nullptr,
                                    as<uint8_t>(5), as<uint8_t>(6), as<uint8_t>(7), as<uint8_t>(8), nullptr,
                                    nullptr, as<float>(9), at(10), mx_rmsnorm_workspace_size(M, axis), nullptr);
    if (M > (1 << 23) || K > (1 << 23) || M * K > (int64_t(1) << 40)) {
        CHECK(st == MX_ERR_SHAPE && g_norm + g_cols + g_any == before);
        return;
    }
    CHECK(st == MX_OK);
    CHECK(g_n.M == M && g_n.K == K && (g_n.q_row != nullptr) == ((axis & 1) != 0));
    CHECK((g_n.h != nullptr) == res);
    const NormShape s = norm_shape(K);
    if (s.chunks) {
        CHECK(s.threads % 64 == 0 && s.threads >= 64 && s.threads <= 1024);
        CHECK((int64_t)s.threads * s.chunks * 8 >= K);
        CHECK(s.threads * norm_back_rows(s) <= (s.threads > 512 ? 1024 : 512));
        // the tile layout's padding blocks have lanes
        CHECK((int64_t)s.threads * s.chunks >= cdiv(cdiv(K, 32), 8) * 32);
    }
    CHECK(norm_back_parts(M, K) >= 1 && norm_back_parts(M, K) <= 256);
    if (!(axis & 2))
        return;
    CHECK(mx_rmsnorm_workspace_size(M, axis) == 8 * (size_t)M && g_n.cut == at(10) && g_n.low == g_n.cut + M);
    CHECK(g_m.row_scale == g_n.cut && g_m.row_low == g_n.low && g_m.x == (res ? at(4) : at(1)) && g_m.aux == at(3) && g_m.ldg == 0);
    const bool any = K % 8 != 0;
    const int64_t tm = any ? kAnyTileM : kTileM, tk = any ? kAnyTileK : kTileK;
    CHECK(g_m.tiles_m == cdiv(M, tm) && g_m.tiles_k == cdiv(K, tk));
    CHECK(g_m.group >= 1 && g_m.group <= (any ? kAnyMaxWalk : M % 16 ? kMaxRagGroup : kMaxGroup));
    CHECK((int64_t)g_m.group * g_m.groups_m >= g_m.tiles_m && (int64_t)g_m.group * (g_m.groups_m - 1) < g_m.tiles_m);
    CHECK(!g_m.tiled || any || g_m.group % 2 == 0);
    if (any || g_rag)
        CHECK(g_t.count == 1 && g_t.len[0] == g_m.group && g_t.walk0[0] == 0 && g_t.walk0[1] == g_m.groups_m &&
              g_t.row0[0] == 0 && g_t.row0[1] == M);
    CHECK(any || g_rag == (M % 16 != 0));
}

static void sort_case(int64_t T, int64_t top, int64_t E, int64_t align)
{
    const int64_t rows = moe_sort_rows(T, top, E, align);
    const size_t ws = moe_sort_workspace_size(T, top, E);
    const bool ok = T * top <= (1 << 23) && top <= 64;
    CHECK((rows != 0) == ok);
    const mx_status st = moe_sort(as<int32_t>(1), T, top, E, align, rows ? rows : 1, as<int32_t>(2), as<int32_t>(3),
                                  as<int32_t>(4), ws ? at(5) : nullptr, ws, nullptr);
    if (!ok || rows > (1 << 24)) {
        CHECK(st == MX_ERR_SHAPE);
        return;
    }
    CHECK(st == MX_OK && g_sort.N == T * top && g_sort.rows == rows);
    CHECK((int64_t)g_sort.blocks * g_sort.chunk >= g_sort.N && (int64_t)(g_sort.blocks - 1) * g_sort.chunk < g_sort.N);
    CHECK((g_sort.ws != nullptr) == (g_sort.N > kSortFew));
    if (g_sort.ws) {
        CHECK(g_sort.blocks <= 256 && g_sort.chunk % kSortThreads == 0 && ws == (size_t)g_sort.blocks * E * 4);
        CHECK(g_sort.chunk <= 65535);              // 16-bit counts
    } else {
        CHECK(g_sort.blocks <= 16 && g_sort.chunk % 1024 == 0 && g_sort.chunk <= 65535);
    }
}

int main()
{
    for (int i = 0; i < 20000; i++) {
        const unsigned axis = 1 + rng() % 3, flags = 4 * (rng() % 8);
        norm_case(size(1 << 24), size(1 << 24), axis | flags, rng() % 2);
    }
    for (int64_t m : {int64_t(1), int64_t(17), int64_t(1) << 23})
        for (int64_t k : {int64_t(1), int64_t(8), int64_t(16384), int64_t(16385), int64_t(131072)})
            for (unsigned axis : {1u, 2u, 3u, 3u | MX_SCALE_TILED})
                norm_case(m, k, axis, true);
    for (int i = 0; i < 20000; i++)
        sort_case(size(1 << 23), 1 + rng() % 66, 1 + rng() % 1024, 1 + rng() % (rng() % 2 ? 32 : 4096));
    sort_case(1 << 17, 64, 1024, 1);
    sort_case(1 << 23, 1, 1, 4096);
    printf("%d checks, %d failed\n", g_checks, g_failed);
    return g_failed != 0;
}
