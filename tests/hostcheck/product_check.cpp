// The products' entry points (csrc/api_matmul.cpp) on the host, with recording
// stand-ins for the kernel launchers: random sizes up to the limits, each launch
// plan checked against the sizes it was made for.  Built under ASan and UBSan by
// tests/test_product_hostcheck.py.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <random>
#include <vector>

#include "launch_mm.h"
#include "mxcast.h"

using namespace mxk;

enum { kNone, kTileL, kTileF32, kSmallL, kAnyL, kMvL };
static int g_kind, g_packs, g_small_rows, g_waves;
static MmArgs g_a;
static MmTable g_t;
static MvArgs g_mv;
static const uint8_t *g_pack_a, *g_pack_b;

namespace mxk {
static hipError_t note(int kind, const MmArgs &a, const MmTable &t)
{
    g_kind = kind, g_a = a, g_t = t;
    return hipSuccess;
}
hipError_t launch_mm_tile(const MmArgs &a, const MmTable &t, hipStream_t) { return note(kTileL, a, t); }
hipError_t launch_mm_tile_f32(const MmArgs &a, const MmTable &t, hipStream_t) { return note(kTileF32, a, t); }
hipError_t launch_mm_any(const MmArgs &a, const MmTable &t, hipStream_t) { return note(kAnyL, a, t); }
hipError_t launch_mm_small(const MmArgs &a, const MmTable &t, int rows, int waves, hipStream_t)
{
    g_small_rows = rows, g_waves = waves;
    return note(kSmallL, a, t);
}
hipError_t launch_mm_pack(const MmArgs &, const MmTable &, uint8_t *qa, uint8_t *qb, hipStream_t)
{
    g_packs++, g_pack_a = qa, g_pack_b = qb;
    return hipSuccess;
}
hipError_t launch_mv(const MvArgs &a, hipStream_t)
{
    g_kind = kMvL, g_mv = a;
    return hipSuccess;
}
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
static int64_t scales(int64_t r, int64_t c, bool tiled)
{
    return tiled ? cdiv(r, 32) * cdiv(cdiv(c, 32), 8) * 256 : r * cdiv(c, 32);
}

template <typename T>
static T *at(int i)
{
    // addresses 2^44 apart, never read
    return reinterpret_cast<T *>((uintptr_t)(i + 1) << 44);
}

int main()
{
    std::mt19937_64 rng(7);
    auto size = [&](int64_t top) {
        const double b = std::uniform_real_distribution<>(0.0, __builtin_log2((double)top))(rng);
        int64_t v = (int64_t)__builtin_exp2(b);
        const int step = (int)(rng() % 4);
        v = step == 0 ? v : step == 1 ? v / 16 * 16 : step == 2 ? v / 128 * 128 : v | 1;
        return v < 1 ? (int64_t)1 : v > top ? top : v;
    };
    int seen[6] = {0, 0, 0, 0, 0, 0}, packed = 0, parts = 0, squares = 0;
    for (int it = 0; it < 20000; it++) {
        const bool wgrad = rng() % 2;
        const int G = it % 3 == 0 ? 1 : 1 + (int)(rng() % 64);
        const int64_t top = it % 5 ? 16384 : (int64_t)1 << 23;
        const int64_t N = size(top), K = size(top);
        std::vector<int64_t> rows(G);
        int64_t M = 0;
        for (auto &r : rows) {
            r = rng() % 4 ? size(top / G + 1) : 0;
            M += r;
        }
        const bool tiled = rng() % 2, f32 = rng() % 2;
        const unsigned flags = (tiled ? MX_SCALE_TILED : 0) | (f32 ? MX_OUT_F32 : 0) |
                               (f32 && rng() % 2 ? MX_OUT_ACCUMULATE : 0) | (rng() % 2 ? MX_A_E5M2 : 0);
        const size_t ws = wgrad ? mx_matmul_wgrad_grouped_workspace_size(N, K, rows.data(), G, flags)
                                : mx_matmul_grouped_workspace_size(N, K, rows.data(), G, flags);
        g_kind = kNone, g_packs = 0;
        const mx_status st = (wgrad ? mx_matmul_wgrad_grouped : mx_matmul_grouped)(
            at<uint8_t>(0), at<uint8_t>(1), at<uint8_t>(2), at<uint8_t>(3), N, K, rows.data(), G, flags,
            at<void>(4), at<void>(5), ws, nullptr);
        const int64_t lim = (int64_t)1 << 40, dim = wgrad ? N : K, cols = wgrad ? K : N;
        const bool ok = M > 0 && M <= (1 << 23) && M * dim <= lim && M * cols <= lim && dim * cols <= lim &&
                        G * (dim * cols) <= lim;
        if (!ok) {
            CHECK(st == MX_ERR_SHAPE && g_kind == kNone && ws == 0);
            continue;
        }
        if (st == MX_ERR_SHAPE) {       // more tiles than a launch has
            CHECK(g_kind == kNone && cdiv(wgrad ? N : M, 256) * cdiv(cols, 256) * G > (1 << 22));
            continue;
        }
        CHECK(st == MX_OK && g_kind != kNone);
        seen[g_kind]++;
        CHECK((g_kind == kTileF32) == (f32 && (g_kind == kTileL || g_kind == kTileF32)));
        CHECK((g_packs != 0) == (ws != 0) && g_packs <= 1 && (g_packs == 0) == (g_a.packed == 0));
        packed += g_packs;
        const bool tiles = g_kind == kTileL || g_kind == kTileF32;
        CHECK(g_t.square == 0 || (tiles && g_t.square == 1 && g_t.parts == 1));
        squares += g_t.square;
        const int64_t tm = g_t.square ? kMmPart : tiles ? kMmTileM : g_kind == kSmallL ? g_small_rows : kMmAnyTile;
        const int64_t tn = g_t.square ? kMmPart : tiles ? kMmTileN : g_kind == kSmallL ? kMmSmallN : kMmAnyTile;
        CHECK(g_kind != kSmallL || ((g_small_rows == 32 || g_small_rows == 64) && (g_waves == 4 || g_waves == 8)));
        CHECK(g_a.dim == dim && g_a.N == cols && g_a.sum_rows == wgrad && g_a.tiled == tiled);
        CHECK(g_t.count == G && g_t.tile0[0] == 0);
        std::vector<char> used(G, 0);
        int64_t pa = 0, pb = 0, qa = 0, qb = 0, sa = 0, sb = 0;
        for (int i = 0; i < G; i++) {
            const int g = g_t.index[i];
            CHECK(g >= 0 && g < G && !used[g]);
            used[g] = 1;
            CHECK(g_t.rows[i] == rows[g]);
            CHECK(!wgrad || i == 0 || g_t.rows[i] <= g_t.rows[i - 1]);
            int64_t r0 = 0, a0 = 0, b0 = 0;
            for (int k = 0; k < g; k++) {
                r0 += rows[k];
                a0 += wgrad ? scales(N, rows[k], tiled) : scales(rows[k], K, tiled);
                b0 += wgrad ? scales(K, rows[k], tiled) : scales(N, K, tiled);
            }
            CHECK(g_t.row0[i] == r0 && g_t.sa_off[i] == a0 && g_t.sb_off[i] == b0);
            CHECK(g_t.tile0[i + 1] - g_t.tile0[i] == cdiv(wgrad ? N : rows[g], tm) * cdiv(cols, tn));
            // packed weight gradient operands stand one after the other
            CHECK(g_t.packed0[i] == pa);
            pa += mm_pitch(wgrad ? rows[g] : K);
        }
        for (int g = 0; g < G; g++) {
            qa += wgrad ? N * rows[g] : rows[g] * K;
            qb += wgrad ? K * rows[g] : N * K;
            sa += wgrad ? scales(N, rows[g], tiled) : scales(rows[g], K, tiled);
            sb += wgrad ? scales(K, rows[g], tiled) : scales(N, K, tiled);
            pb += wgrad ? 0 : N * mm_pitch(K);
        }
        CHECK(g_a.qa_bytes == qa && g_a.qb_bytes == qb && g_a.sa_bytes == sa && g_a.sb_bytes == sb);
        // reads of 16 and 8 bytes fit the operands
        CHECK(g_kind == kAnyL || (qa >= 16 && qb >= 16 && sa >= 8 && sb >= 8));
        const int64_t total = g_t.tile0[G], pieces = g_t.parts;
        CHECK(pieces == 1 || (tiles && (pieces == 2 || pieces == 4)));
        CHECK(total > 0 && g_t.whole >= 0 && g_t.whole <= total);
        CHECK(g_t.whole == total || (pieces > 1 && g_t.whole % kMmCUs == 0 && (total - g_t.whole) * pieces <= kMmCUs));
        parts += g_t.whole < total;
        CHECK((g_t.whole + pieces * (total - g_t.whole)) * 256 < ((int64_t)1 << 32));
        // the tiled kernel's rows start at multiples of 16 bytes
        bool aligned = true;
        for (int g = 0; g < G; g++)
            aligned = aligned && (wgrad ? rows[g] : K) % 16 == 0;
        CHECK(!tiles || aligned || g_packs);
        if (g_packs) {
            const int64_t wa = wgrad ? pa * N : M * mm_pitch(K), wb = wgrad ? pa * K : G * N * mm_pitch(K);
            CHECK(wgrad || pb == wb);
            CHECK((int64_t)ws == wa + wb && g_pack_a == at<uint8_t>(5) && g_pack_b == g_pack_a + wa);
            CHECK(g_a.qa == g_pack_a && g_a.qb == g_pack_b);
            CHECK((wgrad ? mx_matmul_wgrad_grouped : mx_matmul_grouped)(
                      at<uint8_t>(0), at<uint8_t>(1), at<uint8_t>(2), at<uint8_t>(3), N, K, rows.data(), G,
                      flags, at<void>(4), at<void>(5), ws - 1, nullptr) == MX_ERR_WORKSPACE);
        }
    }
    for (int k : {kTileL, kTileF32, kSmallL, kAnyL})
        CHECK(seen[k] > 50);
    CHECK(packed > 50 && parts > 50 && squares > 50);

    for (int it = 0; it < 5000; it++) {
        const int64_t top = it % 2 ? 4096 : (int64_t)1 << 23;
        const int64_t T = size(top), N = size(top), K = size(top), tk = 1 + (int64_t)(rng() % 64);
        const int G = 1 + (int)(rng() % 1024);
        g_kind = kNone;
        const mx_status st = nvfp4_matvec_experts(at<void>(0), at<int32_t>(1), T, tk, at<uint8_t>(2),
                                                  at<uint8_t>(3), at<float>(4), G, N, K, 0, at<void>(5), nullptr);
        const int64_t lim = (int64_t)1 << 40;
        const bool ok = T * K <= lim && N * K <= lim && T * tk <= (1 << 23) && T * tk * N <= lim && G * (N * K) <= lim;
        CHECK(ok ? st == MX_OK && g_kind == kMvL : st == MX_ERR_SHAPE && g_kind == kNone);
        if (ok)
            CHECK(g_mv.T == T && g_mv.N == N && g_mv.K == K && g_mv.top == tk && g_mv.G == G);
    }
    printf("%d checks, %d failed\n", g_checks, g_failed);
    return g_failed != 0;
}
