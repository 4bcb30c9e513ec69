// Which kernel each product takes (csrc/api_matmul.cpp, launch_mm.h), on the host: for
// each line of the standard input one line out.
//   mm M N K flags              -> small <rows> <waves> | any | tile <whole> <parts> <square> <packed>
//   mv T N K                    -> <tokens> <few> <stages of k>
//   mve T top G N K             -> <tokens> <by slot> <stages of k>
// Used by tests/test_product_variants.py.
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include <string>

#include "launch_mm.h"
#include "mxcast.h"

using namespace mxk;

static std::string g_out;
static bool g_packed;

static std::string words(const char *name, long a, long b, long c, long d)
{
    char s[128];
    snprintf(s, sizeof s, "%s %ld %ld %ld %ld", name, a, b, c, d);
    return s;
}

template <int TT, bool EXPERTS>
static int fit(bool few)
{
    return few ? MvPlan<TT, EXPERTS, true>::kFit : MvPlan<TT, EXPERTS, false>::kFit;
}

template <bool EXPERTS>
static int fit_of(int tokens, bool few)
{
    return tokens == 1    ? fit<1, EXPERTS>(few)
           : tokens == 2  ? fit<2, EXPERTS>(few)
           : tokens == 8  ? fit<8, EXPERTS>(few)
           : tokens == 16 ? fit<16, EXPERTS>(few)
           : tokens == 32 ? fit<32, EXPERTS>(few)
                          : fit<64, EXPERTS>(few);
}

namespace mxk {
static hipError_t tile(const MmTable &t)
{
    g_out = words("tile", t.whole, t.whole == t.tile0[t.count] ? 1 : t.parts, t.square, g_packed);
    return hipSuccess;
}
hipError_t launch_mm_tile(const MmArgs &, const MmTable &t, hipStream_t) { return tile(t); }
hipError_t launch_mm_tile_f32(const MmArgs &, const MmTable &t, hipStream_t) { return tile(t); }
hipError_t launch_mm_any(const MmArgs &, const MmTable &, hipStream_t)
{
    g_out = "any";
    return hipSuccess;
}
hipError_t launch_mm_small(const MmArgs &, const MmTable &, int rows, int waves, hipStream_t)
{
    g_out = "small " + std::to_string(rows) + " " + std::to_string(waves);
    return hipSuccess;
}
hipError_t launch_mm_pack(const MmArgs &, const MmTable &, uint8_t *, uint8_t *, hipStream_t)
{
    g_packed = true;
    return hipSuccess;
}
hipError_t launch_mv(const MvArgs &a, hipStream_t)
{
    const MvChoice c = mv_choose(a);
    const int64_t slots = (int64_t)a.T * a.top;
    if (c.tokens == 0) {
        g_out = "tiny";
        return hipSuccess;
    }
    const int k = kMvChunk * (a.experts ? fit_of<true>(c.tokens, false) : fit_of<false>(c.tokens, c.few));
    g_out = std::to_string(c.tokens) + " " + std::to_string(a.experts ? slots <= a.G : c.few) + " " +
            std::to_string((a.K + k - 1) / k);
    return hipSuccess;
}
}  // namespace mxk

template <typename T>
static T *at(int i)
{
    // addresses 2^44 apart, never read
    return reinterpret_cast<T *>((uintptr_t)(i + 1) << 44);
}

int main()
{
    char line[256], op[8];
    long v[5];
    while (fgets(line, sizeof line, stdin)) {
        const int n = sscanf(line, "%7s %ld %ld %ld %ld %ld", op, v, v + 1, v + 2, v + 3, v + 4) - 1;
        g_out = "", g_packed = false;
        mx_status st = MX_ERR_ENUM;
        if (n == 4 && !strcmp(op, "mm"))
            st = mx_matmul(at<uint8_t>(0), at<uint8_t>(1), at<uint8_t>(2), at<uint8_t>(3), v[0], v[1], v[2],
                           (unsigned)v[3], at<void>(4), at<void>(5), (size_t)1 << 42, nullptr);
        else if (n == 3 && !strcmp(op, "mv"))
            st = nvfp4_matvec(at<void>(0), v[0], at<uint8_t>(2), at<uint8_t>(3), at<float>(4), v[1], v[2], 0,
                              at<void>(5), nullptr);
        else if (n == 5 && !strcmp(op, "mve"))
            st = nvfp4_matvec_experts(at<void>(0), at<int32_t>(1), v[0], v[1], at<uint8_t>(2), at<uint8_t>(3),
                                      at<float>(4), (int)v[2], v[3], v[4], 0, at<void>(5), nullptr);
        if (st != MX_OK)
            return 1;
        puts(g_out.c_str());
    }
    return 0;
}
