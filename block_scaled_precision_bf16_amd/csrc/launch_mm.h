// launch_mm.h -- internal interface between the host entry points of the
// products on quantised operands (api_matmul.cpp) and their kernels.  Not
// installed; the public ABI is mxcast.h.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace mxk {

constexpr int kMmMaxGroups = 64;

// One launch of Y_g = A_g B_g^T over G groups.  Group g multiplies its
// operands A_g [m_g][k_g] and B_g [N][k_g] (codes row-major, each row's
// elements along the summed axis) into Y_g [m_g][N].
//   by expert (sum_rows = 0):  m_g = rows of group g, k_g = dim; the operands
//       B_g and their scales stand one after the other;
//   weight gradient (sum_rows = 1):  m_g = dim, k_g = rows of group g; A, B
//       and their scales hold the groups one after the other, Y is [G][dim][N].
struct MmTable {
    int32_t count;                      // the groups, in the order of their tiles
    int32_t whole;                      // tiles not taken in parts
    int32_t parts;                      // of each of the others
    int32_t square;                     // tiles of kMmPart x kMmPart, all whole
    int32_t tile0[kMmMaxGroups + 1];    // first workgroup tile of each
    int32_t rows[kMmMaxGroups];
    int32_t index[kMmMaxGroups];        // its place in the caller's order
    int64_t row0[kMmMaxGroups];         // its first stacked row
    int64_t packed0[kMmMaxGroups];      // packed weight gradient operands: the
                                        // pitches of the groups before it
    int64_t sa_off[kMmMaxGroups];       // byte offsets of its scales
    int64_t sb_off[kMmMaxGroups];
};

struct MmArgs {
    const uint8_t *qa, *sa, *qb, *sb;
    void *y;
    int64_t dim, N;
    int64_t qa_bytes, qb_bytes;         // of all groups' codes and scales
    int64_t sa_bytes, sb_bytes;
    int32_t sum_rows;
    int32_t packed;                     // operands as launch_mm_pack lays them out
    int32_t tiled;                      // scales in MX_SCALE_TILED layout
    int32_t a_e5m2, b_e5m2;
    int32_t out_f32, accumulate;        // fp32 output; added to what it holds
};

// Bytes between the rows of packed operands of K codes: whole 128-byte lines,
// filled up with zeros.
#ifdef __HIPCC__
__host__ __device__
#endif
constexpr int64_t mm_pitch(int64_t K) { return (K + 127) / 128 * 128; }

// The tiled kernel: its tiles, and the sides of the parts (128 x 128 or 256 x 128) in
// which the last ones go.
constexpr int kMmTileM = 256, kMmTileN = 256, kMmPart = 128;
constexpr int kMmCUs = 256;
// The tile of the kernel for tiny operands, and the columns of the small kernel's.
constexpr int kMmAnyTile = 64, kMmSmallN = 32;

hipError_t launch_mm_tile(const MmArgs &a, const MmTable &t, hipStream_t stream);
hipError_t launch_mm_tile_f32(const MmArgs &a, const MmTable &t, hipStream_t stream);
// rows: 32 or 64 of a workgroup's tile; waves: 4 or 8, which share k.
hipError_t launch_mm_small(const MmArgs &a, const MmTable &t, int rows, int waves, hipStream_t stream);
hipError_t launch_mm_any(const MmArgs &a, const MmTable &t, hipStream_t stream);
// Copies the operands' rows to qa and qb, mm_pitch apart.
hipError_t launch_mm_pack(const MmArgs &a, const MmTable &t, uint8_t *qa, uint8_t *qb, hipStream_t stream);

// NVFP4 matrix-vector products.  experts == NULL: y[T][N] = x W^T.  Otherwise
// slot p = t * top + j of y [T * top][N] takes W_e, e = experts[p], G matrices.
struct MvArgs {
    const uint16_t *x;
    const int32_t *experts;
    const uint8_t *qw, *sw;
    const float *sg;
    void *y;
    int32_t T, N, K;                    // each at most 2^23, T * top too
    int32_t top, G;
    int32_t out_f32;
    int32_t by_slot;                    // set by the launcher
};

constexpr int kMvThreads = 512, kMvWaves = 8;
constexpr int kMvChunk = 256;          // k of one step of a wave

// How a kernel for up to TT tokens is laid out: KS waves share the chunks of a
// row, each has D of its chunks under way, a stage holds the tokens of D KS
// chunks.  FEW: for few rows, all 8 waves share them.
template <int TT, bool EXPERTS, bool FEW>
struct MvPlan {
    static constexpr int KS = FEW || (TT <= 2 && EXPERTS) ? 8 : TT <= 16 ? 4 : 2, WN = kMvWaves / KS, D = TT <= 2 && !EXPERTS ? 4 : 2;
    static constexpr int kRows = 16 * WN;                     // weight rows of a block
    static constexpr int kFit = D * KS;                       // chunks of a stage
    static constexpr int kPieces = kFit * 512 * TT / 16 / kMvThreads;   // of a thread
    // 1 or 2 tokens: dot products on the vector units.  Their weights carry the power
    // of two of the block's scale, which the conversion applies, and the block's sum
    // its significand, so that a sum leaves fp32's range only where one of wholly
    // scaled weights, as for more tokens, does: 1.1 (1.6) vector instructions a weight
    static constexpr bool kDot = TT <= 2;
    // LDS: a stage's tokens, then the waves' sums of a token tile
    static constexpr int kTokens = kFit * 512 * TT, kLds = kTokens + kMvWaves * 1024;
};

// The kernel for a product: for up to `tokens` (1, 2, 8, 16, 32, 64) at a time, 0 for
// operands smaller than its loads; few: for few rows.
struct MvChoice {
    int tokens;
    bool few;
};

inline MvChoice mv_choose(const MvArgs &a)
{
    const int64_t rows = (int64_t)a.G * a.N;
    if (rows * ((a.K + 1) / 2) < 16 || rows * ((a.K + 15) / 16) < 4 || (int64_t)a.T * a.K < 8)
        return {0, false};
    // tokens that a weight matrix meets: all, or an expert's fair share twice over
    const int64_t slots = (int64_t)a.T * a.top;
    const int64_t tokens = a.experts ? (2 * slots + a.G - 1) / a.G : a.T;
    int64_t most = slots < tokens ? slots : tokens;
    // Few rows of many tokens: 16 or 32 at a time, the weights read again (from the
    // caches) for each, rather than few workgroups.
    if (!a.experts && a.T > 16) {
        const int64_t by16 = (((int64_t)a.N + 31) / 32) * ((a.T + 15) / 16);
        const int64_t by32 = (((int64_t)a.N + 63) / 64) * ((a.T + 31) / 32);
        most = by16 <= 512 ? 16 : by32 <= 256 ? 32 : 64;
        most = most > a.T ? a.T : most;
    }
    const int at_once = most <= 1 ? 1 : most <= 2 ? 2 : most <= 8 ? 8 : most <= 16 ? 16 : most <= 32 ? 32 : 64;
    // Workgroups of 32 rows that do not fill the CUs: twice as many, of 16 (5 tokens by
    // 1001 x 4095: 7.9 -> 6.7 us, 4096 x 4096: 7.5 -> 5.8 us; but 16384 x 16384: 38 -> 42
    // us, and 512 x 512, where there is nothing to share: 4.1 -> 4.6 us).  For 16 tokens
    // only one of them fits a CU's LDS.
    const int64_t blocks = ((int64_t)a.N + 31) / 32 * (((int64_t)a.T + at_once - 1) / at_once);
    const bool few = !a.experts && at_once <= 16 && blocks <= (at_once == 16 ? 128 : 255) && a.K >= 1024;
    return {at_once, few};
}

hipError_t launch_mv(const MvArgs &a, hipStream_t stream);

}  // namespace mxk
