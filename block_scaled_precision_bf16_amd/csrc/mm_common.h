// mm_common.h -- device code the kernels of the MXFP8 products share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bufio.h"
#include "launch_mm.h"

namespace mxk {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ i32x8_t join(uint4 a, uint4 b)
{
    return i32x8_t{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// How a product is computed.
//   kMx: gfx950's block-scaled MFMA on the codes and scale bytes, 32 x 32 x 64.
//       It sums 8 neighbouring k with the products aligned to the largest one's
//       exponent and cut below 2^-13 of it (measured; everything beyond those 8
//       is summed in fp32): an error of the order of 1.5e-5 of the result, 100
//       times below the rounding of a bf16 output, which is where it is used.
//   kExact: the codes times their scales as bf16 (at most 4 significant bits: exact
//       where the power of two fits, see far_block), products exact, sums in fp32, by
//       the bf16 MFMA, 32 x 32 x 16, at half the rate; for fp32 outputs.  A step with
//       values that bf16 does not hold goes by mfma_far instead.
enum MmMode { kMx, kExact };

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2v_t __attribute__((ext_vector_type(2)));

// Two of the four codes of w (the upper two with HI) times 2^(e - 127), where
// scale holds e in its exponent field.
template <int F, bool HI>
__device__ __forceinline__ uint32_t bf16_of_codes(uint32_t w, float scale)
{
    const bf16x2v_t v = F ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, HI)
                          : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HI);
    return __builtin_bit_cast(uint32_t, v);
}

template <int F>
__device__ __forceinline__ bf16x8_t bf16_of_codes8(uint32_t lo, uint32_t hi, float scale)
{
    typedef uint32_t u32x4v_t __attribute__((ext_vector_type(4)));
    const u32x4v_t v = {bf16_of_codes<F, false>(lo, scale), bf16_of_codes<F, true>(lo, scale),
                        bf16_of_codes<F, false>(hi, scale), bf16_of_codes<F, true>(hi, scale)};
    return __builtin_bit_cast(bf16x8_t, v);
}

// Whether a block has elements that its scale may take out of what bf16 holds, the
// multiples of 2^-133 below 2^128: E4M3's are multiples of 2^-9 up to 448 = 1.75 2^8,
// E5M2's of 2^-16 up to 57344 = 1.75 2^15.  (Scale bytes that the casts write for values
// near the ends of bf16's range; blocks of zeros, whose byte is 0, are not among them.)
// NaN blocks are.
template <int F>
__device__ __forceinline__ bool far_block(uint4 codes, uint32_t byte)
{
    constexpr uint32_t lo = F ? 10 : 3, hi = F ? 239 : 246;
    return ((codes.x | codes.y | codes.z | codes.w) & 0x7F7F7F7Fu) != 0 && byte - lo > hi - lo;
}

// Bit 7 of each byte is set where the byte of w lies in 64 .. 191: no block is far if
// it is in all of them, which is cheaper to look at first.
__device__ __forceinline__ uint32_t middle_bytes(uint32_t w) { return w ^ (w << 1); }
// The same bits for the bytes behind the first `live`, blocks behind the rows' ends.
__device__ __forceinline__ uint32_t dead_bytes(int live)
{
    return live >= 4 ? 0 : live <= 0 ? 0x80808080u : 0x80808080u << (8 * live);
}
// Whether a lane's bits of both, all its words' ANDed, say that a byte is elsewhere.
__device__ __forceinline__ bool any_not_middle(uint32_t middle)
{
    return __ballot((middle & 0x80808080u) != 0x80808080u) != 0;
}

// fp32 to bf16 bits, to nearest even, NaN kept.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const bf16x2_t v = __builtin_convertvector((f32x2_t{lo, hi}), bf16x2_t);
    uint32_t u;
    __builtin_memcpy(&u, &v, 4);
    return u;
}

// A workgroup's tile: its group's operands and the tile's first row and column.
struct MmTile {
    const uint8_t *qa, *sa, *qb, *sb;
    int64_t M, K, nb;       // the group's output rows, summed length, blocks of 32
    int64_t qa_left, qb_left;   // bytes from the group's operands to the arrays' ends
    int64_t sa_left, sb_left;
    int64_t y0;             // first element of the group's output
    int64_t m0, n0;
};

// Tile number of workgroup `id` of n.  Workgroups go to the 8 XCDs in turn; runs
// of kRun consecutive tiles, which share operands in an L2, go to one XCD, the
// next run to the next (so that groups of unequal work are spread).  What is
// left behind the last 8 whole runs stays in order.
constexpr int kRun = 32;
__device__ __forceinline__ int mm_xcd_order(int id, int n)
{
    if (id >= n / (8 * kRun) * (8 * kRun))
        return id;
    const int x = id & 7, s = id >> 3;
    return (s / kRun * 8 + x) * kRun + s % kRun;
}

// Tile number `id` of the launch: the group whose range holds it, and in it
// bands of kBand tile rows, each band's tiles counted down its rows first (so
// that a run of tiles is about square).  A group without output tiles takes
// no ids.
constexpr int kBand = 4;
__device__ __forceinline__ MmTile mm_tile(const MmArgs &a, const MmTable &t, int id, int tile_m,
                                          int tile_n)
{
    // (all lanes look at once: one group after the other is a chain of loads)
    const int L = (int)threadIdx.x & 63;
    const int g = __popcll(__ballot(L < t.count && id >= t.tile0[L + 1 < t.count ? L + 1 : t.count]));
    const int64_t r0 = t.row0[g], rows = t.rows[g];
    MmTile w;
    w.M = a.sum_rows ? a.dim : rows;
    w.K = a.sum_rows ? rows : a.dim;
    w.nb = (w.K + 31) / 32;
    if (a.packed) {
        // the rows' zeros behind the last code count as codes
        w.K = mm_pitch(w.K);
        const int64_t p0 = t.packed0[g];
        w.qa = a.qa + (a.sum_rows ? p0 * a.dim : r0 * w.K);
        w.qb = a.qb + (a.sum_rows ? p0 * a.N : t.index[g] * a.N * w.K);
    } else {
        w.qa = a.qa + r0 * a.dim;
        w.qb = a.qb + (a.sum_rows ? r0 * a.N : t.index[g] * a.N * a.dim);
    }
    w.sa = a.sa + t.sa_off[g];
    w.sb = a.sb + t.sb_off[g];
    w.qa_left = a.qa_bytes - (w.qa - a.qa);
    w.qb_left = a.qb_bytes - (w.qb - a.qb);
    w.sa_left = a.sa_bytes - t.sa_off[g];
    w.sb_left = a.sb_bytes - t.sb_off[g];
    w.y0 = a.sum_rows ? t.index[g] * a.dim * a.N : r0 * a.N;
    const int j = id - t.tile0[g], tm = (int)((w.M + tile_m - 1) / tile_m);
    const int tn = (int)((a.N + tile_n - 1) / tile_n);
    const int band = j / (kBand * tn), in = j - band * (kBand * tn);
    const int high = tm - band * kBand < kBand ? tm - band * kBand : kBand;
    w.m0 = (int64_t)(band * kBand + in % high) * tile_m;
    w.n0 = (int64_t)(in / high) * tile_n;
    return w;
}

// A tile without a sum whose outputs keep what they hold, to the bit (-0 + 0 is 0): an
// empty group's gradient with MX_OUT_ACCUMULATE.
__device__ __forceinline__ bool nothing_to_add(const MmArgs &a, const MmTile &w)
{
    return a.accumulate && w.K == 0;
}

// Scale byte of (row, blk) of an operand [rows][nb]; 0 (2^-127) outside it,
// where every element is 0.
__device__ __forceinline__ int scale_byte(const uint8_t *s, int64_t rows, int64_t nb, int64_t row,
                                          int64_t blk, int tiled)
{
    if (row >= rows || blk >= nb)
        return 0;
    if (!tiled)
        return s[row * nb + blk];
    const int64_t tile = (blk >> 3) * ((rows + 31) >> 5) + (row >> 5);
    return s[tile * 256 + 4 * ((row & 31) + 32 * (blk & 1)) + ((blk & 7) >> 1)];
}

// The fp32 number whose exponent field is the scale byte.
__device__ __forceinline__ float scale_float(int byte) { return __uint_as_float((uint32_t)byte << 23); }

__device__ __forceinline__ void store_out(const MmArgs &a, int64_t i, float v)
{
    if (a.out_f32) {
        float *y = static_cast<float *>(a.y);
        y[i] = a.accumulate ? y[i] + v : v;
    } else {
        static_cast<uint16_t *>(a.y)[i] = (uint16_t)bf16_pair(v, 0.f);
    }
}

// Outputs i and i + 1, at any element (rows of odd lengths): one store.
__device__ __forceinline__ void store_out2(const MmArgs &a, int64_t i, float v0, float v1)
{
    if (a.out_f32) {
        float *y = static_cast<float *>(a.y) + i;
        float2 o = make_float2(0.f, 0.f);
        if (a.accumulate)
            __builtin_memcpy(&o, y, 8);
        o = a.accumulate ? make_float2(o.x + v0, o.y + v1) : make_float2(v0, v1);
        __builtin_memcpy(y, &o, 8);
    } else {
        const uint32_t o = bf16_pair(v0, v1);
        __builtin_memcpy(static_cast<uint16_t *>(a.y) + i, &o, 4);
    }
}

__device__ __forceinline__ uint32_t clip31(int64_t v)
{
    return (uint32_t)(v < kMaxRecords ? v : kMaxRecords);
}

// v moved down by d bytes (d < 16).
__device__ __forceinline__ uint4 bytes_down(uint4 v, uint32_t d)
{
    if (d & 8)
        v = make_uint4(v.z, v.w, 0, 0);
    if (d & 4)
        v = make_uint4(v.y, v.z, v.w, 0);
    const uint32_t b = d & 3;
    return make_uint4(__builtin_amdgcn_alignbyte(v.y, v.x, b), __builtin_amdgcn_alignbyte(v.z, v.y, b),
                      __builtin_amdgcn_alignbyte(v.w, v.z, b), __builtin_amdgcn_alignbyte(0, v.w, b));
}

// The first n of v's 16 bytes, zeros behind them.
__device__ __forceinline__ uint4 bytes_keep(uint4 v, int n)
{
    auto word = [n](uint32_t w, int at) {
        return n >= at + 4 ? w : n <= at ? 0u : w & ((1u << (8 * (n - at))) - 1);
    };
    return make_uint4(word(v.x, 0), word(v.y, 4), word(v.z, 8), word(v.w, 12));
}

// Byte rows that are read B bytes (16 or 8) at a time at any place, the last ones
// of an array too: a base inside the array, up to B bytes before the tile's
// first row, and the last offset from it that B bytes may be read at.  A read
// that would pass it is taken there and moved down.
template <int B>
struct ByteRows {
    const uint8_t *base;
    int64_t last;
    uint32_t lead;             // offset of the tile's first row

    ByteRows() = default;
    // rows of `pitch` bytes from `first` on, of an array that `left` bytes from
    // there on belong to
    __device__ __forceinline__ ByteRows(const uint8_t *array, const uint8_t *first, int64_t left)
        : base(first - array < B ? array : first - B), last(left + (first - base) - B),
          lead((uint32_t)(first - base))
    {
    }
    // B bytes at off + at (at: the part that all lanes share), or the array's last B.
    template <typename V>
    __device__ __forceinline__ V load(uint32_t off, int64_t at) const
    {
        static_assert(sizeof(V) == B, "one read");
        const int64_t to = at < last ? at : last;
        const uint8_t *p = base + to;
        const uint32_t lim = clip31(last - to);
        V v;
        __builtin_memcpy(&v, p + (off < lim ? off : lim), B);
        return v;
    }
    // By how many bytes what load(off, at) read has to move down (more than any
    // row needs: for reads behind the array).
    __device__ __forceinline__ uint32_t behind(uint32_t off, int64_t at) const
    {
        const int64_t d = off + at - last;
        return d <= 0 ? 0 : d < 15 ? (uint32_t)d : 15;
    }
    // What load(off, at) read, with n of its bytes inside the row.
    __device__ __forceinline__ uint4 fix(uint4 v, uint32_t off, int64_t at, int n) const
    {
        return bytes_keep(bytes_down(v, behind(off, at)), n);
    }
};

template <int FA, int FB, int J>
__device__ __forceinline__ f32x16_t mfma_mx(i32x8_t a, i32x8_t b, f32x16_t c, uint32_t sa, uint32_t sb)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, FA, FB, J, (int)sa, J, (int)sb);
}

// c + A B^T over 64 k for fp32 outputs at any scales: the block-scaled MFMA takes the
// powers of two in their whole range, and with one of each 8 neighbouring k at a time,
// the others 0 in both operands, it has nothing to align.  8 instructions, 4 times the
// matrix time of the bf16 ones.
struct Pick {
    uint32_t even, odd;        // of the even and odd words of codes
    __device__ __forceinline__ explicit Pick(int q)
        : even(q < 4 ? 0xFFu << (8 * q) : 0), odd(q < 4 ? 0 : 0xFFu << (8 * (q - 4)))
    {
    }
    __device__ __forceinline__ i32x8_t of(i32x8_t v) const
    {
        const int e = (int)even, o = (int)odd;
        return v & i32x8_t{e, o, e, o, e, o, e, o};
    }
};

template <int FA, int FB, int J>
__device__ __forceinline__ f32x16_t mfma_far(i32x8_t a, i32x8_t b, f32x16_t c, uint32_t sa, uint32_t sb)
{
#pragma unroll 1
    for (int q = 0; q < 8; q++)
        c = mfma_mx<FA, FB, J>(Pick(q).of(a), Pick(q).of(b), c, sa, sb);
    return c;
}

}  // namespace mxk
