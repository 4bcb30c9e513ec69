// norm.hip -- the root-mean-square norm of a residual stream with its row-wise
// outputs, and its gradients (gfx950).
//
//   h = bf16(x + residual), rstd = (mean h^2 + eps)^(-1/2), y = bf16((h w) rstd)
//   dh = dres + rstd (g - xhat c), xhat = h rstd, g = dy w, c = mean(g xhat)
//   dw = sum over rows of dy xhat
//
// Both are bound by memory: a handful of fp32 operations per element against 4 to
// 10 bytes.  A workgroup holds one row in registers (16-byte loads, neighbouring
// chunks in neighbouring lanes), so that every input is read once: the sum over the
// row (in 64 bits: fp32 sums would move y by a step of bf16 in one element of 10^5, and
// cost the same), one barrier, then the outputs.  The loads of the workgroup's next row are
// issued before that sum.  The row-wise MXFP8 blocks (32 elements, 4 lanes) leave in
// the same pass; the column-wise casts need all rows' rstd first and re-read h
// (mx_cast_norm.hip).  The backward's weight gradients are summed in registers over
// the rows that a workgroup's threads take and leave as one row of partial sums per
// workgroup, which a second kernel adds in a fixed order.
//
// Measured (a copy of 1 GiB runs at 5.1 TB/s, one of 118 MB at 5.5 to 7): 16384 x 7168
// with a residual, the row-wise cast and the 8-bit copy 171 us (0.95 GB, 5.6 TB/s),
// 2048 x 8192 with a residual and the row-wise cast 23.5 us (118 MB, 5.0 TB/s), one row
// of 4096 3.5 us.  Backward of 16384 x 7168 with dres from bf16 153 us (0.94 GB, 6.1
// TB/s), from 8 bits 143 us (0.83 GB, 5.8 TB/s), the sums of its partial weight
// gradients 4.5 us more.
#include "bufio.h"
#include "device_math.h"
#include "launch_norm.h"
#include "mx_cast.h"
#include "rows.h"
#include "wave.h"

namespace mxk {

constexpr uint32_t kOnes = 0x3F803F80u;   // two bf16 ones

// The row that workgroup b of n takes in its step-th turn.  With whole groups of
// 256 workgroups, those of one XCD (b mod 8) take 32 rows in a line: their scale
// bytes share the lines of the tile layout.
__device__ __forceinline__ int64_t row_of(int64_t step, int b, int n)
{
    const int at = (n & 255) == 0 ? (b & ~255) + ((b & 7) << 5) + ((b >> 3) & 31) : b;
    return step * n + at;
}

// Sum over `waves` waves of the workgroup, from wave `first` on, the same in each of
// their threads; red: a number for each wave of the workgroup, others for the next
// call.
template <class T>
__device__ __forceinline__ T block_sum(T v, T *red, int waves, int first = 0)
{
    v = wave_sum(v);
    if (waves == 1)
        return v;
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    const int i = (int)threadIdx.x & 15;       // all at once, in each row of 16 lanes
    return row_sum(i < waves ? red[first + i] : T(0));
}

// (sum / K + eps)^(-1/2) in 64 bits, where every element of the row has this factor: the
// hardware's estimate, measured good to 2^-24, and one Newton step, which leaves 2^-47
// (inv_k = 1 / K: a division would be one more of the steps that all waves wait for).
// near, the nearest fp32 number, is for the caller; r and low, as the output's functions
// take them, for y (low is not negative, so that a zero's sign stays).  0 and Inf go
// through fp32, where the step would make NaN of them, and what passes fp32 is Inf.
struct Rstd {
    float near, r, low;
    int wide;                      // as norm_is_wide(r), in a scalar register
};
__device__ __forceinline__ Rstd rstd_of(double sum, double inv_k, float eps)
{
    const double v = __builtin_fma(sum, inv_k, (double)eps);
    const double r = __builtin_amdgcn_rsq(v);
    const double s = __builtin_fma(0.5 * r, __builtin_fma(-v * r, r, 1.0), r);
    Rstd o;
    // (by s's first 32 bits: 2^-64 to 2^10; NaN's and Inf's are larger)
    const uint32_t first = (uint32_t)((uint64_t)__double_as_longlong(s) >> 32);
    o.wide = (uint32_t)__builtin_amdgcn_readfirstlane((int)first) - 0x3BF00000u >= 0x40900000u - 0x3BF00000u;
    o.near = o.r = (float)s;
    o.r = (double)o.r > s ? f32_bits(bits_f32(o.r) - 1u) : o.r;
    o.low = (float)(s - (double)o.r);
    if (__builtin_expect(o.wide != 0, 0)) {
        const double t = s < 0x1p-64 ? s * 0x1p64 : s;
        o.r = (float)t;
        o.r = (double)o.r > t ? f32_bits(bits_f32(o.r) - 1u) : o.r;
        o.low = (float)(t - (double)o.r);
        if (!(v > 0.0 && v < 1e300 && s <= 0x1.fffffep127)) {
            o.near = o.r = 1.0f / sqrtf((float)v);
            o.low = 0.0f;
        }
        o.r = f32_bits(bits_f32(o.r) | 0x80000000u);
    }
    return o;
}

__device__ __forceinline__ uint32_t add_pair(uint32_t a, uint32_t b)
{
    return bf16x2_rne(bf16_lo(a) + bf16_lo(b), bf16_hi(a) + bf16_hi(b));
}

// Largest magnitude of a lane's 8 elements and those of the 3 other lanes of
// its 32-element block.
__device__ __forceinline__ uint32_t block_mag(const uint32_t (&m)[4])
{
    const uint32_t t = pk_max_u16(pk_max_u16(m[0], m[1]), pk_max_u16(m[2], m[3]));
    const uint32_t lo = t & 0xFFFFu, hi = t >> 16;
    return max_xor2(max_xor1(lo > hi ? lo : hi));
}

// MXFP8 of a lane's 8 elements, chunk c of a row: codes to q, the scale byte
// returned.
template <int FMT, int AUX, bool AL>
__device__ __forceinline__ uint32_t cast8(const Row<AL, uint8_t> &q, const uint32_t (&w)[4], uint32_t c)
{
    uint32_t m[4];
#pragma unroll
    for (int d = 0; d < 4; d++)
        m[d] = w[d] & 0x7FFF7FFFu;
    const uint32_t sb = scale_byte<FMT>(block_mag(m));
    uint2 o = encode8_row<FMT>(w, m, sb);
    if (sb == 0xFFu)
        o.x = o.y = 0x7F7F7F7Fu;
    row_store<AUX>(q, c, o);
    return sb;
}

// The scale bytes of 16 lanes (4 blocks, block j in the byte j of every lane's
// word).
__device__ __forceinline__ uint32_t four_scales(uint32_t sb)
{
    uint32_t v = sb << (8 * ((threadIdx.x >> 2) & 3));
    v |= dpp<kDppHalfMirror>(0u, v);
    v |= dpp<kDppMirror>(0u, v);
    return v;
}

// Compact scales of chunk c's blocks: s the descriptor of the row's nb bytes,
// quad whether they start at a multiple of 4.
__device__ __forceinline__ void store_scales(rsrc_t s, uint32_t sb, uint32_t c, uint32_t nb, bool quad)
{
    const uint32_t b = c >> 2;
    if (quad) {
        const uint32_t v = four_scales(sb);
        buf_store4(s, (c & 15) == 0 && b < nb ? b : kDead, v);
    } else {
        buf_store1(s, (c & 3) == 0 && b < nb ? b : kDead, (uint8_t)sb);
    }
}

// The same in the tile layout, s the first tile of row r's row tile and a row's
// block tiles 256 RT bytes apart (64-bit addresses: all of them may pass 2^31
// bytes); blocks b, b + 2 of 4 go to one word's neighbouring bytes.
__device__ __forceinline__ void store_scales_tiled(uint8_t *s, uint32_t sb, uint32_t c, uint32_t r,
                                                   uint32_t RT, uint32_t CT)
{
    const uint32_t v = four_scales(sb), b = c >> 2, odd = b & 1;
    const uint32_t two = odd ? __builtin_amdgcn_perm(0u, v, 0x0C0C0301u)
                             : __builtin_amdgcn_perm(0u, v, 0x0C0C0200u);
    if ((c & 3) == 0 && (b & 2) == 0 && (b >> 3) < CT)
        *reinterpret_cast<uint16_t *>(s + (int64_t)(b >> 3) * RT * 256 + 4 * (32 * odd + (r & 31)) +
                                      ((b & 7) >> 1)) = (uint16_t)two;
}

// Where a row's outputs go: none of them past the last row.
template <bool AL>
struct NormOut {
    Row<AL, uint16_t> h, y;
    Row<AL, uint8_t> q, k;          // codes of y, of h
    rsrc_t s, ks;                   // their compact scales
};

template <bool AL>
__device__ __forceinline__ NormOut<AL> norm_out(const NormArgs &a, int64_t row, uint32_t nb)
{
    const bool live = row < a.M;
    const int64_t at = row * a.K, len = live ? a.K : 0, sat = live ? row * nb : 0;
    NormOut<AL> o;
    o.h = row_at<AL>(a.h, at, a.h ? len : 0);
    o.y = row_at<AL>(a.y, at, a.y ? len : 0);
    o.q = row_at<AL>(a.q_row, at, a.q_row ? len : 0);
    o.k = row_at<AL>(a.q_h, at, a.q_h ? len : 0);
    o.s = make_rsrc(a.s_row + sat, 0, a.s_row && live && !a.tiled ? nb : 0);
    o.ks = make_rsrc(a.s_h + sat, 0, a.s_h && live ? nb : 0);
    return o;
}

// The outputs of chunk c of a row; every lane of a wave takes part.  wide: by 64 bits,
// the same for all of them.
template <int FMT, int NT, bool AL>
__device__ __forceinline__ void norm_write(const NormArgs &a, const NormOut<AL> &o, int64_t row, uint32_t c,
                                           uint32_t nb, const uint32_t (&h)[4], const Rstd &rstd, uint4 wt,
                                           int wide)
{
    const bool quad = (nb & 3) == 0;
    if (a.q_h)
        store_scales(o.ks, cast8<kFmtRoundUp, NT>(o.k, h, c), c, nb, quad);
    if (!a.y && !a.q_row)
        return;
    uint32_t y[4];
    const uint32_t w[4] = {wt.x, wt.y, wt.z, wt.w};
    if (__builtin_expect(wide == 0, 1)) {
#pragma unroll
        for (int d = 0; d < 4; d++)
            y[d] = norm_pair(h[d], rstd.r, rstd.low, w[d]);
    } else {
        const double f = norm_factor(rstd.r, rstd.low);
#pragma unroll
        for (int d = 0; d < 4; d++) {
            y[d] = norm_pair_wide(h[d], f, w[d]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (a.y)
        row_store<0>(o.y, c, make_uint4(y[0], y[1], y[2], y[3]));
    if (!a.q_row)
        return;
    const uint32_t sb = cast8<FMT, NT>(o.q, y, c);
    const uint32_t RT = (uint32_t)((a.M + 31) >> 5);
    if (a.tiled)   // padding is 0, though the zeros there times an Inf or NaN rstd are NaN
        store_scales_tiled(a.s_row + (row >> 5) * 256, row < a.M && (c >> 2) < nb ? sb : 0u, c, (uint32_t)row,
                           RT, (nb + 7) >> 3);
    else
        store_scales(o.s, sb, c, nb, quad);
}

__device__ __forceinline__ void norm_sum(const uint32_t (&x)[4], const uint4 *r, uint32_t (&h)[4], double &s0,
                                         double &s1)
{
    const uint32_t rr[4] = {r ? r->x : 0u, r ? r->y : 0u, r ? r->z : 0u, r ? r->w : 0u};
#pragma unroll
    for (int d = 0; d < 4; d++) {
        h[d] = r ? add_pair(x[d], rr[d]) : x[d];
        const double lo = bf16_lo(h[d]), hi = bf16_hi(h[d]);
        s0 = __builtin_fma(lo, lo, s0);
        s1 = __builtin_fma(hi, hi, s1);
    }
}

template <int CH>
struct NormRow {
    uint4 x[CH], r[CH];
};

// A row outside the tensor reads as zeros, without traffic.
template <int CH, int AUX, bool AL>
__device__ __forceinline__ void norm_load(const NormArgs &a, int64_t row, NormRow<CH> &v)
{
    const int64_t at = row * a.K, len = row < a.M ? a.K : 0;
    const Row<AL, const uint16_t> x = row_at<AL>(a.x, at, len), r = row_at<AL>(a.res, at, a.res ? len : 0);
#pragma unroll
    for (int i = 0; i < CH; i++) {
        v.x[i] = row_raw<AUX>(x, threadIdx.x + i * blockDim.x);
        if (a.res)
            v.r[i] = row_raw<AUX>(r, threadIdx.x + i * blockDim.x);
    }
}

// For the caller, and for the column-wise cast.
__device__ __forceinline__ void put_rstd(const NormArgs &a, int64_t row, const Rstd &rstd)
{
    a.rstd[row] = rstd.near;
    if (a.cut) {
        a.cut[row] = rstd.r;
        a.low[row] = rstd.low;
    }
}

// Rows that the tile layout pads to have scales of 0.
__device__ __forceinline__ int64_t norm_rows(const NormArgs &a)
{
    return a.tiled && a.s_row ? (a.M + 31) & ~(int64_t)31 : a.M;
}

// NT: the policy of what is read and written once (kNT or 0); AL: K is a multiple of
// 8 (other rows start at any byte: 16384 x 7001 with a residual, the row-wise cast and
// the 8-bit copy 232 us, 4.0 TB/s).
template <int FMT, int CH, int NT, bool AL>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a)
{
    __shared__ double red[2][16];
    const int waves = (int)blockDim.x >> 6, n = (int)gridDim.x;
    const uint32_t nb = (uint32_t)((a.K + 31) >> 5);
    const int64_t rows = norm_rows(a);
    const double inv_k = 1.0 / (double)a.K;
    const Row<AL, const uint16_t> w = row_at<AL>(a.w, 0, a.w ? a.K : 0);
    uint4 wt[CH];
#pragma unroll
    for (int i = 0; i < CH; i++)
        wt[i] = a.w ? row_load<0>(w, threadIdx.x + i * blockDim.x) : make_uint4(kOnes, kOnes, kOnes, kOnes);

    NormRow<CH> next;
    int64_t row = row_of(0, (int)blockIdx.x, n);
    norm_load<CH, NT, AL>(a, row, next);
    // (behind the first row's loads, which are on their way meanwhile)
    bool l = false;
#pragma unroll
    for (int i = 0; i < CH; i++)
        l |= norm_is_wide(wt[i]);
    const int large = __builtin_amdgcn_readfirstlane((int)(__builtin_amdgcn_ballot_w64(l) != 0));
    for (int64_t step = 0; row < rows; step++) {
        uint32_t h[CH][4];
        double s0 = 0.0, s1 = 0.0;
#pragma unroll
        for (int i = 0; i < CH; i++) {
            const uint32_t c = threadIdx.x + i * blockDim.x;
            const uint4 u = row_fix<AL>(next.x[i], c, (uint32_t)a.K);
            const uint32_t x[4] = {u.x, u.y, u.z, u.w};
            const uint4 r = row_fix<AL>(next.r[i], c, (uint32_t)a.K);
            norm_sum(x, a.res ? &r : nullptr, h[i], s0, s1);
        }
        const int64_t after = row_of(step + 1, (int)blockIdx.x, n);
        norm_load<CH, NT, AL>(a, after, next);
        __builtin_amdgcn_sched_barrier(0);
        // the weights stay packed: as fp32 they would take 16 registers more, and a wave a
        // SIMD less (16384 x 7168 row-wise 162 us instead of 156)
        if constexpr (CH > 1)
#pragma unroll
            for (int i = 0; i < CH; i++)
                asm("" : "+v"(wt[i].x), "+v"(wt[i].y), "+v"(wt[i].z), "+v"(wt[i].w));
        const Rstd rstd = rstd_of(block_sum(s0 + s1, red[step & 1], waves), inv_k, a.eps);
        if (row < a.M && threadIdx.x == 0)
            put_rstd(a, row, rstd);
        const NormOut<AL> o = norm_out<AL>(a, row, nb);
        const int wide = large | rstd.wide;
#pragma unroll
        for (int i = 0; i < CH; i++) {
            const uint32_t c = threadIdx.x + i * blockDim.x;
            if (a.h)
                row_store<0>(o.h, c, make_uint4(h[i][0], h[i][1], h[i][2], h[i][3]));
            norm_write<FMT, NT, AL>(a, o, row, c, nb, h[i], rstd, wt[i], wide);
        }
        row = after;
    }
}

// Rows of any length, in two passes: the second finds the row in the caches (and
// each thread what it wrote itself).  4096 x 20480 with a residual and the row-wise
// cast 144 us (0.59 GB, 4.1 TB/s; its h read again from the caches), x 20481 164 us.
template <int FMT, bool AL>
__global__ __launch_bounds__(512) void norm_long_kernel(NormArgs a)
{
    __shared__ double red[2][16];
    const uint32_t nb = (uint32_t)((a.K + 31) >> 5), chunks = (uint32_t)((a.K + 7) >> 3), K = (uint32_t)a.K;
    // whole waves, which cover the tile layout's padding blocks too
    const uint32_t upto = (chunks + 63) & ~63u;
    const int64_t rows = norm_rows(a);
    const double inv_k = 1.0 / (double)a.K;
    const Row<AL, const uint16_t> w = row_at<AL>(a.w, 0, a.w ? a.K : 0);
    int step = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, step ^= 1) {
        const int64_t at = row * a.K, len = row < a.M ? a.K : 0;
        const Row<AL, const uint16_t> x = row_at<AL>(a.x, at, len), r = row_at<AL>(a.res, at, a.res ? len : 0);
        const NormOut<AL> o = norm_out<AL>(a, row, nb);
        double s0 = 0.0, s1 = 0.0;
        for (uint32_t c0 = threadIdx.x; c0 < chunks; c0 += 2 * 512) {
            uint4 xv[2], rv[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                xv[i] = row_raw<0>(x, c0 + 512 * i);
                if (a.res)
                    rv[i] = row_raw<0>(r, c0 + 512 * i);
            }
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const uint32_t c = c0 + 512 * i;
                const uint4 v = row_fix<AL>(xv[i], c, K), q = row_fix<AL>(rv[i], c, K);
                const uint32_t xw[4] = {v.x, v.y, v.z, v.w};
                uint32_t h[4];
                norm_sum(xw, a.res ? &q : nullptr, h, s0, s1);
                if (a.h)
                    row_store<0>(o.h, c, make_uint4(h[0], h[1], h[2], h[3]));
            }
        }
        const Rstd rstd = rstd_of(block_sum(s0 + s1, red[step], 8), inv_k, a.eps);
        if (row < a.M && threadIdx.x == 0)
            put_rstd(a, row, rstd);
        const Row<AL, const uint16_t> hr = a.h ? row_at<AL>((const uint16_t *)a.h, at, len) : x;
        for (uint32_t c = threadIdx.x; c < upto; c += 512) {
            uint4 wt = make_uint4(kOnes, kOnes, kOnes, kOnes), v = row_raw<0>(hr, c);
            if (a.w)
                wt = row_raw<0>(w, c);
            v = row_fix<AL>(v, c, K);
            wt = a.w ? row_fix<AL>(wt, c, K) : wt;
            const uint32_t h[4] = {v.x, v.y, v.z, v.w};
            const int wide =
                rstd.wide | __builtin_amdgcn_readfirstlane((int)(__builtin_amdgcn_ballot_w64(norm_is_wide(wt)) != 0));
            norm_write<FMT, 0, AL>(a, o, row, c, nb, h, rstd, wt, wide);
        }
    }
}

template <int FMT>
static hipError_t launch_norm_fmt(const NormArgs &a, hipStream_t s)
{
    const NormShape n = norm_shape(a.K);
    const int64_t rows = a.tiled && a.s_row ? (a.M + 31) / 32 * 32 : a.M;
    // 1024 threads a CU, whose next rows are on their way meanwhile (2048 x 8192 row-wise:
    // 23.7 us, with twice as many that take two rows each 24.7, with half 29.4; 4096 x 8192
    // 41.5, 42.7, 54.4).  From 16384 rows on that are too large for the caches workgroups
    // of two rows, handed out as others end, are faster (whole calls; a trace charges a
    // kernel for the stores of the one before it as well): 16384 x 7168 row-wise 166 -> 158
    // us, with the 8-bit copy 187 -> 171, with both casts too 255 -> 241, 16384 x 8192 to
    // bf16 202 -> 180, 131072 x 1024 row-wise 189 -> 161, 32768 x 2048 78 -> 72, 16384 x 4096
    // 77 -> 74.  Below, it depends on the row: 8192 x 7168 73 -> 78, 8192 x 8192 77 -> 81,
    // 10240 x 8192 to bf16 122 -> 127, but 12288 x 7168 123 -> 117, to bf16 136 -> 123; and
    // one workgroup a CU (16400 x 16384) 341 -> 370, rows at any byte 200 -> 219.
    const bool many = a.stream && rows >= 16384 && a.K % 8 == 0 && n.chunks != 0 && n.threads <= 512;
    const int64_t pairs = (rows + 511) / 512 * 256;
    const int64_t most = n.chunks == 0 ? 1024 : !many ? 256 * (1024 / n.threads) : pairs < 65536 ? pairs : 65536;
    const dim3 grid((unsigned)(rows < most ? rows : most)), block(n.threads);
    if (n.chunks == 0)
        hipLaunchKernelGGL((a.K % 8 == 0 ? norm_long_kernel<FMT, true> : norm_long_kernel<FMT, false>), grid, block,
                           0, s, a);
    else if (a.K % 8 != 0)
        hipLaunchKernelGGL((a.stream ? norm_kernel<FMT, 2, kNT, false> : norm_kernel<FMT, 2, 0, false>), grid,
                           block, 0, s, a);
    else if (n.chunks == 1)
        hipLaunchKernelGGL((a.stream ? norm_kernel<FMT, 1, kNT, true> : norm_kernel<FMT, 1, 0, true>), grid,
                           block, 0, s, a);
    else
        hipLaunchKernelGGL((a.stream ? norm_kernel<FMT, 2, kNT, true> : norm_kernel<FMT, 2, 0, true>), grid,
                           block, 0, s, a);
    return hipGetLastError();
}

hipError_t launch_norm(unsigned fmt, const NormArgs &a, hipStream_t s)
{
    switch (fmt) {
    case 0u: return launch_norm_fmt<0>(a, s);
    case kFmtE5M2: return launch_norm_fmt<kFmtE5M2>(a, s);
    case kFmtRoundUp: return launch_norm_fmt<kFmtRoundUp>(a, s);
    case kFmtE5M2 | kFmtRoundUp: return launch_norm_fmt<kFmtE5M2 | kFmtRoundUp>(a, s);
    default: return hipErrorInvalidValue;
    }
}

// ---- backward -----------------------------------------------------------------

typedef float f32x2_t __attribute__((ext_vector_type(2)));

// Four E4M3 codes times their block's scale: exact (4 significant bits).  sc
// carries the E8M0 byte in its exponent field; byte 0xFF goes with NaN codes.
__device__ __forceinline__ void e4m3x4_values(uint32_t q, float sc, float (&v)[4])
{
    const f32x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, sc, false);
    const f32x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, sc, true);
    v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
}

template <int CH, bool CK>
struct BackRow {
    uint4 dy[CH], dres[CH];
    uint4 h[CK ? 1 : CH];
    uint2 q[CK ? CH : 1];
    uint32_t s[CK ? CH : 1];
    float rstd;
};

// Row `row` of a group of n threads, of which this is the tid-th.
template <int CH, bool CK, int AUX, bool AL>
__device__ __forceinline__ void back_load(const NormBackArgs &a, int64_t row, uint32_t tid, uint32_t n,
                                          BackRow<CH, CK> &v)
{
    const bool live = row < a.M;
    const int64_t at = row * a.K, len = live ? a.K : 0, nb = (a.K + 31) >> 5;
    const Row<AL, const uint16_t> dy = row_at<AL>(a.dy, at, len), dres = row_at<AL>(a.dres, at, a.dres ? len : 0);
    const Row<AL, const uint16_t> h = row_at<AL>(a.h, at, CK ? 0 : len);
    const Row<AL, const uint8_t> q = row_at<AL>(a.q_h, at, CK ? len : 0);
    const rsrc_t s = make_rsrc(a.s_h + (CK && live ? row * nb : 0), 0, CK && live ? nb : 0);
    v.rstd = live ? a.rstd[row] : 0.0f;
#pragma unroll
    for (int i = 0; i < CH; i++) {
        const uint32_t c = tid + i * n;
        v.dy[i] = row_raw<AUX>(dy, c);
        if constexpr (CK) {
            v.q[i] = row_raw<AUX>(q, c);
            v.s[i] = buf_load1(s, c >> 2);
        } else {
            v.h[i] = row_raw<AUX>(h, c);
        }
        if (a.dres)
            v.dres[i] = row_raw<AUX>(dres, c);
    }
}

// The 8 values of h of a chunk: bf16 words, or codes with their block's scale byte.
__device__ __forceinline__ void h_values(uint4 h, float (&v)[8])
{
    const uint32_t w[4] = {h.x, h.y, h.z, h.w};
#pragma unroll
    for (int d = 0; d < 4; d++) {
        v[2 * d] = bf16_lo(w[d]);
        v[2 * d + 1] = bf16_hi(w[d]);
    }
}
__device__ __forceinline__ void h_values(uint2 q, uint32_t s, float (&v)[8])
{
    float lo[4], hi[4];
    e4m3x4_values(q.x, e8m0_operand(s), lo);
    e4m3x4_values(q.y, e8m0_operand(s), hi);
#pragma unroll
    for (int d = 0; d < 4; d++) {
        v[d] = lo[d];
        v[4 + d] = hi[d];
    }
}

// Groups of n threads, a whole number of waves each, take a row each; ROWS is
// whether there may be more than one.  NT: what is read once is read non-temporally,
// and dh written through the caches (SC1), for tensors that do not fit them; from
// the 8-bit copy dh's default policy is faster (16384 x 7168: 143 us and 150, from
// bf16 158 and 149).  T: the most threads of a workgroup (1024 leave 128 registers a
// lane, of which the 8-bit copy's variant spills 4).
template <int CH, bool CK, bool NT, bool AL, bool ROWS, int T>
__global__ __launch_bounds__(T) void norm_back_kernel(NormBackArgs a, int rows)
{
    constexpr int IN = NT ? kNT : 0, OUT = NT && !CK ? kSC1 : 0;
    __shared__ float red[2][16];
    __shared__ __align__(16) float4 parts[ROWS ? 2 * CH * T / 2 : 1];
    const uint32_t n = ROWS ? blockDim.x / rows : blockDim.x;
    const uint32_t group = ROWS ? (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x / n)) : 0u;
    const uint32_t tid = threadIdx.x - group * n;
    const int waves = (int)n >> 6;
    const int64_t step_rows = (int64_t)gridDim.x * rows;
    uint32_t wt[CH][4];
    float dw[CH][8];
#pragma unroll
    for (int i = 0; i < CH; i++) {
        uint4 w = make_uint4(kOnes, kOnes, kOnes, kOnes);
        if (a.w)
            w = row_load<0>(row_at<AL>(a.w, 0, a.K), tid + i * n);
        wt[i][0] = w.x; wt[i][1] = w.y; wt[i][2] = w.z; wt[i][3] = w.w;
#pragma unroll
        for (int d = 0; d < 8; d++)
            dw[i][d] = 0.0f;
    }
    // one turn: a row whose loads are done; all groups of the workgroup take as many
    // (they share barriers)
    const auto turn = [&](const BackRow<CH, CK> &v, int64_t row, int step) {
        float g[CH][8], xh[CH][8], s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; i++) {
            const uint4 u = row_fix<AL>(v.dy[i], tid + i * n, (uint32_t)a.K);
            const uint32_t dy[4] = {u.x, u.y, u.z, u.w};
            float hv[8];
            if constexpr (CK)
                h_values(row_fix<AL>(v.q[i], tid + i * n, (uint32_t)a.K), v.s[i], hv);
            else
                h_values(row_fix<AL>(v.h[i], tid + i * n, (uint32_t)a.K), hv);
#pragma unroll
            for (int d = 0; d < 4; d++) {
                const float y0 = bf16_lo(dy[d]), y1 = bf16_hi(dy[d]);
                xh[i][2 * d] = hv[2 * d] * v.rstd;
                xh[i][2 * d + 1] = hv[2 * d + 1] * v.rstd;
                g[i][2 * d] = y0 * bf16_lo(wt[i][d]);
                g[i][2 * d + 1] = y1 * bf16_hi(wt[i][d]);
                s0 = __builtin_fmaf(g[i][2 * d], xh[i][2 * d], s0);
                s1 = __builtin_fmaf(g[i][2 * d + 1], xh[i][2 * d + 1], s1);
                dw[i][2 * d] = __builtin_fmaf(y0, xh[i][2 * d], dw[i][2 * d]);
                dw[i][2 * d + 1] = __builtin_fmaf(y1, xh[i][2 * d + 1], dw[i][2 * d + 1]);
            }
        }
        const float c = block_sum(s0 + s1, red[step], waves, (int)group * waves) / (float)a.K;
        const Row<AL, uint16_t> ro = row_at<AL>(a.dh, row * a.K, row < a.M ? a.K : 0);
#pragma unroll
        for (int i = 0; i < CH; i++) {
            const uint4 u = row_fix<AL>(v.dres[i], tid + i * n, (uint32_t)a.K);
            const uint32_t dr[4] = {u.x, u.y, u.z, u.w};
            uint32_t o[4];
#pragma unroll
            for (int d = 0; d < 4; d++) {
                float e0 = v.rstd * __builtin_fmaf(-xh[i][2 * d], c, g[i][2 * d]);
                float e1 = v.rstd * __builtin_fmaf(-xh[i][2 * d + 1], c, g[i][2 * d + 1]);
                if (a.dres) {
                    e0 += bf16_lo(dr[d]);
                    e1 += bf16_hi(dr[d]);
                }
                o[d] = bf16x2_rne(e0, e1);
            }
            row_store<OUT>(ro, tid + i * n, make_uint4(o[0], o[1], o[2], o[3]));
        }
    };
    const int64_t all = a.M + (int64_t)group;   // rows `row` < all: the workgroup's turns
    int64_t row = (int64_t)blockIdx.x * rows + group;
    if constexpr (T <= 512 && AL) {
        // three sets of registers in turn: two rows are under way while one is worked
        // on
        BackRow<CH, CK> v0, v1, v2;
        back_load<CH, CK, IN, AL>(a, row, tid, n, v0);
        back_load<CH, CK, IN, AL>(a, row + step_rows, tid, n, v1);
        for (int step = 0; row < all;) {
            back_load<CH, CK, IN, AL>(a, row + 2 * step_rows, tid, n, v2);
            __builtin_amdgcn_sched_barrier(0);
            turn(v0, row, step);
            row += step_rows, step ^= 1;
            if (row >= all)
                break;
            back_load<CH, CK, IN, AL>(a, row + 2 * step_rows, tid, n, v0);
            __builtin_amdgcn_sched_barrier(0);
            turn(v1, row, step);
            row += step_rows, step ^= 1;
            if (row >= all)
                break;
            back_load<CH, CK, IN, AL>(a, row + 2 * step_rows, tid, n, v1);
            __builtin_amdgcn_sched_barrier(0);
            turn(v2, row, step);
            row += step_rows, step ^= 1;
        }
    } else {
        BackRow<CH, CK> next;
        back_load<CH, CK, IN, AL>(a, row, tid, n, next);
        for (int step = 0; row < all; row += step_rows, step ^= 1) {
            const BackRow<CH, CK> v = next;
            back_load<CH, CK, IN, AL>(a, row + step_rows, tid, n, next);
            __builtin_amdgcn_sched_barrier(0);
            turn(v, row, step);
        }
    }
    if (!a.partials)
        return;
    if constexpr (ROWS) {
        // the groups' sums, halves to halves: group g adds that of g + half
        for (int left = rows; left > 1;) {
            const int half = (left + 1) / 2;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2 * CH; i++)
                if ((int)group >= half && (int)group < left)
                    parts[(i * (rows / 2) + group - half) * n + tid] =
                        make_float4(dw[i / 2][4 * (i & 1)], dw[i / 2][4 * (i & 1) + 1],
                                    dw[i / 2][4 * (i & 1) + 2], dw[i / 2][4 * (i & 1) + 3]);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 2 * CH; i++)
                if ((int)group < left - half) {
                    const float4 p = parts[(i * (rows / 2) + group) * n + tid];
                    dw[i / 2][4 * (i & 1)] += p.x;
                    dw[i / 2][4 * (i & 1) + 1] += p.y;
                    dw[i / 2][4 * (i & 1) + 2] += p.z;
                    dw[i / 2][4 * (i & 1) + 3] += p.w;
                }
            left = half;
        }
        if (group != 0)
            return;
    }
    const rsrc_t rp = make_rsrc(a.partials + (int64_t)blockIdx.x * a.K, 0, 4 * a.K);
#pragma unroll
    for (int i = 0; i < CH; i++) {
        const uint32_t off = 32 * (tid + i * n);
        if constexpr (!AL) {
#pragma unroll
            for (int d = 0; d < 8; d++)
                buf_store4(rp, off + 4 * d, bits_f32(dw[i][d]));
            continue;
        }
#pragma unroll
        for (int q = 0; q < 2; q++)
            buf_store16(rp, off + 16 * q,
                        make_uint4(bits_f32(dw[i][4 * q]), bits_f32(dw[i][4 * q + 1]),
                                   bits_f32(dw[i][4 * q + 2]), bits_f32(dw[i][4 * q + 3])));
    }
}

// Rows of any length, in two passes, and their weight gradients in a third.  Chunk c
// of a row: dy, g = dy w and xhat.
template <bool AL>
struct LongRow {
    Row<AL, const uint16_t> dy, h, dres;
    Row<AL, const uint8_t> q;
    rsrc_t s;
};

template <bool AL>
__device__ __forceinline__ LongRow<AL> long_row(const NormBackArgs &a, int64_t row)
{
    const int64_t at = row * a.K, nb = (a.K + 31) >> 5;
    LongRow<AL> v;
    v.dy = row_at<AL>(a.dy, at, a.K);
    v.h = row_at<AL>(a.h, at, a.h ? a.K : 0);
    v.dres = row_at<AL>(a.dres, at, a.dres ? a.K : 0);
    v.q = row_at<AL>(a.q_h, at, a.h ? 0 : a.K);
    v.s = make_rsrc(a.s_h + (a.h ? 0 : row * nb), 0, a.h ? 0 : nb);
    return v;
}

template <bool AL>
__device__ __forceinline__ void long_chunk(const NormBackArgs &a, const LongRow<AL> &v,
                                           const Row<AL, const uint16_t> &wr, uint32_t c, float rstd,
                                           float (&dy)[8], float (&g)[8], float (&xh)[8])
{
    const uint32_t K = (uint32_t)a.K;
    uint4 w = make_uint4(kOnes, kOnes, kOnes, kOnes), h;
    uint2 q;
    uint32_t sb;
    const uint4 d = row_raw<0>(v.dy, c);
    if (a.h) {
        h = row_raw<0>(v.h, c);
    } else {
        q = row_raw<0>(v.q, c);
        sb = buf_load1(v.s, c >> 2);
    }
    if (a.w)
        w = row_raw<0>(wr, c);
    h_values(row_fix<AL>(d, c, K), dy);
    if (a.h)
        h_values(row_fix<AL>(h, c, K), xh);
    else
        h_values(row_fix<AL>(q, c, K), sb, xh);
    float wv[8];
    h_values(a.w ? row_fix<AL>(w, c, K) : w, wv);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        xh[i] *= rstd;
        g[i] = dy[i] * wv[i];
    }
}

template <bool AL>
__global__ __launch_bounds__(512) void norm_back_long_kernel(NormBackArgs a)
{
    __shared__ float red[2][16];
    const uint32_t chunks = (uint32_t)((a.K + 7) >> 3);
    const Row<AL, const uint16_t> w = row_at<AL>(a.w, 0, a.w ? a.K : 0);
    int step = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, step ^= 1) {
        const float rstd = a.rstd[row];
        const LongRow<AL> v = long_row<AL>(a, row);
        const Row<AL, uint16_t> dh = row_at<AL>(a.dh, row * a.K, a.K);
        float s = 0.0f, dy[8], g[8], xh[8];
#pragma unroll 4
        for (uint32_t c = threadIdx.x; c < chunks; c += 512) {
            long_chunk<AL>(a, v, w, c, rstd, dy, g, xh);
#pragma unroll
            for (int d = 0; d < 8; d++)
                s = __builtin_fmaf(g[d], xh[d], s);
        }
        const float mean = block_sum(s, red[step], 8) / (float)a.K;
        for (uint32_t c = threadIdx.x; c < chunks; c += 512) {
            float r[8] = {};
            uint4 dr;
            if (a.dres)
                dr = row_raw<0>(v.dres, c);
            long_chunk<AL>(a, v, w, c, rstd, dy, g, xh);
            if (a.dres)
                h_values(row_fix<AL>(dr, c, (uint32_t)a.K), r);
            uint32_t o[4];
#pragma unroll
            for (int d = 0; d < 4; d++)
                o[d] = bf16x2_rne(rstd * __builtin_fmaf(-xh[2 * d], mean, g[2 * d]) + r[2 * d],
                                  rstd * __builtin_fmaf(-xh[2 * d + 1], mean, g[2 * d + 1]) + r[2 * d + 1]);
            row_store<0>(dh, c, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
}

// Their partial weight gradients: slice blockIdx.y of the rows, a chunk per thread, four
// rows' loads under way (at any byte 168 registers, with a few of them spilled: x 20481
// from bf16 276 us, with the 187 that it would take, two waves a SIMD, 301).  Both and
// their sums, 4096 x 20480 with dres: from bf16 209 us, from 8 bits 191 us (0.67 GB; 1.2 GB
// with what is read twice).
template <bool AL>
__global__ __launch_bounds__(256, AL ? 1 : 3) void norm_dweight_long_kernel(NormBackArgs a)
{
    const uint32_t c = blockIdx.x * 256 + threadIdx.x;
    if (8 * (int64_t)c >= a.K)
        return;
    const Row<AL, const uint16_t> w = row_at<AL>(a.w, 0, a.w ? a.K : 0);
    // in fp32 over 64 rows at a time, those sums in 64 bits: a slice of 2^17 rows in one
    // line would be off by 2^-7 of its terms' magnitudes at worst
    double sum[8] = {};
    for (int64_t row0 = blockIdx.y; row0 < a.M; row0 += 64 * (int64_t)gridDim.y) {
        const int64_t end = row0 + 64 * (int64_t)gridDim.y < a.M ? row0 + 64 * (int64_t)gridDim.y : a.M;
        float run[8] = {};
#pragma unroll 4
        for (int64_t row = row0; row < end; row += gridDim.y) {
            float dy[8], g[8], xh[8];
            long_chunk<AL>(a, long_row<AL>(a, row), w, c, a.rstd[row], dy, g, xh);
#pragma unroll
            for (int d = 0; d < 8; d++)
                run[d] = __builtin_fmaf(dy[d], xh[d], run[d]);
        }
#pragma unroll
        for (int d = 0; d < 8; d++)
            sum[d] += (double)run[d];
    }
#pragma unroll
    for (int d = 0; d < 8; d++)
        if (8 * (int64_t)c + d < a.K)
            a.partials[(int64_t)blockIdx.y * a.K + 8 * (int64_t)c + d] = (float)sum[d];
}

// dweight[k] = sum of partials[p][k]: 32 columns by 32 slices of p a workgroup,
// each slice in order, then the slices in order.
__global__ __launch_bounds__(1024) void norm_dweight_kernel(const float *partials, int parts, int64_t K,
                                                            float *dweight)
{
    __shared__ float red[32][33];
    const int c = threadIdx.x & 31, p0 = threadIdx.x >> 5;
    const int64_t k = (int64_t)blockIdx.x * 32 + c;
    float s = 0.0f;
    if (k < K) {
#pragma unroll 8
        for (int p = p0; p < parts; p += 32)
            s += partials[(int64_t)p * K + k];
    }
    red[p0][c] = s;
    __syncthreads();
    if (p0 == 0 && k < K) {
        for (int p = 1; p < 32; p++)
            s += red[p][c];
        dweight[k] = s;
    }
}

template <int CH, bool AL, bool ROWS, int T>
static void launch_back(const NormBackArgs &a, unsigned grid, int threads, int rows, hipStream_t s)
{
    auto *const kernel = a.h ? (a.stream ? norm_back_kernel<CH, false, true, AL, ROWS, T>
                                         : norm_back_kernel<CH, false, false, AL, ROWS, T>)
                             : (a.stream ? norm_back_kernel<CH, true, true, AL, ROWS, T>
                                         : norm_back_kernel<CH, true, false, AL, ROWS, T>);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads * rows), 0, s, a, rows);
}

hipError_t launch_norm_back(const NormBackArgs &a, hipStream_t s)
{
    const NormShape n = norm_shape(a.K);
    const unsigned parts = (unsigned)norm_back_parts(a.M, a.K);
    const int rows = norm_back_rows(n);
    const bool al = a.K % 8 == 0;
    if (n.chunks == 0) {
        hipLaunchKernelGGL((al ? norm_back_long_kernel<true> : norm_back_long_kernel<false>),
                           dim3((unsigned)(a.M < 1024 ? a.M : 1024)), dim3(512), 0, s, a);
        if (a.partials)
            hipLaunchKernelGGL((al ? norm_dweight_long_kernel<true> : norm_dweight_long_kernel<false>),
                               dim3((unsigned)((a.K + 2047) / 2048), parts), dim3(256), 0, s, a);
    } else if (rows > 1) {
        (!al             ? launch_back<2, false, true, 512>
         : n.chunks == 1 ? launch_back<1, true, true, 512>
                         : launch_back<2, true, true, 512>)(a, parts, n.threads, rows, s);
    } else if (n.threads <= 512) {
        (al ? launch_back<2, true, false, 512> : launch_back<2, false, false, 512>)(a, parts, n.threads, rows, s);
    } else {
        (al ? launch_back<2, true, false, 1024> : launch_back<2, false, false, 1024>)(a, parts, n.threads, rows, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.partials)
        return e;
    hipLaunchKernelGGL(norm_dweight_kernel, dim3((unsigned)((a.K + 31) / 32)), dim3(1024), 0, s,
                       a.partials, (int)parts, a.K, a.dweight);
    return hipGetLastError();
}

}  // namespace mxk
