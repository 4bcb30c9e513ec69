// norm.hip -- the root-mean-square norm of a residual stream with its row-wise
// outputs, and its gradients (gfx950).
//
//   h = bf16(x + residual), rstd = (mean h^2 + eps)^(-1/2), y = bf16((h w) rstd)
//   dh = dres + rstd (g - xhat c), xhat = h rstd, g = dy w, c = mean(g xhat)
//   dw = sum over rows of dy xhat
//
// Both are bound by memory: a handful of fp32 operations per element against 4 to
// 9 bytes.  A workgroup holds one row in registers (16-byte loads, a lane's chunks
// 64 lanes apart), so that every input is read once: the sum over the row, one
// barrier, then the outputs.  The loads of the workgroup's next row are issued
// before that sum.  The row-wise MXFP8 blocks (32 elements, 4 lanes) leave in the
// same pass; the column-wise casts need all rows' rstd first and re-read h
// (mx_cast_norm.hip).  The backward's weight gradients are summed in registers
// over the workgroup's rows and leave as one row of partial sums per workgroup,
// which a second kernel adds in a fixed order.
#include "bufio.h"
#include "device_math.h"
#include "launch_norm.h"
#include "mx_cast.h"
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
// their threads; red: a float for each wave of the workgroup, others for the next
// call.
__device__ __forceinline__ float block_sum(float v, float *red, int waves, int first = 0)
{
    v = wave_sum(v);
    if (waves == 1)
        return v;
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[first];
    for (int i = 1; i < waves; i++)
        s += red[first + i];
    return s;
}

// (sum / K + eps)^(-1/2) in 64 bits, rounded once (in fp32 the mean, the root and
// the reciprocal would each add their rounding, and every element of the row has
// this factor): the hardware's estimate, measured good to 2^-24, and one Newton step,
// which leaves 2^-47.  0 and Inf go through fp32, where the step would make NaN of them.
__device__ __forceinline__ float rstd_of(float sum, int64_t K, float eps)
{
    const double v = (double)sum / (double)K + (double)eps;
    const double r = __builtin_amdgcn_rsq(v);
    const double s = __builtin_fma(0.5 * r, __builtin_fma(-v * r, r, 1.0), r);
    return v > 0.0 && v < 1e300 ? (float)s : 1.0f / sqrtf((float)v);
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

// MXFP8 of a lane's 8 elements of row r, chunk c: codes to q (the row's
// descriptor), the scale byte returned.
template <int FMT, int AUX>
__device__ __forceinline__ uint32_t cast8(rsrc_t q, const uint32_t (&w)[4], uint32_t c)
{
    uint32_t m[4];
#pragma unroll
    for (int d = 0; d < 4; d++)
        m[d] = w[d] & 0x7FFF7FFFu;
    const uint32_t sb = scale_byte<FMT>(block_mag(m));
    uint2 o = encode8_row<FMT>(w, m, sb);
    if (sb == 0xFFu)
        o.x = o.y = 0x7F7F7F7Fu;
    buf_store8<AUX>(q, 8 * c, o);
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

template <int CH>
struct NormRow {
    uint4 x[CH], r[CH];
};

template <int CH, int AUX>
__device__ __forceinline__ void norm_load(const NormArgs &a, int64_t row, NormRow<CH> &v)
{
    // a row outside the tensor reads as zeros, without traffic
    const bool live = row < a.M;
    const rsrc_t rx = make_rsrc(a.x, 0, 0), none = rx;
    const rsrc_t dx = live ? make_rsrc(a.x + row * a.K, 0, 2 * a.K) : none;
    const rsrc_t dr = live && a.res ? make_rsrc(a.res + row * a.K, 0, 2 * a.K) : none;
#pragma unroll
    for (int i = 0; i < CH; i++) {
        const uint32_t off = 16 * (threadIdx.x + i * blockDim.x);
        v.x[i] = buf_load16<AUX>(dx, off);
        if (a.res)
            v.r[i] = buf_load16<AUX>(dr, off);
    }
}

// NT: the policy of what is read and written once (kNT or 0).
template <int FMT, int CH, int NT>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a)
{
    __shared__ float red[2][16];
    const int waves = (int)blockDim.x >> 6, n = (int)gridDim.x;
    const uint32_t nb = (uint32_t)((a.K + 31) >> 5), RT = (uint32_t)((a.M + 31) >> 5), CT = (nb + 7) >> 3;
    const bool tiled = a.tiled && a.s_row, quad = (nb & 3) == 0;
    const int64_t rows = tiled ? 32 * (int64_t)RT : a.M;   // of padding, scales of 0
    uint4 wt[CH];
#pragma unroll
    for (int i = 0; i < CH; i++)
        wt[i] = a.w ? buf_load16(make_rsrc(a.w, 0, 2 * a.K), 16 * (threadIdx.x + i * blockDim.x))
                    : make_uint4(kOnes, kOnes, kOnes, kOnes);

    NormRow<CH> next;
    int64_t row = row_of(0, (int)blockIdx.x, n);
    norm_load<CH, NT>(a, row, next);
    for (int64_t step = 0; row < rows; step++) {
        uint32_t h[CH][4];
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; i++) {
            h[i][0] = next.x[i].x; h[i][1] = next.x[i].y; h[i][2] = next.x[i].z; h[i][3] = next.x[i].w;
            if (a.res) {
                h[i][0] = add_pair(h[i][0], next.r[i].x);
                h[i][1] = add_pair(h[i][1], next.r[i].y);
                h[i][2] = add_pair(h[i][2], next.r[i].z);
                h[i][3] = add_pair(h[i][3], next.r[i].w);
            }
#pragma unroll
            for (int d = 0; d < 4; d++) {
                s0 = __builtin_fmaf(bf16_lo(h[i][d]), bf16_lo(h[i][d]), s0);
                s1 = __builtin_fmaf(bf16_hi(h[i][d]), bf16_hi(h[i][d]), s1);
            }
        }
        const int64_t after = row_of(step + 1, (int)blockIdx.x, n);
        norm_load<CH, NT>(a, after, next);
        __builtin_amdgcn_sched_barrier(0);
        const float rstd = rstd_of(block_sum(s0 + s1, red[step & 1], waves), a.K, a.eps);

        const bool live = row < a.M;
        const int64_t at = live ? row * a.K : 0, len = live ? a.K : 0;
        if (live && threadIdx.x == 0)
            a.rstd[row] = rstd;
        const rsrc_t rh = make_rsrc(a.h + at, 0, a.h ? 2 * len : 0);
        const rsrc_t ry = make_rsrc(a.y + at, 0, a.y ? 2 * len : 0);
        const rsrc_t rq = make_rsrc(a.q_row + at, 0, a.q_row ? len : 0);
        const rsrc_t rk = make_rsrc(a.q_h + at, 0, a.q_h ? len : 0);
        const rsrc_t rks = make_rsrc(a.s_h + (live ? row * nb : 0), 0, a.s_h && live ? nb : 0);
        const rsrc_t rs = make_rsrc(a.s_row + (live ? row * nb : 0), 0, live && !tiled ? nb : 0);
#pragma unroll
        for (int i = 0; i < CH; i++) {
            const uint32_t c = threadIdx.x + i * blockDim.x;
            if (a.h)
                buf_store16(rh, 16 * c, make_uint4(h[i][0], h[i][1], h[i][2], h[i][3]));
            if (a.q_h)
                store_scales(rks, cast8<kFmtRoundUp, NT>(rk, h[i], c), c, nb, quad);
            if (!a.y && !a.q_row)
                continue;
            uint32_t y[4] = {norm_pair(h[i][0], rstd, wt[i].x), norm_pair(h[i][1], rstd, wt[i].y),
                             norm_pair(h[i][2], rstd, wt[i].z), norm_pair(h[i][3], rstd, wt[i].w)};
            if (a.y)
                buf_store16(ry, 16 * c, make_uint4(y[0], y[1], y[2], y[3]));
            if (a.q_row) {
                const uint32_t sb = cast8<FMT, NT>(rq, y, c);
                if (tiled)
                    store_scales_tiled(a.s_row + (row >> 5) * 256, live ? sb : 0u, c, (uint32_t)row, RT,
                                       CT);
                else
                    store_scales(rs, sb, c, nb, quad);
            }
        }
        row = after;
    }
}

// Any row length, rows at any byte: lane by lane over the columns, in two passes
// over the row (the second finds it in the caches).  Columns past K count as 0.
template <int FMT>
__device__ __forceinline__ void any_cast(uint8_t *q, uint32_t y, int64_t k, int64_t K, uint32_t &sb)
{
    uint32_t mag = y & 0x7FFFu;
    mag = max_xor2(max_xor1(mag));
    const uint32_t a = dpp<kDppHalfMirror>(0u, mag);
    mag = mag > a ? mag : a;
    const uint32_t b = dpp<kDppMirror>(0u, mag);
    mag = mag > b ? mag : b;
    const uint32_t c = (uint32_t)__shfl_xor((int)mag, 16, 64);
    mag = mag > c ? mag : c;
    sb = scale_byte<FMT>(mag);
    const uint32_t code = mx_pair<FMT, false>(y, y & 0x7FFFu, sat_limit2<FMT>(sb), e8m0_operand(sb), 0u);
    if (k < K)
        q[k] = (uint8_t)(sb == 0xFFu ? 0x7Fu : code);
}

template <int FMT>
__global__ __launch_bounds__(256) void norm_any_kernel(NormArgs a)
{
    __shared__ float red[2][16];
    const int64_t K = a.K, nb = (K + 31) >> 5, RT = (a.M + 31) >> 5, CT = (nb + 7) >> 3;
    const bool tiled = a.tiled && a.s_row;
    const int64_t rows = tiled ? 32 * RT : a.M;
    int step = 0;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, step ^= 1) {
        const bool live = row < a.M;
        const int64_t at = row * K;
        float s = 0.0f;
        for (int64_t k = threadIdx.x; live && k < K; k += 256) {
            uint32_t v = a.x[at + k];
            if (a.res) {
                v = bf16x2_rne(bf16_lo(v) + bf16_lo(a.res[at + k]), 0.0f) & 0xFFFFu;
                a.h[at + k] = (uint16_t)v;
            }
            s = __builtin_fmaf(bf16_lo(v), bf16_lo(v), s);
        }
        const float rstd = rstd_of(block_sum(s, red[step], 4), K, a.eps);
        if (live && threadIdx.x == 0)
            a.rstd[row] = rstd;
        const uint16_t *src = a.res ? a.h : a.x;
        // whole blocks of 32 lanes, and the tile layout's padding blocks
        const int64_t upto = tiled ? 256 * CT : 32 * nb;
        for (int64_t k = threadIdx.x; k < ((upto + 63) & ~63); k += 256) {
            const bool in = live && k < K;
            const uint32_t h = in ? src[at + k] : 0u, wt = !a.w ? 0x3F80u : in ? a.w[k] : 0u;
            const uint32_t y = in ? norm_pair(h, rstd, wt) & 0xFFFFu : 0u;
            const int64_t b = k >> 5;
            uint32_t sb;
            if (a.y && in)
                a.y[at + k] = (uint16_t)y;
            if (a.q_h) {
                any_cast<kFmtRoundUp>(a.q_h + at, h, k, live ? K : 0, sb);
                if (live && (k & 31) == 0 && b < nb)
                    a.s_h[row * nb + b] = (uint8_t)sb;
            }
            if (!a.q_row)
                continue;
            any_cast<FMT>(a.q_row + at, y, k, live ? K : 0, sb);
            if ((k & 31) != 0)
                continue;
            if (tiled) {
                if (b < 8 * CT)
                    a.s_row[((b >> 3) * RT + (row >> 5)) * 256 + 4 * (32 * (b & 1) + (row & 31)) +
                            ((b & 7) >> 1)] = (uint8_t)sb;
            } else if (live && b < nb) {
                a.s_row[row * nb + b] = (uint8_t)sb;
            }
        }
    }
}

template <int FMT>
static hipError_t launch_norm_fmt(const NormArgs &a, hipStream_t s)
{
    const NormShape n = norm_shape(a.K);
    const int64_t rows = a.tiled && a.s_row ? (a.M + 31) / 32 * 32 : a.M;
    if (n.chunks == 0) {
        const dim3 grid((unsigned)(rows < 2048 ? rows : 2048));
        hipLaunchKernelGGL(norm_any_kernel<FMT>, grid, dim3(256), 0, s, a);
        return hipGetLastError();
    }
    // 1024 threads a CU, whose next rows are on their way meanwhile (2048 x 8192: 21.4
    // us, with twice as many that take two rows each 23.2, with half 26.2)
    const int64_t most = 256 * (1024 / n.threads);
    const dim3 grid((unsigned)(rows < most ? rows : most)), block(n.threads);
    auto *const kernel = n.chunks == 1 ? (a.stream ? norm_kernel<FMT, 1, kNT> : norm_kernel<FMT, 1, 0>)
                                       : (a.stream ? norm_kernel<FMT, 2, kNT> : norm_kernel<FMT, 2, 0>);
    hipLaunchKernelGGL(kernel, grid, block, 0, s, a);
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
template <int CH, bool CK, int AUX>
__device__ __forceinline__ void back_load(const NormBackArgs &a, int64_t row, uint32_t tid, uint32_t n,
                                          BackRow<CH, CK> &v)
{
    const bool live = row < a.M;
    const int64_t at = live ? row * a.K : 0, len = live ? a.K : 0, nb = (a.K + 31) >> 5;
    const rsrc_t rd = make_rsrc(a.dy + at, 0, 2 * len), rr = make_rsrc(a.dres + at, 0, a.dres ? 2 * len : 0);
    const rsrc_t rh = CK ? make_rsrc(a.q_h + at, 0, len) : make_rsrc(a.h + at, 0, 2 * len);
    v.rstd = live ? a.rstd[row] : 0.0f;
#pragma unroll
    for (int i = 0; i < CH; i++) {
        const uint32_t c = tid + i * n;
        v.dy[i] = buf_load16<AUX>(rd, 16 * c);
        if constexpr (CK) {
            v.q[i] = buf_load8<AUX>(rh, 8 * c);
            v.s[i] = buf_load1(make_rsrc(a.s_h + (live ? row * nb : 0), 0, live ? nb : 0), c >> 2);
        } else {
            v.h[i] = buf_load16<AUX>(rh, 16 * c);
        }
        if (a.dres)
            v.dres[i] = buf_load16<AUX>(rr, 16 * c);
    }
}

// Groups of n threads, a whole number of waves each, take a row each; ROWS is
// whether there may be more than one.  NT: what is read once is read non-temporally,
// and dh written through the caches (SC1), for tensors that do not fit them; from
// the 8-bit copy dh's default policy is faster (16384 x 7168: 143 us and 150, from
// bf16 158 and 149).  T: the most threads of a workgroup (1024 leave 128 registers a
// lane, of which the 8-bit copy's variant spills 4).
template <int CH, bool CK, bool NT, bool ROWS, int T>
__global__ __launch_bounds__(T) void norm_back_kernel(NormBackArgs a, int rows)
{
    constexpr int IN = NT ? kNT : 0, OUT = NT && !CK ? kSC1 : 0;
    __shared__ float red[2][16];
    __shared__ __align__(16) float4 parts[ROWS ? 2 * CH * T / 2 : 1];
    const uint32_t n = ROWS ? blockDim.x / rows : blockDim.x;
    const uint32_t group = ROWS ? (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x / n)) : 0u;
    const uint32_t tid = threadIdx.x - group * n;
    const int waves = (int)n >> 6, step_rows = (int)gridDim.x * rows;
    uint32_t wt[CH][4];
    float dw[CH][8];
#pragma unroll
    for (int i = 0; i < CH; i++) {
        uint4 w = make_uint4(kOnes, kOnes, kOnes, kOnes);
        if (a.w)
            w = buf_load16(make_rsrc(a.w, 0, 2 * a.K), 16 * (tid + i * n));
        wt[i][0] = w.x; wt[i][1] = w.y; wt[i][2] = w.z; wt[i][3] = w.w;
#pragma unroll
        for (int d = 0; d < 8; d++)
            dw[i][d] = 0.0f;
    }
    // two rows under way, one where registers are short (2001 x 5120 from the 8-bit
    // copy 22.3 -> 21.5 us, 16384 x 7168 155.4 -> 153.8 us)
    constexpr bool TWO = T <= 512;
    BackRow<CH, CK> next, after;
    int64_t row = (int64_t)blockIdx.x * rows + group;
    back_load<CH, CK, IN>(a, row, tid, n, next);
    if constexpr (TWO)
        back_load<CH, CK, IN>(a, row + step_rows, tid, n, after);
    int step = 0;
    // all groups of the workgroup take as many turns: they share barriers
    for (int64_t row0 = (int64_t)blockIdx.x * rows; row0 < a.M; row0 += step_rows, row += step_rows, step ^= 1) {
        const BackRow<CH, CK> v = next;
        if constexpr (TWO) {
            next = after;
            back_load<CH, CK, IN>(a, row + 2 * (int64_t)step_rows, tid, n, after);
        } else {
            back_load<CH, CK, IN>(a, row + step_rows, tid, n, next);
        }
        __builtin_amdgcn_sched_barrier(0);
        float g[CH][8], xh[CH][8], s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; i++) {
            const uint32_t dy[4] = {v.dy[i].x, v.dy[i].y, v.dy[i].z, v.dy[i].w};
            float hv[8];
            if constexpr (CK) {
                float lo[4], hi[4];
                const float sc = e8m0_operand(v.s[i]);
                e4m3x4_values(v.q[i].x, sc, lo);
                e4m3x4_values(v.q[i].y, sc, hi);
#pragma unroll
                for (int d = 0; d < 4; d++) {
                    hv[d] = lo[d];
                    hv[4 + d] = hi[d];
                }
            } else {
                const uint32_t h[4] = {v.h[i].x, v.h[i].y, v.h[i].z, v.h[i].w};
#pragma unroll
                for (int d = 0; d < 4; d++) {
                    hv[2 * d] = bf16_lo(h[d]);
                    hv[2 * d + 1] = bf16_hi(h[d]);
                }
            }
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
        const bool live = row < a.M;
        const rsrc_t ro = make_rsrc(a.dh + (live ? row * a.K : 0), 0, live ? 2 * a.K : 0);
#pragma unroll
        for (int i = 0; i < CH; i++) {
            const uint32_t dr[4] = {v.dres[i].x, v.dres[i].y, v.dres[i].z, v.dres[i].w};
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
            buf_store16<OUT>(ro, 16 * (tid + i * n), make_uint4(o[0], o[1], o[2], o[3]));
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
#pragma unroll
        for (int q = 0; q < 2; q++)
            buf_store16(rp, off + 16 * q,
                        make_uint4(bits_f32(dw[i][4 * q]), bits_f32(dw[i][4 * q + 1]),
                                   bits_f32(dw[i][4 * q + 2]), bits_f32(dw[i][4 * q + 3])));
    }
}

// h's element of a row (bf16, or the 8-bit copy's value).
__device__ __forceinline__ float any_h(const NormBackArgs &a, int64_t row, int64_t k)
{
    if (a.h)
        return bf16_lo(a.h[row * a.K + k]);
    float v[4];
    e4m3x4_values(a.q_h[row * a.K + k], e8m0_operand(a.s_h[row * ((a.K + 31) >> 5) + (k >> 5)]), v);
    return v[0];
}

__global__ __launch_bounds__(256) void norm_back_any_kernel(NormBackArgs a)
{
    __shared__ float red[2][16];
    int step = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, step ^= 1) {
        const float rstd = a.rstd[row];
        float s = 0.0f;
        for (int64_t k = threadIdx.x; k < a.K; k += 256) {
            const float g = bf16_lo(a.dy[row * a.K + k]) * (a.w ? bf16_lo(a.w[k]) : 1.0f);
            s = __builtin_fmaf(g, any_h(a, row, k) * rstd, s);
        }
        const float c = block_sum(s, red[step], 4) / (float)a.K;
        for (int64_t k = threadIdx.x; k < a.K; k += 256) {
            const float g = bf16_lo(a.dy[row * a.K + k]) * (a.w ? bf16_lo(a.w[k]) : 1.0f);
            float e = rstd * __builtin_fmaf(-(any_h(a, row, k) * rstd), c, g);
            if (a.dres)
                e += bf16_lo(a.dres[row * a.K + k]);
            a.dh[row * a.K + k] = (uint16_t)(bf16x2_rne(e, 0.0f) & 0xFFFFu);
        }
    }
}

// Partial weight gradients of any row length: slice blockIdx.y of the rows,
// one column per thread.
__global__ __launch_bounds__(256) void norm_dweight_any_kernel(NormBackArgs a)
{
    const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (k >= a.K)
        return;
    float s = 0.0f;
    for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y)
        s = __builtin_fmaf(bf16_lo(a.dy[row * a.K + k]), any_h(a, row, k) * a.rstd[row], s);
    a.partials[(int64_t)blockIdx.y * a.K + k] = s;
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

template <int CH, bool ROWS, int T>
static void launch_back(const NormBackArgs &a, unsigned grid, int threads, int rows, hipStream_t s)
{
    auto *const kernel = a.h ? (a.stream ? norm_back_kernel<CH, false, true, ROWS, T>
                                         : norm_back_kernel<CH, false, false, ROWS, T>)
                             : (a.stream ? norm_back_kernel<CH, true, true, ROWS, T>
                                         : norm_back_kernel<CH, true, false, ROWS, T>);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(threads * rows), 0, s, a, rows);
}

hipError_t launch_norm_back(const NormBackArgs &a, hipStream_t s)
{
    const NormShape n = norm_shape(a.K);
    const unsigned parts = (unsigned)norm_back_parts(a.M, a.K);
    const int rows = norm_back_rows(n);
    switch (n.chunks) {
    case 0:
        hipLaunchKernelGGL(norm_back_any_kernel, dim3((unsigned)(a.M < 2048 ? a.M : 2048)), dim3(256), 0,
                           s, a);
        if (a.partials)
            hipLaunchKernelGGL(norm_dweight_any_kernel, dim3((unsigned)((a.K + 255) / 256), parts),
                               dim3(256), 0, s, a);
        break;
    case 1: launch_back<1, true, 512>(a, parts, n.threads, rows, s); break;
    default:
        (rows > 1           ? launch_back<2, true, 512>
         : n.threads <= 512 ? launch_back<2, false, 512>
                            : launch_back<2, false, 1024>)(a, parts, n.threads, rows, s);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.partials)
        return e;
    hipLaunchKernelGGL(norm_dweight_kernel, dim3((unsigned)((a.K + 31) / 32)), dim3(1024), 0, s,
                       a.partials, (int)parts, a.K, a.dweight);
    return hipGetLastError();
}

}  // namespace mxk
