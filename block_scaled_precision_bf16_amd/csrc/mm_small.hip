// mm_small.hip -- small products of MXFP8 operands: few rows, or few outputs.
//
// Here the operands are read about once and there is too little work for the
// tiled kernel, whose workgroups walk along k alone.  A workgroup of KW waves owns
// 32 MT x 32 outputs, and its waves take pieces of 128 k in turn, two under way
// per wave, without barriers.  A wave loads a piece's rows as whole 128-byte lines
// (rows at any byte) and turns them into fragment order through LDS of its own: 16
// bytes of 32 rows per load, straight into the fragments, cost the memory pipeline
// four times the lines (16 x 512 outputs with 8192 k: 17.5 us, with LDS 12.1 us).  The
// KW partial sums are added through LDS in a fixed order.
//
// 8 waves where those workgroups do not fill the CUs more than once (the same product
// 10.2 us, 64 x 8192 outputs 22.7 us for 23.3), else 4 (16 experts' 64 rows by 4096 x
// 2048 each: 25 - 29 us with 105 MB of weights, some of them from the MALL, 3.6 - 4.3
// TB/s; with 8 waves 36 us).
#include "mm_common.h"

namespace mxk {
namespace {

// A wave's share of a piece, 32 rows of 128 k, as it is loaded: lane L holds 16-byte
// chunk L % 8 of rows L / 8, 8 + L / 8, ...; and the four scale bytes of row L % 32.
struct Load {
    uint4 q[4];
    uint32_t s, odd;           // tiled: the words of even and of odd blocks
};

// In fragment order: chunks 2 s + h and 2 s + 2 + h of row r in f[s].
struct Piece {
    i32x8_t f[2];
    uint32_t s;
};

__device__ __forceinline__ uint4 half_of(const i32x8_t &f, int i)
{
    return make_uint4((uint32_t)f[4 * i], (uint32_t)f[4 * i + 1], (uint32_t)f[4 * i + 2], (uint32_t)f[4 * i + 3]);
}

// One operand's rows for a wave's 32-row tile.
struct Rows {
    ByteRows<16> q;
    ByteRows<4> sc;            // compact scales
    const uint8_t *stile;      // tiled ones
    uint32_t qoff[4], soff;
    int64_t K, nb;
    int32_t tiled;
    int64_t rt;                // tiled: bytes from one block tile to the next

    __device__ __forceinline__ Rows(const uint8_t *qarray, const uint8_t *qg, int64_t qleft,
                                    const uint8_t *sarray, const uint8_t *sg, int64_t sleft, int64_t rows,
                                    int64_t r0, int64_t K_, int64_t nb_, int32_t tiled_, int lane)
        : q(qarray, qg + r0 * K_, qleft - r0 * K_), sc(sarray, sg + r0 * nb_, sleft - r0 * nb_),
          stile(sg + (r0 >> 5) * 256), K(K_), nb(nb_), tiled(tiled_), rt(((rows + 31) >> 5) * 256)
    {
        const int last = (int)(rows - 1 - r0 < 31 ? rows - 1 - r0 : 31);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int r = 8 * i + (lane >> 3);
            qoff[i] = q.lead + (uint32_t)((r < last ? r : last) * (int)K) + 16 * (lane & 7);
        }
        const int r = (lane & 31) < last ? lane & 31 : last;
        soff = tiled ? 4 * r : sc.lead + (uint32_t)(r * (int)nb);
    }
    // Piece u (128 k from 128 u on; u inside the rows).
    __device__ __forceinline__ void load(Load &p, int u) const
    {
#pragma unroll
        for (int i = 0; i < 4; i++)
            p.q[i] = q.load<uint4>(qoff[i], 128 * (int64_t)u);
        if (tiled) {
            const uint8_t *s = stile + (u >> 1) * rt + soff;
            __builtin_memcpy(&p.s, s, 4);
            __builtin_memcpy(&p.odd, s + 128, 4);
        } else {
            p.s = sc.load<uint32_t>(soff, 4 * (int64_t)u);
        }
    }
    // The scale bytes of piece u, once they are here.
    __device__ __forceinline__ uint32_t scales(const Load &p, int u) const
    {
        // bytes 2 (u % 2), + 1 of each: blocks 4u, 4u + 2 and 4u + 1, 4u + 3
        return tiled ? __builtin_amdgcn_perm(p.odd, p.s, u & 1 ? 0x07030602u : 0x05010400u) : p.s;
    }
    // The last piece: what lies behind the row's end becomes 0 (tiled scales there
    // are 0).
    __device__ __forceinline__ void fix(Load &p, int u, int lane) const
    {
        const int left = (int)(K - 128 * (int64_t)u);
#pragma unroll
        for (int i = 0; i < 4; i++)
            p.q[i] = q.fix(p.q[i], qoff[i], 128 * (int64_t)u, left - 16 * (lane & 7));
        if (!tiled) {
            const int keep = (int)(nb - 4 * (int64_t)u);
            const uint32_t d = sc.behind(soff, 4 * (int64_t)u);
            p.s = d < 4 ? p.s >> (8 * d) : 0;
            if (keep < 4)
                p.s &= (1u << (8 * keep)) - 1;
        }
    }
};

// Through the wave's own 4 KB of LDS (whose accesses come in order): chunk c of row
// R lies in slot c ^ (R / 2 mod 8) of the row, so that 16 lanes that are served
// together use all 64 banks, writing and reading.
__device__ __forceinline__ void turn(const Rows &rows, const Load &p, int u, Piece &o, uint4 *lds, int lane)
{
#pragma unroll
    for (int i = 0; i < 4; i++)
        lds[64 * i + (lane & 56) + ((lane & 7) ^ ((4 * i + (lane >> 4)) & 7))] = p.q[i];
    asm volatile("" ::: "memory");
    const uint4 *row = lds + 8 * (lane & 31);
    const int h = lane >> 5, x = lane >> 1 & 7;
#pragma unroll
    for (int i = 0; i < 2; i++)
        o.f[i] = join(row[(4 * i + h) ^ x], row[(4 * i + 2 + h) ^ x]);
    asm volatile("" ::: "memory");
    o.s = rows.scales(p, u);
}

// The scale bytes that a lane gives the block-scaled MFMA: blocks h and 2 + h, for steps
// 0 and 1.
__device__ __forceinline__ uint32_t lane_scales(uint32_t s, int h)
{
    return __builtin_amdgcn_perm(0, s, h ? 0x00000301u : 0x00000200u);
}

template <int F>
__device__ __forceinline__ bool far_piece(const Piece &p)
{
    bool far = false;
#pragma unroll
    for (int b = 0; b < 4; b++)
        far |= far_block<F>(half_of(p.f[b >> 1], b & 1), (p.s >> (8 * b)) & 255);
    return far;
}

// kExact: a piece (of `blocks` blocks, or more) with far blocks goes by mfma_far, and
// leaves zeros for multiply().
template <int FA, int FB, int MT>
__device__ __forceinline__ void multiply_far(Piece (&x)[MT], Piece &y, f32x16_t (&acc)[MT], int h, int blocks)
{
    uint32_t middle = middle_bytes(y.s);
#pragma unroll
    for (int m = 0; m < MT; m++)
        middle &= middle_bytes(x[m].s);
    if (__builtin_expect(!any_not_middle(middle | dead_bytes(blocks)), 1))
        return;
    bool far = far_piece<FB>(y);
#pragma unroll
    for (int m = 0; m < MT; m++)
        far |= far_piece<FA>(x[m]);
    if (__builtin_expect(__ballot(far) == 0, 1))
        return;
    const uint32_t sy = lane_scales(y.s, h);
#pragma unroll
    for (int m = 0; m < MT; m++) {
        const uint32_t sx = lane_scales(x[m].s, h);
        acc[m] = mfma_far<FA, FB, 0>(x[m].f[0], y.f[0], acc[m], sx, sy);
        acc[m] = mfma_far<FA, FB, 1>(x[m].f[1], y.f[1], acc[m], sx, sy);
        x[m].f[0] = x[m].f[1] = i32x8_t{};
    }
    y.f[0] = y.f[1] = i32x8_t{};
}

// acc += A B^T over a piece: two steps of 64 k.  Chunk 2 s + b of a lane (r, h)
// holds k 16 h .. + 15 of block 2 s + b.
template <MmMode MODE, int FA, int FB>
__device__ __forceinline__ void multiply(const Piece &x, const Piece &y, f32x16_t &acc, int h)
{
    if constexpr (MODE == kMx) {
        const uint32_t sx = lane_scales(x.s, h), sy = lane_scales(y.s, h);
        acc = mfma_mx<FA, FB, 0>(x.f[0], y.f[0], acc, sx, sy);
        acc = mfma_mx<FA, FB, 1>(x.f[1], y.f[1], acc, sx, sy);
    } else {
#pragma unroll
        for (int b = 0; b < 4; b++) {
            const float sx = scale_float((x.s >> (8 * b)) & 255), sy = scale_float((y.s >> (8 * b)) & 255);
            const uint4 cx = half_of(x.f[b >> 1], b & 1), cy = half_of(y.f[b >> 1], b & 1);
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf16_of_codes8<FA>(cx.x, cx.y, sx),
                                                          bf16_of_codes8<FB>(cy.x, cy.y, sy), acc, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf16_of_codes8<FA>(cx.z, cx.w, sx),
                                                          bf16_of_codes8<FB>(cy.z, cy.w, sy), acc, 0, 0, 0);
        }
    }
}

template <MmMode MODE, int FA, int FB, int MT, int KW>
__global__ __launch_bounds__(64 * KW, MT == 1 && KW == 4 ? 3 : 2) void mm_small_kernel(const MmArgs a, const MmTable t)
{
    __shared__ uint4 lds[KW * (MT + 1) * 256];
    float *const part = reinterpret_cast<float *>(lds);    // the partial sums, at the end
    const int tid = (int)threadIdx.x, L = tid & 63, h = L >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const MmTile w = mm_tile(a, t, (int)blockIdx.x, 32 * MT, 32);
    if (nothing_to_add(a, w))
        return;
    const int pieces = (int)((w.K + 127) >> 7), whole = (int)(w.K >> 7);
    f32x16_t acc[MT];
#pragma unroll
    for (int i = 0; i < MT; i++)
        acc[i] = f32x16_t{};
    if (wave < pieces) {
        const Rows rb(a.qb, w.qb, w.qb_left, a.sb, w.sb, w.sb_left, a.N, w.n0, w.K, w.nb, a.tiled, L);
        const Rows ra0(a.qa, w.qa, w.qa_left, a.sa, w.sa, w.sa_left, w.M, w.m0, w.K, w.nb, a.tiled, L);
        const int64_t m1 = w.m0 + 32 < w.M ? w.m0 + 32 : w.m0;
        const Rows ra1(a.qa, w.qa, w.qa_left, a.sa, w.sa, w.sa_left, w.M, m1, w.K, w.nb, a.tiled, L);
        Load pa[2][MT], pb[2];
        uint4 *const mine = lds + wave * (MT + 1) * 256;
        auto load = [&](int i, int u) {
            rb.load(pb[i], u);
            ra0.load(pa[i][0], u);
            if constexpr (MT == 2)
                ra1.load(pa[i][MT - 1], u);
        };
        auto work = [&](int i, int u) {
            Piece x[MT], y;
            turn(rb, pb[i], u, y, mine, L);
#pragma unroll
            for (int m = 0; m < MT; m++)
                turn(m ? ra1 : ra0, pa[i][m], u, x[m], mine + 256 * (m + 1), L);
            if constexpr (MODE == kExact)
                multiply_far<FA, FB, MT>(x, y, acc, h, (int)w.nb - 4 * u);
#pragma unroll
            for (int m = 0; m < MT; m++)
                multiply<MODE, FA, FB>(x[m], y, acc[m], h);
        };
        // the partial piece, by the wave whose turn it is, first
        const bool partial = whole < pieces && wave == whole % KW;
        if (partial)
            load(1, whole);
        if (wave < whole)
            load(0, wave);
        if (partial) {
            rb.fix(pb[1], whole, L);
            ra0.fix(pa[1][0], whole, L);
            if constexpr (MT == 2)
                ra1.fix(pa[1][MT - 1], whole, L);
            work(1, whole);
        }
        for (int u = wave; u < whole; u += 2 * KW) {
            if (u + KW < whole)
                load(1, u + KW);
            work(0, u);
            if (u + 2 * KW < whole)
                load(0, u + 2 * KW);
            if (u + KW < whole)
                work(1, u + KW);
        }
    }
    __syncthreads();
    // the upper half of the waves hands its sums to the lower
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int e = 0; e < 16; e++)
            if (wave >= KW / 2)
                part[((wave - KW / 2) * MT + i) * 1024 + 64 * e + L] = acc[i][e];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int e = 0; e < 16; e++)
            if (wave < KW / 2)
                part[(wave * MT + i) * 1024 + 64 * e + L] += acc[i][e];
    __syncthreads();
    // register e of lane (r, h) is row 8 (e / 4) + 4 h + e % 4, column r
    for (int o = tid; o < MT * 512; o += 64 * KW) {
        const int i = o >> 9, m = o >> 4 & 31, n = 2 * (o & 15);
        const int e = (m >> 3) * 4 + (m & 3), lane = n + 32 * (m >> 2 & 1);
        float v0 = 0.f, v1 = 0.f;
#pragma unroll
        for (int k = 0; k < KW / 2; k++) {
            const float2 p = *reinterpret_cast<const float2 *>(part + (k * MT + i) * 1024 + 64 * e + lane);
            v0 += p.x;
            v1 += p.y;
        }
        const int64_t row = w.m0 + 32 * i + m, col = w.n0 + n;
        if (row < w.M && col + 1 < a.N)
            store_out2(a, w.y0 + row * a.N + col, v0, v1);
        else if (row < w.M && col < a.N)
            store_out(a, w.y0 + row * a.N + col, v0);
    }
}

template <MmMode MODE, int MT, int KW>
hipError_t launch(const MmArgs &a, const MmTable &t, hipStream_t stream)
{
    const dim3 grid((unsigned)t.tile0[t.count]), block(64 * KW);
    if (!a.a_e5m2 && !a.b_e5m2)
        hipLaunchKernelGGL((mm_small_kernel<MODE, 0, 0, MT, KW>), grid, block, 0, stream, a, t);
    else if (a.a_e5m2 && !a.b_e5m2)
        hipLaunchKernelGGL((mm_small_kernel<MODE, 1, 0, MT, KW>), grid, block, 0, stream, a, t);
    else if (!a.a_e5m2)
        hipLaunchKernelGGL((mm_small_kernel<MODE, 0, 1, MT, KW>), grid, block, 0, stream, a, t);
    else
        hipLaunchKernelGGL((mm_small_kernel<MODE, 1, 1, MT, KW>), grid, block, 0, stream, a, t);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mm_small(const MmArgs &a, const MmTable &t, int rows, int waves, hipStream_t stream)
{
    if (a.out_f32)
        return rows == 32 ? waves == 8 ? launch<kExact, 1, 8>(a, t, stream) : launch<kExact, 1, 4>(a, t, stream)
               : waves == 8 ? launch<kExact, 2, 8>(a, t, stream)
                            : launch<kExact, 2, 4>(a, t, stream);
    return rows == 32 ? waves == 8 ? launch<kMx, 1, 8>(a, t, stream) : launch<kMx, 1, 4>(a, t, stream)
           : waves == 8 ? launch<kMx, 2, 8>(a, t, stream)
                        : launch<kMx, 2, 4>(a, t, stream);
}

}  // namespace mxk
