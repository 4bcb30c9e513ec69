// mm_small.hip -- small products of MXFP8 operands: few rows, or few outputs.
//
// Here the operands are read about once and there is too little work for the
// tiled kernel, whose workgroups walk along k alone and pay a memory latency per
// 128 k.  A workgroup of 4 waves owns 32 MT x 32 outputs, and its waves take
// pieces of 128 k in turn, straight from memory into the fragments (rows at any
// byte), two pieces under way per wave.  The 4 partial sums are added through LDS
// in a fixed order.
#include "mm_common.h"

namespace mxk {
namespace {

constexpr int kWavesK = 4;

// A row's share of a piece: the lane's four 16-byte chunks and the scale bytes of
// the piece's four blocks.
struct Piece {
    i32x8_t f[2];              // chunks 2 s and 2 s + 1: step s
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
    uint32_t qoff, soff;
    int64_t K, nb;
    int32_t tiled;
    int64_t rt;                // tiled: bytes from one block tile to the next

    __device__ __forceinline__ Rows(const uint8_t *qarray, const uint8_t *qg, int64_t qleft,
                                    const uint8_t *sarray, const uint8_t *sg, int64_t sleft, int64_t rows,
                                    int64_t r0, int64_t K_, int64_t nb_, int32_t tiled_, int lane)
        : q(qarray, qg + r0 * K_, qleft - r0 * K_), sc(sarray, sg + r0 * nb_, sleft - r0 * nb_),
          stile(sg + (r0 >> 5) * 256), K(K_), nb(nb_), tiled(tiled_), rt(((rows + 31) >> 5) * 256)
    {
        const int h = lane >> 5;
        int r = lane & 31;
        r = r0 + r < rows ? r : (int)(rows - 1 - r0);
        qoff = q.lead + (uint32_t)(r * (int)K) + 16 * h;
        soff = tiled ? 4 * r : sc.lead + (uint32_t)(r * (int)nb);
    }
    // Piece u (128 k from 128 u on; u inside the rows).
    __device__ __forceinline__ void load(Piece &p, int u) const
    {
#pragma unroll
        for (int i = 0; i < 2; i++)
            p.f[i] = join(q.load<uint4>(qoff + 64 * i, 128 * (int64_t)u),
                          q.load<uint4>(qoff + 64 * i + 32, 128 * (int64_t)u));
        if (tiled) {
            const uint8_t *s = stile + (u >> 1) * rt + soff;
            uint32_t even, odd;
            __builtin_memcpy(&even, s, 4);
            __builtin_memcpy(&odd, s + 128, 4);
            // bytes 2 (u % 2), + 1 of each: blocks 4u, 4u + 2 and 4u + 1, 4u + 3
            p.s = __builtin_amdgcn_perm(odd, even, u & 1 ? 0x07030602u : 0x05010400u);
        } else {
            p.s = sc.load<uint32_t>(soff, 4 * (int64_t)u);
        }
    }
    // The last piece: what lies behind the row's end becomes 0.
    __device__ __forceinline__ void fix(Piece &p, int u, int h) const
    {
        const int left = (int)(K - 128 * (int64_t)u);
#pragma unroll
        for (int i = 0; i < 2; i++)
            p.f[i] = join(q.fix(half_of(p.f[i], 0), qoff + 64 * i, 128 * (int64_t)u, left - 64 * i - 16 * h),
                          q.fix(half_of(p.f[i], 1), qoff + 64 * i + 32, 128 * (int64_t)u,
                                left - 64 * i - 32 - 16 * h));
        const int keep = (int)(nb - 4 * (int64_t)u);
        if (!tiled) {
            const uint32_t d = sc.behind(soff, 4 * (int64_t)u);
            p.s = d < 4 ? p.s >> (8 * d) : 0;
        }
        if (keep < 4)
            p.s &= (1u << (8 * keep)) - 1;
    }
};

// acc += A B^T over a piece: two steps of 64 k.  Chunk 2 s + b of a lane (r, h)
// holds k 16 h .. + 15 of block 2 s + b.
template <MmMode MODE, int FA, int FB>
__device__ __forceinline__ void multiply(const Piece &x, const Piece &y, f32x16_t &acc, int h)
{
    if constexpr (MODE == kMx) {
        // the lane's scale bytes: blocks h and 2 + h, for steps 0 and 1
        const uint32_t sel = h ? 0x00000301u : 0x00000200u;
        const uint32_t sx = __builtin_amdgcn_perm(0, x.s, sel), sy = __builtin_amdgcn_perm(0, y.s, sel);
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

template <MmMode MODE, int FA, int FB, int MT>
__global__ __launch_bounds__(64 * kWavesK, MT == 1 ? 3 : 2) void mm_small_kernel(const MmArgs a, const MmTable t)
{
    __shared__ float part[kWavesK / 2 * MT * 1024];
    const int tid = (int)threadIdx.x, L = tid & 63, h = L >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const MmTile w = mm_tile(a, t, (int)blockIdx.x, 32 * MT, 32);
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
        Piece pa[2][MT], pb[2];
        auto load = [&](int i, int u) {
            rb.load(pb[i], u);
            ra0.load(pa[i][0], u);
            if constexpr (MT == 2)
                ra1.load(pa[i][MT - 1], u);
        };
        auto work = [&](int i) {
#pragma unroll
            for (int m = 0; m < MT; m++)
                multiply<MODE, FA, FB>(pa[i][m], pb[i], acc[m], h);
        };
        // the partial piece, by the wave whose turn it is, first
        const bool partial = whole < pieces && wave == whole % kWavesK;
        if (partial)
            load(1, whole);
        if (wave < whole)
            load(0, wave);
        if (partial) {
            rb.fix(pb[1], whole, h);
            ra0.fix(pa[1][0], whole, h);
            if constexpr (MT == 2)
                ra1.fix(pa[1][MT - 1], whole, h);
            work(1);
        }
        for (int u = wave; u < whole; u += 2 * kWavesK) {
            if (u + kWavesK < whole)
                load(1, u + kWavesK);
            work(0);
            if (u + 2 * kWavesK < whole)
                load(0, u + 2 * kWavesK);
            if (u + kWavesK < whole)
                work(1);
        }
    }
    // the upper half of the waves hands its sums to the lower
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int e = 0; e < 16; e++)
            if (wave >= kWavesK / 2)
                part[((wave - kWavesK / 2) * MT + i) * 1024 + 64 * e + L] = acc[i][e];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int e = 0; e < 16; e++)
            if (wave < kWavesK / 2)
                part[(wave * MT + i) * 1024 + 64 * e + L] += acc[i][e];
    __syncthreads();
    // register e of lane (r, h) is row 8 (e / 4) + 4 h + e % 4, column r
    for (int o = tid; o < MT * 1024; o += 64 * kWavesK) {
        const int i = o >> 10, m = o >> 5 & 31, n = o & 31;
        const int e = (m >> 3) * 4 + (m & 3), lane = n + 32 * (m >> 2 & 1);
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kWavesK / 2; k++)
            v += part[(k * MT + i) * 1024 + 64 * e + lane];
        const int64_t row = w.m0 + 32 * i + m, col = w.n0 + n;
        if (row < w.M && col < a.N)
            store_out(a, w.y0 + row * a.N + col, v);
    }
}

template <MmMode MODE, int MT>
hipError_t launch(const MmArgs &a, const MmTable &t, hipStream_t stream)
{
    const dim3 grid((unsigned)t.tile0[t.count]), block(64 * kWavesK);
    if (!a.a_e5m2 && !a.b_e5m2)
        hipLaunchKernelGGL((mm_small_kernel<MODE, 0, 0, MT>), grid, block, 0, stream, a, t);
    else if (a.a_e5m2 && !a.b_e5m2)
        hipLaunchKernelGGL((mm_small_kernel<MODE, 1, 0, MT>), grid, block, 0, stream, a, t);
    else if (!a.a_e5m2)
        hipLaunchKernelGGL((mm_small_kernel<MODE, 0, 1, MT>), grid, block, 0, stream, a, t);
    else
        hipLaunchKernelGGL((mm_small_kernel<MODE, 1, 1, MT>), grid, block, 0, stream, a, t);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mm_small(const MmArgs &a, const MmTable &t, int rows, hipStream_t stream)
{
    if (rows == 32)
        return a.out_f32 ? launch<kExact, 1>(a, t, stream) : launch<kMx, 1>(a, t, stream);
    return a.out_f32 ? launch<kExact, 2>(a, t, stream) : launch<kMx, 2>(a, t, stream);
}

}  // namespace mxk
