// mm_any.hip -- products of MXFP8 operands too small for the other kernels' loads:
// fewer than 16 bytes of codes or 8 of scales in one of them.
//
// Y_g[m][n] = sum_k A_g[m][k] B_g[n][k], each operand's value being its
// element times 2^(byte - 127) of its 32-element block along k.  (MmMode has the
// two ways to compute it; fp32 outputs all go by mfma_far here.)  Such an operand
// has at most 7 blocks, so time is a launch (3 us) and the output; nothing here is
// tuned.
//
// A workgroup of 4 waves owns 64 x 64 outputs, a wave 32 x 32.  Codes come through
// registers (16 bytes inside a row, else byte by byte, zeros behind it) into LDS,
// 128 k at a time.
#include "launch_mm.h"
#include "mm_common.h"

namespace mxk {
namespace {

constexpr int kT = kMmAnyTile;
constexpr int kBK = 128;

// 16 codes of row `row` from k on; zeros outside the operand.
__device__ __forceinline__ uint4 load_chunk(const uint8_t *q, int64_t rows, int64_t K, int64_t row,
                                            int64_t k)
{
    uint4 v = make_uint4(0, 0, 0, 0);
    if (row >= rows || k >= K)
        return v;
    const uint8_t *p = q + row * K + k;
    if (k + 16 <= K) {
        __builtin_memcpy(&v, p, 16);
        return v;
    }
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; i++)
        if (k + i < K)
            w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <MmMode MODE, int FA, int FB>
__global__ __launch_bounds__(256) void mm_any_kernel(const MmArgs a, const MmTable t)
{
    __shared__ uint4 lds[2][kT * kBK / 16];
    const int tid = (int)threadIdx.x, L = tid & 63, wave = tid >> 6;
    const MmTile w = mm_tile(a, t, (int)blockIdx.x, kT, kT);
    if (nothing_to_add(a, w))
        return;
    const int h = L >> 5, r = L & 31;
    const int wm = 32 * (wave >> 1), wn = 32 * (wave & 1);

    f32x16_t acc = {};
    for (int64_t k0 = 0; k0 < w.K; k0 += kBK) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int row = (tid >> 3) + 32 * i, c = tid & 7;
            lds[0][row * 8 + (c ^ (row & 7))] = load_chunk(w.qa, w.M, w.K, w.m0 + row, k0 + 16 * c);
            lds[1][row * 8 + (c ^ (row & 7))] = load_chunk(w.qb, a.N, w.K, w.n0 + row, k0 + 16 * c);
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; s++) {
            // lane (r, h): bytes 0-15 hold k 16h .. 16h + 15 of the step's
            // first block, bytes 16-31 those of its second
            const int c0 = 4 * s + h, c1 = 4 * s + 2 + h;
            const uint4 a0 = lds[0][(wm + r) * 8 + (c0 ^ (r & 7))];
            const uint4 a1 = lds[0][(wm + r) * 8 + (c1 ^ (r & 7))];
            const uint4 b0 = lds[1][(wn + r) * 8 + (c0 ^ (r & 7))];
            const uint4 b1 = lds[1][(wn + r) * 8 + (c1 ^ (r & 7))];
            const int64_t blk = k0 / 32 + 2 * s, m = w.m0 + wm + r, n = w.n0 + wn + r;
            // the lane's scale byte is block h's
            const uint32_t sa = (uint32_t)scale_byte(w.sa, w.M, w.nb, m, blk + h, a.tiled);
            const uint32_t sb = (uint32_t)scale_byte(w.sb, a.N, w.nb, n, blk + h, a.tiled);
            acc = MODE == kMx ? mfma_mx<FA, FB, 0>(join(a0, a1), join(b0, b1), acc, sa, sb)
                              : mfma_far<FA, FB, 0>(join(a0, a1), join(b0, b1), acc, sa, sb);
        }
    }
    // lane (r, h), register i: row 8 (i / 4) + 4 h + i % 4, column r
#pragma unroll
    for (int i = 0; i < 16; i++) {
        const int64_t m = w.m0 + wm + 8 * (i >> 2) + 4 * h + (i & 3), n = w.n0 + wn + r;
        if (m < w.M && n < a.N)
            store_out(a, w.y0 + m * a.N + n, acc[i]);
    }
}

template <MmMode MODE>
hipError_t launch(const MmArgs &a, const MmTable &t, hipStream_t stream)
{
    const dim3 grid((unsigned)t.tile0[t.count]), block(256);
    if (!a.a_e5m2 && !a.b_e5m2)
        hipLaunchKernelGGL((mm_any_kernel<MODE, 0, 0>), grid, block, 0, stream, a, t);
    else if (a.a_e5m2 && !a.b_e5m2)
        hipLaunchKernelGGL((mm_any_kernel<MODE, 1, 0>), grid, block, 0, stream, a, t);
    else if (!a.a_e5m2)
        hipLaunchKernelGGL((mm_any_kernel<MODE, 0, 1>), grid, block, 0, stream, a, t);
    else
        hipLaunchKernelGGL((mm_any_kernel<MODE, 1, 1>), grid, block, 0, stream, a, t);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mm_any(const MmArgs &a, const MmTable &t, hipStream_t stream)
{
    return a.out_f32 ? launch<kExact>(a, t, stream) : launch<kMx>(a, t, stream);
}

}  // namespace mxk
