// nvfp4_matvec.hip -- matrix-vector products with NVFP4 weights.
//
// y[p][n] = S_g sum_k x[p][k] E2M1(qw[n][k]) E4M3(sw[n][k / 16]), x bf16.
// A wave owns one weight row; its lanes take the row's 16-element blocks in
// turn, sum a block's products in fp32, scale the block's sum and add it.
#include "launch_mm.h"
#include "mm_common.h"

namespace mxk {
namespace {

__device__ __forceinline__ float e2m1_value(uint32_t code)
{
    const uint32_t e = (code >> 1) & 3, m = code & 1;
    const float v = e == 0 ? 0.5f * (float)m : (float)((2 + m) << (e - 1)) * 0.5f;
    return code & 8 ? -v : v;
}

__global__ __launch_bounds__(256) void mv_any_kernel(const MvArgs a)
{
    const int lane = (int)threadIdx.x & 63;
    const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (n >= a.N)
        return;
    const int64_t nb = (a.K + 15) / 16, pitch = (a.K + 1) / 2, slots = a.T * a.top;
    for (int64_t p = blockIdx.y; p < slots; p += gridDim.y) {
        const int e = a.experts ? a.experts[p] : 0;
        float sum = 0.f;
        if (e >= 0 && e < a.G) {
            const uint8_t *q = a.qw + (e * a.N + n) * pitch, *s = a.sw + (e * a.N + n) * nb;
            const uint16_t *x = a.x + (p / a.top) * a.K;
            for (int64_t b = lane; b < nb; b += 64) {
                float part = 0.f;
                for (int i = 0; i < 16; i++) {
                    const int64_t k = 16 * b + i;
                    if (k < a.K)
                        part += __uint_as_float((uint32_t)x[k] << 16) *
                                e2m1_value(q[k >> 1] >> (4 * (k & 1)) & 15);
                }
                sum += part * __builtin_amdgcn_cvt_f32_fp8((int)s[b], 0);
            }
#pragma unroll
            for (int d = 32; d; d >>= 1)
                sum += __shfl_xor(sum, d);
            sum *= a.sg[e];
        }
        if (lane == 0) {
            if (a.out_f32)
                static_cast<float *>(a.y)[p * a.N + n] = sum;
            else
                static_cast<uint16_t *>(a.y)[p * a.N + n] = (uint16_t)bf16_pair(sum, 0.f);
        }
    }
}

}  // namespace

hipError_t launch_mv(const MvArgs &a, hipStream_t stream)
{
    const int64_t slots = a.T * a.top;
    const dim3 grid((unsigned)((a.N + 3) / 4), (unsigned)(slots < 65535 ? slots : 65535));
    hipLaunchKernelGGL(mv_any_kernel, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace mxk
