// nvfp4_matvec.hip -- matrix-vector products with NVFP4 weights.
//
// y[p][n] = S_g sum_k x[p][k] E2M1(qw[n][k]) E4M3(sw[n][k / 16]), x bf16.
//
// Reading the weights is the work: N K (1/2 + 1/16) bytes for any number of
// tokens up to 64, so the kernel streams them once, from HBM straight into
// registers, and does the rest beside that.  E2M1 times E4M3 has at most 6
// significant bits, so a scaled weight is exact in bf16: weights are converted
// to fp32 pairs, multiplied by their block's scale and packed to bf16 (2 vector
// instructions a weight; at 64 lanes a clock and CU that feeds about 9 TB/s of
// weights, more than HBM gives), and the matrix cores (16 x 16 x 32) multiply
// them with up to 16 tokens at once and sum in fp32.  One token costs what 16
// do.
//
// A wave takes R tiles of 16 weight rows.  It walks over k in chunks of 256; the
// 4 lanes of a row read 64 k each, as two 16-byte loads and one 4-byte load of 4
// scales, so a row's chunk is a whole 128-byte line.  KS waves of a workgroup
// take the chunks in turn (more loads in flight, and N rows alone would leave
// most of the chip idle); WN waves take different rows.  Tokens come through
// LDS, in the order in which the fragments want them.  The KS partial sums are
// added through LDS in a fixed order.
#include "launch_mm.h"
#include "mm_common.h"

namespace mxk {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2v_t __attribute__((ext_vector_type(2)));

constexpr int kMvThreads = 512, kMvWaves = 8;
constexpr int kChunk = 256;            // k of one step of a wave
constexpr int kMvStage = 65536;        // LDS bytes for tokens: two workgroups per CU
constexpr int kMvMaxSlots = 64;

// 8 E2M1 codes times their scale, as bf16 (exact).
__device__ __forceinline__ bf16x8_t weights8(uint32_t w, float s)
{
    const f32x2v_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    const f32x2v_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const f32x2v_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    const f32x2v_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    typedef uint32_t u32x4v_t __attribute__((ext_vector_type(4)));
    const u32x4v_t v = {bf16_pair(p0[0] * s, p0[1] * s), bf16_pair(p1[0] * s, p1[1] * s),
                        bf16_pair(p2[0] * s, p2[1] * s), bf16_pair(p3[0] * s, p3[1] * s)};
    return __builtin_bit_cast(bf16x8_t, v);
}

// A lane's share of a chunk of one row: 64 codes and 4 scale bytes.
struct Share {
    uint4 q[2];
    uint32_t s;
};

// v shifted down by d bytes (d < 16; anything above leaves any codes).
__device__ __forceinline__ uint4 shift_down(uint4 v, uint32_t d)
{
    if (d & 8)
        v = make_uint4(v.z, v.w, 0, 0);
    if (d & 4)
        v = make_uint4(v.y, v.z, v.w, 0);
    const uint32_t b = d & 3;
    return make_uint4(__builtin_amdgcn_alignbyte(v.y, v.x, b), __builtin_amdgcn_alignbyte(v.z, v.y, b),
                      __builtin_amdgcn_alignbyte(v.w, v.z, b), __builtin_amdgcn_alignbyte(0, v.w, b));
}

// TT: tokens at once.  EXPERTS: blockIdx.y is the expert (G: the slots without
// one, whose rows become zeros); else the tile of TT tokens.
template <int TT, int R, bool EXPERTS>
__global__ __launch_bounds__(kMvThreads, 4) void mv_kernel(const MvArgs a)
{
    constexpr int TB = TT / 16;                   // token tiles
    constexpr int KS = TT == 16 ? 8 : TT == 32 ? 4 : 2, WN = kMvWaves / KS;
    constexpr int kRows = 16 * R * WN;            // weight rows of a workgroup
    __shared__ __attribute__((aligned(16))) uint8_t lds[kMvStage];
    __shared__ int32_t slot[kMvMaxSlots];
    __shared__ int32_t wave_count[kMvWaves];

    const int tid = (int)threadIdx.x, L = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = L & 15, g = L >> 4;
    const int ks = wave % KS, wn = wave / KS;
    const int64_t n0 = (int64_t)blockIdx.x * kRows;
    const int64_t nb = (a.K + 15) >> 4, pitch = (a.K + 1) >> 1;
    const int nchunk = (int)((a.K + kChunk - 1) / kChunk);
    const int e = EXPERTS ? (int)blockIdx.y : 0;
    const int64_t slots = a.T * a.top;
    int64_t from = EXPERTS ? 0 : (int64_t)blockIdx.y * TT;    // next slot to look at

    // the workgroup's first row, the lanes' offsets from it (at most 128 rows of
    // 2^22 bytes), and how far the arrays reach from there
    const int64_t first = (EXPERTS && e == a.G ? 0 : (int64_t)e * a.N) + n0;
    const uint8_t *const qbase = a.qw + first * pitch, *const sbase = a.sw + first * nb;
    const int64_t qleft = ((int64_t)a.G * a.N - first) * pitch - 16;
    const int64_t sleft = ((int64_t)a.G * a.N - first) * nb - 4;
    uint32_t qoff[R], soff[R];
#pragma unroll
    for (int i = 0; i < R; i++) {
        int n = 16 * (wn * R + i) + r;
        n = n0 + n < a.N ? n : (int)(a.N - 1 - n0);
        qoff[i] = (uint32_t)(n * pitch) + 32 * g;
        soff[i] = (uint32_t)(n * nb) + 4 * g;
    }
    auto fetch = [&](Share (&w)[R], int c) {
        // a chunk inside the rows: as it lies there
        if ((c + 1) * kChunk <= a.K) {
#pragma unroll
            for (int i = 0; i < R; i++) {
                const uint8_t *q = qbase + c * (kChunk / 2) + qoff[i];
                __builtin_memcpy(&w[i].q[0], q, 16);
                __builtin_memcpy(&w[i].q[1], q + 16, 16);
                __builtin_memcpy(&w[i].s, sbase + c * (kChunk / 16) + soff[i], 4);
            }
            return;
        }
        // the last, partial one: never read behind the arrays; codes behind a
        // row's end meet zero tokens, scales there become 0
#pragma unroll
        for (int i = 0; i < R; i++) {
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int64_t q = (int64_t)c * (kChunk / 2) + qoff[i] + 16 * h;
                const int64_t p = q < qleft ? q : qleft;
                __builtin_memcpy(&w[i].q[h], qbase + p, 16);
                w[i].q[h] = shift_down(w[i].q[h], (uint32_t)(q - p < 15 ? q - p : 15));
            }
            const int64_t s = (int64_t)c * (kChunk / 16) + soff[i];
            const int64_t p = s < sleft ? s : sleft;
            __builtin_memcpy(&w[i].s, sbase + p, 4);
            const int64_t d = s - p, keep = nb - (int64_t)c * (kChunk / 16) - 4 * g;
            w[i].s = d < 4 ? w[i].s >> (8 * d) : 0;
            if (keep < 4)
                w[i].s = keep <= 0 ? 0 : w[i].s & ((1u << (8 * keep)) - 1);
        }
    };

    for (;;) {
        Share w[2][R];
        // this pass's tokens: count of them, their slots in slot[]
        int count;
        if (EXPERTS) {
            // the next TT slots of the expert, in order
            count = 0;
            int64_t base = from;
            while (base < slots && count < TT) {
                const int64_t p = base + tid;
                int32_t v = -1;
                if (p < slots)
                    v = a.experts[p];
                const bool none = v < 0 || v >= a.G;
                const bool hit = p < slots && (e < a.G ? v == e : none);
                const uint64_t m = __ballot(hit);
                if (L == 0)
                    wave_count[wave] = __popcll(m);
                __syncthreads();
                int at = count, all = count;
#pragma unroll
                for (int i = 0; i < kMvWaves; i++) {
                    at += i < wave ? wave_count[i] : 0;
                    all += wave_count[i];
                }
                at += __popcll(m & ((1ull << L) - 1));
                if (hit && at < TT)
                    slot[at] = (int32_t)p;
                count = all;
                base += kMvThreads;
                __syncthreads();
            }
            if (count > TT)
                count = TT;
            if (count == 0)
                return;
            from = slot[count - 1] + 1;
            if (e == a.G) {
                for (int64_t i = tid; i < (int64_t)count * kRows; i += kMvThreads) {
                    const int64_t n = n0 + i % kRows, o = (int64_t)slot[i / kRows] * a.N + n;
                    if (n >= a.N)
                        continue;
                    if (a.out_f32)
                        static_cast<float *>(a.y)[o] = 0.f;
                    else
                        static_cast<uint16_t *>(a.y)[o] = 0;
                }
                __syncthreads();
                continue;
            }
        } else {
            if (from >= a.T)
                return;
            count = (int)(a.T - from < TT ? a.T - from : TT);
            __syncthreads();
        }
        if (ks < nchunk)
            fetch(w[0], ks);

        f32x4_t acc[TB][R];
#pragma unroll
        for (int t = 0; t < TB; t++)
#pragma unroll
            for (int i = 0; i < R; i++)
                acc[t][i] = f32x4_t{};

        // chunks whose tokens fit the stage at once: a multiple of KS
        const int fit = kMvStage / (512 * count) / KS * KS;
        for (int c0 = 0; c0 < nchunk; c0 += fit) {
            const int nc = nchunk - c0 < fit ? nchunk - c0 : fit;
            __syncthreads();
            // 8 k of one token per 16 bytes; k = 64 g + 32 h + 8 d of a chunk
            // lies in fragment 4 h + d at lane group g
            for (int i = tid; i < nc * 32 * count; i += kMvThreads) {
                const int q = i & 31, t = (i >> 5) % count, c = (i >> 5) / count;
                const int64_t row = EXPERTS ? slot[t] / a.top : from + t;
                const int64_t k = (int64_t)(c0 + c) * kChunk + 8 * q;
                const uint16_t *x = a.x + row * a.K + k;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (k + 8 <= a.K) {
                    __builtin_memcpy(&v, x, 16);
                } else if (k < a.K) {
                    uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < 7; j++)
                        if (k + j < a.K)
                            u[j >> 1] |= (uint32_t)x[j] << (16 * (j & 1));
                    v = make_uint4(u[0], u[1], u[2], u[3]);
                }
                const int frag = 8 * c + (q & 7), lg = q >> 3;
                reinterpret_cast<uint4 *>(lds)[(frag * 4 + lg) * count + t] = v;
            }
            __syncthreads();
            const uint4 *xs = reinterpret_cast<const uint4 *>(lds);
            auto work = [&](const Share (&u)[R], int c) {
#pragma unroll
                for (int f = 0; f < 8; f++) {
                    bf16x8_t xf[TB];
#pragma unroll
                    for (int t = 0; t < TB; t++) {
                        // a lane behind the last token repeats it: its column
                        // is not stored
                        const int tt = 16 * t + r < count ? 16 * t + r : count - 1;
                        xf[t] = __builtin_bit_cast(bf16x8_t, xs[((8 * c + f) * 4 + g) * count + tt]);
                    }
#pragma unroll
                    for (int i = 0; i < R; i++) {
                        const uint4 q = u[i].q[f >> 2];
                        const uint32_t d = (f & 3) == 0 ? q.x : (f & 3) == 1 ? q.y : (f & 3) == 2 ? q.z : q.w;
                        const float s = (f >> 1) == 0   ? __builtin_amdgcn_cvt_f32_fp8((int)u[i].s, 0)
                                        : (f >> 1) == 1 ? __builtin_amdgcn_cvt_f32_fp8((int)u[i].s, 1)
                                        : (f >> 1) == 2 ? __builtin_amdgcn_cvt_f32_fp8((int)u[i].s, 2)
                                                        : __builtin_amdgcn_cvt_f32_fp8((int)u[i].s, 3);
                        const bf16x8_t wf = weights8(d, s);
#pragma unroll
                        for (int t = 0; t < TB; t++)
                            acc[t][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[t], acc[t][i], 0, 0, 0);
                    }
                    __builtin_amdgcn_sched_barrier(0);   // keeps the conversions of few fragments alive
                }
            };
            for (int c = ks; c < nc; c += 2 * KS) {
                if (c0 + c + KS < nchunk)
                    fetch(w[1], c0 + c + KS);
                work(w[0], c);
                if (c + KS < nc) {
                    if (c0 + c + 2 * KS < nchunk)
                        fetch(w[0], c0 + c + 2 * KS);
                    work(w[1], c + KS);
                } else {
#pragma unroll
                    for (int i = 0; i < R; i++)
                        w[0][i] = w[1][i];
                }
            }
        }

        // the KS partial sums, token tile by token tile; lane (r, g), register
        // j of a tile: weight row 4 g + j, token r
        float sg = a.sg[e];
#pragma unroll
        for (int t = 0; t < TB; t++) {
            __syncthreads();
            f32x4_t *part = reinterpret_cast<f32x4_t *>(lds);
#pragma unroll
            for (int i = 0; i < R; i++)
                part[(wave * R + i) * 64 + L] = acc[t][i];
            __syncthreads();
            for (int u = tid; u < WN * R * 64; u += kMvThreads) {
                const int i = (u >> 6) % R, v = (u >> 6) / R, l = u & 63;
                f32x4_t sum = part[(v * KS * R + i) * 64 + l];
                for (int k = 1; k < KS; k++)
                    sum += part[((v * KS + k) * R + i) * 64 + l];
                const int tok = 16 * t + (l & 15);
                const int64_t n = n0 + 16 * (v * R + i) + 4 * (l >> 4);
                if (tok >= count || n >= a.N)
                    continue;
                const int64_t o = (EXPERTS ? slot[tok] : from + tok) * a.N + n;
                sum *= sg;
                if ((a.N & 3) == 0) {
                    if (a.out_f32)
                        *reinterpret_cast<f32x4_t *>(static_cast<float *>(a.y) + o) = sum;
                    else
                        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.y) + o) =
                            make_uint2(bf16_pair(sum[0], sum[1]), bf16_pair(sum[2], sum[3]));
                } else {
                    for (int j = 0; j < 4 && n + j < a.N; j++) {
                        if (a.out_f32)
                            static_cast<float *>(a.y)[o + j] = sum[j];
                        else
                            static_cast<uint16_t *>(a.y)[o + j] = (uint16_t)bf16_pair(sum[j], 0.f);
                    }
                }
            }
        }
        if (!EXPERTS)
            from += (int64_t)gridDim.y * TT;
        __syncthreads();
    }
}

// Weights of fewer than 16 bytes of codes or 4 of scales, which the loads above
// do not fit: a wave per output row, bytes one by one.
__global__ __launch_bounds__(64) void mv_tiny_kernel(const MvArgs a)
{
    const int lane = (int)threadIdx.x;
    const int64_t nb = (a.K + 15) / 16, pitch = (a.K + 1) / 2, slots = a.T * a.top;
    for (int64_t p = (int64_t)blockIdx.x * 64 + lane; p < slots; p += (int64_t)gridDim.x * 64)
        for (int64_t n = 0; n < a.N; n++) {
            const int e = a.experts ? a.experts[p] : 0;
            float sum = 0.f;
            if (e >= 0 && e < a.G) {
                const int64_t row = e * a.N + n;
                for (int64_t k = 0; k < a.K; k++) {
                    const uint32_t code = a.qw[row * pitch + (k >> 1)] >> (4 * (k & 1));
                    const float s = __builtin_amdgcn_cvt_f32_fp8((int)a.sw[row * nb + (k >> 4)], 0);
                    const f32x2v_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 0);
                    sum += __uint_as_float((uint32_t)a.x[p / a.top * a.K + k] << 16) * (v[0] * s);
                }
                sum *= a.sg[e];
            }
            if (a.out_f32)
                static_cast<float *>(a.y)[p * a.N + n] = sum;
            else
                static_cast<uint16_t *>(a.y)[p * a.N + n] = (uint16_t)bf16_pair(sum, 0.f);
        }
}

template <int TT, int R>
hipError_t launch(const MvArgs &a, hipStream_t stream)
{
    constexpr int KS = TT == 16 ? 8 : TT == 32 ? 4 : 2, rows = 16 * R * (kMvWaves / KS);
    const unsigned nx = (unsigned)((a.N + rows - 1) / rows);
    if (a.experts)
        hipLaunchKernelGGL((mv_kernel<TT, R, true>), dim3(nx, (unsigned)a.G + 1), dim3(kMvThreads), 0,
                           stream, a);
    else
        hipLaunchKernelGGL((mv_kernel<TT, R, false>),
                           dim3(nx, (unsigned)(a.T < 4096 * TT ? (a.T + TT - 1) / TT : 4096)),
                           dim3(kMvThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mv(const MvArgs &a, hipStream_t stream)
{
    if (a.G * a.N * ((a.K + 1) / 2) < 16 || a.G * a.N * ((a.K + 15) / 16) < 4) {
        const int64_t n = (a.T * a.top + 63) / 64;
        hipLaunchKernelGGL(mv_tiny_kernel, dim3((unsigned)(n < 4096 ? n : 4096)), dim3(64), 0, stream, a);
        return hipGetLastError();
    }
    // tokens that a weight matrix meets: all, or an expert's fair share twice over
    const int64_t slots = a.T * a.top;
    const int64_t tokens = a.experts ? (2 * slots + a.G - 1) / a.G : a.T;
    const int64_t most = slots < tokens ? slots : tokens;
    if (most > 32)
        return launch<64, 1>(a, stream);
    if (most > 16)
        return launch<32, 2>(a, stream);
    // more rows per wave where that leaves two workgroups per CU: the tokens
    // are then staged for more rows at once
    const int64_t tiles = (a.N + 15) / 16 * (a.experts ? (slots < a.G ? slots : a.G) : 1);
    if (tiles >= 2048)
        return launch<16, 4>(a, stream);
    if (tiles >= 1024)
        return launch<16, 2>(a, stream);
    return launch<16, 1>(a, stream);
}

}  // namespace mxk
