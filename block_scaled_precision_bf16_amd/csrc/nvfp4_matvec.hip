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
// A wave takes 16 weight rows.  It walks over k in chunks of 256; the 4 lanes of a
// row read 64 k each, as two 16-byte loads and one 4-byte load of 4 scales, so a
// row's chunk is a whole 128-byte line.  KS waves of a workgroup take the chunks
// in turn (more loads in flight, and N rows alone would leave most of the chip
// idle); WN waves take different rows.  Tokens come through LDS, in the order in
// which the fragments want them, a stage of chunks at a time.  The KS partial
// sums are added through LDS in a fixed order.
//
// Measured, 16384 x 16384 (151 MB of weights, some of them from the MALL): 1 token 31 us,
// 4.9 TB/s; 16 tokens 41 - 43 us (from HBM alone, 131072 rows: 3.4 TB/s, where 1 token
// reaches 4.4 and the absmax pass, which only reads, 6.8 - 7.2); the vector units are
// busy 53% of the time, and waves wait for weights and at the stages' barriers.  32
// tokens 50 us, 64 tokens 69 us, where the conversions, the reads of the tokens from
// LDS and the MFMAs come one after the other in too few waves.  One token by 14336 x
// 4096: 9.8 us, of which 3.2 are an empty launch's.
#include "launch_mm.h"
#include "mm_common.h"

namespace mxk {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2v_t __attribute__((ext_vector_type(2)));

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

__device__ __forceinline__ float dot2(bf16x2v_t w, uint32_t x, float c)
{
    return __builtin_amdgcn_fdot2_f32_bf16(w, __builtin_bit_cast(bf16x2v_t, x), c, false);
}

// A lane's share of a chunk of one row: 64 codes and 4 scale bytes.
struct Share {
    uint4 q[2];
    uint32_t s;
};

__device__ __forceinline__ void store_mv(const MvArgs &a, int64_t i, float v)
{
    if (a.out_f32)
        static_cast<float *>(a.y)[i] = v;
    else
        static_cast<uint16_t *>(a.y)[i] = (uint16_t)bf16_pair(v, 0.f);
}

// Up to TT slots that take expert e (with e = G: that take none), in order from
// slot `from` on, into slot[]; returns how many.  Called by all waves; slot[] is
// there after the caller's next barrier.
template <int TT>
__device__ __forceinline__ int gather_slots(const MvArgs &a, int e, int from, int32_t *slot,
                                            int32_t *wave_count)
{
    const int slots = a.T * a.top;
    const int tid = (int)threadIdx.x, L = tid & 63, wave = tid >> 6;
    const uint64_t below = (1ull << L) - 1;
    auto takes = [&](int p) {
        if (p >= slots)
            return false;
        const int32_t v = a.experts[p];
        return e < a.G ? v == e : v < 0 || v >= a.G;
    };
    if (slots - from <= 64) {
        // every wave looks for itself
        const bool hit = takes(from + L);
        const uint64_t m = __ballot(hit);
        const int at = __popcll(m & below), all = __popcll(m);
        if (wave == 0 && hit && at < TT)
            slot[at] = from + L;
        return all < TT ? all : TT;
    }
    int count = 0;
    for (int base = from; base < slots && count < TT; base += kMvThreads) {
        const bool hit = takes(base + tid);
        const uint64_t m = __ballot(hit);
        if (L == 0)
            wave_count[wave] = __popcll(m);
        __syncthreads();
        int at = count + __popcll(m & below);
#pragma unroll
        for (int i = 0; i < kMvWaves; i++) {
            at += i < wave ? wave_count[i] : 0;
            count += wave_count[i];
        }
        if (hit && at < TT)
            slot[at] = base + tid;
        __syncthreads();
    }
    return count < TT ? count : TT;
}

// Zeros in the workgroup's share of the rows of slots p + 0 .. or slot[0] ...
__device__ __forceinline__ void zero_rows(const MvArgs &a, const int32_t *slot, int p, int count)
{
    for (int t = 0; t < count; t++)
        for (int n = (int)(blockIdx.x * kMvThreads + threadIdx.x); n < a.N; n += (int)gridDim.x * kMvThreads)
            store_mv(a, (int64_t)(slot ? slot[t] : p + t) * a.N + n, 0.f);
}

// Waves per SIMD: two workgroups per CU, or one that takes 136 KB of LDS.
constexpr int mv_occupancy(int tokens, bool few) { return tokens == 64 || (tokens == 16 && few) ? 2 : 4; }

// Where a workgroup finds the weights of a block of rows.
struct Aim {
    const uint8_t *q, *s;       // bases a little before the block's first row
    uint32_t qlast, slast;      // the last offsets that a load of 16 (4) bytes may have
    uint32_t qoff, soff;        // the lane's (at most 64 rows of 2^22 bytes)

    __device__ __forceinline__ Aim(const MvArgs &a, int e, int n0, int row, int g)
    {
        const int nb = (a.K + 15) >> 4, pitch = (a.K + 1) >> 1;
        const int64_t first = (int64_t)e * a.N + n0, all = (int64_t)a.G * a.N;
        const int64_t q0 = first * pitch < 16 ? 0 : first * pitch - 16;
        const int64_t s0 = first * nb < 4 ? 0 : first * nb - 4;
        q = a.qw + q0;
        s = a.sw + s0;
        const int64_t qreach = all * pitch - 16 - q0, sreach = all * nb - 4 - s0;
        qlast = (uint32_t)(qreach < INT32_MAX ? qreach : INT32_MAX);
        slast = (uint32_t)(sreach < INT32_MAX ? sreach : INT32_MAX);
        row = row < a.N - 1 - n0 ? row : a.N - 1 - n0;
        qoff = (uint32_t)(first * pitch - q0) + (uint32_t)(row * pitch) + 32 * g;
        soff = (uint32_t)(first * nb - s0) + (uint32_t)(row * nb) + 4 * g;
    }
    // A chunk's bytes, never from behind the arrays' ends: there, those before
    // the end, which settle() moves where they belong.
    __device__ __forceinline__ void fetch(Share &w, int c) const
    {
        const uint32_t o = qoff + c * (kMvChunk / 2), p = soff + c * (kMvChunk / 16);
        __builtin_memcpy(&w.q[0], q + (o < qlast ? o : qlast), 16);
        __builtin_memcpy(&w.q[1], q + (o + 16 < qlast ? o + 16 : qlast), 16);
        __builtin_memcpy(&w.s, s + (p < slast ? p : slast), 4);
    }
    // The last, partial chunk: codes behind a row's end are some codes and meet
    // zero tokens, scales there (from block nb on) become 0.
    __device__ __forceinline__ void settle(Share &w, int c, int nb, int g) const
    {
        const int o = (int)(qoff + c * (kMvChunk / 2) - qlast), p = (int)(soff + c * (kMvChunk / 16) - slast);
        if (o > 0)
            w.q[0] = bytes_down(w.q[0], o < 15 ? o : 15);
        if (o + 16 > 0)
            w.q[1] = bytes_down(w.q[1], o + 16 < 15 ? o + 16 : 15);
        const int keep = nb - c * (kMvChunk / 16) - 4 * g;
        uint32_t v = p > 0 ? (p < 4 ? w.s >> (8 * p) : 0) : w.s;
        if (keep < 4)
            v = keep <= 0 ? 0 : v & ((1u << (8 * keep)) - 1);
        w.s = v;
    }
};

// A workgroup takes row block blockIdx.x, with EXPERTS and tokens that fit one stage
// also + gridDim.x, ... (which costs registers, and gains where a workgroup's own work
// is short).
// EXPERTS: blockIdx.y is the expert (G: the slots without one, whose rows become zeros)
// or, with a.by_slot, a slot, whose workgroups serve its expert if no earlier
// slot has the same; else the tile of TT tokens.
template <int TT, bool EXPERTS, bool FEW>
__global__ __launch_bounds__(kMvThreads, mv_occupancy(TT, FEW)) void mv_kernel(const MvArgs a)
{
    using Plan = MvPlan<TT, EXPERTS, FEW>;
    constexpr int TB = (TT + 15) / 16;            // token tiles
    constexpr int KS = Plan::KS, P = Plan::kPieces, D = Plan::D;
    constexpr int kMix = TT == 1 ? 3 : 7;         // within a fragment's 4 TT slots
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ int32_t slot[EXPERTS ? TT : 1];
    __shared__ int32_t wave_count[kMvWaves];

    const int blocks = (a.N + Plan::kRows - 1) / Plan::kRows, step = (int)gridDim.x;
    const int nb = (a.K + 15) >> 4, nchunk = (a.K + kMvChunk - 1) / kMvChunk;
    const int partial = a.K % kMvChunk ? nchunk - 1 : nchunk;    // the first chunk to settle
    const int stages = (nchunk + Plan::kFit - 1) / Plan::kFit;
    // Rows some kilobytes apart lie in few of the memory's channels at any one k, and
    // the workgroups walk along k at about the same pace: neighbouring ones start
    // at different stages.  (Not where a workgroup lives for a few chunks only: one
    // token through 2 of 8 experts of 5120 x 4096 11.3 -> 11.0 us without, of 4096 x
    // 14336 19.7 -> 19.0, of 4096 x 8192 13.2 -> 13.4.)
    const int first = (TT <= 2 && EXPERTS) || stages <= 1
                          ? 0
                          : (int)((blockIdx.x + blockIdx.x / 8) % (unsigned)stages);
    auto turned = [&](int st) { return st + first < stages ? st + first : st + first - stages; };
    int from = 0;                                 // the next slot to look at
    int e = 0;
    if (EXPERTS) {
        e = (int)blockIdx.y;
        if (a.by_slot) {
            from = e;
            e = __builtin_amdgcn_readfirstlane(a.experts[from]);
            if (e < 0 || e >= a.G) {
                zero_rows(a, nullptr, from, 1);
                return;
            }
            bool earlier = false;
            for (int p = threadIdx.x & 63; p < from; p += 64)
                earlier |= a.experts[p] == e;
            if (__ballot(earlier))
                return;
        }
    } else {
        from = (int)blockIdx.y * TT;
    }

    for (;;) {
        // (the lane's places are worked out in each pass: kept over passes they
        // cost more registers than there are)
        int tid = (int)threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int L = tid & 63, r = L & 15, g = L >> 4;
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int ks = wave % KS, wn = wave / KS;
        int count;                                // this pass's tokens
        if (EXPERTS) {
            count = gather_slots<TT>(a, e, from, slot, wave_count);
            if (count == 0)
                return;
            if (e == a.G) {
                __syncthreads();
                zero_rows(a, slot, 0, count);
                from = slot[count - 1] + 1;
                __syncthreads();
                continue;
            }
        } else {
            if (from >= a.T)
                return;
            count = a.T - from < TT ? a.T - from : TT;
        }
        Share w[D];
        Aim next(a, e, (int)blockIdx.x * Plan::kRows, 16 * wn + r, g);
#pragma unroll
        for (int j = 0; j < D; j++)
            if (turned(0) * Plan::kFit + ks + j * KS < nchunk)
                next.fetch(w[j], turned(0) * Plan::kFit + ks + j * KS);
        if (EXPERTS)
            __syncthreads();                      // slot[]

        // The tokens of a stage, in fragment order: 8 k of one token per 16
        // bytes; k = 64 g + 32 h + 8 d of a chunk belongs to fragment f = 4 h + d
        // at lane group g, and lies in slot (g TT + token) ^ f of the fragment's
        // 4 TT (one token: ^ f % 4; the writes of 8 neighbouring pieces go to 8
        // fragments, the reads stay in one: both touch all banks).  A thread
        // moves P pieces, at the same places in every stage, through registers:
        // all loads before the first store, and those of the next stage while
        // this one is used.
        // Thread tid: piece tid % 32 of a chunk; the 16 rows tid / 32 are
        // tokens (TT < 16: TT tokens of 16 / TT chunks), TB times over.
        constexpr int kSide = TT < 16 ? 16 / TT : 1;
        const int q = tid & 31, c_side = (tid >> 5) / (TT < 16 ? TT : 16);
        const int xk = c_side * kMvChunk + 8 * q;
        int64_t xo[TB];                           // element offset in x
#pragma unroll
        for (int b = 0; b < TB; b++) {
            int t = (tid >> 5) % TT + 16 * b;
            t = t < count ? t : count - 1;        // a place of no token: any
            xo[b] = (int64_t)(EXPERTS ? slot[t] / a.top : from + t) * a.K + xk;
        }
        uint4 *const xl = reinterpret_cast<uint4 *>(lds) + (8 * c_side + (q & 7)) * 4 * TT +
                          (((q >> 3) * TT + (tid >> 5) % TT) ^ (q & kMix));
        uint4 xv[P];
        // never from behind x's end: there, the 16 bytes before it
        const int64_t x_end = (int64_t)a.T * a.K - 8;
        auto load_tokens = [&](int st) {
#pragma unroll
            for (int j = 0; j < P; j++) {
                const int64_t o = xo[j % TB] + (st * Plan::kFit + j / TB * kSide) * kMvChunk;
                __builtin_memcpy(&xv[j], a.x + (o < x_end ? o : x_end), 16);
            }
        };
        auto store_tokens = [&](int st) {
            if ((st + 1) * Plan::kFit * kMvChunk > a.K) {
                // what lies behind a row's end becomes 0
#pragma unroll
                for (int j = 0; j < P; j++) {
                    const int k0 = (st * Plan::kFit + j / TB * kSide) * kMvChunk;
                    const int64_t d = 2 * (xo[j % TB] + k0 - x_end);
                    const int keep = a.K - k0 - xk;
                    uint4 v = xv[j];
                    if (d > 0)
                        v = bytes_down(v, d < 15 ? (uint32_t)d : 15);
                    const uint32_t half = keep & 1 ? 0xFFFFu : 0;
                    v.x &= keep >= 2 ? ~0u : keep > 0 ? half : 0;
                    v.y &= keep >= 4 ? ~0u : keep > 2 ? half : 0;
                    v.z &= keep >= 6 ? ~0u : keep > 4 ? half : 0;
                    v.w &= keep >= 8 ? ~0u : keep > 6 ? half : 0;
                    xv[j] = v;
                }
            }
#pragma unroll
            for (int j = 0; j < P; j++)
                xl[j / TB * kSide * 32 * TT + 16 * (j % TB)] = xv[j];
        };
        load_tokens(turned(0));
        const float sg = a.sg[e];

        for (int block = (int)blockIdx.x; block < blocks; block += EXPERTS ? step : blocks) {
            Aim aim = next;
            // (what depends on these is computed where it is used: kept over the
            // loop it costs more registers than there are)
            if (EXPERTS)
                asm volatile("" : "+v"(aim.qoff), "+v"(aim.soff));
            const int n0 = block * Plan::kRows;
            const bool more = EXPERTS && block + step < blocks;
            if (more)
                next = Aim(a, e, n0 + step * Plan::kRows, 16 * wn + r, g);
            f32x4_t acc[TB];                      // kDot: acc[0][t] of token t
#pragma unroll
            for (int t = 0; t < TB; t++)
                acc[t] = f32x4_t{};
            // chunk number `chunk`, chunk c of the stage
            auto work = [&](Share &u, int c, int chunk) {
                if (chunk >= partial)
                    aim.settle(u, chunk, nb, g);
                const uint4 *xs = reinterpret_cast<const uint4 *>(lds) + 32 * TT * c;
                // token fragment f of tile t; columns behind the last token are of any
                // value and not stored
                auto tokens = [&](int f, int t) {
                    return __builtin_bit_cast(
                        bf16x8_t, xs[4 * f * TT + ((g * TT + (r < TT ? r : 0)) ^ (f & kMix)) + 16 * t]);
                };
                // read one fragment ahead of their use
                bf16x8_t xf[2][TB];
                if constexpr (!Plan::kDot) {
#pragma unroll
                    for (int t = 0; t < TB; t++)
                        xf[0][t] = tokens(0, t);
                }
#pragma unroll
                for (int b = 0; b < 4; b++) {     // block b of the lane's 4: fragments 2b, 2b + 1
                    const float s = b == 0   ? __builtin_amdgcn_cvt_f32_fp8((int)u.s, 0)
                                    : b == 1 ? __builtin_amdgcn_cvt_f32_fp8((int)u.s, 1)
                                    : b == 2 ? __builtin_amdgcn_cvt_f32_fp8((int)u.s, 2)
                                             : __builtin_amdgcn_cvt_f32_fp8((int)u.s, 3);
                    // kDot: s = 2 rest * 2^e (s = 0: rest = 0; NaN: NaN), and the conversion
                    // takes e from s, whose other bits it does not look at
                    const float rest = __builtin_amdgcn_frexp_mantf(s);
                    float sum[2] = {0.f, 0.f};
#pragma unroll
                    for (int f = 2 * b; f < 2 * b + 2; f++) {
                        const uint4 v = u.q[f >> 2];
                        const uint32_t d = (f & 3) == 0 ? v.x : (f & 3) == 1 ? v.y : (f & 3) == 2 ? v.z : v.w;
                        if constexpr (Plan::kDot) {
                            const bf16x2v_t w0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 0);
                            const bf16x2v_t w1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 1);
                            const bf16x2v_t w2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 2);
                            const bf16x2v_t w3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, s, 3);
#pragma unroll
                            for (int t = 0; t < TT; t++) {
                                const uint4 x = xs[4 * f * TT + ((g * TT + t) ^ (f & kMix))];
                                sum[t] = dot2(w0, x.x, sum[t]);
                                sum[t] = dot2(w1, x.y, sum[t]);
                                sum[t] = dot2(w2, x.z, sum[t]);
                                sum[t] = dot2(w3, x.w, sum[t]);
                            }
                        } else {
                            if (f < 7) {
#pragma unroll
                                for (int t = 0; t < TB; t++)
                                    xf[(f + 1) & 1][t] = tokens(f + 1, t);
                            }
                            const bf16x8_t wf = weights8(d, s);
#pragma unroll
                            for (int t = 0; t < TB; t++)
                                acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[f & 1][t], acc[t], 0, 0, 0);
                            if (TB > 1)
                                __builtin_amdgcn_sched_barrier(0);   // and not all reads first
                        }
                    }
                    if constexpr (Plan::kDot) {
#pragma unroll
                        for (int t = 0; t < TT; t++)
                            acc[0][t] = __builtin_fmaf(sum[t], rest, acc[0][t]);
                        if (TT == 2)
                            __builtin_amdgcn_sched_barrier(0);
                    }
                }
            };
            for (int st = 0; st < stages; st++) {
                // tokens that fit one stage stay for all blocks
                if (stages > 1 || block == (int)blockIdx.x) {
                    __syncthreads();
                    store_tokens(turned(st));
                    __syncthreads();
                    if (st + 1 < stages)
                        load_tokens(turned(st + 1));
                }
#pragma unroll
                for (int j = 0; j < D; j++) {
                    const int c = turned(st) * Plan::kFit + ks + j * KS;
                    if (c < nchunk)
                        work(w[j], ks + j * KS, c);
                    if (Plan::kDot)
                        __builtin_amdgcn_sched_barrier(0);   // one chunk's fragments at a time
                    // the next stage's chunk, or the next block's
                    const int ahead = turned(st + 1 < stages ? st + 1 : 0) * Plan::kFit + ks + j * KS;
                    if (st + 1 < stages && ahead < nchunk)
                        aim.fetch(w[j], ahead);
                    else if (st + 1 == stages && more && ahead < nchunk)
                        next.fetch(w[j], ahead);
                }
            }

            if constexpr (Plan::kDot) {
                // lane (r, g): row r's sums over its k; over g, then over KS
#pragma unroll
                for (int t = 0; t < TT; t++) {
                    acc[0][t] += __shfl_xor(acc[0][t], 16);
                    acc[0][t] += __shfl_xor(acc[0][t], 32);
                    acc[0][t] *= 2.f;            // (rest)
                }
                float *part = reinterpret_cast<float *>(lds + Plan::kTokens);
                __syncthreads();
                if (g < TT)
                    part[(wave * TT + g) * 16 + r] = g ? acc[0][1] : acc[0][0];
                __syncthreads();
                const int v = tid / (16 * TT), t = tid / 16 % TT, n = 16 * v + tid % 16;
                if (v < Plan::WN && t < count && n0 + n < a.N) {
                    float sum = part[(v * KS * TT + t) * 16 + tid % 16];
#pragma unroll
                    for (int k = 1; k < KS; k++)
                        sum += part[((v * KS + k) * TT + t) * 16 + tid % 16];
                    store_mv(a, (int64_t)(EXPERTS ? slot[t] : from + t) * a.N + n0 + n, sum * sg);
                }
            }
            // the KS partial sums, token tile by token tile; lane (r, g), register
            // j of a tile: weight row 4 g + j, token r
#pragma unroll
            for (int t = 0; t < (Plan::kDot ? 0 : TB); t++) {
                f32x4_t *part = reinterpret_cast<f32x4_t *>(lds + Plan::kTokens);
                __syncthreads();
                part[tid] = acc[t];
                __syncthreads();
                if (tid < Plan::WN * 64) {
                    const int v = tid >> 6;
                    f32x4_t sum = part[v * KS * 64 + L];
#pragma unroll
                    for (int k = 1; k < KS; k++)
                        sum += part[(v * KS + k) * 64 + L];
                    const int tok = 16 * t + r;
                    const int n = n0 + 16 * v + 4 * g;
                    if (tok < count && n < a.N) {
                        const int64_t o = (int64_t)(EXPERTS ? slot[tok] : from + tok) * a.N + n;
                        sum *= sg;
                        if ((a.N & 3) == 0) {
                            if (a.out_f32)
                                *reinterpret_cast<f32x4_t *>(static_cast<float *>(a.y) + o) = sum;
                            else
                                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.y) + o) =
                                    make_uint2(bf16_pair(sum[0], sum[1]), bf16_pair(sum[2], sum[3]));
                        } else {
                            for (int j = 0; j < 4 && n + j < a.N; j++)
                                store_mv(a, o + j, sum[j]);
                        }
                    }
                }
            }
        }
        if (EXPERTS)
            from = slot[count - 1] + 1;
        else
            from += (int)gridDim.y * TT;
        __syncthreads();
    }
}

// Weights of fewer than 16 bytes of codes or 4 of scales, or fewer than 8 token
// elements, which the loads above do not fit: a lane per output, bytes one by one (K is
// 48 at most).  There may be many outputs: one token of 7 by 2^23 rows.
constexpr int kTinyThreads = 256;
__global__ __launch_bounds__(kTinyThreads) void mv_tiny_kernel(const MvArgs a)
{
    const int64_t nb = (a.K + 15) / 16, pitch = (a.K + 1) / 2, all = (int64_t)a.T * a.top * a.N;
    for (int64_t i = (int64_t)blockIdx.x * kTinyThreads + threadIdx.x; i < all;
         i += (int64_t)gridDim.x * kTinyThreads) {
        const int64_t p = i / a.N, n = i - p * a.N;
        const int e = a.experts ? a.experts[p] : 0;
        float sum = 0.f;
        if (e >= 0 && e < a.G) {
            const int64_t row = (int64_t)e * a.N + n;
            for (int k = 0; k < a.K; k++) {
                const uint32_t code = a.qw[row * pitch + (k >> 1)] >> (4 * (k & 1));
                const float s = __builtin_amdgcn_cvt_f32_fp8((int)a.sw[row * nb + (k >> 4)], 0);
                const f32x2v_t v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 0);
                sum += __uint_as_float((uint32_t)a.x[p / a.top * a.K + k] << 16) * (v[0] * s);
            }
            sum *= a.sg[e];
        }
        store_mv(a, i, sum);
    }
}

template <int TT, bool EXPERTS, bool FEW>
hipError_t launch_one(MvArgs a, hipStream_t stream)
{
    using Plan = MvPlan<TT, EXPERTS, FEW>;
    const int64_t slots = (int64_t)a.T * a.top, blocks = (a.N + Plan::kRows - 1) / Plan::kRows;
    if (Plan::kLds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(mv_kernel<TT, EXPERTS, FEW>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, Plan::kLds);
        if (e != hipSuccess)
            return e;
    }
    // Few slots: by slot, so that no workgroup is started for an expert that
    // nobody picked.
    a.by_slot = EXPERTS && slots <= a.G;
    const int64_t tiles = (a.T + TT - 1) / TT;
    const int64_t ny = !EXPERTS ? (tiles < 4096 ? tiles : 4096) : a.by_slot ? slots : a.G + 1;
    // Experts' tokens whose k fits one stage are staged once for all of a
    // workgroup's blocks: then as many workgroups as fit the CUs (two each), so
    // that weights are always under way.  Otherwise a workgroup per block.
    int64_t nx = blocks;
    if (EXPERTS && a.K <= Plan::kFit * kMvChunk) {
        const int64_t each_y = a.by_slot ? slots : a.G;      // (zero rows take no time)
        const int64_t fill = 2 * 256 / each_y > 1 ? 2 * 256 / each_y : 1;
        const int64_t each = (blocks + fill - 1) / fill;
        nx = (blocks + each - 1) / each;
    }
    hipLaunchKernelGGL((mv_kernel<TT, EXPERTS, FEW>), dim3((unsigned)nx, (unsigned)ny), dim3(kMvThreads),
                       Plan::kLds, stream, a);
    return hipGetLastError();
}

template <int TT>
hipError_t launch(const MvArgs &a, bool few, hipStream_t stream)
{
    if (a.experts)
        return launch_one<TT, true, false>(a, stream);
    if constexpr (TT <= 16) {
        if (few)
            return launch_one<TT, false, true>(a, stream);
    }
    return launch_one<TT, false, false>(a, stream);
}

}  // namespace

hipError_t launch_mv(const MvArgs &a, hipStream_t stream)
{
    const MvChoice c = mv_choose(a);
    if (c.tokens == 0) {
        const int64_t n = ((int64_t)a.T * a.top * a.N + kTinyThreads - 1) / kTinyThreads;
        hipLaunchKernelGGL(mv_tiny_kernel, dim3((unsigned)(n < 65536 ? n : 65536)), dim3(kTinyThreads), 0,
                           stream, a);
        return hipGetLastError();
    }
    return c.tokens == 1    ? launch<1>(a, c.few, stream)
           : c.tokens == 2  ? launch<2>(a, c.few, stream)
           : c.tokens == 8  ? launch<8>(a, c.few, stream)
           : c.tokens == 16 ? launch<16>(a, c.few, stream)
           : c.tokens == 32 ? launch<32>(a, c.few, stream)
                            : launch<64>(a, c.few, stream);
}

}  // namespace mxk
