// mm_tile.h -- the tiled kernel of the MXFP8 products: rows aligned to 16 bytes.
//
// Y_g[m][n] = sum_k A_g[m][k] B_g[n][k] over blocks of 32 k that share a scale.
// gfx950's block-scaled MFMA (32 x 32 x 64) takes the codes and scale bytes as
// the casts wrote them.  A workgroup of 4 waves (2 x 2) owns TM x TN outputs.
// The codes come into LDS 128 k at a time by loads that write LDS directly (no
// registers), two buffers in turn; fragments are double buffered in registers,
// so that a step's MFMAs run while the next step's fragments are read:
//
//   step 0 of tile t:  MFMAs on F0, reads of F1 (step 1 of tile t)
//   wait for the loads of tile t + 1 and the reads of F1; barrier: every wave is
//   done with tile t's buffer, and tile t + 1 is there; load tile t + 2
//   step 1 of tile t:  MFMAs on F1, reads of F0 (step 0 of tile t + 1)
//
// LDS holds rows of 128 bytes; 16-byte chunk c of a row sits in slot c ^ s(row),
// so that the 8 lanes a read serves together take 8 different slots.  The
// direct loads place lanes' 16 bytes one after the other, so the exchange is
// done on the global side: a lane loads the chunk that belongs in its slot.
//
// B's rows are dealt to the lanes in pairs: of two neighbouring 32-column
// tiles, lane r holds columns 2r (first tile) and 2r + 1 (second), so that the
// outputs leave as whole 128-byte lines from registers.
#pragma once

#include "bufio.h"
#include "mm_common.h"

namespace mxk {

// Waits until at most the given counts are outstanding, with no motion of
// memory operations across.
__device__ __forceinline__ void wait_all_and_barrier()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

typedef unsigned int mm_rsrc_t __attribute__((ext_vector_type(4)));

// 64 lanes x 16 bytes from base + voff + soff into LDS at lds + 16 * lane.
// Asynchronous: counted by vmcnt, which the caller waits for.  Written in
// assembly because the compiler otherwise waits for every outstanding load
// before the next read of any LDS.  (m0 is reserved: the compiler sets it right
// before any use of its own.)
__device__ __forceinline__ void load_to_lds(mm_rsrc_t rsrc, uint32_t voff, uint32_t soff,
                                            uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc), "s"(soff));
}

__device__ __forceinline__ mm_rsrc_t rows_rsrc(const uint8_t *p)
{
    // no bound but kDeadRow: every other offset lies in the operand
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    return mm_rsrc_t{(uint32_t)u, (uint32_t)(u >> 32) & 0xFFFFu, 0xFFFFFF00u, 0x00020000u};
}
constexpr uint32_t kDeadRow = 0xFFFFFFF0u;   // out of every range: loads zeros

// Where the scales of one operand's rows lie for a workgroup tile, 8 blocks
// (256 k) at a time: two 4-byte loads per row, `second` bytes apart, at a lane's
// offset from a base that moves by `move` bytes per 8 blocks.  Compact, they are
// the row's 8 bytes, taken from up to 7 bytes before where the array would end
// inside them; tiled, the words of the row's two lanes (blocks 2j, 2j + 1).
struct ScaleRows {
    const uint8_t *base;
    int64_t left;              // compact: bytes from base to 8 before the array's end
    uint32_t second;
    int64_t move;

    __device__ __forceinline__ ScaleRows(const uint8_t *s, int64_t bytes, int64_t rows, int64_t nb,
                                         int64_t r0, int tiled)
        : base(s + (tiled ? (r0 >> 5) * 256 : r0 * nb)),
          left(tiled ? kMaxRecords : bytes - 8 - r0 * nb), second(tiled ? 128 : 4),
          move(tiled ? ((rows + 31) >> 5) * 256 : 8)
    {
    }
    // Offset of row r0 + d from the base.
    __device__ __forceinline__ static uint32_t row(int64_t rows, int64_t nb, int64_t r0, int d, int tiled)
    {
        const int last = (int)(rows - 1 - r0 < 1024 ? rows - 1 - r0 : 1024);
        d = d < last ? d : last;
        return tiled ? (uint32_t)((d >> 5) * 256 + 4 * (d & 31)) : (uint32_t)(d * nb);
    }
    __device__ __forceinline__ uint32_t limit(int bt) const
    {
        const int64_t room = left - bt * 8;
        return (uint32_t)(room < kMaxRecords ? room : kMaxRecords);
    }
    __device__ __forceinline__ void load(uint32_t off, int bt, uint32_t &x, uint32_t &y) const
    {
        const uint8_t *p = base + bt * move;
        const uint32_t lim = limit(bt), o = off < lim ? off : lim;
        __builtin_memcpy(&x, p + o, 4);
        __builtin_memcpy(&y, p + (o + second), 4);
    }
    // The row's 8 bytes (the lanes' two words) of what load gave.
    __device__ __forceinline__ uint64_t value(uint32_t off, int bt, uint32_t x, uint32_t y) const
    {
        const uint32_t lim = limit(bt), d = off < lim ? 0 : off - lim;
        return ((uint64_t)y << 32 | x) >> (8 * d);
    }
};

template <int FA, int FB, int J>
__device__ __forceinline__ f32x16_t mfma_mx(i32x8_t a, i32x8_t b, f32x16_t c, uint32_t sa, uint32_t sb)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, FA, FB, J, (int)sa, J, (int)sb);
}

template <MmMode MODE, int FA, int FB, int TM, int TN>
struct MmKernel {
    static constexpr int MT = TM / 64, NT = TN / 64;      // 32-row tiles of a wave
    static constexpr int kBuf = (TM + TN) * 128;          // bytes of an LDS buffer
    static constexpr int kLoads = (TM + TN) / 32;         // loads of a wave per tile
    static_assert(NT % 2 == 0, "column tiles come in pairs");

    struct Frags {
        i32x8_t a[MT], b[NT];
    };

    const MmArgs &a;
    const MmTile &w;
    const ScaleRows ssa, ssb;
    uint8_t *lds;
    uint32_t lds0;                 // its LDS address
    int L, wave, h, r;
    int wm, wn;                    // the wave's rows and columns in the tile
    uint32_t voff[kLoads];
    mm_rsrc_t ra, rb;
    uint32_t sel, sel1;            // how the words come out of a row's 8 scale bytes
    f32x16_t acc[MT][NT];
    uint32_t off_a[MT], off_b[NT];
    uint32_t raw_a[MT][2], raw_b[NT][2];
    // kMx: the words of the lane's blocks (byte j: step j of the next four);
    // kExact: those of even blocks and of odd ones
    static constexpr int W = MODE == kMx ? 1 : 2;
    uint32_t sa[MT][W], sb[NT][W];

    // Row of B in the workgroup tile that lane r of the wave's column tile j
    // holds.
    __device__ __forceinline__ int brow(int j) const { return wn + 64 * (j >> 1) + 2 * r + (j & 1); }

    // Load i of the wave for tile t (zeros for one behind the last).
    __device__ __forceinline__ void issue(int t, int i) const
    {
        const uint32_t k0 = 128u * (uint32_t)t;
        const uint32_t dst = lds0 + (uint32_t)(t & 1) * kBuf;
        // 16-byte chunks behind the rows' ends are zeros
        const uint32_t left = k0 < w.K ? (uint32_t)(w.K - k0) : 0;
        const uint32_t v = 16 * chunk(i) < left ? voff[i] : kDeadRow;
        load_to_lds(is_a(i) ? ra : rb, v, k0, dst + (uint32_t)row8(i) * 128);
    }
    // The wave's load i fills 8 rows of LDS, from row8(i) on: a share of A's TM
    // rows, then of B's TN rows behind them.
    static constexpr int kLoadsA = TM / 32;
    __device__ static constexpr bool is_a(int i) { return i < kLoadsA; }
    __device__ __forceinline__ int row8(int i) const
    {
        return 8 * (is_a(i) ? wave * kLoadsA + i : TM / 8 + wave * (TN / 32) + i - kLoadsA);
    }
    // The chunk of its row that lane L loads (the slot's exchange, above).
    __device__ __forceinline__ uint32_t chunk(int i) const
    {
        const int row = row8(i) + (L >> 3);
        return (uint32_t)((L & 7) ^ ((is_a(i) ? row : row >> 1) & 7));
    }

    __device__ __forceinline__ i32x8_t frag_a(int t, int s, int i) const
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(lds + (t & 1) * kBuf) + (wm + 32 * i + r) * 8;
        return join(p[(4 * s + h) ^ (r & 7)], p[(4 * s + 2 + h) ^ (r & 7)]);
    }
    __device__ __forceinline__ i32x8_t frag_b(int t, int s, int j) const
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(lds + (t & 1) * kBuf) + (TM + brow(j)) * 8;
        return join(p[(4 * s + h) ^ (r & 7)], p[(4 * s + 2 + h) ^ (r & 7)]);
    }
    // One of a step's MT + NT fragments.
    __device__ __forceinline__ void read(Frags &f, int t, int s, int i) const
    {
        if (i < NT)
            f.b[i] = frag_b(t, s, i);
        else
            f.a[i - NT] = frag_a(t, s, i - NT);
    }

    __device__ __forceinline__ void fetch_scales(int bt)
    {
#pragma unroll
        for (int i = 0; i < MT; i++)
            ssa.load(off_a[i], bt, raw_a[i][0], raw_a[i][1]);
#pragma unroll
        for (int j = 0; j < NT; j++)
            ssb.load(off_b[j], bt, raw_b[j][0], raw_b[j][1]);
    }
    __device__ __forceinline__ void settle_scales()
    {
#pragma unroll
        for (int i = 0; i < MT; i++)
            asm volatile("" : "+v"(raw_a[i][0]), "+v"(raw_a[i][1]));
#pragma unroll
        for (int j = 0; j < NT; j++)
            asm volatile("" : "+v"(raw_b[j][0]), "+v"(raw_b[j][1]));
    }
    // The words of blocks 8 bt on; bytes of blocks behind the last one become 0.
    __device__ __forceinline__ void take_scales(int bt)
    {
        const int64_t keep = w.nb - 8 * bt;
        const uint64_t mask = keep >= 8 || a.tiled ? ~0ull : (1ull << (8 * keep)) - 1;
#pragma unroll
        for (int i = 0; i < MT; i++)
            words(sa[i], ssa.value(off_a[i], bt, raw_a[i][0], raw_a[i][1]) & mask);
#pragma unroll
        for (int j = 0; j < NT; j++)
            words(sb[j], ssb.value(off_b[j], bt, raw_b[j][0], raw_b[j][1]) & mask);
    }
    __device__ __forceinline__ void words(uint32_t (&o)[W], uint64_t v) const
    {
        const uint32_t hi = (uint32_t)(v >> 32), lo = (uint32_t)v;
        if (MODE == kMx) {
            o[0] = __builtin_amdgcn_perm(hi, lo, sel);
        } else {
            o[0] = __builtin_amdgcn_perm(hi, lo, sel);
            o[W - 1] = __builtin_amdgcn_perm(hi, lo, sel1);
        }
    }

    // The MFMAs of one step on f, with the reads of the next step's fragments
    // between them.
    template <int J, bool LOAD>
    __device__ __forceinline__ void step(const Frags &f, Frags &next, int tn, int sn, int tl)
    {
        if (MODE == kMx) {
            int k = 0;
#pragma unroll
            for (int i = 0; i < MT; i++)
#pragma unroll
                for (int j = 0; j < NT; j++) {
                    acc[i][j] = mfma_mx<FA, FB, J>(f.a[i], f.b[j], acc[i][j], sa[i][0], sb[j][0]);
                    if (LOAD && k < kLoads)
                        issue(tl, k);
                    if (k < MT + NT)
                        read(next, tn, sn, k);
                    k++;
                    __builtin_amdgcn_sched_barrier(0);
                }
            return;
        }
        // four parts of 8 codes per lane: block p, half q.  A part's B
        // fragments and the next A fragment are converted between the MFMAs
        // before them.
        bf16x8_t b[2][NT], ca = conv_a<J>(f, 0, 0);
#pragma unroll
        for (int j = 0; j < NT; j++)
            b[0][j] = conv_b<J>(f, j, 0);
#pragma unroll
        for (int part = 0; part < 4; part++)
#pragma unroll
            for (int i = 0; i < MT; i++) {
                const bf16x8_t x = ca;
#pragma unroll
                for (int j = 0; j < NT; j++) {
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, b[part & 1][j], acc[i][j],
                                                                        0, 0, 0);
                    if (j == 0 && i + 1 < MT)
                        ca = conv_a<J>(f, i + 1, part);
                    if (j == 0 && i + 1 == MT && part < 3)
                        ca = conv_a<J>(f, 0, part + 1);
                    if (j == 1 && part < 3) {
#pragma unroll
                        for (int jj = 0; jj < NT; jj++)
                            if (jj * MT / NT == i)
                                b[(part & 1) ^ 1][jj] = conv_b<J>(f, jj, part + 1);
                    }
                    if (LOAD && part * MT * NT + i * NT + j < kLoads)
                        issue(tl, part * MT * NT + i * NT + j);
                    if (j == NT - 1) {
#pragma unroll
                        for (int k = 0; k < MT + NT; k++)
                            if (k * 4 * MT / (MT + NT) == part * MT + i)
                                read(next, tn, sn, k);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
    }
    template <int J>
    __device__ __forceinline__ bf16x8_t conv_a(const Frags &f, int i, int part) const
    {
        const float s = scale_float((sa[i][(part >> 1) * (W - 1)] >> (8 * J)) & 255);
        return bf16_of_codes8<FA>((uint32_t)f.a[i][2 * part], (uint32_t)f.a[i][2 * part + 1], s);
    }
    template <int J>
    __device__ __forceinline__ bf16x8_t conv_b(const Frags &f, int j, int part) const
    {
        const float s = scale_float((sb[j][(part >> 1) * (W - 1)] >> (8 * J)) & 255);
        return bf16_of_codes8<FB>((uint32_t)f.b[j][2 * part], (uint32_t)f.b[j][2 * part + 1], s);
    }

    template <int J>
    __device__ __forceinline__ void tile(Frags &f0, Frags &f1, int t)
    {
        step<J, false>(f0, f1, t, 1, 0);
        wait_all_and_barrier();
        // the scale bytes fetched for the next four steps are here: say so
        // before more loads are under way, which the compiler would wait for
        if (J == 2)
            settle_scales();
        step<J + 1, true>(f1, f0, t + 1, 0, t + 2);
    }

    __device__ __forceinline__ void run()
    {
        // an even number of tiles: one behind the last k holds zeros
        const int nt = 2 * (int)((w.K + 255) / 256);
        const uint32_t even = a.tiled ? 0x03020100u : 0x06040200u;
        const uint32_t odd = a.tiled ? 0x07060504u : 0x07050301u;
        sel = MODE == kMx && h ? odd : even;
        sel1 = odd;
        ra = rows_rsrc(w.qa + w.m0 * w.K);
        rb = rows_rsrc(w.qb + w.n0 * w.K);
#pragma unroll
        for (int i = 0; i < kLoads; i++) {
            const int64_t last = is_a(i) ? w.M - 1 - w.m0 : a.N - 1 - w.n0;
            const int64_t rr = row8(i) + (L >> 3) - (is_a(i) ? 0 : TM);
            voff[i] = (uint32_t)((rr < last ? rr : last) * w.K) + 16 * chunk(i);
        }
#pragma unroll
        for (int i = 0; i < MT; i++) {
            off_a[i] = ScaleRows::row(w.M, w.nb, w.m0, wm + 32 * i + r, a.tiled);
#pragma unroll
            for (int j = 0; j < NT; j++)
                acc[i][j] = f32x16_t{};
        }
#pragma unroll
        for (int j = 0; j < NT; j++)
            off_b[j] = ScaleRows::row(a.N, w.nb, w.n0, brow(j), a.tiled);
        if (nt > 0) {
            Frags f0, f1;
            fetch_scales(0);
            take_scales(0);
#pragma unroll
            for (int i = 0; i < kLoads; i++)
                issue(0, i);
            wait_all_and_barrier();
#pragma unroll
            for (int i = 0; i < kLoads; i++)
                issue(1, i);
#pragma unroll
            for (int i = 0; i < MT + NT; i++)
                read(f0, 0, 0, i);
            int t = 0;
            do {
                const int next = t + 2 < nt ? (t >> 1) + 1 : t >> 1;
                tile<0>(f0, f1, t);
                fetch_scales(next);
                tile<2>(f0, f1, t + 1);
                take_scales(next);
                t += 2;
            } while (t < nt);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the loads of no tile
        store();
    }

    // Writes the outputs (kMx: bf16, kExact: fp32, with ADD added to what is
    // there); PAIR: a lane's two neighbouring columns in one store, where rows
    // start at an even element.
    template <bool PAIR, bool ADD>
    __device__ __forceinline__ void store_form() const
    {
        // lane (r, h), register e: row 8 (e / 4) + 4 h + e % 4.  One descriptor
        // per 32 rows, which ends with the group's last row; columns from N on
        // get an offset behind it.
        constexpr int size = MODE == kMx ? 2 : 4;
        const uint32_t pitch = (uint32_t)a.N * size;
#pragma unroll
        for (int i = 0; i < MT; i++) {
            const int64_t m = w.m0 + wm + 32 * i;
            const int64_t at = w.y0 + m * a.N, end = w.y0 + (w.M < m + 32 ? w.M : m + 32) * a.N;
            const rsrc_t y = make_rsrc(a.y, at * size, end * size);
#pragma unroll
            for (int j = 0; j < NT; j += 2) {
                const int64_t n = w.n0 + brow(j);
                const uint32_t off = n < a.N ? (uint32_t)n * size + 4 * h * pitch : kDead;
                const uint32_t off1 = n + 1 < a.N ? off + size : kDead;
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    const float v0 = acc[i][j][e], v1 = acc[i][j + 1][e];
                    const uint32_t down = (uint32_t)(8 * (e >> 2) + (e & 3)) * pitch;
                    if (MODE == kMx && PAIR) {
                        buf_store4(y, off + down, bf16_pair(v0, v1));
                    } else if (MODE == kMx) {
                        buf_store2(y, off + down, (uint16_t)bf16_pair(v0, 0.f));
                        buf_store2(y, off1 + down, (uint16_t)bf16_pair(v1, 0.f));
                    } else if (PAIR) {
                        float2 o = make_float2(0.f, 0.f);
                        if (ADD)
                            o = buf_load_f2(y, off + down);
                        buf_store8(y, off + down, make_uint2(__float_as_uint(ADD ? o.x + v0 : v0),
                                                             __float_as_uint(ADD ? o.y + v1 : v1)));
                    } else {
                        const float o0 = ADD ? buf_load_f(y, off + down) : 0.f;
                        const float o1 = ADD ? buf_load_f(y, off1 + down) : 0.f;
                        buf_store4(y, off + down, __float_as_uint(ADD ? o0 + v0 : v0));
                        buf_store4(y, off1 + down, __float_as_uint(ADD ? o1 + v1 : v1));
                    }
                }
            }
        }
    }
    __device__ __forceinline__ static float2 buf_load_f2(rsrc_t y, uint32_t off)
    {
        const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(y, (int)off, 0, 0);
        return make_float2(__uint_as_float(v[0]), __uint_as_float(v[1]));
    }
    __device__ __forceinline__ static float buf_load_f(rsrc_t y, uint32_t off)
    {
        return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(y, (int)off, 0, 0));
    }

    __device__ __forceinline__ void store() const
    {
        const bool pair = (a.N & 1) == 0;
        if (MODE == kMx)
            pair ? store_form<true, false>() : store_form<false, false>();
        else if (a.accumulate)
            pair ? store_form<true, true>() : store_form<false, true>();
        else
            pair ? store_form<true, false>() : store_form<false, false>();
    }
};

template <MmMode MODE, int FA, int FB, int TM, int TN>
__global__ __launch_bounds__(256, 1) void mm_tile_kernel(const MmArgs a, const MmTable t)
{
    extern __shared__ uint8_t mm_lds[];
    typedef __attribute__((address_space(3))) uint8_t lds_byte_t;
    const MmTile w = mm_tile(a, t, mm_xcd_order((int)blockIdx.x, (int)gridDim.x), TM, TN);
    MmKernel<MODE, FA, FB, TM, TN> k{a, w, ScaleRows(w.sa, w.sa_left, w.M, w.nb, w.m0, a.tiled),
                               ScaleRows(w.sb, w.sb_left, a.N, w.nb, w.n0, a.tiled)};
    k.lds = mm_lds;
    k.lds0 = (uint32_t)(uintptr_t)(lds_byte_t *)mm_lds;
    k.L = (int)threadIdx.x & 63;
    k.wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    k.h = k.L >> 5;
    k.r = k.L & 31;
    k.wm = (k.wave >> 1) * (TM / 2);
    k.wn = (k.wave & 1) * (TN / 2);
    k.run();
}

template <MmMode MODE, int FA, int FB, int TM, int TN>
hipError_t launch_mm_tile_one(const MmArgs &a, const MmTable &t, hipStream_t stream)
{
    constexpr int lds = 2 * (TM + TN) * 128;
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void *>(mm_tile_kernel<MODE, FA, FB, TM, TN>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL((mm_tile_kernel<MODE, FA, FB, TM, TN>), dim3((unsigned)t.tile0[t.count]),
                       dim3(256), lds, stream, a, t);
    return hipGetLastError();
}

template <MmMode MODE, int TM, int TN>
hipError_t launch_mm_tile_mode(const MmArgs &a, const MmTable &t, hipStream_t stream)
{
    if (!a.a_e5m2 && !a.b_e5m2)
        return launch_mm_tile_one<MODE, 0, 0, TM, TN>(a, t, stream);
    if (a.a_e5m2 && !a.b_e5m2)
        return launch_mm_tile_one<MODE, 1, 0, TM, TN>(a, t, stream);
    if (!a.a_e5m2)
        return launch_mm_tile_one<MODE, 0, 1, TM, TN>(a, t, stream);
    return launch_mm_tile_one<MODE, 1, 1, TM, TN>(a, t, stream);
}

}  // namespace mxk
