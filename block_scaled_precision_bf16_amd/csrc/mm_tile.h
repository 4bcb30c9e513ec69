// mm_tile.h -- the tiled kernel of the MXFP8 products: rows aligned to 16 bytes.
//
// Y_g[m][n] = sum_k A_g[m][k] B_g[n][k] over blocks of 32 k that share a scale.
// gfx950's block-scaled MFMA (32 x 32 x 64) takes the codes and scale bytes as
// the casts wrote them.  A workgroup of 4 waves (2 x 2) owns TM x TN outputs.
// The codes come into LDS 128 k at a time by loads that write LDS directly (no
// registers), into NB buffers in turn; fragments are double buffered in registers,
// so that a step's MFMAs run while the next step's fragments are read:
//
//   step 0 of tile t:  MFMAs on F0, reads of F1 (step 1 of tile t)
//   wait for the loads of tile t + 1 and the reads of F1; barrier: every wave is
//   done with tile t's buffer, and tile t + 1 is there; load tile t + NB
//   step 1 of tile t:  MFMAs on F1, reads of F0 (step 0 of tile t + 1)
//
// LDS holds rows of 128 bytes, two of which use its 64 banks once; 16-byte chunk c of
// row R sits in slot c ^ (R / 2 mod 8), so that the 16 lanes (rows) a read serves
// together use all banks.  The direct loads place lanes' 16 bytes one after the other, so
// the exchange is done on the global side: a lane loads the chunk that belongs in
// its slot.
//
// B's rows are dealt to the lanes in pairs: of two neighbouring 32-column
// tiles, lane r holds columns 2r (first tile) and 2r + 1 (second), so that the
// outputs leave as whole 128-byte lines from registers.  In LDS the first tile's rows
// come first.
//
// Measured: 8192^3 to bf16 in 440 - 460 us back to back, by the card, 2.4 - 2.5 PFLOP/s
// (a library's fp8 product without block scales reaches 2.8 - 2.96), 397 in short
// bursts; the matrix cores are busy 70% of the time at the clock that the power limit
// leaves them (1.7 - 2.0 GHz).  To fp32 (twice the MFMA time) 762 us in bursts, of which
// the look for far blocks takes 11; with one in every step it takes 3.4 times as long,
// with zeros for half of A's rows, whose scale bytes have to be told from those, 9 %
// longer.  A round of 256 tiles takes 8 us + 1.5 us for 128 k; its outputs alone are 34
// MB, about 7 us.  A last round of 128 x 128 parts takes
// 0.55 us for 128 k, one of 256 x 128 parts 1.0 us: 64 tiles of 8192 k take 39 us in
// parts and 92 us whole.  With two buffers instead of four they take 50 us.
#pragma once

#include "mm_common.h"

namespace mxk {

// Waits until at most N loads (and no LDS reads) are outstanding and for the other
// waves, with no motion of memory operations across.
template <int N>
__device__ __forceinline__ void wait_and_barrier()
{
    static_assert(N < 64, "vmcnt");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(N) : "memory");
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

// The same with 4 bytes a lane.
__device__ __forceinline__ void load_words_to_lds(mm_rsrc_t rsrc, uint32_t voff, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds"
                 :
                 : "s"(lds), "v"(voff), "s"(rsrc));
}

// `bytes` bytes at p.
__device__ __forceinline__ mm_rsrc_t bytes_rsrc(const uint8_t *p, uint32_t bytes)
{
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    return mm_rsrc_t{(uint32_t)u, (uint32_t)(u >> 32) & 0xFFFFu, bytes, 0x00020000u};
}

// Rows of `pitch` bytes at p, of which `rows` exist: a load's voff is a place in
// them, its soff a step along k that stays inside the row, so whether or not the
// bound is compared with soff too, rows behind the last one load zeros.
__device__ __forceinline__ mm_rsrc_t rows_rsrc(const uint8_t *p, int64_t rows, int64_t pitch)
{
    return bytes_rsrc(p, (uint32_t)(rows < 256 ? rows : 256) * (uint32_t)pitch);
}
constexpr uint32_t kDeadRow = 0xFFFFFFF0u;   // behind every bound: loads zeros

// PAIRED: two workgroups share a CU and its LDS.
template <MmMode MODE, int FA, int FB, int TM, int TN, bool TILED, bool PAIRED = false>
struct MmKernel {
    static constexpr int MT = TM / 64, NT = TN / 64;      // 32-row tiles of a wave
    static constexpr int kBuf = (TM + TN) * 128;          // bytes of an LDS buffer
    static constexpr int kLoads = (TM + TN) / 32;         // loads of a wave per tile
    // LDS buffers: smaller tiles take less time, and have more of them under way.
    // (Compact scales come through registers, which the compiler waits for with
    // all loads: two buffers.)
    static constexpr int NB = !TILED || PAIRED ? 2 : TM == 128 ? 4 : TN == 128 ? 3 : 2;
    // Scales of 8 blocks and all rows; of the tiled ones, (NB + 1) / 2 buffers and
    // a wave's share of the loads, which go with those of the first of two tiles.
    static constexpr int kScales = (TM + TN) * 8;
    static constexpr int kScaleLoads = TILED ? (TM + TN) / 128 : 0;
    static constexpr int kLds = NB * kBuf + (TILED ? (NB + 1) / 2 : 2) * kScales;
    // Loads of the tiles from..to (relative to an even one).
    static constexpr int loads(int from, int to)
    {
        int n = 0;
        for (int u = from; u <= to; u++)
            n += kLoads + (u % 2 == 0 ? kScaleLoads : 0);
        return n;
    }
    static_assert(NT % 2 == 0, "column tiles come in pairs");

    struct Frags {
        i32x8_t a[MT], b[NT];
    };

    const MmArgs &a;
    const MmTile &w;
    const ByteRows<8> sra, srb;    // !TILED: the scales
    uint8_t *lds;
    uint32_t lds0;                 // its LDS address
    int L, wave, h, r;
    int wm, wn;                    // the wave's rows and columns in the tile
    uint32_t voff[4];              // A's loads of even and odd numbers, and B's
    mm_rsrc_t ra, rb;
    uint32_t last_a, last_b;       // the operands' last rows in the tile
    int nt, phase;                 // tiles of k, the first one
    uint32_t sel;                  // compact: how a word comes out of 8 scale bytes
    // Scales, for 4 steps (2 tiles) at a time, in LDS.  Tiled: direct loads of the
    // words as they lie.  Compact: a thread loads the 8 bytes of one row of A and of
    // one of B and puts them there, from where the lanes make their words.
    uint32_t off_a, off_b, raw_a[2], raw_b[2];     // compact
    static constexpr int W = MODE == kMx ? 1 : 2;
    // kMx: the words of the lane's blocks (byte j: step j of the next four);
    // kExact: those of even blocks and of odd ones
    uint32_t sa[MT][W], sb[NT][W];
    int at_a[MT], at_b[NT];        // kExact, tiled: where a lane's words are
    bool odd_scales;               // kExact: some of them may make a block far (wave-uniform)
    f32x16_t acc[MT][NT];

    // Row of B in the workgroup tile that lane r of the wave's column tile j
    // holds.
    __device__ __forceinline__ int brow(int j) const { return wn + 64 * (j >> 1) + 2 * r + (j & 1); }

    // The tile of k that comes in place t: workgroups start at different ones
    // (see run()).
    __device__ __forceinline__ int turned(int t) const
    {
        return t >= nt ? t : t + phase < nt ? t + phase : t + phase - nt;
    }
    // Where in LDS the tile in place t goes.
    __device__ __forceinline__ uint32_t buf(int t) const { return (uint32_t)t % NB * kBuf; }
    // Tiled: where the scales of the tiles in places t (even) and t + 1 go.
    __device__ __forceinline__ uint32_t scale_buf(int t) const
    {
        return NB * kBuf + (uint32_t)(t >> 1) % ((NB + 1) / 2) * kScales;
    }
    // Load i of the wave for the tile in place t (zeros behind the last).
    __device__ __forceinline__ void issue(int t, int i) const
    {
        const uint32_t k0 = 128u * (uint32_t)turned(t), dst = lds0 + buf(t);
        // 16-byte chunks behind the rows' ends are zeros
        const uint32_t left = k0 < w.K ? (uint32_t)(w.K - k0) : 0;
        const uint32_t v = 16 * chunk(i) < left ? offset(i) : kDeadRow;
        load_to_lds(is_a(i) ? ra : rb, v, k0, dst + (uint32_t)row8(i) * 128);
    }
    // The wave's loads of the scales for the tiles in places t and t + 1: of each
    // operand's 32-row tiles, one load each.
    __device__ __forceinline__ void issue_scales(int t) const
    {
        const int bt = turned(t) >> 1;
        const bool live = t < nt;
        const int64_t ta = (w.M + 31) >> 5, tb = (a.N + 31) >> 5;
        const mm_rsrc_t qa = bytes_rsrc(w.sa + (live ? bt * ta + (w.m0 >> 5) : 0) * 256, live ? last_a / 32 * 256 + 256 : 0);
        const mm_rsrc_t qb = bytes_rsrc(w.sb + (live ? bt * tb + (w.n0 >> 5) : 0) * 256, live ? last_b / 32 * 256 + 256 : 0);
        const uint32_t dst = lds0 + scale_buf(t);
#pragma unroll
        for (int i = 0; i < TM / 128; i++) {
            const uint32_t x = 256 * (uint32_t)(wave * (TM / 128) + i);
            load_words_to_lds(qa, x + 4 * (uint32_t)L, dst + x);
        }
#pragma unroll
        for (int i = 0; i < TN / 128; i++) {
            const uint32_t x = 256 * (uint32_t)(wave * (TN / 128) + i);
            load_words_to_lds(qb, x + 4 * (uint32_t)L, dst + TM * 8 + x);
        }
    }
    // The loads that go with MFMA k of n.
    __device__ __forceinline__ void issue_share(int t, int k, int n) const
    {
#pragma unroll
        for (int i = 0; i < kLoads; i++)
            if (i * n / kLoads == k)
                issue(t, i);
    }
    // The wave's load i fills 8 rows of LDS, from row8(i) on: a share of A's TM
    // rows, then of B's TN rows behind them.
    static constexpr int kLoadsA = TM / 32;
    __device__ static constexpr bool is_a(int i) { return i < kLoadsA; }
    __device__ __forceinline__ int row8(int i) const
    {
        return 8 * (is_a(i) ? wave * kLoadsA + i : TM / 8 + wave * (TN / 32) + i - kLoadsA);
    }
    // Where in the tile's rows lane L's load i starts.
    __device__ __forceinline__ uint32_t offset(int i) const
    {
        const int nth = is_a(i) ? i : i - kLoadsA;
        const int row = is_a(i) ? 8 * nth : 64 * (nth >> 3) + (nth >> 2 & 1) + 16 * (nth & 3);
        return voff[(is_a(i) ? 0 : 2) + (nth & 1)] + row * (uint32_t)w.K;
    }
    // The chunk of its row that lane L loads (the slot's exchange, above).
    __device__ __forceinline__ uint32_t chunk(int i) const
    {
        static_assert(kLoadsA % 2 == 0 && TN / 32 % 2 == 0, "rows 16 n + 0 .. 7 by even loads");
        return (uint32_t)((L & 7) ^ (4 * ((is_a(i) ? i : i - kLoadsA) & 1) + (L >> 4)));
    }

    __device__ __forceinline__ i32x8_t frag_a(int t, int s, int i) const
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(lds + buf(t)) + (wm + 32 * i + r) * 8;
        return join(p[(4 * s + h) ^ (r >> 1 & 7)], p[(4 * s + 2 + h) ^ (r >> 1 & 7)]);
    }
    __device__ __forceinline__ i32x8_t frag_b(int t, int s, int j) const
    {
        const uint4 *p = reinterpret_cast<const uint4 *>(lds + buf(t)) + (TM + wn + 32 * j + r) * 8;
        return join(p[(4 * s + h) ^ (r >> 1 & 7)], p[(4 * s + 2 + h) ^ (r >> 1 & 7)]);
    }
    // One of a step's MT + NT fragments.
    __device__ __forceinline__ void read(Frags &f, int t, int s, int i) const
    {
        if (i < NT)
            f.b[i] = frag_b(t, s, i);
        else
            f.a[i - NT] = frag_a(t, s, i - NT);
    }

    // The words of the tiles in places t (even) and t + 1.
    struct Words {
        uint32_t a[MT][W], b[NT][W];
        uint32_t middle[W];            // kExact: of those looked at

        __device__ __forceinline__ void look(int i)
        {
            if (i < MT * W)
                middle[i % W] &= middle_bytes(a[i / W][i % W]);
            else if (i < (MT + NT) * W)
                middle[i % W] &= middle_bytes(b[i / W - MT][i % W]);
        }
        __device__ __forceinline__ void look_at_none()
        {
            middle[0] = middle[W - 1] = ~0u;
        }
    };
    // (kExact: rows behind the last one, whose elements are zeros, take that one's
    // words, so that only scales that count are looked at.)
    __device__ __forceinline__ static int word_at(int row) { return (row >> 5) * 256 + 4 * (row & 31); }
    __device__ __forceinline__ int word_a(int i) const
    {
        return MODE == kExact ? at_a[i] : ((wm >> 5) + i) * 256 + 4 * r;
    }
    __device__ __forceinline__ int word_b(int j) const { return MODE == kExact ? at_b[j] : word_at(brow(j)); }
    __device__ __forceinline__ void read_words(Words &o, int t) const
    {
        const uint8_t *p = lds + scale_buf(t);
#pragma unroll
        for (int k = 0; k < W; k++) {
            const int at = 128 * (MODE == kMx ? h : k);
#pragma unroll
            for (int j = 0; j < NT; j++)
                o.b[j][k] = *reinterpret_cast<const uint32_t *>(p + TM * 8 + word_b(j) + at);
#pragma unroll
            for (int i = 0; i < MT; i++)
                o.a[i][k] = *reinterpret_cast<const uint32_t *>(p + word_a(i) + at);
        }
    }
    // The words of the tiles in places 2 place and 2 place + 1 in use.
    __device__ __forceinline__ void take_words(const Words &o, int place)
    {
#pragma unroll
        for (int k = 0; k < W; k++) {
#pragma unroll
            for (int i = 0; i < MT; i++)
                sa[i][k] = o.a[i][k];
#pragma unroll
            for (int j = 0; j < NT; j++)
                sb[j][k] = o.b[j][k];
        }
        if (MODE == kExact) {
            // (byte j of word k: block 2 j + k)
            const int live = (int)w.nb - 8 * (turned(2 * place) >> 1);
            odd_scales = any_not_middle((o.middle[0] | dead_bytes((live + 1) >> 1)) &
                                        (o.middle[W - 1] | dead_bytes(live >> 1)));
        }
    }

    // Compact: offset of the scales of the tile's row d of an operand (rows behind
    // the last one: the last one's).
    __device__ __forceinline__ uint32_t scale_offset(uint32_t last, int d) const
    {
        return (uint32_t)((d < (int)last ? d : (int)last) * (int)w.nb);
    }
    // Compact: loads the scales of 8 blocks, those of the two tiles in places
    // 2 place and on (for a place behind the last: some).
    __device__ __forceinline__ void fetch_scales(int place)
    {
        const int bt = turned(2 * place) >> 1;
        const int64_t at = 8 * bt < w.nb ? 8 * bt : 0;
        const uint2 x = sra.load<uint2>(off_a, at), y = srb.load<uint2>(off_b, at);
        raw_a[0] = x.x, raw_a[1] = x.y;
        raw_b[0] = y.x, raw_b[1] = y.y;
    }
    // Says that the fetched scales are here (they are: after a wait for every
    // load), before more loads are under way that the compiler would wait for.
    __device__ __forceinline__ void settle_scales()
    {
#pragma unroll
        for (int k = 0; k < 2; k++) {
            asm volatile("" : "+v"(raw_a[k]));
            asm volatile("" : "+v"(raw_b[k]));
        }
    }
    // Compact: the scales fetched for `place` into LDS buffer place % 2; those
    // behind the last block become 0.
    __device__ __forceinline__ void write_scales(int place)
    {
        const int bt = turned(2 * place) >> 1;
        uint2 x = make_uint2(raw_a[0], raw_a[1]), y = make_uint2(raw_b[0], raw_b[1]);
        const int64_t keep = w.nb - 8 * bt;
        if (keep < 8) {
            x = keep8(x, sra, off_a, 8 * bt, (int)keep);
            y = keep8(y, srb, off_b, 8 * bt, (int)keep);
        }
        uint2 *p = reinterpret_cast<uint2 *>(lds + NB * kBuf) + (place & 1) * (TM + TN) + 64 * wave + L;
        if (TM == 256 || wave < TM / 64)
            p[0] = x;
        if (TN == 256 || wave < TN / 64)
            p[TM] = y;
    }
    __device__ __forceinline__ static uint2 keep8(uint2 v, const ByteRows<8> &rows, uint32_t off, int64_t at,
                                                  int n)
    {
        if (n <= 0)
            return make_uint2(0, 0);
        const uint4 u = rows.fix(make_uint4(v.x, v.y, 0, 0), off, at, n);
        return make_uint2(u.x, u.y);
    }
    // Compact: the words of the four steps of `place`.
    __device__ __forceinline__ void read_scales(Words &o, int place) const
    {
        const uint2 *p = reinterpret_cast<const uint2 *>(lds + NB * kBuf) + (place & 1) * (TM + TN);
#pragma unroll
        for (int i = 0; i < MT; i++)
            words(o.a[i], p[wm + 32 * i + r]);
#pragma unroll
        for (int j = 0; j < NT; j++)
            words(o.b[j], p[TM + brow(j)]);
    }
    __device__ __forceinline__ void words(uint32_t (&o)[W], uint2 v) const
    {
        o[0] = __builtin_amdgcn_perm(v.y, v.x, sel);
        if (MODE == kExact)
            o[W - 1] = __builtin_amdgcn_perm(v.y, v.x, 0x07050301u);
    }

    template <int F, int J>
    __device__ __forceinline__ static bool far_of(const i32x8_t &f, const uint32_t (&s)[W])
    {
        return far_block<F>(make_uint4((uint32_t)f[0], (uint32_t)f[1], (uint32_t)f[2], (uint32_t)f[3]),
                            (s[0] >> (8 * J)) & 255) ||
               far_block<F>(make_uint4((uint32_t)f[4], (uint32_t)f[5], (uint32_t)f[6], (uint32_t)f[7]),
                            (s[W - 1] >> (8 * J)) & 255);
    }
    // kExact, a step with odd scales: if it has a far block, its MFMAs as in mfma_far,
    // and then zeros for the usual ones.  (Those instead of these, in two branches,
    // spill 1900 registers.)
    template <int J>
    __device__ __forceinline__ void step_far(Frags &f)
    {
        bool far = false;
#pragma unroll
        for (int i = 0; i < MT; i++)
            far |= far_of<FA, J>(f.a[i], sa[i]);
#pragma unroll
        for (int j = 0; j < NT; j++)
            far |= far_of<FB, J>(f.b[j], sb[j]);
        if (__builtin_expect(__ballot(far) == 0, 1))
            return;
#pragma unroll 1
        for (int q = 0; q < 8; q++) {
            const Pick pick(q);
            i32x8_t y[NT];
#pragma unroll
            for (int j = 0; j < NT; j++)
                y[j] = pick.of(f.b[j]);
#pragma unroll
            for (int i = 0; i < MT; i++) {
                const i32x8_t x = pick.of(f.a[i]);
#pragma unroll
                for (int j = 0; j < NT; j++)
                    acc[i][j] = mfma_mx<FA, FB, J>(x, y[j], acc[i][j], h ? sa[i][W - 1] : sa[i][0],
                                                   h ? sb[j][W - 1] : sb[j][0]);
            }
        }
#pragma unroll
        for (int i = 0; i < MT; i++)
            f.a[i] = i32x8_t{};
#pragma unroll
        for (int j = 0; j < NT; j++)
            f.b[j] = i32x8_t{};
    }

    // The MFMAs of one step on f, with the reads of the next step's fragments
    // between them, and in kExact the look at the next scale words.
    template <int J, bool LOAD>
    __device__ __forceinline__ void step(Frags &f, Frags &next, int tn, int sn, int tl, Words &scales)
    {
        if (MODE == kMx) {
            int k = 0;
#pragma unroll
            for (int i = 0; i < MT; i++)
#pragma unroll
                for (int j = 0; j < NT; j++) {
                    acc[i][j] = mfma_mx<FA, FB, J>(f.a[i], f.b[j], acc[i][j], sa[i][0], sb[j][0]);
                    if (LOAD)
                        issue_share(tl, k, MT * NT);
                    if (k < MT + NT)
                        read(next, tn, sn, k);
                    k++;
                    __builtin_amdgcn_sched_barrier(0);
                }
            return;
        }
        if (__builtin_expect(odd_scales, 0))
            step_far<J>(f);
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
                    if (LOAD && part < 2)
                        issue_share(tl, part * MT * NT + i * NT + j, 2 * MT * NT);
                    if (j == NT - 1) {
#pragma unroll
                        for (int k = 0; k < MT + NT; k++)
                            if (k * 4 * MT / (MT + NT) == part * MT + i)
                                read(next, tn, sn, k);
                        if (J == 3)
                            scales.look(part * MT + i);
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

    // The tile in place t, steps J and J + 1 of the scale words (J: 0 in even
    // places, 2 in odd ones).
    template <int J>
    __device__ __forceinline__ void tile(Frags &f0, Frags &f1, Words &next, int t)
    {
        constexpr int odd = J / 2;
        step<J, false>(f0, f1, t, 1, 0, next);
        wait_and_barrier<loads(odd + 2, odd + NB - 1)>();
        if constexpr (TILED) {
            if (odd)
                read_words(next, t + 1);
            if ((odd + NB) % 2 == 0)
                issue_scales(t + NB);
        } else if (odd) {
            settle_scales();       // fetched before: no more loads than here
            if (MODE == kExact)
                read_scales(next, (t >> 1) + 1);
        }
        next.look_at_none();
        step<J + 1, true>(f1, f0, t + 1, 0, t + NB, next);
    }

    __device__ __forceinline__ void run()
    {
        // an even number of tiles: one behind the last k holds zeros
        nt = 2 * (int)((w.K + 255) / 256);
        // Rows a multiple of 256 bytes apart lie in few of the L2's channels at
        // any one k, and the workgroups of an XCD walk along k at about the same
        // pace: columns of tiles start in four different places, 256 k apart.
        phase = 2 * (int)((w.n0 / TN) & 3);
        phase = phase < nt ? phase : 0;
        sel = MODE == kMx && h ? 0x07050301u : 0x06040200u;
        ra = rows_rsrc(w.qa + w.m0 * w.K, w.M - w.m0, w.K);
        rb = rows_rsrc(w.qb + w.n0 * w.K, a.N - w.n0, w.K);
        last_a = (uint32_t)(w.M - w.m0 < TM ? w.M - w.m0 : TM) - 1;
        last_b = (uint32_t)(a.N - w.n0 < TN ? a.N - w.n0 : TN) - 1;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int ra = 8 * wave * kLoadsA + (L >> 3), p = wave * (TN / 32);
            const int rb = 64 * (p >> 3) + (p >> 2 & 1) + 2 * (L >> 3);
            voff[i] = (uint32_t)(ra * (int)w.K) + 16 * chunk(i);
            voff[2 + i] = (uint32_t)(rb * (int)w.K) + 16 * chunk(kLoadsA + i);
        }
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int j = 0; j < NT; j++)
                acc[i][j] = f32x16_t{};
        if (TILED && MODE == kExact) {
#pragma unroll
            for (int i = 0; i < MT; i++)
                at_a[i] = word_at(wm + 32 * i + r < (int)last_a ? wm + 32 * i + r : (int)last_a);
#pragma unroll
            for (int j = 0; j < NT; j++)
                at_b[j] = word_at(brow(j) < (int)last_b ? brow(j) : (int)last_b);
        }
        static_assert(TM <= 256 && TN <= 256, "compact scales: a thread per row");
        if constexpr (!TILED) {
            off_a = scale_offset(last_a, 64 * wave + L) + sra.lead;
            off_b = scale_offset(last_b, 64 * wave + L) + srb.lead;
        }
        if (nt > 0) {
            Frags f0, f1;
            Words next;
            uint32_t behind[4];
            if constexpr (!TILED) {
                fetch_scales(1);
                behind[0] = raw_a[0], behind[1] = raw_a[1], behind[2] = raw_b[0], behind[3] = raw_b[1];
                fetch_scales(0);
            }
#pragma unroll
            for (int t = 0; t < NB; t++) {
                if (TILED && t % 2 == 0)
                    issue_scales(t);
#pragma unroll
                for (int i = 0; i < kLoads; i++)
                    issue(t, i);
                if (!TILED && t == 0) {
                    write_scales(0);
                    raw_a[0] = behind[0], raw_a[1] = behind[1], raw_b[0] = behind[2], raw_b[1] = behind[3];
                    settle_scales();
                }
            }
            wait_and_barrier<loads(1, NB - 1)>();
            if constexpr (TILED) {
                read_words(next, 0);
            } else {
                read_scales(next, 0);
            }
            next.look_at_none();
#pragma unroll
            for (int i = 0; i < (MT + NT) * W; i++)
                next.look(i);
            take_words(next, 0);
#pragma unroll
            for (int i = 0; i < MT + NT; i++)
                read(f0, 0, 0, i);
            int t = 0;
            do {
                // scale words of two tiles at a time.  Tiled: read from LDS behind
                // the second one's barrier.  Compact: fetched two tiles earlier, put
                // into LDS before the first tile's barrier and taken from there
                // after the second's (kMx: after its MFMAs, for the registers).
                const int place = (t >> 1) + 1;
                if constexpr (!TILED)
                    write_scales(place);
                tile<0>(f0, f1, next, t);
                if constexpr (!TILED)
                    fetch_scales(place + 1);
                tile<2>(f0, f1, next, t + 1);
                if (!TILED && MODE == kMx)
                    read_scales(next, place);
                take_words(next, place);
                t += 2;
            } while (t < nt);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the loads of no tile
        store();
    }

    // Writes the outputs (kMx: bf16, kExact: fp32, with ADD added to what is
    // there); PAIR: a lane's two neighbouring columns in one store.
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
        // (rows of an odd length: pairs at any element, which memory takes, where
        // none holds the last column alone)
        const bool pair = (a.N & 1) == 0 || w.n0 + TN <= a.N;
        if (MODE == kMx)
            pair ? store_form<true, false>() : store_form<false, false>();
        else if (a.accumulate)
            pair ? store_form<true, true>() : store_form<false, true>();
        else
            pair ? store_form<true, false>() : store_form<false, false>();
    }
};

template <MmMode MODE, int FA, int FB, int TM, int TN, bool TILED, bool PAIRED = false>
__device__ __forceinline__ void mm_tile_run(const MmArgs &a, const MmTile &w, uint8_t *lds)
{
    if (nothing_to_add(a, w))
        return;
    typedef __attribute__((address_space(3))) uint8_t lds_byte_t;
    MmKernel<MODE, FA, FB, TM, TN, TILED, PAIRED> k{
        a, w,
        ByteRows<8>(a.sa, w.sa + w.m0 * w.nb, w.sa_left - w.m0 * w.nb),
        ByteRows<8>(a.sb, w.sb + w.n0 * w.nb, w.sb_left - w.n0 * w.nb)};
    k.lds = lds;
    k.lds0 = (uint32_t)(uintptr_t)(lds_byte_t *)lds;
    k.L = (int)threadIdx.x & 63;
    k.wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    k.h = k.L >> 5;
    k.r = k.L & 31;
    k.wm = (k.wave >> 1) * (TM / 2);
    k.wn = (k.wave & 1) * (TN / 2);
    k.run();
}

// The first t.whole workgroups take a whole tile each.  The tiles behind them,
// too few to fill the CUs once more, go in t.parts parts.
template <MmMode MODE, int FA, int FB, int TM, int TN, bool TILED>
__global__ __launch_bounds__(256, 1) void mm_tile_kernel(const MmArgs a, const MmTable t)
{
    extern __shared__ uint8_t mm_lds[];
    constexpr int S = kMmPart;
    static_assert(TM == 2 * S && TN == 2 * S, "parts: halves of the sides");
    const int id = (int)blockIdx.x, q = id - t.whole;
    if (q < 0) {
        const MmTile w = mm_tile(a, t, mm_xcd_order(id, t.whole), TM, TN);
        mm_tile_run<MODE, FA, FB, TM, TN, TILED>(a, w, mm_lds);
        return;
    }
    MmTile w = mm_tile(a, t, t.whole + q / t.parts, TM, TN);
    w.n0 += q & 1 ? S : 0;
    w.m0 += q & 2 && t.parts == 4 ? S : 0;
    if (w.m0 >= w.M || w.n0 >= a.N)
        return;
    if (t.parts == 2)
        mm_tile_run<MODE, FA, FB, TM, S, TILED>(a, w, mm_lds);
    else
        mm_tile_run<MODE, FA, FB, S, S, TILED>(a, w, mm_lds);
}

// Tiles of 128 x 128 only, two workgroups per CU.
template <MmMode MODE, int FA, int FB, bool TILED>
__global__ __launch_bounds__(256, 2) void mm_square_kernel(const MmArgs a, const MmTable t)
{
    extern __shared__ uint8_t mm_lds[];
    constexpr int S = kMmPart;
    const MmTile w = mm_tile(a, t, mm_xcd_order((int)blockIdx.x, t.whole), S, S);
    mm_tile_run<MODE, FA, FB, S, S, TILED, true>(a, w, mm_lds);
}

template <MmMode MODE, int FA, int FB, int TM, int TN, bool TILED>
hipError_t launch_mm_tile_one(const MmArgs &a, const MmTable &t, hipStream_t stream)
{
    constexpr int S = kMmPart;
    if (t.square) {
        constexpr int bytes = MmKernel<MODE, FA, FB, S, S, TILED, true>::kLds;
        const hipError_t e =
            hipFuncSetAttribute(reinterpret_cast<const void *>(mm_square_kernel<MODE, FA, FB, TILED>),
                                hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess)
            return e;
        hipLaunchKernelGGL((mm_square_kernel<MODE, FA, FB, TILED>), dim3((unsigned)t.whole), dim3(256), bytes,
                           stream, a, t);
        return hipGetLastError();
    }
    constexpr int l0 = MmKernel<MODE, FA, FB, TM, TN, TILED>::kLds, l1 = MmKernel<MODE, FA, FB, TM, S, TILED>::kLds,
                  l2 = MmKernel<MODE, FA, FB, S, S, TILED>::kLds;
    constexpr int lds = l0 > l1 ? (l0 > l2 ? l0 : l2) : l1 > l2 ? l1 : l2;
    static_assert(lds <= 160 * 1024, "a CU's LDS");
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void *>(mm_tile_kernel<MODE, FA, FB, TM, TN, TILED>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess)
        return e;
    const unsigned n = (unsigned)(t.whole + t.parts * (t.tile0[t.count] - t.whole));
    hipLaunchKernelGGL((mm_tile_kernel<MODE, FA, FB, TM, TN, TILED>), dim3(n), dim3(256), lds, stream, a, t);
    return hipGetLastError();
}

template <MmMode MODE, int TM, int TN, bool TILED>
hipError_t launch_mm_tile_mode(const MmArgs &a, const MmTable &t, hipStream_t stream)
{
    if (!a.a_e5m2 && !a.b_e5m2)
        return launch_mm_tile_one<MODE, 0, 0, TM, TN, TILED>(a, t, stream);
    if (a.a_e5m2 && !a.b_e5m2)
        return launch_mm_tile_one<MODE, 1, 0, TM, TN, TILED>(a, t, stream);
    if (!a.a_e5m2)
        return launch_mm_tile_one<MODE, 0, 1, TM, TN, TILED>(a, t, stream);
    return launch_mm_tile_one<MODE, 1, 1, TM, TN, TILED>(a, t, stream);
}

}  // namespace mxk
