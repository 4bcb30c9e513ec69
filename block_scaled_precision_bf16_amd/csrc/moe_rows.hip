// moe_rows.hip -- the tokens' rows to their experts and back (gfx950): a stable
// sort of the slots (token, choice) by expert, the rows in that order, and the
// weighted sum of the experts' rows with its gradients.
//
// The sort counts.  A workgroup's slots are taken in order, a run of them by each
// wave; a wave counts 64 slots at a time, the lanes of one expert found by a
// ballot for each bit of its index, so that ranks are those of the slots' order
// and nothing depends on the order of atomics.  Few slots take one workgroup; more
// take up to 16 in one launch, each of which counts everything; still more take two
// launches, counts of each workgroup and then their sums and the ranks.  What bounds
// it is the chain of its steps, not bytes: in a graph 1024 slots of 256 experts 4.9 us,
// 16384 of 8 7.3 us, 32768 of 256 11.2 us, 131072 of 256 13.7 us.
//
// The rest moves rows and is bound by memory: 16-byte accesses, at any byte, several
// in flight for each lane.
#include "bufio.h"
#include "device_math.h"
#include "launch_moe.h"
#include "rows.h"
#include "wave.h"

namespace mxk {

constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortE = 1024;

// Lanes of the wave whose e is this lane's (e < 2^bits).
__device__ __forceinline__ uint64_t same_lanes(int e, int bits)
{
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; b++) {
        const bool one = (e >> b) & 1;
        const uint64_t v = __builtin_amdgcn_ballot_w64(one);
        m &= one ? v : ~v;
    }
    return m;
}

// Rank of this lane's slot among its expert's slots of the run so far, whose
// counts are in cnt (one wave's own); -1 without an expert (e = E).
template <class C>
__device__ __forceinline__ int rank_and_count(C *cnt, int e, int E, int bits, int lane)
{
    const uint64_t m = same_lanes(e, bits);
    const int before = __builtin_popcountll(m & ((1ull << lane) - 1));
    int at = -1;
    if (e < E)
        at = cnt[e] + before;
    __builtin_amdgcn_wave_barrier();
    if (e < E && before == 0)
        cnt[e] = (C)(cnt[e] + __builtin_popcountll(m));
    __builtin_amdgcn_wave_barrier();
    return at;
}

__device__ __forceinline__ int expert_of(const SortArgs &a, int64_t slot, int64_t end)
{
    int e = a.E;
    if (slot < end) {
        const int v = a.experts[slot];
        e = v >= 0 && v < a.E ? v : a.E;
    }
    return e;
}

// Sum of v over the workgroup's threads before this one (red: a word per wave, used
// once), and over all of them.
template <int WAVES>
__device__ __forceinline__ int before_sum(int v, int32_t *red, int &total)
{
    const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int s = (int)wave_scan((uint32_t)v);
    if (lane == 63)
        red[wave] = s;
    __syncthreads();
    int base = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < WAVES; w++) {
        const int n = red[w];
        base += w < wave ? n : 0;
        total += n;
    }
    return base + s - v;
}

// -1 in the rows between expert e's last and the next expert's first, for the
// workgroup's share of the experts, and behind the last one's (from `total` on).
__device__ __forceinline__ void fill_rows(const SortArgs &a, const int32_t *start, const int32_t *counts,
                                          int64_t total, int block, int blocks)
{
    if (a.align > 1)   // 16 threads for each expert
        for (int e = block * (int)(blockDim.x / 16) + (int)(threadIdx.x >> 4); e < a.E;
             e += blocks * (int)(blockDim.x / 16)) {
            const int64_t from = (int64_t)start[e] + counts[e], to = e + 1 < a.E ? start[e + 1] : total;
            for (int64_t r = from + (threadIdx.x & 15); r < to; r += 16)
                a.slots[r] = -1;
        }
    for (int64_t r = total + (int64_t)block * blockDim.x + threadIdx.x; r < a.rows;
         r += (int64_t)blocks * blockDim.x)
        a.slots[r] = -1;
}

__device__ __forceinline__ int index_bits(int E) { return 32 - __builtin_clz((unsigned)E); }

// One workgroup of 64 WAVES threads sorts up to 64 WAVES RUN slots: a wave's run,
// 64 at a time, with each slot's rank within the run kept in registers; the runs'
// counts (16 bits) summed over the waves and the experts; the rows.
template <int WAVES, int RUN>
__global__ __launch_bounds__(64 * WAVES) void sort_alone_kernel(SortArgs a)
{
    extern __shared__ int32_t lds[];                  // start [E], counts [E], runs [WAVES][E]
    __shared__ int32_t red[WAVES];
    constexpr int THREADS = 64 * WAVES;
    int32_t *const start = lds, *const counts = lds + a.E;
    uint16_t *const runs = reinterpret_cast<uint16_t *>(counts + a.E);
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6, bits = index_bits(a.E);
    const int64_t first = (int64_t)wave * (64 * RUN);
    const int64_t end = first + 64 * RUN < a.N ? first + 64 * RUN : a.N;
    uint16_t *const cnt = runs + wave * a.E;
    int e[RUN], rank[RUN];
#pragma unroll
    for (int i = 0; i < RUN; i++)
        e[i] = expert_of(a, first + 64 * i + lane, end);
    for (int i = lane; i < a.E; i += 64)
        cnt[i] = 0;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < RUN; i++)
        rank[i] = first + 64 * i < end ? rank_and_count(cnt, e[i], a.E, bits, lane) : -1;
    __syncthreads();
    // each thread's experts are neighbours, so that the threads' sums are in order
    const int per = (a.E + THREADS - 1) / THREADS, e0 = (int)threadIdx.x * per;
    int mine = 0;
    for (int k = e0; k < e0 + per && k < a.E; k++) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < WAVES; w++) {
            const int c = runs[w * a.E + k];
            runs[w * a.E + k] = (uint16_t)n;
            n += c;
        }
        counts[k] = n;
        a.counts[k] = n;
        mine += (n + a.align - 1) / a.align * a.align;
    }
    int total;
    int at = before_sum<WAVES>(mine, red, total);
    for (int k = e0; k < e0 + per && k < a.E; k++) {
        start[k] = at;
        at += (counts[k] + a.align - 1) / a.align * a.align;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < RUN; i++) {
        const int64_t s = first + 64 * i + lane;
        if (s >= end)
            continue;
        const int row = rank[i] < 0 ? -1 : start[e[i]] + cnt[e[i]] + rank[i];
        a.pos[s] = row;
        if (row >= 0)
            a.slots[row] = (int32_t)s;
    }
    fill_rows(a, start, counts, total, 0, 1);
}

// The first slots of this wave's run of a workgroup's a.chunk, whose first is `first`.
template <int WAVES>
__device__ __forceinline__ int first_of_run(const SortArgs &a, int64_t first)
{
    const int64_t run = a.chunk / WAVES, from = first + (threadIdx.x >> 6) * run;
    return expert_of(a, from + (threadIdx.x & 63), from + run < a.N ? from + run : a.N);
}

// Rows of a workgroup's slots, its waves' runs of a.chunk / WAVES one after the
// other from `first` on, e0 = first_of_run: base[e], the row of the first of expert
// e's among them; runs: 16-bit counts [WAVES][E], any values.  Each run is ranked
// twice where it is longer than 64 (the first ranks are not kept), once otherwise.
template <int WAVES>
__device__ __forceinline__ void place_slots(const SortArgs &a, int64_t first, int e0, const int32_t *base,
                                            uint16_t *runs)
{
    constexpr int THREADS = 64 * WAVES;
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6, bits = index_bits(a.E);
    const int64_t run = a.chunk / WAVES, from = first + wave * run;
    const int64_t end = from + run < a.N ? from + run : a.N;
    uint16_t *const cnt = runs + wave * a.E;
    for (int k = lane; k < a.E; k += 64)
        cnt[k] = 0;
    __builtin_amdgcn_wave_barrier();
    int e = e0, rank = -1;
    for (int64_t s = from; s < end; s += 64) {
        const int next = run > 64 ? expert_of(a, s + 64 + lane, end) : a.E;
        rank = rank_and_count(cnt, e, a.E, bits, lane);
        e = next;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < a.E; k += THREADS) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < WAVES; w++) {
            const int c = runs[w * a.E + k];
            runs[w * a.E + k] = (uint16_t)n;
            n += c;
        }
    }
    __syncthreads();
    e = e0;
    for (int64_t s = from; s < end; s += 64) {
        const int next = run > 64 ? expert_of(a, s + 64 + lane, end) : a.E;
        if (run > 64)
            rank = rank_and_count(cnt, e, a.E, bits, lane);
        else if (rank >= 0)
            rank += cnt[e];
        if (s + lane < end) {
            const int row = rank < 0 ? -1 : base[e] + rank;
            a.pos[s + lane] = row;
            if (row >= 0)
                a.slots[row] = (int32_t)(s + lane);
        }
        e = next;
    }
}

// Up to 16 workgroups in one launch: each counts all slots (wave w those of
// workgroup w, at most 2048), so that it knows what comes before its own.  All of a
// lane's loads are under way at once.  Few experts are counted in several copies, by
// neighbouring lanes, or these would queue for the same words.
constexpr int kFewWaves = 16, kFewLoads = 8;
static_assert(kSortFew <= 16 * 64 * 4 * kFewLoads, "a wave's slots in one step");
static int few_copies(int E)
{
    int n = 1;
    while (n < 32 && 2 * n * E <= 512)
        n *= 2;
    return n;
}
// 32-bit words of one copy, two experts of a wave in each; one more, so that the
// copies' words lie in different banks.
__host__ __device__ inline int few_words(int E) { return kFewWaves * ((E + 1) / 2) + 1; }

__global__ __launch_bounds__(64 * kFewWaves) void sort_few_kernel(SortArgs a, int copies)
{
    extern __shared__ int32_t lds[];       // base [E], start [E], counts [E], copies of [16][E] (16 bits)
    __shared__ int32_t red[kFewWaves];
    constexpr int THREADS = 64 * kFewWaves;
    const int E2 = (a.E + 1) & ~1;
    int32_t *const base = lds, *const start = base + E2, *const counts = start + E2;
    uint32_t *const words = reinterpret_cast<uint32_t *>(counts + E2);
    uint16_t *const runs = reinterpret_cast<uint16_t *>(words);
    const int lane = (int)threadIdx.x & 63, wave = (int)threadIdx.x >> 6, me = (int)blockIdx.x;
    const int64_t from = (int64_t)wave * a.chunk + 4 * lane;
    const int64_t end = (int64_t)(wave + 1) * a.chunk < a.N ? (int64_t)(wave + 1) * a.chunk : a.N;
    int4 v[kFewLoads];
#pragma unroll
    for (int i = 0; i < kFewLoads; i++) {
        const int64_t s = from + 256 * i;
        if (s + 4 <= end)
            v[i] = *reinterpret_cast<const int4 *>(a.experts + s);
        else
            v[i] = make_int4(s < end ? a.experts[s] : -1, s + 1 < end ? a.experts[s + 1] : -1,
                             s + 2 < end ? a.experts[s + 2] : -1, -1);
    }
    const int e0 = first_of_run<kFewWaves>(a, (int64_t)me * a.chunk);
    for (int i = threadIdx.x; i < copies * few_words(a.E); i += THREADS)
        words[i] = 0;
    __syncthreads();
    uint32_t *const mine_at = words + (lane & (copies - 1)) * few_words(a.E) + wave * (E2 / 2);
#pragma unroll
    for (int i = 0; i < kFewLoads; i++) {
        if (wave * a.chunk + 256 * i >= a.N || 256 * i >= a.chunk)
            break;
        const int e[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; j++)
            if (e[j] >= 0 && e[j] < a.E)   // sums of ones: the same in any order
                atomicAdd(mine_at + (e[j] >> 1), 1u << (16 * (e[j] & 1)));
    }
    __syncthreads();
    // the copies into the first one, two counts a word (none passes 16 bits)
    for (int i = threadIdx.x; copies > 1 && i < kFewWaves * E2 / 2; i += THREADS) {
        uint32_t n = words[i];
#pragma unroll 4
        for (int c = 1; c < copies; c++)
            n += words[c * few_words(a.E) + i];
        words[i] = n;
    }
    __syncthreads();
    // each thread's experts are neighbours, so that the threads' sums are in order
    const int per = (a.E + THREADS - 1) / THREADS, k0 = (int)threadIdx.x * per;
    int mine = 0;
    for (int k = k0; k < k0 + per && k < a.E; k++) {
        int n = 0, before = 0;
#pragma unroll
        for (int w = 0; w < kFewWaves; w++) {
            const int c = runs[w * E2 + k];
            before += w < me ? c : 0;
            n += c;
        }
        base[k] = before;
        counts[k] = n;
        if (me == 0)
            a.counts[k] = n;
        mine += (n + a.align - 1) / a.align * a.align;
    }
    int total;
    int at = before_sum<kFewWaves>(mine, red, total);
    for (int k = k0; k < k0 + per && k < a.E; k++) {
        start[k] = at;
        base[k] += at;
        at += (counts[k] + a.align - 1) / a.align * a.align;
    }
    __syncthreads();
    place_slots<kFewWaves>(a, (int64_t)me * a.chunk, e0, base, runs);
    fill_rows(a, start, counts, total, me, (int)gridDim.x);
}

// Counts of each workgroup's slots: ws[block][E].
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a)
{
    __shared__ int32_t cnt[kSortE];
    for (int e = threadIdx.x; e < a.E; e += kSortThreads)
        cnt[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * a.chunk;
    const int64_t end = first + a.chunk < a.N ? first + a.chunk : a.N;
    for (int64_t s = first + threadIdx.x; s < end; s += kSortThreads) {
        const int e = expert_of(a, s, end);
        if (e < a.E)
            atomicAdd(&cnt[e], 1);   // sums of ones: the same in any order
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kSortThreads)
        a.ws[(int64_t)blockIdx.x * a.E + e] = cnt[e];
}

// Each workgroup adds all workgroups' counts, those before it apart.
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a)
{
    extern __shared__ int32_t lds[];       // base [E], start [E], counts [E], runs [waves][E] (16 bits)
    __shared__ int32_t red[kSortWaves];
    int32_t *const base = lds, *const start = base + a.E, *const counts = start + a.E;
    const int per = (a.E + kSortThreads - 1) / kSortThreads, e0 = (int)threadIdx.x * per;
    const int me = (int)blockIdx.x;
    const int e1 = first_of_run<kSortWaves>(a, (int64_t)me * a.chunk);
    // a thread's share: experts k, k + 512, .. when they are many, or a part of the
    // workgroups' counts of one expert when they are few
    for (int k = threadIdx.x; k < a.E; k += kSortThreads)
        base[k] = counts[k] = 0;
    __syncthreads();
    const int parts = a.E >= kSortThreads ? 1 : kSortThreads / a.E;
    const int part = parts == 1 ? 0 : (int)threadIdx.x / a.E;
    for (int k = parts == 1 ? (int)threadIdx.x : (int)threadIdx.x - part * a.E; k < a.E && part < parts;
         k += parts == 1 ? kSortThreads : a.E) {
        int n = 0, before = 0;
#pragma unroll 8
        for (int b = part; b < a.blocks; b += parts) {
            const int c = a.ws[(int64_t)b * a.E + k];
            before += b < me ? c : 0;
            n += c;
        }
        atomicAdd(&counts[k], n);      // whole numbers: the same in any order
        atomicAdd(&base[k], before);
    }
    __syncthreads();
    int mine = 0;
    for (int k = e0; k < e0 + per && k < a.E; k++)
        mine += (counts[k] + a.align - 1) / a.align * a.align;
    int total;
    int at = before_sum<kSortWaves>(mine, red, total);
    for (int k = e0; k < e0 + per && k < a.E; k++) {
        start[k] = at;
        base[k] += at;
        at += (counts[k] + a.align - 1) / a.align * a.align;
        if (me == 0)
            a.counts[k] = counts[k];
    }
    __syncthreads();
    place_slots<kSortWaves>(a, (int64_t)me * a.chunk, e1, base, reinterpret_cast<uint16_t *>(counts + a.E));
    fill_rows(a, start, counts, total, me, (int)gridDim.x);
}

hipError_t launch_sort(const SortArgs &a, hipStream_t s)
{
    const size_t sums = 3 * (size_t)((a.E + 1) & ~1) * sizeof(int32_t);
    const size_t run = (size_t)((a.E + 1) & ~1) * sizeof(uint16_t);
    if (a.N <= 1024) {
        hipLaunchKernelGGL((sort_alone_kernel<4, 4>), dim3(1), dim3(256), sums + 4 * run, s, a);
    } else if (!a.ws) {
        const int copies = few_copies(a.E);
        hipLaunchKernelGGL(sort_few_kernel, dim3(a.blocks), dim3(64 * kFewWaves),
                           sums + (size_t)copies * few_words(a.E) * sizeof(uint32_t), s, a, copies);
    } else {
        hipLaunchKernelGGL(sort_count_kernel, dim3(a.blocks), dim3(kSortThreads), 0, s, a);
        hipLaunchKernelGGL(sort_place_kernel, dim3(a.blocks), dim3(kSortThreads), sums + kSortWaves * run,
                           s, a);
    }
    return hipGetLastError();
}

// ---- rows ---------------------------------------------------------------------

// Rows of out, `per` threads (a power of two) to each, four pieces of 16 bytes a thread
// under way at once; a row's last bytes one by one.  A workgroup's rows are one unit.
// A token's row is read `top` times, and where each time comes from the last cache
// this bounds the kernel (4096 tokens to 4 of 8 experts, rows of 14336 bytes: 68 us
// with the units in order).  So with stretch > 0 the units are cut into kSlices slices,
// each slice into 8 stretches, and XCD x (workgroups b mod 8) takes the x-th stretch of
// all slices side by side: where up to 8 experts are loaded alike these are the same
// tokens, found in the XCD's L2 (48 us, 6.2 TB/s; unevenly loaded 67 us).
constexpr int kSlices = 8, kGatherThreads = 256;

__global__ __launch_bounds__(kGatherThreads) void gather_kernel(GatherArgs a, int per, int64_t stretch)
{
    const int64_t n = a.row_bytes >> 4;
    const int rows = kGatherThreads / per, tid = (int)threadIdx.x & (per - 1);
    const int64_t units = stretch ? 8 * kSlices * stretch : (a.rows + rows - 1) / rows;
    for (int64_t b = blockIdx.x; b < units; b += gridDim.x) {
        const int64_t turn = b >> 3;
        const int64_t unit = stretch ? ((turn % kSlices) * 8 + (b & 7)) * stretch + turn / kSlices : b;
        const int64_t r = unit * rows + threadIdx.x / per;
        if (r >= a.rows)
            continue;
        const int32_t slot = a.slots[r];
        const bool live = slot >= 0 && slot < a.T * a.top;
        uint8_t *const ob = a.out + r * a.row_bytes;
        const uint8_t *const xb = a.x + (live ? (int64_t)(slot / a.top) * a.row_bytes : 0);
        u32x4_bytes *const o = reinterpret_cast<u32x4_bytes *>(ob);
        const u32x4_bytes *const x = reinterpret_cast<const u32x4_bytes *>(xb);
        for (int64_t i = tid; i < n; i += 4 * per) {
            u32x4_t v[4];
#pragma unroll
            for (int j = 0; j < 4; j++)
                v[j] = live && i + per * j < n ? (u32x4_t)x[i + per * j] : u32x4_t{};
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (i + per * j < n)
                    __builtin_nontemporal_store((u32x4_bytes)v[j], &o[i + per * j]);
        }
        for (int64_t i = 16 * n + tid; i < a.row_bytes; i += per)
            ob[i] = live ? xb[i] : (uint8_t)0;
    }
}

hipError_t launch_gather(const GatherArgs &a, hipStream_t s)
{
    int per = 1;
    while (per < kGatherThreads && 64 * (int64_t)per < a.row_bytes)
        per *= 2;
    const int64_t rows = kGatherThreads / per, units = (a.rows + rows - 1) / rows;
    // Tokens that the last cache does not keep are read from memory, where rows in order
    // are read faster; with few reads of each that is more than the L2 saves (of 8
    // experts, in order and in stretches: 64 MiB of tokens to 2 experts 38.5 and 31 us,
    // 112 MiB 67 and 73 us, 128 MiB 78 and 88 us; to 4, 64 MiB 75 and 54 us, 112 MiB 133
    // and 125 us, 224 MiB 273 and 250 us).  With many experts it matters little: 56 MiB of
    // tokens to 8 of 64 133.7 and 134.8 us, of 256 137.9 and 136.4, to 2 of 64 36.7 and 36.1;
    // 128 MiB to 4 of 64 152.6 and 147.8, to 8 of 256 304.9 and 304.8, to 4 of 256 in rows of
    // 2048 bytes 153.4 and 155.2.
    const bool near = a.T * a.row_bytes <= int64_t(1) << 26 || a.top >= 4;
    const int64_t stretch = near ? (units + 8 * kSlices - 1) / (8 * kSlices) : 0;
    const int64_t blocks = near ? 8 * kSlices * stretch : units;
    hipLaunchKernelGGL(gather_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(kGatherThreads),
                       0, s, a, per, stretch);
    return hipGetLastError();
}

// Row of slot s in y, or -1.
__device__ __forceinline__ int64_t row_of_slot(const CombineArgs &a, int64_t s)
{
    if (!a.pos)
        return s;
    const int32_t r = a.pos[s];
    return r >= 0 && r < a.rows ? r : -1;
}

__device__ __forceinline__ void widen(uint4 u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int d = 0; d < 4; d++) {
        v[2 * d] = bf16_lo(w[d]);
        v[2 * d + 1] = bf16_hi(w[d]);
    }
}
__device__ __forceinline__ uint4 narrow(const float (&v)[8])
{
    return make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]),
                      bf16x2_rne(v[6], v[7]));
}

// One chunk of 8 elements of one token per thread; J rows' loads under way.  4096
// tokens from 4 experts each, rows of 7168: 56 us (294 MB, 5.2 TB/s).
template <int J>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a, int64_t parts)
{
    for (int64_t b = blockIdx.x; b < a.T * parts; b += gridDim.x) {
        const int64_t t = b / parts, c = (b - t * parts) * 256 + threadIdx.x;
        if (8 * c >= a.K)
            continue;
        float acc[8] = {};
        for (int j0 = 0; j0 < a.top; j0 += J) {
            int64_t r[J];
            float w[J];
            uint4 y[J];
#pragma unroll
            for (int j = 0; j < J; j++) {
                const int64_t s = t * a.top + j0 + j;
                r[j] = j0 + j < a.top ? row_of_slot(a, s) : -1;
                w[j] = a.weights && r[j] >= 0 ? a.weights[s] : 1.0f;
            }
#pragma unroll
            for (int j = 0; j < J; j++) {
                const int64_t len = r[j] < 0 ? 0 : a.K;
                const uint16_t *const yr = a.y + (r[j] < 0 ? 0 : r[j]) * a.K;
                y[j] = 8 * c + 8 <= len ? whole_chunk<false>(yr, c) : load_chunk<false>(yr, c, len);
            }
#pragma unroll
            for (int j = 0; j < J; j++) {
                float v[8];
                widen(y[j], v);
#pragma unroll
                for (int d = 0; d < 8; d++)
                    acc[d] = r[j] < 0 ? acc[d] : __builtin_fmaf(w[j], v[d], acc[d]);
            }
        }
        store_chunk<false>(a.out + t * a.K, c, a.K, narrow(acc));
    }
}

hipError_t launch_combine(const CombineArgs &a, hipStream_t s)
{
    const int64_t parts = (a.K + 2047) / 2048;
    const dim3 grid((unsigned)(a.T * parts < (1 << 22) ? a.T * parts : 1 << 22));
    // (what is left of four is not free: 4096 tokens of 4096 from 2 experts 16.4 and, by
    // four, 19.3 us; from 8 by two 29.3 and by four 29.0 us)
    hipLaunchKernelGGL((a.top <= 2 ? combine_kernel<2> : combine_kernel<4>), grid, dim3(256), 0, s, a, parts);
    return hipGetLastError();
}

// Rows of more than 64 MiB are read and written non-temporally, which leaves the
// caches to the tokens' rows that are read once for each slot (16384 rows of 7168: 117
// -> 108 us; 4100 of them 39 us both ways; 2050, still in the caches, 24.9 and 27.5 us).
static bool rows_stream(const CombineArgs &a) { return 2 * a.rows * a.K > int64_t(1) << 26; }

// First a wave per kZeroRows rows for those without a slot (first, and few to a wave:
// the rows behind the last expert's lie together, and a wave that has 64 of them
// ends long after all others), then a wave per slot.  4096 tokens from 4 experts each,
// rows of 7168: 99 us (0.53 GB, 5.3 TB/s).
constexpr int kZeroRows = 8;

template <bool NT>
__global__ __launch_bounds__(256) void combine_back_kernel(CombineArgs a, int64_t zeros)
{
    const int lane = (int)threadIdx.x & 63;
    const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), s = w - zeros;
    if (s < 0) {
        const int64_t r0 = w * kZeroRows;
        bool empty = false;
        if (lane < kZeroRows && r0 + lane < a.rows) {
            const int32_t slot = a.slots[r0 + lane];
            empty = slot < 0 || slot >= a.T * a.top;
        }
        for (uint64_t m = __builtin_amdgcn_ballot_w64(empty); m; m &= m - 1) {
            uint16_t *const out = a.out + (r0 + __builtin_ctzll(m)) * a.K;
            int64_t c = lane;
            for (; 8 * c + 8 <= a.K; c += 64)
                put_chunk<NT>(out, c, make_uint4(0u, 0u, 0u, 0u));
            if (8 * c < a.K)
                store_chunk<false>(out, c, a.K, make_uint4(0u, 0u, 0u, 0u));
        }
        return;
    }
    if (s >= a.T * a.top)
        return;
    const int64_t r = row_of_slot(a, s), t = s / a.top;
    float dot = 0.0f;
    if (r >= 0) {
        const float wt = a.weights ? a.weights[s] : 1.0f;
        const bool mine = !a.slots || a.slots[r] == s;   // the row's only writer
        const uint16_t *const gr = a.dout + t * a.K, *const yr = a.y + r * a.K;
        uint16_t *const out = a.out + r * a.K;
        const auto chunk = [&](uint4 gw, uint4 yw) {
            float g[8], y[8], o[8];
            widen(gw, g);
            widen(yw, y);
#pragma unroll
            for (int d = 0; d < 8; d++) {
                dot = __builtin_fmaf(g[d], y[d], dot);
                o[d] = wt * g[d];
            }
            return narrow(o);
        };
        // whole chunks, then the rest
        int64_t c = lane;
        for (; 8 * c + 8 <= a.K; c += 64) {
            const uint4 o = chunk(whole_chunk<false>(gr, c), whole_chunk<NT>(yr, c));
            if (mine)
                put_chunk<NT>(out, c, o);
        }
        if (8 * c < a.K) {
            const uint4 o = chunk(load_chunk<false>(gr, c, a.K), load_chunk<false>(yr, c, a.K));
            if (mine)
                store_chunk<false>(out, c, a.K, o);
        }
        dot = wave_sum(dot);
    }
    if (a.dweights && lane == 0)
        a.dweights[s] = dot;
}

hipError_t launch_combine_back(const CombineArgs &a, hipStream_t s)
{
    const int64_t zeros = a.slots ? (a.rows + kZeroRows - 1) / kZeroRows : 0;
    const dim3 grid((unsigned)((zeros + a.T * a.top + 3) / 4));
    if (rows_stream(a))
        hipLaunchKernelGGL(combine_back_kernel<true>, grid, dim3(256), 0, s, a, zeros);
    else
        hipLaunchKernelGGL(combine_back_kernel<false>, grid, dim3(256), 0, s, a, zeros);
    return hipGetLastError();
}

}  // namespace mxk
