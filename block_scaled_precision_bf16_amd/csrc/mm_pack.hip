// mm_pack.hip -- operands of the MXFP8 products with their rows moved to 128-byte
// boundaries.
//
// Rows of a length that is no multiple of 16 bytes start anywhere, and reading
// them 16 bytes at a time in the product's order costs the memory pipeline about
// three times the requests of aligned rows (a variant of the tiled kernel that
// did so took 1014 us for the weight gradients of 8 experts with 2050 rows each,
// 4096 x 7168).  Copying them once, read row by row, is cheaper: 535 us with 2049
// rows, of which the copy of 185 MB is about 95 (3.9 TB/s read and written); aligned,
// 2048 rows take 430 us.  Rows are filled up with zeros.
#include "mm_common.h"

namespace mxk {
namespace {

constexpr int kPackWaves = 4, kPackRows = 4;

// Where row `id` of A's rows and then B's (weight gradients: of each group's) is and
// goes.
struct PackRow {
    ByteRows<16> row;
    uint8_t *dst;
    int64_t K;
};

__device__ __forceinline__ PackRow pack_row(const MmArgs &a, const MmTable &t, uint8_t *qa, uint8_t *qb,
                                            int64_t id)
{
    if (a.sum_rows) {
        const int64_t each = a.dim + a.N;
        const int g = (int)(id / each);
        const int64_t r = id - g * each, K = t.rows[g], pitch = mm_pitch(K);
        if (r < a.dim) {
            const uint8_t *src = a.qa + t.row0[g] * a.dim + r * K;
            return {ByteRows<16>(a.qa, src, a.qa + a.qa_bytes - src), qa + t.packed0[g] * a.dim + r * pitch, K};
        }
        const uint8_t *src = a.qb + t.row0[g] * a.N + (r - a.dim) * K;
        return {ByteRows<16>(a.qb, src, a.qb + a.qb_bytes - src), qb + t.packed0[g] * a.N + (r - a.dim) * pitch, K};
    }
    const int64_t K = a.dim, ra = a.qa_bytes / K;
    if (id < ra)
        return {ByteRows<16>(a.qa, a.qa + id * K, a.qa_bytes - id * K), qa + id * mm_pitch(K), K};
    return {ByteRows<16>(a.qb, a.qb + (id - ra) * K, a.qb_bytes - (id - ra) * K), qb + (id - ra) * mm_pitch(K), K};
}

__host__ __device__ inline int64_t pack_rows(const MmArgs &a, const MmTable &t)
{
    return a.sum_rows ? t.count * (a.dim + a.N) : (a.qa_bytes + a.qb_bytes) / a.dim;
}

__global__ __launch_bounds__(64 * kPackWaves) void mm_pack_kernel(const MmArgs a, const MmTable t,
                                                                 uint8_t *qa, uint8_t *qb)
{
    // a wave's kPackRows rows at a time, all loads before the first store
    const int lane = (int)threadIdx.x & 63;
    const int64_t rows = pack_rows(a, t), step = (int64_t)gridDim.x * kPackWaves * kPackRows;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    for (int64_t id = ((int64_t)blockIdx.x * kPackWaves + wave) * kPackRows; id < rows; id += step) {
        PackRow p[kPackRows];
        int64_t most = 0;
#pragma unroll
        for (int i = 0; i < kPackRows; i++) {
            p[i] = pack_row(a, t, qa, qb, id + i < rows ? id + i : rows - 1);
            most = p[i].K > most ? p[i].K : most;
        }
        for (int64_t k = 16 * lane; k < mm_pitch(most); k += 16 * 64) {
            uint4 v[kPackRows];
#pragma unroll
            for (int i = 0; i < kPackRows; i++)
                v[i] = p[i].row.load<uint4>(p[i].row.lead, k < p[i].K ? k : 0);
#pragma unroll
            for (int i = 0; i < kPackRows; i++) {
                const int64_t K = p[i].K;
                if (k + 16 > K)
                    v[i] = k < K ? p[i].row.fix(v[i], p[i].row.lead, k, (int)(K - k)) : make_uint4(0, 0, 0, 0);
                if (k < mm_pitch(K) && id + i < rows)
                    *reinterpret_cast<uint4 *>(p[i].dst + k) = v[i];
            }
        }
    }
}

}  // namespace

hipError_t launch_mm_pack(const MmArgs &a, const MmTable &t, uint8_t *qa, uint8_t *qb, hipStream_t stream)
{
    constexpr int each = kPackWaves * kPackRows;
    const int64_t groups = (pack_rows(a, t) + each - 1) / each, most = int64_t(1) << 20;
    hipLaunchKernelGGL(mm_pack_kernel, dim3((unsigned)(groups < most ? groups : most)),
                       dim3(64 * kPackWaves), 0, stream, a, t, qa, qb);
    return hipGetLastError();
}

}  // namespace mxk
