// mm_pack.hip -- operands of the MXFP8 products with their rows moved to 128-byte
// boundaries.
//
// Rows of a length that is no multiple of 16 bytes start anywhere, and reading
// them 16 bytes at a time in the product's order costs the memory pipeline about
// three times the requests of aligned rows (a variant of the tiled kernel that
// did so took 1014 us for the weight gradients of 8 experts with 2050 rows each,
// 4096 x 7168; aligned, 2048 rows take 459 us).  Copying them once, read row by
// row, is cheaper than that: 589 us with 2049 rows, the copy and the product.
// Rows are filled up with zeros.
#include "mm_common.h"

namespace mxk {
namespace {

constexpr int kPackWaves = 4;

// One row, by a wave: row `id` of A's rows and then B's (weight gradients: of each
// group's).
__device__ __forceinline__ void pack_row(const MmArgs &a, const MmTable &t, uint8_t *qa, uint8_t *qb,
                                         int64_t id)
{
    const int lane = (int)threadIdx.x & 63;
    const uint8_t *array, *src;
    uint8_t *dst;
    int64_t K, left;
    if (a.sum_rows) {
        const int64_t each = a.dim + a.N;
        const int g = (int)(id / each);
        const int64_t r = id - g * each;
        K = t.rows[g];
        const int64_t pitch = mm_pitch(K);
        if (r < a.dim) {
            array = a.qa;
            src = a.qa + t.row0[g] * a.dim + r * K;
            dst = qa + t.packed0[g] * a.dim + r * pitch;
            left = a.qa + a.qa_bytes - src;
        } else {
            array = a.qb;
            src = a.qb + t.row0[g] * a.N + (r - a.dim) * K;
            dst = qb + t.packed0[g] * a.N + (r - a.dim) * pitch;
            left = a.qb + a.qb_bytes - src;
        }
    } else {
        K = a.dim;
        const int64_t ra = a.qa_bytes / K, pitch = mm_pitch(K);
        const bool second = id >= ra;
        const int64_t r = second ? id - ra : id;
        array = second ? a.qb : a.qa;
        src = array + r * K;
        dst = (second ? qb : qa) + r * pitch;
        left = array + (second ? a.qb_bytes : a.qa_bytes) - src;
    }
    const ByteRows<16> row(array, src, left);
    for (int64_t k = 16 * lane; k < mm_pitch(K); k += 16 * 64) {
        const int64_t at = k < K ? k : 0;
        uint4 v = row.load<uint4>(row.lead, at);
        if (k + 16 > K)
            v = k < K ? row.fix(v, row.lead, at, (int)(K - k)) : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4 *>(dst + k) = v;
    }
}

__host__ __device__ inline int64_t pack_rows(const MmArgs &a, const MmTable &t)
{
    return a.sum_rows ? t.count * (a.dim + a.N) : (a.qa_bytes + a.qb_bytes) / a.dim;
}

__global__ __launch_bounds__(64 * kPackWaves) void mm_pack_kernel(const MmArgs a, const MmTable t,
                                                                 uint8_t *qa, uint8_t *qb)
{
    const int64_t rows = pack_rows(a, t);
    for (int64_t id = (int64_t)blockIdx.x * kPackWaves + (threadIdx.x >> 6); id < rows;
         id += (int64_t)gridDim.x * kPackWaves)
        pack_row(a, t, qa, qb, id);
}

}  // namespace

hipError_t launch_mm_pack(const MmArgs &a, const MmTable &t, uint8_t *qa, uint8_t *qb, hipStream_t stream)
{
    const int64_t groups = (pack_rows(a, t) + kPackWaves - 1) / kPackWaves, most = int64_t(1) << 20;
    hipLaunchKernelGGL(mm_pack_kernel, dim3((unsigned)(groups < most ? groups : most)),
                       dim3(64 * kPackWaves), 0, stream, a, t, qa, qb);
    return hipGetLastError();
}

}  // namespace mxk
