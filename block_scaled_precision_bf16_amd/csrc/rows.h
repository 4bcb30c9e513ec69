// rows.h -- chunks of 8 elements of rows that start at any element: bf16 rows of a
// length that is no multiple of 8, and the 8-bit codes of such rows.  gfx950 takes
// vector accesses at any byte; a chunk that its row ends inside goes element by
// element, so that nothing outside the row is touched.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bufio.h"

namespace mxk {

typedef u32x4_t __attribute__((aligned(2))) u32x4_any;
typedef u32x2_t __attribute__((aligned(1))) u32x2_any;
typedef u32x4_t __attribute__((aligned(1))) u32x4_bytes;

// A chunk, elements 8 c .. 8 c + 7 of the row at p, that is wholly inside the row; NT:
// non-temporally.
template <bool NT>
__device__ __forceinline__ uint4 whole_chunk(const uint16_t *p, int64_t c)
{
    const u32x4_any *const q = reinterpret_cast<const u32x4_any *>(p + 8 * c);
    const u32x4_t v = NT ? (u32x4_t)__builtin_nontemporal_load(q) : (u32x4_t)*q;
    return make_uint4(v[0], v[1], v[2], v[3]);
}
template <bool NT>
__device__ __forceinline__ void put_chunk(uint16_t *p, int64_t c, uint4 v)
{
    u32x4_any *const q = reinterpret_cast<u32x4_any *>(p + 8 * c);
    const u32x4_any u = {v.x, v.y, v.z, v.w};
    if constexpr (NT)
        __builtin_nontemporal_store(u, q);
    else
        *q = u;
}

// The same of any chunk of a row of `len` elements (0 past the end).
template <bool NT>
__device__ __forceinline__ uint4 load_chunk(const uint16_t *p, int64_t c, int64_t len)
{
    if (8 * c + 8 <= len)
        return whole_chunk<NT>(p, c);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 7; i++)
        if (8 * c + i < len)
            w[i >> 1] |= (uint32_t)p[8 * c + i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool NT>
__device__ __forceinline__ void store_chunk(uint16_t *p, int64_t c, int64_t len, uint4 v)
{
    if (8 * c + 8 <= len) {
        put_chunk<NT>(p, c, v);
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 7; i++)
        if (8 * c + i < len)
            p[8 * c + i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}

// The same of 8-bit codes.
template <bool NT>
__device__ __forceinline__ uint2 load_codes(const uint8_t *p, int64_t c, int64_t len)
{
    if (8 * c + 8 <= len) {
        const u32x2_any *const q = reinterpret_cast<const u32x2_any *>(p + 8 * c);
        const u32x2_t v = NT ? (u32x2_t)__builtin_nontemporal_load(q) : (u32x2_t)*q;
        return make_uint2(v[0], v[1]);
    }
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 7; i++)
        if (8 * c + i < len)
            w[i >> 2] |= (uint32_t)p[8 * c + i] << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}

template <bool NT>
__device__ __forceinline__ void store_codes(uint8_t *p, int64_t c, int64_t len, uint2 v)
{
    if (8 * c + 8 <= len) {
        u32x2_any *const q = reinterpret_cast<u32x2_any *>(p + 8 * c);
        const u32x2_any u = {v.x, v.y};
        if constexpr (NT)
            __builtin_nontemporal_store(u, q);
        else
            *q = u;
        return;
    }
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 7; i++)
        if (8 * c + i < len)
            p[8 * c + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
}

// A row of bf16 (T = uint16_t) or codes (uint8_t) of `len` elements, none of them
// where len is 0: by a buffer descriptor where every chunk is whole and aligned (AL),
// which masks those past the end, or by its address.
template <bool AL, class T>
struct Row {
    rsrc_t r;
    T *p;
    int64_t len;
};

template <bool AL, class T>
__device__ __forceinline__ Row<AL, T> row_at(T *p, int64_t at, int64_t len)
{
    Row<AL, T> v;
    if constexpr (AL)
        v.r = make_rsrc(p + (len ? at : 0), 0, (int64_t)sizeof(T) * len);
    else
        v.p = p + (len ? at : 0);
    v.len = len;
    return v;
}

// AUX: the descriptors' policy; without one, any policy but 0 is non-temporal.
template <int AUX, bool AL>
__device__ __forceinline__ uint4 row_load(const Row<AL, const uint16_t> &v, uint32_t c)
{
    if constexpr (AL)
        return buf_load16<AUX>(v.r, 16 * c);
    else
        return load_chunk<AUX != 0>(v.p, c, v.len);
}
template <int AUX, bool AL>
__device__ __forceinline__ uint2 row_load(const Row<AL, const uint8_t> &v, uint32_t c)
{
    if constexpr (AL)
        return buf_load8<AUX>(v.r, 8 * c);
    else
        return load_codes<AUX != 0>(v.p, c, v.len);
}
template <int AUX, bool AL>
__device__ __forceinline__ void row_store(const Row<AL, uint16_t> &v, uint32_t c, uint4 w)
{
    if constexpr (AL)
        buf_store16<AUX>(v.r, 16 * c, w);
    else
        store_chunk<AUX != 0>(v.p, c, v.len, w);
}
template <int AUX, bool AL>
__device__ __forceinline__ void row_store(const Row<AL, uint8_t> &v, uint32_t c, uint2 w)
{
    if constexpr (AL)
        buf_store8<AUX>(v.r, 8 * c, w);
    else
        store_codes<AUX != 0>(v.p, c, v.len, w);
}

}  // namespace mxk
