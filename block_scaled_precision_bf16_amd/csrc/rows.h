// rows.h -- chunks of 8 elements of rows that start at any element: bf16 rows of a
// length that is no multiple of 8, and the 8-bit codes of such rows.  gfx950 takes
// vector accesses at any byte; a chunk that its row ends inside is loaded with the
// elements before it and stored element by element, so that nothing outside the row is
// touched.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "bufio.h"

namespace mxk {

typedef u32x4_t __attribute__((aligned(2))) u32x4_any;
typedef u32x2_t __attribute__((aligned(1))) u32x2_any;
typedef u32x4_t __attribute__((aligned(1))) u32x4_bytes;

// Rows are at most 2^24 bytes long: 32-bit offsets from a row's (uniform) address.
template <class V, class T>
__device__ __forceinline__ V *at_of(T *p, uint32_t i)
{
    typedef typename std::conditional<std::is_const<T>::value, const char, char>::type byte;
    return reinterpret_cast<V *>(reinterpret_cast<byte *>(p) + (uint32_t)(sizeof(T) * i));
}
template <bool NT, class V>
__device__ __forceinline__ auto load_any(const V *q)
{
    return NT ? __builtin_nontemporal_load(q) : *q;
}

// A chunk, elements 8 c .. 8 c + 7 of the row at p, that is wholly inside the row; NT:
// non-temporally.
template <bool NT>
__device__ __forceinline__ uint4 eight_at(const uint16_t *p, uint32_t i)
{
    const u32x4_t v = load_any<NT>(at_of<const u32x4_any>(p, i));
    return make_uint4(v[0], v[1], v[2], v[3]);
}
template <bool NT>
__device__ __forceinline__ uint4 whole_chunk(const uint16_t *p, uint32_t c)
{
    return eight_at<NT>(p, 8 * c);
}
template <bool NT>
__device__ __forceinline__ void put_chunk(uint16_t *p, uint32_t c, uint4 v)
{
    u32x4_any *const q = at_of<u32x4_any>(p, 8 * c);
    const u32x4_any u = {v.x, v.y, v.z, v.w};
    if constexpr (NT)
        __builtin_nontemporal_store(u, q);
    else
        *q = u;
}

// The same of any chunk of a row of `len` elements (0 past the end), in two steps: the
// load, which takes the row's last 8 elements for a chunk that it ends inside, and,
// once they are there, their way down to the chunk's first places.  (Element by element
// the wave would wait for each.)
template <bool NT>
__device__ __forceinline__ uint4 raw_chunk(const uint16_t *p, uint32_t c, uint32_t len)
{
    if (len >= 8)
        return 8 * c < len ? eight_at<NT>(p, 8 * c + 8 <= len ? 8 * c : len - 8) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (uint32_t i = 0; i < 7; i++)
        if (8 * c + i < len)
            w[i >> 1] |= (uint32_t)*at_of<const uint16_t>(p, 8 * c + i) << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 fix_chunk(uint4 v, uint32_t c, uint32_t len)
{
    const int past = (int)(8 * c + 8 - len);      // 1 to 7 elements in the row's last chunk
    if (len < 8 || past <= 0 || past >= 8)
        return v;
    const int bits = 16 * past;
    uint64_t lo = ((uint64_t)v.y << 32) | v.x, hi = ((uint64_t)v.w << 32) | v.z;
    lo = bits >= 64 ? hi >> (bits - 64) : (lo >> bits) | (hi << (64 - bits));
    hi = bits >= 64 ? 0u : hi >> bits;
    return make_uint4((uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32));
}
template <bool NT>
__device__ __forceinline__ uint4 load_chunk(const uint16_t *p, uint32_t c, uint32_t len)
{
    return fix_chunk(raw_chunk<NT>(p, c, len), c, len);
}

template <bool NT>
__device__ __forceinline__ void store_chunk(uint16_t *p, uint32_t c, uint32_t len, uint4 v)
{
    if (8 * c + 8 <= len) {
        put_chunk<NT>(p, c, v);
        return;
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (uint32_t i = 0; i < 7; i++)
        if (8 * c + i < len)
            *at_of<uint16_t>(p, 8 * c + i) = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
}

// The same of 8-bit codes.
template <bool NT>
__device__ __forceinline__ uint2 raw_codes(const uint8_t *p, uint32_t c, uint32_t len)
{
    if (len >= 8) {
        if (8 * c >= len)
            return make_uint2(0u, 0u);
        const u32x2_t v = load_any<NT>(at_of<const u32x2_any>(p, 8 * c + 8 <= len ? 8 * c : len - 8));
        return make_uint2(v[0], v[1]);
    }
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (uint32_t i = 0; i < 7; i++)
        if (8 * c + i < len)
            w[i >> 2] |= (uint32_t)*at_of<const uint8_t>(p, 8 * c + i) << (8 * (i & 3));
    return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ uint2 fix_codes(uint2 v, uint32_t c, uint32_t len)
{
    const int past = (int)(8 * c + 8 - len);
    if (len < 8 || past <= 0 || past >= 8)
        return v;
    const uint64_t u = (((uint64_t)v.y << 32) | v.x) >> (8 * past);
    return make_uint2((uint32_t)u, (uint32_t)(u >> 32));
}
template <bool NT>
__device__ __forceinline__ uint2 load_codes(const uint8_t *p, uint32_t c, uint32_t len)
{
    return fix_codes(raw_codes<NT>(p, c, len), c, len);
}

template <bool NT>
__device__ __forceinline__ void store_codes(uint8_t *p, uint32_t c, uint32_t len, uint2 v)
{
    if (8 * c + 8 <= len) {
        u32x2_any *const q = at_of<u32x2_any>(p, 8 * c);
        const u32x2_any u = {v.x, v.y};
        if constexpr (NT)
            __builtin_nontemporal_store(u, q);
        else
            *q = u;
        return;
    }
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (uint32_t i = 0; i < 7; i++)
        if (8 * c + i < len)
            *at_of<uint8_t>(p, 8 * c + i) = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
}

// A row of bf16 (T = uint16_t) or codes (uint8_t) of `len` elements, none of them
// where len is 0: by a buffer descriptor where every chunk is whole and aligned (AL),
// which masks those past the end, or by its address.
template <bool AL, class T>
struct Row {
    rsrc_t r;
    T *p;
    uint32_t len;
};

template <bool AL, class T>
__device__ __forceinline__ Row<AL, T> row_at(T *p, int64_t at, int64_t len)
{
    Row<AL, T> v;
    if constexpr (AL)
        v.r = make_rsrc(p + (len ? at : 0), 0, (int64_t)sizeof(T) * len);
    else
        v.p = p + (len ? at : 0);
    v.len = (uint32_t)len;
    return v;
}

// AUX: the descriptors' policy; without one, any policy but 0 is non-temporal.  raw:
// without the second step, row_fix, which takes the row's length.
template <int AUX, bool AL>
__device__ __forceinline__ uint4 row_raw(const Row<AL, const uint16_t> &v, uint32_t c)
{
    if constexpr (AL)
        return buf_load16<AUX>(v.r, 16 * c);
    else
        return raw_chunk<AUX != 0>(v.p, c, v.len);
}
template <int AUX, bool AL>
__device__ __forceinline__ uint2 row_raw(const Row<AL, const uint8_t> &v, uint32_t c)
{
    if constexpr (AL)
        return buf_load8<AUX>(v.r, 8 * c);
    else
        return raw_codes<AUX != 0>(v.p, c, v.len);
}
template <bool AL>
__device__ __forceinline__ uint4 row_fix(uint4 v, uint32_t c, uint32_t len)
{
    return AL ? v : fix_chunk(v, c, len);
}
template <bool AL>
__device__ __forceinline__ uint2 row_fix(uint2 v, uint32_t c, uint32_t len)
{
    return AL ? v : fix_codes(v, c, len);
}
template <int AUX, bool AL>
__device__ __forceinline__ uint4 row_load(const Row<AL, const uint16_t> &v, uint32_t c)
{
    return row_fix<AL>(row_raw<AUX>(v, c), c, v.len);
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
