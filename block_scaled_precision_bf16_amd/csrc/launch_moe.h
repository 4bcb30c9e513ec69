// launch_moe.h -- internal interface between the host API of the router and of
// the rows' way to the experts and back (api_moe.cpp) and their kernels.  Not
// installed.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace mxk {

struct RouteArgs {
    const void *logits;
    const float *bias;              // may be null
    int64_t T;
    int E, top, groups, top_groups;
    float scale;
    int sigmoid, renorm, pair, f32;
    int32_t *experts;
    float *weights, *scores;        // scores may be null
};

struct RouteBackArgs {
    const void *logits;
    const int32_t *experts;
    const float *dweights, *dscores;   // dscores may be null
    int64_t T;
    int E, top;
    float scale;
    int sigmoid, renorm, f32;
    void *dlogits;
};

struct SortArgs {
    const int32_t *experts;
    int64_t N;                      // slots
    int E, align;
    int64_t rows;
    int32_t *counts, *pos, *slots;
    int32_t *ws;                    // [blocks][E], or null for one launch
    int blocks, chunk;              // workgroups and slots of each
};

// Slots up to which one launch sorts, in up to 16 workgroups of 1024 threads and a
// whole number of 1024 slots each; beyond, workgroups of 512 threads take a whole
// number of 512 slots, at least 2048, and are at most 256.
constexpr int64_t kSortFew = 32768;
constexpr int kSortThreads = 512;
inline int64_t sort_chunk(int64_t N)
{
    if (N <= kSortFew)
        return 1024 * ((N + 16 * 1024 - 1) / (16 * 1024));
    const int64_t per = (N + 256 * kSortThreads - 1) / (256 * kSortThreads);
    return kSortThreads * (per < 4 ? 4 : per);
}

struct GatherArgs {
    const uint8_t *x;
    const int32_t *slots;
    int64_t T, rows, row_bytes;
    int top;
    uint8_t *out;
};

struct CombineArgs {
    const uint16_t *y, *dout;       // dout: the backward
    const int32_t *pos, *slots;     // null: slot i is row i
    const float *weights;           // may be null
    int64_t T, rows, K;
    int top;
    uint16_t *out;                  // forward: tokens; backward: dy
    float *dweights;                // may be null
};

hipError_t launch_route(const RouteArgs &a, hipStream_t s);
hipError_t launch_route_back(const RouteBackArgs &a, hipStream_t s);
hipError_t launch_sort(const SortArgs &a, hipStream_t s);
hipError_t launch_gather(const GatherArgs &a, hipStream_t s);
hipError_t launch_combine(const CombineArgs &a, hipStream_t s);
hipError_t launch_combine_back(const CombineArgs &a, hipStream_t s);

}  // namespace mxk
