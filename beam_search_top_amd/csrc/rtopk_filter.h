// Internal interface between the host side (rtopk_filter.cpp) of filtered
// sampling and its kernels (rtopk_filter.hip). Not part of the ABI.
#pragma once

#include "rtopk_internal.h"

namespace rtopk {

constexpr int kFilterMaxV = 1 << 24; // 38 bits behind a weight's binary point
constexpr int kFilterMaxR = 1 << 20; // a workgroup of 1024 threads each: a launch counts its threads in 32 bits

struct FilterArgs {
    const void *logits;  // [R][ld]
    int R, V;
    int64_t ld;
    int frac;            // bits of a weight behind the binary point (filter_frac)
    const float *temperature, *top_p, *min_p; // [R] or null
    const int32_t *top_k; // [R] or null
    const float *u;      // [R]
    int32_t *out_token;
    float *out_logprob;
};

// Weights are whole numbers, exp((x - max) / T) times 2^frac, the largest 2^frac: V of
// them stay below 2^62, so that sums are exact and do not depend on their order.
constexpr int filter_frac(int V)
{
    int l = 0;
    while ((1ll << l) < V)
        ++l;
    return 62 - l < 50 ? 62 - l : 50;
}

// Workgroups per row (1: no workspace is needed).
constexpr int kFilterChunks = 64;
constexpr size_t kFilterRowBytes = 49920; // workspace of a row that is cut
inline int filter_chunks(int R, int V)
{
    const int slots = 512 / R, most = V / 4096; // two workgroups on each of 256 CUs
    const int c = slots < most ? slots : most;
    return c < 2 ? 1 : c < kFilterChunks ? c : kFilterChunks;
}
hipError_t launch_filter(const FilterArgs &a, int dtype, int chunks, void *ws, hipStream_t s);

} // namespace rtopk
