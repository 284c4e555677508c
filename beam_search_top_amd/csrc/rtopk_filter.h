// Internal interface between the host side (rtopk_filter.cpp) of filtered
// sampling and its kernels (rtopk_filter.hip), and arithmetic of theirs that a plain
// C++ compiler reads too, so that tests run it on the CPU. Not part of the ABI.
#pragma once

#include "rtopk_pages.h"

#if !defined(RTOPK_ARITHMETIC_ONLY)
#include "rtopk_internal.h"
#endif

namespace rtopk {

constexpr int kFilterMaxV = 1 << 24; // 38 bits behind a weight's binary point
constexpr int kFilterMaxR = 1 << 20; // a workgroup of 512 threads each: a launch counts its threads in 32 bits

#if !defined(RTOPK_ARITHMETIC_ONLY)
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
#endif

// Weights are whole numbers, exp((x - max) / T) times 2^frac, the largest 2^frac: V of
// them stay below 2^62, so that sums are exact and do not depend on their order.
constexpr int filter_frac(int V)
{
    int l = 0;
    while ((1ll << l) < V)
        ++l;
    return 62 - l < 50 ? 62 - l : 50;
}

// f times total, rounded down, or up: exact, where a double would drop the product's bits below
// the 53rd and with them a border between two sums. f (by its float32 bits) is in [0, 1), so that it is
// m 2^-(d + 32) with m < 2^32 and d >= 0; total <= 2^62. The product is high 2^32 + (lows mod 2^32).
RTOPK_HD uint64_t part_of(uint32_t f, uint64_t total, bool up)
{
    const uint32_t e = f >> 23, m = (e ? (f & 0x7fffffu) | 0x800000u : f) << 8;
    const int d = 126 - (int)(e ? e : 1u);
    const uint64_t lows = m * (total & 0xffffffffu), high = m * (total >> 32) + (lows >> 32);
    const uint64_t whole = d < 64 ? high >> d : 0;
    return whole + (up && ((d < 64 ? whole << d : 0) != high || (uint32_t)lows != 0));
}

// Workgroups per row (1: no workspace is needed).
constexpr int kFilterChunks = 64;
constexpr size_t kFilterRowBytes = 49920; // workspace of a row that is cut
// counts: top-k without top-p
inline int filter_chunks(int R, int V, bool counts)
{
    // Three launches and the workspace between them cost about 15 us whatever the size; a row's own workgroup takes
    // 20 to 40 us per 40000 logits, and leaves CUs idle up to 256 rows. us cut / not, bfloat16, every filter: 1 x 16000
    // 17 / 11, 16 x 24000 25 / 24, 64 x 24000 34 / 27; 1 x 28672 16 / 17, 32 x 32000 29 / 31, 64 x 40000 35 / 37,
    // 128 x 32000 37 / 38, 128 x 100000 62 / 81, 8 x 250000 34 / 182. With 129 to 170 rows, of three chunks each, it pays from
    // longer rows on: 160 x 60000 56 / 55, 160 x 70000 62 / 61, 160 x 80000 66 / 70, 160 x 150000 101 / 140, 170 x 250000
    // 150 / 189 (top-p alone 57 / 59, 57 / 62, 61 / 81, 92 / 141, 135 / 192); with two chunks it does not: 200 x 60000 69 / 56,
    // 200 x 100000 99 / 89, 200 x 250000 206 / 190, 256 x 100000 99 / 83.
    // Top-k alone weighs only what it keeps, and a row's own workgroup takes half as long: 1 x 30000 17 / 15,
    // 8 x 30000 20 / 18, 8 x 60000 21 / 26, 32 x 30000 22 / 18, 32 x 60000 26 / 27, 64 x 60000 29 / 27, 64 x 100000 35 / 38,
    // 96 x 100000 41 / 39, 128 x 100000 46 / 39, 128 x 250000 86 / 90, 160 x 250000 105 / 91.
    const int most = V / 4096;
    if (R > 170 || most < 7 || (R > 128 && (counts || V < 1 << 16)) || (counts && V < 1024 * (R + 32)))
        return 1;
    const int slots = 512 / R, c = slots < most ? slots : most; // two workgroups on each of 256 CUs
    return c < kFilterChunks ? c : kFilterChunks;
}
#if !defined(RTOPK_ARITHMETIC_ONLY)
hipError_t launch_filter(const FilterArgs &a, int dtype, int chunks, void *ws, hipStream_t s);
#endif

} // namespace rtopk
