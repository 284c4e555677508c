// Rows of a head in registers: loads and stores of one element or of 16 bytes, as
// float32, and sums and maxima over the lanes of a group. For the kernels of the
// rotation and of the 8-bit cache.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace rtopk {

typedef uint32_t row_u32x4 __attribute__((ext_vector_type(4)));

// The types by their codes: 0 float32, 1 float16, 2 bfloat16.
template <int DT> struct RowType;
template <> struct RowType<0> { typedef float T; };
template <> struct RowType<1> { typedef _Float16 T; };
template <> struct RowType<2> { typedef __bf16 T; };

template <int DT> struct Row {
    typedef typename RowType<DT>::T T;
    static constexpr int kWide = 16 / (int)sizeof(T); // elements of 16 bytes
    // N elements at p, 16 bytes at a time where N is at least that many, else one element
    template <int N> static __device__ __forceinline__ void load(const T *p, float (&x)[N])
    {
        if constexpr (N == 1) {
            x[0] = (float)*p;
        } else {
            static_assert(N % kWide == 0, "whole loads");
#pragma unroll
            for (int i = 0; i < N / kWide; ++i) {
                typedef T V __attribute__((ext_vector_type(kWide)));
                const V v = __builtin_bit_cast(V, __builtin_nontemporal_load(reinterpret_cast<const row_u32x4 *>(p) + i));
#pragma unroll
                for (int e = 0; e < kWide; ++e)
                    x[i * kWide + e] = (float)v[e];
            }
        }
    }
    template <int N> static __device__ __forceinline__ void store(T *p, const float (&x)[N])
    {
        if constexpr (N == 1) {
            *p = (T)x[0];
        } else {
#pragma unroll
            for (int i = 0; i < N / kWide; ++i) {
                typedef T V __attribute__((ext_vector_type(kWide)));
                V v;
#pragma unroll
                for (int e = 0; e < kWide; ++e)
                    v[e] = (T)x[i * kWide + e];
                reinterpret_cast<row_u32x4 *>(p)[i] = __builtin_bit_cast(row_u32x4, v);
            }
        }
    }
};

// x of the lane that DPP control CTRL names (every lane has one here)
template <int CTRL> __device__ __forceinline__ uint32_t lane_by(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, false);
}

// f over the lanes of a group of G = 4 ... 64 that all run, by exchanges within
// four lanes, mirrored halves of 8 and 16, and swaps of the rows of 16. Every lane
// gets the same bits: at each step two lanes combine the same two values.
template <int G, typename F> __device__ __forceinline__ uint32_t group_all(uint32_t x, F f)
{
    x = f(x, lane_by<0xb1>(x)); // quad_perm 1 0 3 2
    x = f(x, lane_by<0x4e>(x)); // quad_perm 2 3 0 1
    if (G >= 8)
        x = f(x, lane_by<0x141>(x)); // row_half_mirror
    if (G >= 16)
        x = f(x, lane_by<0x140>(x)); // row_mirror
    if (G >= 32) {
        const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        x = f(s[0], s[1]);
    }
    if (G >= 64) {
        const auto s = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        x = f(s[0], s[1]);
    }
    return x;
}
template <int G> __device__ __forceinline__ float group_sum(float x)
{
    return __uint_as_float(group_all<G>(__float_as_uint(x), [](uint32_t p, uint32_t q) {
        return __float_as_uint(__uint_as_float(p) + __uint_as_float(q));
    }));
}
// The same for a sum in 64 bits, whose halves move one after the other.
template <int CTRL> __device__ __forceinline__ double plus_lane(double x)
{
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    return x + __builtin_bit_cast(double, (uint64_t)lane_by<CTRL>((uint32_t)(b >> 32)) << 32 | lane_by<CTRL>((uint32_t)b));
}
template <int G> __device__ __forceinline__ double group_sum(double x)
{
    const auto halves = [](uint32_t hi, uint32_t lo) { return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo); };
    x = plus_lane<0x4e>(plus_lane<0xb1>(x));
    if (G >= 8)
        x = plus_lane<0x141>(x);
    if (G >= 16)
        x = plus_lane<0x140>(x);
    if (G >= 32) {
        const uint64_t b = __builtin_bit_cast(uint64_t, x);
        const auto hi = __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
        const auto lo = __builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false);
        x = halves(hi[0], lo[0]) + halves(hi[1], lo[1]);
    }
    if (G >= 64) {
        const uint64_t b = __builtin_bit_cast(uint64_t, x);
        const auto hi = __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false);
        const auto lo = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false);
        x = halves(hi[0], lo[0]) + halves(hi[1], lo[1]);
    }
    return x;
}
template <int G> __device__ __forceinline__ uint32_t group_max(uint32_t x)
{
    return group_all<G>(x, [](uint32_t p, uint32_t q) { return p > q ? p : q; });
}

} // namespace rtopk
