// gfx950 kernels of the paged cache in 8 bits: the store that quantises keys
// and values as it writes them, and the reading back. Format: rtopk_cache8.h.
#include <hip/hip_runtime.h>

#include "rtopk_cache8.h"
#include "rtopk_internal.h"
#include "rtopk_rows.h"

namespace rtopk {
namespace {

constexpr int kC8Threads = 256;

// Where token `slot`'s row of head h lies: codes at .at, its scale at .scale; false: nowhere
struct Place8 {
    int64_t at, scale;
};
__device__ __forceinline__ bool place8(const Cache8Args &a, int32_t slot, int h, Place8 &p)
{
    if ((uint32_t)slot >= (uint32_t)a.nslots)
        return false;
    const uint32_t pg = page_of(a.page, (uint32_t)slot), off = (uint32_t)slot - pg * a.page.d;
    p.at = (int64_t)pg * a.cs[0] + (int64_t)off * a.cs[1] + (int64_t)h * a.cs[2];
    p.scale = (int64_t)slot * a.Hkv + h;
    return true;
}

// Four values, each at most 448 or NaN, as e4m3 codes (round to nearest, ties to even).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}
__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// One row of a tensor: N elements per lane of a group of LPH, the lane's first at
// e0, the others behind it (N of 16 bytes and more) or LPH apart (one at a time).
template <int DT, int LPH> struct Quantise {
    template <int N> static __device__ __forceinline__ uint32_t scale(const float (&x)[N])
    {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const uint32_t y = __float_as_uint(x[e]) & 0x7fffffffu;
            m = finite(x[e]) && y > m ? y : m;
        }
        return scale_of(group_max<LPH>(m));
    }
    // x over the power of two; an infinity or a NaN becomes NaN
    static __device__ __forceinline__ float scaled(float x, float inverse)
    {
        const float lim = stored_limit(DT);
        const float y = x > lim ? lim : x < -lim ? -lim : x;
        return finite(x) ? y * inverse : __builtin_nanf("");
    }
};

// A workgroup takes `tpw` tokens; every row (a head of a token) is a group of LPH
// lanes, 16 elements each, which takes the key's and the value's row together, so that the
// largest element is found by lane moves alone. Bound by HBM: 130001 tokens of 8 heads of 128, bfloat16, 152 us,
// 5.25 TB/s read and written; 200 tokens of 16 x 64 3.6 us, the call on the host 8.
template <int DT, int LPH> __global__ __launch_bounds__(kC8Threads) void cache8_store(const Cache8Args a)
{
    typedef Row<DT> X;
    typedef typename X::T T;
    typedef Quantise<DT, LPH> Q;
    const int64_t t0 = (int64_t)blockIdx.x * a.tpw;
    const int nt = (int)(t0 + a.tpw < a.T ? a.tpw : a.T - t0), rows = nt * a.Hkv;
    const int j = threadIdx.x % LPH, e0 = 16 * j;
    for (int r = threadIdx.x / LPH; r < rows; r += kC8Threads / LPH) {
        const int t = (int)page_of(a.heads, (uint32_t)r), h = r - t * a.Hkv;
        Place8 p;
        if (!place8(a, a.slots[t0 + t], h, p))
            continue; // the same for the lanes of a row
        float x[2][16] = {};
        if (e0 < a.D) {
            X::load(static_cast<const T *>(a.k) + (t0 + t) * a.ks[0] + h * a.ks[1] + e0, x[0]);
            X::load(static_cast<const T *>(a.v) + (t0 + t) * a.vs[0] + h * a.vs[1] + e0, x[1]);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const uint32_t s = Q::scale(x[y]);
            const float inv = __uint_as_float(inverse_bits(s));
            row_u32x4 c;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                c[e] = codes4(Q::scaled(x[y][4 * e], inv), Q::scaled(x[y][4 * e + 1], inv), Q::scaled(x[y][4 * e + 2], inv),
                              Q::scaled(x[y][4 * e + 3], inv));
            if (e0 < a.D)
                *reinterpret_cast<row_u32x4 *>((y ? a.vc : a.kc) + p.at + e0) = c;
            if (j == 0)
                (y ? a.vsc : a.ksc)[p.scale] = (uint8_t)s;
        }
    }
}

// The same for other strides, alignments and sizes: a wave per row, one element at a time.
template <int DT> __global__ __launch_bounds__(kC8Threads) void cache8_store_any(const Cache8Args a)
{
    typedef Row<DT> X;
    typedef typename X::T T;
    typedef Quantise<DT, 64> Q;
    constexpr int N = kMaxRowDim / 64;
    const int64_t t0 = (int64_t)blockIdx.x * a.tpw;
    const int nt = (int)(t0 + a.tpw < a.T ? a.tpw : a.T - t0), rows = nt * a.Hkv;
    const int lane = threadIdx.x % 64;
    for (int r = threadIdx.x / 64; r < rows; r += kC8Threads / 64) {
        const int t = (int)page_of(a.heads, (uint32_t)r), h = r - t * a.Hkv;
        Place8 p;
        if (!place8(a, a.slots[t0 + t], h, p))
            continue;
        for (int y = 0; y < 2; ++y) {
            const T *from = static_cast<const T *>(y ? a.v : a.k) + (t0 + t) * (y ? a.vs : a.ks)[0] + h * (y ? a.vs : a.ks)[1];
            float x[N];
#pragma unroll
            for (int i = 0; i < N; ++i)
                x[i] = lane + 64 * i < a.D ? (float)from[lane + 64 * i] : 0.f;
            const uint32_t s = Q::scale(x);
            const float inv = __uint_as_float(inverse_bits(s));
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (lane + 64 * i < a.D)
                    (y ? a.vc : a.kc)[p.at + lane + 64 * i] = (uint8_t)codes4(Q::scaled(x[i], inv), 0.f, 0.f, 0.f);
            if (lane == 0)
                (y ? a.vsc : a.ksc)[p.scale] = (uint8_t)s;
        }
    }
}

// The way back: the same groups; codes are read once (non-temporal), rows written 16 bytes at a time. Bound by HBM:
// 100001 tokens of 8 x 128, pages of 24, 125 us, 4.93 TB/s; 500 tokens of 16 x 64 3.3 us.
template <int DT, int LPH> __global__ __launch_bounds__(kC8Threads) void cache8_load(const Cache8Args a)
{
    typedef Row<DT> X;
    typedef typename X::T T;
    const int64_t t0 = (int64_t)blockIdx.x * a.tpw;
    const int nt = (int)(t0 + a.tpw < a.T ? a.tpw : a.T - t0), rows = nt * a.Hkv;
    const int e0 = 16 * (threadIdx.x % LPH);
    if (e0 >= a.D)
        return;
    for (int r = threadIdx.x / LPH; r < rows; r += kC8Threads / LPH) {
        const int t = (int)page_of(a.heads, (uint32_t)r), h = r - t * a.Hkv;
        Place8 p{0, 0};
        const bool in = place8(a, a.slots[t0 + t], h, p);
        const int64_t to = ((t0 + t) * a.Hkv + h) * a.D + e0;
        row_u32x4 c[2] = {};
        uint32_t s[2] = {kMinScale, kMinScale};
        if (in) {
            c[0] = __builtin_nontemporal_load(reinterpret_cast<const row_u32x4 *>(a.kc + p.at + e0));
            c[1] = __builtin_nontemporal_load(reinterpret_cast<const row_u32x4 *>(a.vc + p.at + e0));
            s[0] = a.ksc[p.scale];
            s[1] = a.vsc[p.scale];
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const float by = __uint_as_float(scale_bits(held_scale(s[y])));
            float x[16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[y][e], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[y][e], true);
                x[4 * e] = lo[0] * by;
                x[4 * e + 1] = lo[1] * by;
                x[4 * e + 2] = hi[0] * by;
                x[4 * e + 3] = hi[1] * by;
            }
            X::store(static_cast<T *>(y ? a.v_out : a.k_out) + to, x);
        }
    }
}

template <int DT> __global__ __launch_bounds__(kC8Threads) void cache8_load_any(const Cache8Args a)
{
    typedef typename Row<DT>::T T;
    const int64_t t0 = (int64_t)blockIdx.x * a.tpw;
    const int nt = (int)(t0 + a.tpw < a.T ? a.tpw : a.T - t0), rows = nt * a.Hkv;
    for (int r = threadIdx.x / 64; r < rows; r += kC8Threads / 64) {
        const int t = (int)page_of(a.heads, (uint32_t)r), h = r - t * a.Hkv;
        Place8 p{0, 0};
        const bool in = place8(a, a.slots[t0 + t], h, p);
        const int64_t to = ((t0 + t) * a.Hkv + h) * a.D;
        for (int y = 0; y < 2; ++y) {
            const float by = __uint_as_float(scale_bits(held_scale(in ? (y ? a.vsc : a.ksc)[p.scale] : kMinScale)));
            for (int e = threadIdx.x % 64; e < a.D; e += 64) {
                const int c = in ? (y ? a.vc : a.kc)[p.at + e] : 0;
                static_cast<T *>(y ? a.v_out : a.k_out)[to + e] = (T)(__builtin_amdgcn_cvt_pk_f32_fp8(c, false)[0] * by);
            }
        }
    }
}

// Kernels by the lanes of a row of 16 elements each, or the one for any row
#define RTOPK_C8(KERNEL, DT)                                                                                           \
    do {                                                                                                               \
        const int64_t blocks = (a.T + a.tpw - 1) / a.tpw;                                                              \
        const dim3 grid((unsigned)blocks), block(kC8Threads);                                                          \
        if (!wide)                                                                                                     \
            hipLaunchKernelGGL(KERNEL##_any<DT>, grid, block, 0, s, a);                                                \
        else if (a.D <= 64)                                                                                            \
            hipLaunchKernelGGL((KERNEL<DT, 4>), grid, block, 0, s, a);                                                 \
        else if (a.D <= 128)                                                                                           \
            hipLaunchKernelGGL((KERNEL<DT, 8>), grid, block, 0, s, a);                                                 \
        else                                                                                                           \
            hipLaunchKernelGGL((KERNEL<DT, 16>), grid, block, 0, s, a);                                                \
        return hipGetLastError();                                                                                      \
    } while (0)

template <int DT> hipError_t store_type(const Cache8Args &a, bool wide, hipStream_t s) { RTOPK_C8(cache8_store, DT); }
template <int DT> hipError_t load_type(const Cache8Args &a, bool wide, hipStream_t s) { RTOPK_C8(cache8_load, DT); }

} // namespace

hipError_t launch_cache8_store(Cache8Args a, int dtype, bool wide, hipStream_t s)
{
    a.tpw = (int)store_tokens(a.T, (int64_t)a.Hkv * a.D / 16 + 1, kC8Threads);
    return dtype == 0 ? store_type<0>(a, wide, s) : dtype == 1 ? store_type<1>(a, wide, s) : store_type<2>(a, wide, s);
}

hipError_t launch_cache8_load(Cache8Args a, int dtype, bool wide, hipStream_t s)
{
    a.tpw = (int)store_tokens(a.T, (int64_t)a.Hkv * a.D / 16 + 1, kC8Threads);
    return dtype == 0 ? load_type<0>(a, wide, s) : dtype == 1 ? load_type<1>(a, wide, s) : load_type<2>(a, wide, s);
}

} // namespace rtopk
