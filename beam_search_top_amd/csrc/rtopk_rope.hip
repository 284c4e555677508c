// gfx950 kernel of the norms of queries and keys and of their rotation by
// position, in one pass: every element is read once and written once, and
// rounded once.
//
//     y_d = x_d / sqrt(mean(x^2) + eps) * w_d             (without weights: y = x)
//     (a, b) -> (a cos t - b sin t, b cos t + a sin t),   t = position * freqs[i],
//
// for the pairs i < rot / 2: elements (i, i + rot / 2), or (2i, 2i + 1) where
// they are interleaved. Elements from rot on are not rotated.
#include <hip/hip_runtime.h>

#include "rtopk_cache8.h"
#include "rtopk_internal.h"
#include "rtopk_rows.h"

namespace rtopk {
namespace {

constexpr int kRopeThreads = 256;

// A workgroup takes `tpw` tokens with all their heads. It first puts the sines and
// cosines of its tokens into LDS, once for all heads. Then every row (a head of
// a token) is a group of LPH lanes; a unit of a lane is two chunks of VE elements that
// hold both members of their pairs, so that nothing is exchanged but the sum
// of squares. VE is 16 bytes where pointers, strides and sizes allow it, else one element.
//
// An angle is the product of the position and the frequency in 64 bits, taken off
// whole turns there: position 10^6 at frequency 1 would lose 2^-4 of a radian in 32 bits.
//
// Bound by HBM: 60001 tokens of 32 + 8 heads of 128, bfloat16 with norms, 245 us, 4.93 TB/s read and
// written (a device copy: 5.01). 200 tokens of 16 + 16 heads of 64 take 4.0 us, a chain of a position, an
// angle and a row; the call on the host takes 8.8.
template <int DT, int VE, int LPH>
__global__ __launch_bounds__(kRopeThreads) void qk_norm_rope(const RopeArgs a)
{
    typedef Row<DT> X;
    typedef typename X::T T;
    constexpr int NU = VE > 1 ? 1 : kMaxRowDim / 2 / LPH; // units per lane
    extern __shared__ float2 s_turn[];                    // [tpw][rot / 2] cosine, sine
    const int tid = threadIdx.x, half = a.rot / 2;
    const int64_t t0 = (int64_t)blockIdx.x * a.tpw;
    const int nt = (int)(t0 + a.tpw < a.T ? a.tpw : a.T - t0);
    for (int i = tid; i < nt * half; i += kRopeThreads) {
        const int t = i / half;
        const double turns = (double)a.positions[t0 + t] * (double)a.freqs[i - t * half] * 0.15915494309189535;
        float s, c;
        sincospif(2.f * (float)(turns - __builtin_rint(turns)), &s, &c);
        s_turn[i] = make_float2(c, s);
    }
    __syncthreads();
    const int j = tid % LPH, rows = nt * (int)a.heads.d;
    for (int r = tid / LPH; r < rows; r += kRopeThreads / LPH) {
        const int t = (int)page_of(a.heads, (uint32_t)r);
        int h = r - t * (int)a.heads.d;
        const bool key = h >= a.Hq;
        h -= key ? a.Hq : 0;
        if (a.positions[t0 + t] < 0)
            continue; // the same for the lanes of a row
        const T *from = static_cast<const T *>(key ? a.k : a.q) + (t0 + t) * (key ? a.ks[0] : a.qs[0]) + h * (key ? a.ks[1] : a.qs[1]);
        T *to = static_cast<T *>(key ? a.k_out : a.q_out) + (t0 + t) * (key ? a.kos[0] : a.qos[0]) + h * (key ? a.kos[1] : a.qos[1]);
        const T *w = static_cast<const T *>(key ? a.kw : a.qw);
        float x[NU][2][VE];
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int at = (j + n * LPH) * VE; // pairs before this unit's
            const bool turn = at < half;
            const int o0 = turn && !a.interleaved ? at : 2 * at, o1 = turn && !a.interleaved ? half + at : 2 * at + VE;
#pragma unroll
            for (int e = 0; e < VE; ++e)
                x[n][0][e] = x[n][1][e] = 0.f;
            if (o0 < a.D)
                X::template load<VE>(from + o0, x[n][0]);
            if (o1 < a.D)
                X::template load<VE>(from + o1, x[n][1]);
#pragma unroll
            for (int e = 0; e < VE; ++e)
                sum += x[n][0][e] * x[n][0][e] + x[n][1][e] * x[n][1][e];
        }
        float f = 1.f;
        if (w) {
            const float mean = group_sum<LPH>(sum) / (float)a.D + a.eps;
            if (mean >= 0x1p-100f && mean <= 0x1.fffffep127f) {
                f = 1.f / sqrtf(mean);
            } else {
                // squares that leave float32's range, or lose bits at its lower end (up to 2^-150 of each, which a
                // mean of 2^-100 does not feel): the row is normalised in 64 bits, and rounded once on the way
                double wide = 0.;
#pragma unroll
                for (int n = 0; n < NU; ++n)
#pragma unroll
                    for (int e = 0; e < VE; ++e)
                        wide += (double)x[n][0][e] * x[n][0][e] + (double)x[n][1][e] * x[n][1][e];
                const double by = 1. / sqrt(group_sum<LPH>(wide) / a.D + (double)a.eps);
#pragma unroll
                for (int n = 0; n < NU; ++n)
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        x[n][0][e] = (float)(x[n][0][e] * by);
                        x[n][1][e] = (float)(x[n][1][e] * by);
                    }
            }
        }
#pragma unroll
        for (int n = 0; n < NU; ++n) {
            const int at = (j + n * LPH) * VE;
            const bool turn = at < half;
            const int o0 = turn && !a.interleaved ? at : 2 * at, o1 = turn && !a.interleaved ? half + at : 2 * at + VE;
            if (w) {
                float g[2][VE] = {};
                if (o0 < a.D)
                    X::template load<VE>(w + o0, g[0]);
                if (o1 < a.D)
                    X::template load<VE>(w + o1, g[1]);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    x[n][0][e] = x[n][0][e] * f * g[0][e];
                    x[n][1][e] = x[n][1][e] * f * g[1][e];
                }
            }
            if (turn) {
                const float2 *cs = s_turn + t * half + at;
                if (VE > 1 && a.interleaved) { // pairs of neighbours: the first half of them in x[0], the others in x[1]
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int e = 0; e < VE; e += 2) {
                            const float2 z = cs[(y * VE + e) / 2];
                            const float p = x[n][y][e], q = x[n][y][e + (VE > 1)];
                            x[n][y][e] = p * z.x - q * z.y;
                            x[n][y][e + (VE > 1)] = q * z.x + p * z.y;
                        }
                } else {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float2 z = cs[e];
                        const float p = x[n][0][e], q = x[n][1][e];
                        x[n][0][e] = p * z.x - q * z.y;
                        x[n][1][e] = q * z.x + p * z.y;
                    }
                }
            }
            if (o0 < a.D)
                X::template store<VE>(to + o0, x[n][0]);
            if (o1 < a.D)
                X::template store<VE>(to + o1, x[n][1]);
        }
    }
}

template <int DT, int VE, int LPH> hipError_t go(const RopeArgs &a, hipStream_t s)
{
    const int64_t blocks = (a.T + a.tpw - 1) / a.tpw;
    hipLaunchKernelGGL((qk_norm_rope<DT, VE, LPH>), dim3((unsigned)blocks), dim3(kRopeThreads),
                       sizeof(float2) * a.tpw * (a.rot / 2), s, a);
    return hipGetLastError();
}

template <int DT> hipError_t go_type(const RopeArgs &a, bool wide, hipStream_t s)
{
    constexpr int VE = DT == 0 ? 4 : 8;
    if (!wide)
        return go<DT, 1, 64>(a, s);
    const int lanes = a.D / (2 * VE);
    if (lanes <= 4)
        return go<DT, VE, 4>(a, s);
    if (lanes <= 8)
        return go<DT, VE, 8>(a, s);
    if (lanes <= 16)
        return go<DT, VE, 16>(a, s);
    return go<DT, VE, 32>(a, s);
}

} // namespace

hipError_t launch_rope(RopeArgs a, int dtype, bool wide, hipStream_t s)
{
    a.tpw = rope_tokens(a.T, (int64_t)(a.Hq + a.Hkv) * a.D);
    return dtype == 0 ? go_type<0>(a, wide, s) : dtype == 1 ? go_type<1>(a, wide, s) : go_type<2>(a, wide, s);
}

} // namespace rtopk
