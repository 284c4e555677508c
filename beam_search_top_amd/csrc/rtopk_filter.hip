// gfx950 kernel of sampling with temperature, top-k, top-p and min-p from
// given random numbers.
//
// Row r's candidates are its logits above -infinity, in the order "larger logit
// first, equal logits by the lower token". With w_i = exp((x_i - max x) / T):
//   top-k keeps the first k of them; top-p the shortest beginning of those whose
//   weights sum to at least p of theirs; min-p those with w_i >= min_p.
// Each is a beginning of the order, so all together are the shortest of them, a
// cut (key, ties): everything above a logit, and the first few equal to it. The
// draw takes the first kept token i, in the order of tokens, whose running sum of
// kept weights exceeds u times their sum S, and its log(w_i / S).
//
// Sums at a border decide about whole numbers, so they must be the same in any
// order and exact: weights are computed in 64 bits and held as whole numbers
// (rtopk_filter.h).
#include <hip/hip_runtime.h>

#include <cmath>

#include "rtopk_filter.h"

namespace rtopk {
namespace {

constexpr int kFThreads = 1024, kFWaves = kFThreads / 64;
constexpr int kBits = 11, kBins = 1 << kBits;

typedef uint32_t f_u32x4 __attribute__((ext_vector_type(4)));

// Logits by their order: a key is larger where the logit is; -0 is +0, a NaN is -infinity.
template <int DT> struct Logit;
template <> struct Logit<0> {
    typedef uint32_t Raw;
    static constexpr int kKeyBits = 32, kPer = 4;
    static constexpr uint32_t kNone = 0x007fffffu; // -infinity
    static __device__ __forceinline__ float value(uint32_t r) { return __uint_as_float(r); }
    static __device__ __forceinline__ uint32_t key(uint32_t r)
    {
        if ((r & 0x7fffffffu) > 0x7f800000u)
            return kNone;
        r = r == 0x80000000u ? 0u : r;
        return r >> 31 ? ~r : r | 0x80000000u;
    }
    static __device__ __forceinline__ uint32_t raw(uint32_t k) { return k >> 31 ? k & 0x7fffffffu : ~k; }
};
template <int DT> struct Logit16 {
    typedef uint16_t Raw;
    static constexpr int kKeyBits = 16, kPer = 8;
    static constexpr uint32_t kInf = DT == 1 ? 0x7c00u : 0x7f80u, kNone = 0xffffu ^ (kInf | 0x8000u);
    static __device__ __forceinline__ float value(uint32_t r)
    {
        if constexpr (DT == 1)
            return (float)__builtin_bit_cast(_Float16, (uint16_t)r);
        else
            return __uint_as_float(r << 16);
    }
    static __device__ __forceinline__ uint32_t key(uint32_t r)
    {
        if ((r & 0x7fffu) > kInf)
            return kNone;
        r = r == 0x8000u ? 0u : r;
        return r >> 15 ? 0xffffu ^ r : r | 0x8000u;
    }
    static __device__ __forceinline__ uint32_t raw(uint32_t k) { return k >> 15 ? k & 0x7fffu : 0xffffu ^ k; }
};
template <> struct Logit<1> : Logit16<1> {};
template <> struct Logit<2> : Logit16<2> {};

// exp((x - top) / T) 2^frac, rounded to a whole number: 2^t by the Taylor series of
// e^y, |y| <= ln 2 / 2, up to y^13 / 13! < 2^-52, in 64 bits.
struct Weigh {
    double top, by; // by = log2(e) / T
    int frac;
    __device__ __forceinline__ uint64_t operator()(float x) const
    {
        const double d = (double)x - top;
        double t = d == 0. ? 0. : d * by;
        if ((double)x == top)
            t = 0.; // infinities among them
        if (!(t >= -70.) || x == -INFINITY)
            return 0;
        const double n = __builtin_rint(t), y = (t - n) * 0.6931471805599453;
        double p = 1. / 479001600.;
        p = __builtin_fma(p, y, 1. / 39916800.);
        p = __builtin_fma(p, y, 1. / 3628800.);
        p = __builtin_fma(p, y, 1. / 362880.);
        p = __builtin_fma(p, y, 1. / 40320.);
        p = __builtin_fma(p, y, 1. / 5040.);
        p = __builtin_fma(p, y, 1. / 720.);
        p = __builtin_fma(p, y, 1. / 120.);
        p = __builtin_fma(p, y, 1. / 24.);
        p = __builtin_fma(p, y, 1. / 6.);
        p = __builtin_fma(p, y, 0.5);
        p = __builtin_fma(p, y, 1.);
        p = __builtin_fma(p, y, 1.);
        const uint64_t bits = __builtin_bit_cast(uint64_t, p); // in [0.7, 1.42]
        const int down = 52 - ((int)(bits >> 52) - 1023 + (int)n + frac); // >= 1: frac <= 50, and p < 2 at n = 0
        const uint64_t m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
        return down > 60 ? 0 : (m + (1ull << (down - 1))) >> down;
    }
};

template <typename T> __device__ __forceinline__ T wave_sum(T x)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        x += __shfl_xor(x, o);
    return x;
}
template <typename T> __device__ __forceinline__ T scan_up(T x, int lane) // inclusive
{
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const T y = __shfl_up(x, o);
        x += lane >= o ? y : 0;
    }
    return x;
}

struct Bin {
    uint32_t at;        // the bin that the border lies in
    uint64_t above_n, n; // logits above it, in it
    uint64_t above_w, w; // their weights
};

template <int DT> __global__ __launch_bounds__(kFThreads) void filter_sample(const FilterArgs a)
{
    typedef Logit<DT> L;
    typedef typename L::Raw Raw;
    constexpr int PER = L::kPer;
    __shared__ uint64_t s_w[kBins];
    __shared__ uint32_t s_n[kBins];
    __shared__ uint64_t s_part[3][kFWaves];
    __shared__ Bin s_bin;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row = blockIdx.x, V = a.V;
    const Raw *x = static_cast<const Raw *>(a.logits) + (int64_t)row * a.ld;
    // 16-byte pieces from the boundary at or below the row on; piece i holds elements i * PER - lead ...
    const int lead = (int)(((uintptr_t)x & 15) / sizeof(Raw)), pieces = (int)(((int64_t)V + lead + PER - 1) / PER);
    const f_u32x4 *base = reinterpret_cast<const f_u32x4 *>((uintptr_t)x & ~(uintptr_t)15);
    auto element = [&](const f_u32x4 &v, int e) -> uint32_t {
        return sizeof(Raw) == 4 ? v[e] : (e & 1 ? v[e / 2] >> 16 : v[e / 2] & 0xffffu);
    };
    // f(token, raw bits) for every logit of pieces i0 + lane', in steps of all threads
    auto each = [&](auto f) {
        for (int i = tid; i < pieces; i += kFThreads) {
            const f_u32x4 v = base[i];
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int t = i * PER + e - lead;
                if (t >= 0 && t < V)
                    f(t, element(v, e));
            }
        }
    };

    // ---- the largest
    uint32_t best = 0;
    each([&](int, uint32_t r) {
        const uint32_t k = L::key(r);
        best = k > best ? k : best;
    });
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const uint32_t y = __shfl_xor(best, o);
        best = y > best ? y : best;
    }
    if (lane == 0)
        s_part[0][wave] = best;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kFWaves; ++w)
        best = s_part[0][w] > best ? (uint32_t)s_part[0][w] : best;
    __syncthreads();
    if (best == L::kNone) { // no candidate
        if (tid == 0) {
            a.out_token[row] = -1;
            a.out_logprob[row] = -INFINITY;
        }
        return;
    }
    const float T = a.temperature ? a.temperature[row] : 1.f;
    const bool greedy = !(T > 0.f);
    const Weigh weigh{(double)L::value(L::raw(best)), greedy ? 0. : 1.4426950408889634 / (double)T, a.frac};
    const int k = greedy ? 1 : a.top_k ? a.top_k[row] : 0;
    float p = greedy || !a.top_p ? 1.f : a.top_p[row];
    const bool by_k = k > 0 && k < V, by_p = p < 1.f;
    p = p > 0.f ? p : 0.f;
    float mp = greedy || !a.min_p ? 0.f : a.min_p[row];
    mp = mp > 0.f ? mp < 1.f ? mp : 1.f : 0.f; // NaN: 0
    const uint64_t least = (uint64_t)__builtin_ceil((double)mp * (double)(1ull << a.frac));

    // ---- the cut
    // Counts and weights by the next kBits bits of the keys that begin with `prefix`.
    auto histogram = [&](uint32_t prefix, int done) {
        for (int i = tid; i < kBins; i += kFThreads) {
            s_w[i] = 0;
            s_n[i] = 0;
        }
        __syncthreads();
        const int left = L::kKeyBits - done, take = left < kBits ? left : kBits;
        each([&](int, uint32_t r) {
            const uint32_t key = L::key(r);
            if (done == 0 || key >> left == prefix) {
                const uint32_t b = key >> (left - take) & ((1u << take) - 1);
                atomicAdd(&s_n[b], 1u);
                atomicAdd((unsigned long long *)&s_w[b], (unsigned long long)weigh(L::value(r)));
            }
        });
        __syncthreads();
    };
    // The first bin from the top at which the count (or the weight) reaches `want`, given what lies above.
    auto border = [&](bool weights, uint64_t want, uint64_t above_n, uint64_t above_w) -> Bin {
        constexpr int EACH = kBins / kFThreads;
        uint64_t n = 0, w = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            n += s_n[kBins - 1 - (tid * EACH + i)];
            w += s_w[kBins - 1 - (tid * EACH + i)];
        }
        uint64_t cn = scan_up(n, lane), cw = scan_up(w, lane);
        if (lane == 63) {
            s_part[0][wave] = cn;
            s_part[1][wave] = cw;
        }
        __syncthreads();
        cn += above_n;
        cw += above_w;
        for (int i = 0; i < wave; ++i) {
            cn += s_part[0][i];
            cw += s_part[1][i];
        }
        cn -= n;
        cw -= w;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int b = kBins - 1 - (tid * EACH + i);
            const uint64_t bn = s_n[b], bw = s_w[b];
            if (weights ? cw < want && cw + bw >= want : cn < want && cn + bn >= want)
                s_bin = Bin{(uint32_t)b, cn, bn, cw, bw};
            cn += bn;
            cw += bw;
        }
        __syncthreads();
        const Bin got = s_bin;
        __syncthreads();
        return got;
    };
    // The key at which the count (or the weight) reaches `want`, from the first histogram on.
    auto search = [&](bool weights, uint64_t want, uint32_t &key) -> Bin {
        Bin b = border(weights, want, 0, 0);
        key = b.at;
        for (int done = kBits; done < L::kKeyBits; done += kBits) {
            const int take = L::kKeyBits - done < kBits ? L::kKeyBits - done : kBits;
            histogram(key, done);
            b = border(weights, want, b.above_n, b.above_w);
            key = key << take | b.at;
        }
        return b;
    };
    // kept: keys above `cut`, and the first `ties` of those equal to it
    uint32_t cut = L::kNone;
    uint64_t ties = 0, total = 0;
    if (by_k || by_p) {
        histogram(0, 0);
        if (by_p && !by_k) {
            uint64_t w = 0;
            for (int i = tid; i < kBins; i += kFThreads)
                w += s_w[i];
            w = wave_sum(w);
            if (lane == 0)
                s_part[2][wave] = w;
            __syncthreads();
            for (int i = 0; i < kFWaves; ++i)
                total += s_part[2][i];
        }
        if (by_k) {
            const Bin b = search(false, (uint64_t)k, cut);
            ties = (uint64_t)k - b.above_n;
            total = b.above_w + ties * weigh(L::value(L::raw(cut)));
        }
        if (by_p) {
            const double want = __builtin_ceil((double)p * (double)total);
            uint64_t goal = want < 1. ? 1 : (uint64_t)want;
            goal = goal < total ? goal : total;
            if (by_k)
                histogram(0, 0);
            const Bin b = search(true, goal, cut);
            const uint64_t w = weigh(L::value(L::raw(cut)));
            ties = (goal - b.above_w + w - 1) / w; // w > 0: the border lies in its bin
        }
    }

    // ---- the draw. A wave takes a run of consecutive pieces.
    const uint64_t cut_w = weigh(L::value(L::raw(cut))), tie_w = cut_w >= least ? cut_w : 0;
    const int per = (pieces + kFWaves - 1) / kFWaves, p0 = wave * per, p1 = p0 + per < pieces ? p0 + per : pieces;
    uint64_t sum = 0, equal = 0;
    for (int i = p0 + lane; i < p1; i += 64) {
        const f_u32x4 v = base[i];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int t = i * PER + e - lead;
            if (t >= 0 && t < V) {
                const uint32_t r = element(v, e), key = L::key(r);
                if (key > cut) {
                    const uint64_t w = weigh(L::value(r));
                    sum += w >= least ? w : 0;
                }
                equal += key == cut;
            }
        }
    }
    sum = wave_sum(sum);
    equal = wave_sum(equal);
    if (lane == 0) {
        s_part[0][wave] = sum;
        s_part[1][wave] = equal;
    }
    __syncthreads();
    uint64_t S = 0, before = 0, ties_before = 0, seen = 0;
    uint64_t start[kFWaves];
#pragma unroll
    for (int i = 0; i < kFWaves; ++i) {
        start[i] = S;
        if (i == wave)
            ties_before = seen;
        const uint64_t room = ties > seen ? ties - seen : 0, mine = s_part[1][i] < room ? s_part[1][i] : room;
        S += s_part[0][i] + mine * tie_w;
        seen += s_part[1][i];
    }
    float u = a.u[row];
    u = u > 0.f ? u : 0.f; // NaN: 0
    uint64_t goal = u < 1.f ? (uint64_t)((double)u * (double)S) : S; // S > 0: the best is kept
    goal = goal < S ? goal : S - 1;
    // the run that the running sum passes the goal in
    bool mine = false;
#pragma unroll
    for (int i = 0; i < kFWaves; ++i)
        if (i == wave) {
            before = start[i];
            mine = start[i] <= goal && (i + 1 < kFWaves ? start[i + 1 < kFWaves ? i + 1 : i] : S) > goal;
        }
    if (!mine)
        return;
    for (int i0 = p0; i0 < p1; i0 += 64) {
        const int i = i0 + lane;
        f_u32x4 v = {0, 0, 0, 0};
        if (i < p1)
            v = base[i];
        uint64_t w[PER], n = 0;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int t = i * PER + e - lead;
            const bool in = i < p1 && t >= 0 && t < V;
            n += in && L::key(element(v, e)) == cut;
        }
        const uint64_t upto = scan_up(n, lane);
        uint64_t rank = ties_before + upto - n, own = 0;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int t = i * PER + e - lead;
            const bool in = i < p1 && t >= 0 && t < V;
            const uint32_t r = element(v, e), key = L::key(r);
            w[e] = 0;
            if (in && key > cut) {
                w[e] = weigh(L::value(r));
                w[e] = w[e] >= least ? w[e] : 0;
            } else if (in && key == cut) {
                w[e] = rank < ties ? tie_w : 0;
                ++rank;
            }
            own += w[e];
        }
        const uint64_t sums = scan_up(own, lane);
        const uint64_t hit = __ballot(before + sums > goal);
        if (hit) {
            if (lane == __ffsll((unsigned long long)hit) - 1) {
                uint64_t c = before + sums - own;
                int e = 0;
                while (e < PER - 1 && c + w[e] <= goal)
                    c += w[e++];
                a.out_token[row] = i * PER + e - lead;
                a.out_logprob[row] = (float)log((double)w[e] / (double)S);
            }
            return;
        }
        before += __shfl(sums, 63);
        ties_before += __shfl(upto, 63);
    }
}

} // namespace

hipError_t launch_filter(const FilterArgs &a, int dtype, hipStream_t s)
{
    const dim3 grid((unsigned)a.R), block(kFThreads);
    if (dtype == 0)
        hipLaunchKernelGGL(filter_sample<0>, grid, block, 0, s, a);
    else if (dtype == 1)
        hipLaunchKernelGGL(filter_sample<1>, grid, block, 0, s, a);
    else
        hipLaunchKernelGGL(filter_sample<2>, grid, block, 0, s, a);
    return hipGetLastError();
}

} // namespace rtopk
