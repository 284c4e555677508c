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
#include "rtopk_rows.h"

namespace rtopk {
namespace {

constexpr int kFThreads = 512, kFWaves = kFThreads / 64;
constexpr int kBins = 2048;
constexpr int kOctaves = 32;        // factors of two of weight that the bins span, at most
constexpr int kList = 8192;          // logits that the filters may keep, of which a list is made, at most
constexpr int kWaveList = kList / kFWaves;
constexpr int kZone = 2 * kFThreads; // logits around the borders that are ordered one by one, at most

typedef uint32_t f_u32x4 __attribute__((ext_vector_type(4)));

// Logits as they are stored: raw bits, and how many 16 bytes hold.
template <int DT> struct Logit;
template <> struct Logit<0> {
    typedef uint32_t Raw;
    static constexpr int kPer = 4;
    static __device__ __forceinline__ float value(uint32_t r) { return __uint_as_float(r); }
};
template <> struct Logit<1> {
    typedef uint16_t Raw;
    static constexpr int kPer = 8;
    static __device__ __forceinline__ float value(uint32_t r) { return (float)__builtin_bit_cast(_Float16, (uint16_t)r); }
};
template <> struct Logit<2> {
    typedef uint16_t Raw;
    static constexpr int kPer = 8;
    static __device__ __forceinline__ float value(uint32_t r) { return __uint_as_float(r << 16); }
};

constexpr int kSteps = 512; // table entries per factor of two

// exp((x - top) / T) 2^frac as a whole number, from t = (x - top) log2(e) / T in steps of
// 1/512: 2^t = 2^(n / 512) 2^(r / 512), the first factor's fraction from a table, its whole
// part added to the exponent, the second, |r| <= 1/2, by the Taylor series up to r^3, where
// r^2 stands in for r^4 as 0.207 r^2, which is within 0.172 / 16 of it: off by 2^-49 at most,
// and exact at r = 0. All in 64 bits. Adding 1.5 2^52 rounds t to a whole number, and adding
// 2^52 the weight, which the lower bits then hold. Every pass over a row spends most
// of its instructions here: 19 in 64 bits or for them.
struct Weigh {
    double top, by, low; // by = 512 log2(e) / T; what lies further below top than -low weighs nothing
    const double *table; // 2^(frac + i / 512), LDS; frac <= 50
    __device__ __forceinline__ void scale(double t, double per_T)
    {
        top = t;
        by = __builtin_fmax(kSteps * 1.4426950408889634 * per_T, 0x1p-900); // T may be infinite
        // The largest float32 stands for infinity (value()): whatever T, the next number below it, 2^104 away,
        // weighs nothing beside it.
        if (t == 0x1.fffffep127)
            by = __builtin_fmax(by, 200. * kSteps * 0x1p-104);
        low = -200. * kSteps / by;
    }
    __device__ __forceinline__ uint64_t operator()(float x) const
    {
        const double d = __builtin_fmax((double)x - top, low); // -infinity: 2^-200, which rounds to 0
        const double n = __builtin_fma(d, by, 0x1.8p52), r = __builtin_fma(d, by, 0x1.8p52 - n);
        constexpr double c = 0.6931471805599453 / kSteps;
        double p = __builtin_fma(c * c * c / 6., r, c * c / 2. + 0.207 * c * c * c * c / 24.);
        p = __builtin_fma(p, r, c);
        p = __builtin_fma(p, r, 1.);
        const uint32_t m = (uint32_t)__builtin_bit_cast(uint64_t, n); // modulo 2^32
        const uint64_t first = __builtin_bit_cast(uint64_t, table[m & (kSteps - 1)]) + ((uint64_t)((m & ~(uint32_t)(kSteps - 1)) << 11) << 32);
        const double w = __builtin_fma(p, __builtin_bit_cast(double, first), 0x1p52);
        return __builtin_bit_cast(uint64_t, w) & 0xfffffffffffffull;
    }
};
static_assert(kSteps == 1 << 9, "m / kSteps goes to bit 52");

// x of the lane that DPP control CTRL names, 0 where it names none or ROWS leaves the row of 16 out
template <int CTRL, int ROWS> __device__ __forceinline__ uint32_t moved(uint32_t x)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS> __device__ __forceinline__ uint64_t moved(uint64_t x)
{
    return (uint64_t)moved<CTRL, ROWS>((uint32_t)(x >> 32)) << 32 | moved<CTRL, ROWS>((uint32_t)x);
}
__device__ __forceinline__ uint32_t of_lane(uint32_t x, int lane) { return (uint32_t)__builtin_amdgcn_readlane((int)x, lane); }
__device__ __forceinline__ uint64_t of_lane(uint64_t x, int lane)
{
    return (uint64_t)of_lane((uint32_t)(x >> 32), lane) << 32 | of_lane((uint32_t)x, lane);
}
// Sums over the lanes up to each and over all; every lane runs. (By exchanges through LDS a sum's six steps took
// 0.4 us, and a row waits for eight of them.)
template <typename T> __device__ __forceinline__ T scan_up(T x)
{
    x += moved<0x111, 0xf>(x); // the lane below in the row of 16, then 2, 4 and 8 below
    x += moved<0x112, 0xf>(x);
    x += moved<0x114, 0xf>(x);
    x += moved<0x118, 0xf>(x);
    x += moved<0x142, 0xa>(x); // the last lane of the row below, for rows 1 and 3
    x += moved<0x143, 0xc>(x); // lane 31, for rows 2 and 3
    return x;
}
template <typename T> __device__ __forceinline__ T wave_sum(T x) { return of_lane(scan_up(x), 63); }

// What a workgroup keeps in LDS.
struct Shared {
    double table[kSteps];
    union {
        uint64_t w[kBins + 64]; // weights by bins, and the last bin's by lanes
        uint32_t n[kBins + 64]; // or counts
    };
    uint64_t zone[kZone], parts[kZone];
    uint32_t list[kFWaves][kWaveList]; // tokens
    uint64_t scan[kFWaves];
    float2 ends[kFWaves];
    uint32_t part32[kFWaves];
    uint32_t count;
    int found[2];
    uint64_t value[4];
};

// Where the borders of top-k and top-p lie: bins below `sure` are kept whole, the
// zones [p0, p1] and kb hold the borders.
struct Borders {
    int sure, p0, p1, kb;
    uint32_t rest_k;  // logits of bin kb that top-k keeps
    uint64_t above_k; // weight above bin kb
    uint64_t above_p; // weight above bin p0
    uint64_t all;     // of the row (or of what the list holds)
};
constexpr Borders kNoBorders{kBins, kBins, -1, kBins, 0, 0, 0, 0};

// What keeps everything but -infinity.
constexpr uint64_t kKeepAll = 0x00800000ull << 32;

// One row and what its filters are. SHORT: the loop over the logits of 16 bytes is not unrolled. A lane of a
// launch of few rows has one or two pieces, for which unrolled code takes as long (the last launch of 8 x 250000: 19.8
// us, 19.2 as it is; of 32 x 32000 15.8 both) and is more to fetch for a call that finds it nowhere.
template <int DT, bool SHORT> struct RowFilter {
    typedef Logit<DT> L;
    typedef typename L::Raw Raw;
    static constexpr int PER = L::kPer;
    const FilterArgs &a;
    Shared &sh;
    int row, tid, lane, wave, lead, pieces;
    const __attribute__((address_space(1))) f_u32x4 *base;
    float top, bin_by, bin_top; // the largest logit; bins per unit below it, and their product
    Weigh weigh;
    bool greedy, by_k, by_p;
    int k;
    float p, m;
    uint64_t least; // min-p
    int from, to;   // the pieces that this workgroup reads
    int mine;       // length of this wave's list, -1: none
    int shift;      // a run is 2^shift pieces: kBins runs hold the row
    f_u32x4 ready;  // piece ready_at, loaded ahead
    int ready_at;

    __device__ __forceinline__ RowFilter(const FilterArgs &args, Shared &shared, int r) : a(args), sh(shared), row(r)
    {
        tid = threadIdx.x;
        lane = tid & 63;
        wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const Raw *x = static_cast<const Raw *>(a.logits) + (int64_t)row * a.ld;
        // 16-byte pieces from the boundary at or below the row on; piece i holds tokens i * PER - lead ...
        lead = (int)(((uintptr_t)x & 15) / sizeof(Raw));
        pieces = (int)(((int64_t)a.V + lead + PER - 1) / PER);
        base = (const __attribute__((address_space(1))) f_u32x4 *)((uintptr_t)x & ~(uintptr_t)15);
        from = 0;
        to = pieces;
        mine = ready_at = -1;
        shift = 0;
        while ((pieces - 1) >> shift >= kBins)
            ++shift;
    }
    __device__ __forceinline__ float at(int token) const // of the list
    {
        typedef const __attribute__((address_space(1))) Raw graw;
        f_u32x4 v = {0, 0, 0, 0};
        v[0] = reinterpret_cast<graw *>(base)[token + lead];
        return value(v, 0);
    }
    static __device__ __forceinline__ uint32_t raw(const f_u32x4 &v, int e)
    {
        return sizeof(Raw) == 4 ? v[e] : (e & 1 ? v[e / 2] >> 16 : v[e / 2] & 0xffffu);
    }
    // A NaN is -infinity, and +infinity the largest float32, so that differences are numbers.
    static __device__ __forceinline__ float value(const f_u32x4 &v, int e)
    {
        return fminf(fmaxf(L::value(raw(v, e)), -INFINITY), 0x1.fffffep127f);
    }
    // piece i, with -infinity in the place of what is not the row's
    __device__ __forceinline__ f_u32x4 piece(int i) const
    {
        f_u32x4 v;
        if (SHORT && i == ready_at)
            v = ready;
        else
            v = base[i];
        if (i == 0 || i == pieces - 1) {
            constexpr uint32_t none = sizeof(Raw) == 4 ? 0xff800000u : DT == 1 ? 0xfc00u : 0xff80u;
#pragma unroll
            for (int e = 0; e < PER; ++e) {
                const int t = i * PER + e - lead;
                const bool in = t >= 0 && t < a.V;
                if (sizeof(Raw) == 4)
                    v[e] = in ? v[e] : none;
                else if (e & 1)
                    v[e / 2] = in ? v[e / 2] : (v[e / 2] & 0xffffu) | none << 16;
                else
                    v[e / 2] = in ? v[e / 2] : (v[e / 2] & 0xffff0000u) | none;
            }
        }
        return v;
    }
    // f(token, value) for every logit of the pieces i0 + at, i0 + at + step, ... below i1, and
    // after each piece end(piece); the next piece is on its way while one is worked on
    template <typename F> __device__ __forceinline__ void each(int i0, int i1, int at, int step, F f) const
    {
        each(i0, i1, at, step, f, [](int) {});
    }
    template <typename F, typename G> __device__ __forceinline__ void each(int i0, int i1, int at, int step, F f, G end) const
    {
        int i = i0 + at;
        if (i >= i1)
            return;
        f_u32x4 v = piece(i);
        while (true) {
            const int next = i + step;
            f_u32x4 ahead = v;
            if (next < i1)
                ahead = piece(next);
            if constexpr (SHORT) {
#pragma unroll 1
                for (int e = 0; e < PER; e += PER / 4) {
                    f(i * PER + e - lead, value(v, 0));
                    if constexpr (PER == 8)
                        f(i * PER + e + 1 - lead, value(v, 1));
                    v = __builtin_shufflevector(v, v, 1, 2, 3, 0);
                }
            } else {
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    f(i * PER + e - lead, value(v, e));
            }
            end(i);
            if (next >= i1)
                break;
            i = next;
            v = ahead;
        }
    }
    // the largest and the smallest value of its pieces (-infinity apart), for every thread
    __device__ __forceinline__ void range(float &hi, float &lo)
    {
        float x = -INFINITY, y = INFINITY;
        each(from, to, tid, kFThreads, [&](int, float v) {
            x = fmaxf(x, v);
            y = fminf(y, v > -INFINITY ? v : INFINITY);
        });
        all_range(x, y);
        hi = x;
        lo = y;
    }
    __device__ __forceinline__ void all_range(float &x, float &y) // of the workgroup
    {
        x = __uint_as_float(group_all<64>(__float_as_uint(x), [](uint32_t p, uint32_t q) {
            return __float_as_uint(fmaxf(__uint_as_float(p), __uint_as_float(q)));
        }));
        y = __uint_as_float(group_all<64>(__float_as_uint(y), [](uint32_t p, uint32_t q) {
            return __float_as_uint(fminf(__uint_as_float(p), __uint_as_float(q)));
        }));
        __syncthreads();
        if (lane == 0)
            sh.ends[wave] = make_float2(x, y);
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kFWaves; ++w) {
            x = fmaxf(x, sh.ends[w].x);
            y = fminf(y, sh.ends[w].y);
        }
    }
    // what is asked of the row, given its largest value and its smallest
    __device__ __forceinline__ void ask(float hi, float lo)
    {
        top = hi;
        const float T = a.temperature ? a.temperature[row] : 1.f;
        greedy = !(T > 0.f);
        weigh.scale((double)top, greedy ? 0. : 1. / (double)T);
        weigh.table = sh.table;
        // the bins span the row, or the logits with weights down to 2^-32 of the largest
        const float by_weight = greedy ? 0.f : (float)((kBins / kOctaves) * 1.4426950408889634 / (double)T);
        bin_by = fminf(fmaxf(by_weight, (float)(kBins - 1) / (hi - lo)), 0x1p126f);
        bin_top = top * bin_by;
        k = greedy || !a.top_k ? 0 : a.top_k[row];
        p = greedy || !a.top_p ? 1.f : a.top_p[row];
        by_k = k > 0 && k < a.V;
        by_p = p < 1.f;
        p = p > 0.f ? p : 0.f;
        m = greedy || !a.min_p ? 0.f : a.min_p[row];
        m = m > 0.f ? m < 1.f ? m : 1.f : 0.f; // NaN: 0
        least = (uint64_t)__builtin_ceil((double)m * (double)(1ull << a.frac));
        for (int i = tid; i < kSteps; i += kFThreads)
            sh.table[i] = __builtin_ldexp(exp2((double)i / kSteps), a.frac);
    }
    // No logit behind this bin has the weight that min-p asks for.
    __device__ __forceinline__ int lowest_bin() const
    {
        if (m == 0.f)
            return kBins - 1;
        const float T = a.temperature ? a.temperature[row] : 1.f;
        const float x = -__builtin_log2f(m) * 0.6931472f * T * bin_by * (1.f + 0x1p-18f) + 2.f;
        return x < (float)(kBins - 1) ? (int)x : kBins - 1; // (NaN: the last)
    }
    // A logit's bin: larger logits in lower ones. The same in every pass, since it rounds the
    // same; far from the top, or with numbers that bin_top rounds, it is a coarse one.
    __device__ __forceinline__ int bin(float x) const
    {
        return (int)__builtin_amdgcn_fmed3f(__builtin_fmaf(-x, bin_by, bin_top), 0.f, (float)(kBins - 1));
    }
    // The order of logits as whole numbers: larger logit first, then lower token.
    static __device__ __forceinline__ uint64_t order(float x, int t)
    {
        uint32_t u = __float_as_uint(x + 0.f); // -0 is +0
        u = u >> 31 ? ~u : u | 0x80000000u;
        return (uint64_t)u << 32 | (uint32_t)~t;
    }
    static __device__ __forceinline__ float value_of(uint64_t o)
    {
        const uint32_t u = (uint32_t)(o >> 32);
        return __uint_as_float(u >> 31 ? u & 0x7fffffffu : ~u);
    }
    static __device__ __forceinline__ int token_of(uint64_t o) { return (int)~(uint32_t)o; }
    // u times S as a whole number below S; S is the same for every thread
    __device__ __forceinline__ uint64_t point(uint64_t S) const
    {
        const float u = a.u[row];
        const uint32_t part = __float_as_uint(u > 0.f ? u : 0.f); // NaN: 0
        S = of_lane(S, 0);
        return u < 1.f || part == 0 ? part_of(part, S, false) : S - 1; // S > 0: the best is kept
    }
    // What top-p (p < 1) asks of a beginning, of a weight of `total`
    __device__ __forceinline__ uint64_t goal_of(uint64_t total) const
    {
        const uint64_t g = part_of(__float_as_uint(p), total, true);
        return g > 0 ? g : 1;
    }
    // The sum over the workgroup, for every thread.
    __device__ __forceinline__ uint64_t all_sum(uint64_t x)
    {
        x = wave_sum(x);
        __syncthreads();
        if (lane == 0)
            sh.scan[wave] = x;
        __syncthreads();
        x = 0;
#pragma unroll
        for (int i = 0; i < kFWaves; ++i)
            x += sh.scan[i];
        return x;
    }
    // The sum over the threads before this one.
    __device__ __forceinline__ uint64_t before_me(uint64_t x)
    {
        const uint64_t upto = scan_up(x);
        __syncthreads();
        if (lane == 63)
            sh.scan[wave] = upto;
        __syncthreads();
        uint64_t b = upto - x;
#pragma unroll
        for (int i = 0; i < kFWaves; ++i)
            b += i < wave ? sh.scan[i] : 0;
        return b;
    }

    // The sum over the workgroup of what before_me has just scanned.
    __device__ __forceinline__ uint64_t scanned() const
    {
        uint64_t x = 0;
#pragma unroll
        for (int i = 0; i < kFWaves; ++i)
            x += sh.scan[i];
        return x;
    }

    // ---- histograms of the pieces; the last bin is summed by lanes first, for it may hold most
    __device__ __forceinline__ void clear_bins()
    {
        __syncthreads();
        for (int i = tid; i < kBins + 64; i += kFThreads)
            sh.w[i] = 0;
        __syncthreads();
    }
    __device__ __forceinline__ int bin_or_lane(float x) const
    {
        const int b = bin(x);
        return b < kBins - 1 ? b : kBins + lane;
    }
    __device__ __forceinline__ void count_bins()
    {
        clear_bins();
        each(from, to, tid, kFThreads, [&](int, float x) { atomicAdd(&sh.n[bin_or_lane(x)], 1u); });
        __syncthreads();
        if (wave == 0) {
            const uint32_t far = wave_sum(sh.n[kBins + lane]);
            if (lane == 0)
                sh.n[kBins - 1] = far;
        }
        __syncthreads();
    }
    __device__ __forceinline__ void weigh_bins()
    {
        clear_bins();
        auto add = [&](int, float x) { atomicAdd((unsigned long long *)&sh.w[bin_or_lane(x)], (unsigned long long)weigh(x)); };
        if (mine >= 0)
            each_listed(add);
        else
            each(from, to, tid, kFThreads, add);
        __syncthreads();
        if (wave == 0) {
            const uint64_t far = wave_sum(sh.w[kBins + lane]);
            if (lane == 0)
                sh.w[kBins - 1] = far;
        }
        __syncthreads();
    }
    // From the counts: the bin in which the first `want` logits end (found[0], kBins if there are fewer),
    // how many of it (value[0]) they take, and the number of logits through bin `through` (value[1]).
    __device__ __forceinline__ void find_count(uint32_t want, int through)
    {
        constexpr int EACH = kBins / kFThreads;
        uint32_t n[EACH], sum = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            n[i] = sh.n[tid * EACH + i];
            sum += n[i];
        }
        uint32_t c = (uint32_t)before_me(sum);
        if (tid == 0) {
            sh.found[0] = kBins;
            sh.value[0] = sh.value[1] = 0;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int b = tid * EACH + i;
            if (c < want && c + n[i] >= want) {
                sh.found[0] = b;
                sh.value[0] = want - c;
                if (through < 0)
                    sh.value[1] = c + n[i];
            }
            c += n[i];
            if (b == through)
                sh.value[1] = c;
        }
        __syncthreads();
    }
    // From the weights: the bin in which their running sum reaches `goal` (found[at]); value[2 at] is what
    // lies above it.
    __device__ __forceinline__ void find_weight(const uint64_t (&w)[kBins / kFThreads], uint64_t before, uint64_t goal, int at)
    {
        constexpr int EACH = kBins / kFThreads;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            if (before < goal && before + w[i] >= goal) {
                sh.found[at] = tid * EACH + i;
                sh.value[2 * at] = before;
            }
            before += w[i];
        }
    }
    // The smallest value whose bin is `b` or below, or a little less.
    __device__ __forceinline__ float floor_of(int b) const
    {
        if (b >= kBins - 1)
            return -0x1.fffffep127f; // every number
        const float x = (bin_top - (float)(b + 1)) / bin_by; // infinite or NaN where bin_by is 0
        const float slack = (fabsf(bin_top) + (float)kBins) / bin_by * 0x1p-21f;
        const float y = x - slack;
        return y > -0x1.fffffep127f ? y < top ? y : top : -0x1.fffffep127f;
    }
    // From the counts in sh.n: where top-k's border lies. Returns the number of logits through its bin, or without
    // top-k through bin `low`.
    __device__ __forceinline__ uint64_t border_of_count(Borders &b, int low)
    {
        find_count(by_k ? (uint32_t)k : ~0u, by_k ? -1 : low);
        if (by_k) {
            b.kb = sh.found[0];
            b.rest_k = (uint32_t)sh.value[0];
        }
        return sh.value[1];
    }
    // From the weights in sh.w: where top-p's border may lie.
    __device__ __forceinline__ void border_of_weight(Borders &b)
    {
        constexpr int EACH = kBins / kFThreads;
        uint64_t w[EACH], sum = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            w[i] = sh.w[tid * EACH + i];
            sum += w[i];
        }
        const uint64_t before = before_me(sum);
        b.all = scanned();
        uint64_t least_left = b.all, most_left = b.all; // by top-k
        if (by_k) {
            uint64_t c = before;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                if (tid * EACH + i == b.kb) {
                    sh.value[1] = c;
                    sh.value[3] = w[i];
                }
                c += w[i];
            }
            __syncthreads();
            b.above_k = sh.value[1];
            least_left = b.above_k > 0 ? b.above_k : 1; // (something is left)
            most_left = b.above_k + sh.value[3];
        }
        const uint64_t goals = goal_of(lane & 1 ? most_left : least_left); // both at once: the code is long
        find_weight(w, before, of_lane(goals, 0), 0);
        find_weight(w, before, of_lane(goals, 1), 1);
        __syncthreads();
        b.p0 = sh.found[0];
        b.p1 = sh.found[1];
        b.above_p = sh.value[0];
    }
    // From the weights in sh.w: about how many logits lie through bin `last`.
    __device__ __forceinline__ float number_through(int last)
    {
        const float octaves = (float)weigh.by * (1.f / kSteps) / bin_by; // of a bin
        float n = 0.f;
#pragma unroll
        for (int i = 0; i < kBins / kFThreads; ++i) {
            const int at = i * kFThreads + tid;
            if (at <= last) // its weight over that of its middle
                n += (float)sh.w[at] * __builtin_amdgcn_exp2f(((float)at + 0.5f) * octaves - (float)a.frac);
        }
        return (float)all_sum((uint64_t)fminf(n, 1e9f));
    }
    // Sums the kept weights of its pieces (or list) by runs in sh.w, and takes the logits of the zones down in sh.zone
    // (sh.count of them, or more than it holds).
    __device__ __forceinline__ void weigh_kept(const Borders &b)
    {
        __syncthreads();
        if (tid == 0)
            sh.count = 0;
        const bool zones = b.sure < kBins;
        weigh_runs([&](int t, float x) -> uint64_t {
            const int at = bin(x);
            const uint64_t w = weigh(x);
            if (zones && ((at >= b.p0 && at <= b.p1) || at == b.kb) && x > -INFINITY) {
                const uint32_t i = atomicAdd(&sh.count, 1u);
                if (i < kZone)
                    sh.zone[i] = order(x, t);
            }
            return at < b.sure && w >= least ? w : 0;
        });
    }
    // The draw, given the row's runs and zones.
    __device__ __forceinline__ void finish(const Borders &b)
    {
        uint64_t cut = kKeepAll;
        if (sh.count > kZone) {
            cut = by_values();
            weigh_runs([&](int t, float x) -> uint64_t {
                const uint64_t w = order(x, t) >= cut ? weigh(x) : 0;
                return w >= least ? w : 0;
            });
        } else if (by_k || by_p) {
            const int kept = kept_of_zone(b, (int)sh.count);
            if (kept > 0)
                cut = sh.zone[kept - 1];
            for (int i = tid; i < kept; i += kFThreads) {
                const uint64_t o = sh.zone[i], w = weigh(value_of(o));
                add_to_run((token_of(o) + lead) / PER, w >= least ? w : 0);
            }
            __syncthreads();
        }
        draw_from_runs(cut);
    }

    // ---- few logits that the filters may keep: the tokens of all from `floor` on go to lists, one
    // of each wave's. False: too many.
    __device__ __forceinline__ bool collect(float floor)
    {
        int n = 0;
        uint32_t *list = sh.list[wave];
        each(from, to, tid, kFThreads, [&](int t, float x) {
            const uint64_t hit = __ballot(x >= floor);
            if (hit) {
                const int at = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(hit >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)hit, 0));
                if (x >= floor && at < kWaveList)
                    list[at] = (uint32_t)t;
                n += __popcll(hit);
            }
        });
        // lanes whose pieces end earlier have missed the last hits
        n = (int)group_max<64>((uint32_t)n);
        __syncthreads();
        if (tid == 0)
            sh.count = 0;
        __syncthreads();
        if (n > kWaveList)
            sh.count = 1;
        __syncthreads();
        mine = sh.count ? -1 : n;
        return mine >= 0;
    }
    // f(token, value) for every logit of the lists, each wave its own
    template <typename F> __device__ __forceinline__ void each_listed(F f) const
    {
        for (int i = lane; i < mine; i += 64) {
            const int t = (int)sh.list[wave][i];
            f(t, at(t));
        }
    }
    // The zone in its order. A wave orders 64 logits by counting the larger ones of them; a logit's place is the
    // number of larger ones in all such parts, eight of which are searched together, by halves. (Counting
    // over the whole zone: 8 us for 480 logits.) Short loops, as above.
    __device__ __forceinline__ void sort_zone(int n)
    {
        constexpr int PARTS = 8, STEP = 16;
        static_assert(kZone % (64 * PARTS) == 0 && 64 * PARTS % kFThreads == 0, "whole groups of parts");
        const int filled = n <= 64 ? 64 : (n + 64 * PARTS - 1) & ~(64 * PARTS - 1);
        uint64_t *to = n <= 64 ? sh.zone : sh.parts;
        __syncthreads();
#pragma unroll 1
        for (int first = wave * 64; first < filled; first += kFThreads) {
            const uint64_t o = first + lane < n ? sh.zone[first + lane] : 0; // below every logit
            int larger = 0;
#pragma unroll 1
            for (int j = 0; first + j < n && j < 64; j += STEP)
#pragma unroll
                for (int e = 0; e < STEP; ++e) // (behind the last: 0)
                    larger += of_lane(o, j + e) > o;
            to[first + (o ? larger : lane)] = o; // (behind the last in their own places)
        }
        __syncthreads();
        if (n <= 64)
            return;
#pragma unroll 1
        for (int first = wave * 64; first < n; first += kFThreads) {
            const uint64_t o = sh.parts[first + lane];
            int place = 0;
#pragma unroll 1
            for (int q = 0; q < n; q += 64 * PARTS) {
                const uint64_t *part = sh.parts + q;
                uint32_t larger[PARTS] = {};
#pragma unroll 1
                for (uint32_t by = 32; by > 0; by >>= 1)
#pragma unroll
                    for (int c = 0; c < PARTS; ++c)
                        larger[c] += part[64 * c + larger[c] + by - 1] > o ? by : 0;
#pragma unroll
                for (int c = 0; c < PARTS; ++c) // up to 63 so far
                    place += (int)larger[c] + (part[64 * c + larger[c]] > o);
            }
            if (o)
                sh.zone[place] = o;
        }
        __syncthreads();
    }
    // How many of the n logits of the zones top-k and top-p keep; sh.zone is in its order then.
    __device__ __forceinline__ int kept_of_zone(const Borders &b, int n)
    {
        constexpr int EACH = kZone / kFThreads;
        sort_zone(n);
        if (!by_p)
            return (int64_t)b.rest_k < n ? (int)b.rest_k : n;
        uint64_t w[EACH], sum = 0;
        uint32_t above = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            const int at = tid * EACH + i;
            const float x = at < n ? value_of(sh.zone[at]) : -INFINITY;
            w[i] = at < n ? weigh(x) : 0;
            above += at < n && bin(x) < b.kb;
            sum += w[i];
        }
        uint64_t c = before_me(sum), all = b.all;
        if (by_k) {
            const int k0 = (int)all_sum(above); // in front of bin kb
            const int k1 = (int)((int64_t)k0 + b.rest_k < n ? k0 + (int)b.rest_k : n);
            uint64_t x = 0;
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                x += tid * EACH + i >= k0 && tid * EACH + i < k1 ? w[i] : 0;
            all = b.above_k + all_sum(x);
        }
        const uint64_t goal = goal_of(all) - b.above_p; // above 0: the border lies in the zone
        uint32_t less = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            c += w[i];
            less += tid * EACH + i < n && c < goal;
        }
        const int kept = (int)all_sum(less) + 1;
        return kept < n ? kept : n;
    }

    // ---- the draw: kept weights by runs of the row, then the run that the draw falls in
    __device__ __forceinline__ void add_to_run(int piece_index, uint64_t w)
    {
        if (w)
            atomicAdd((unsigned long long *)&sh.w[piece_index >> shift], (unsigned long long)w);
    }
    // weight(token, value) of every logit to its run, of the list or the row
    template <typename F> __device__ __forceinline__ void weigh_runs(F weight)
    {
        clear_bins();
        if (mine >= 0) {
            each_listed([&](int t, float x) { add_to_run((t + lead) / PER, weight(t, x)); });
        } else {
            uint64_t w = 0;
            each(from, to, tid, kFThreads, [&](int t, float x) { w += weight(t, x); },
                 [&](int i) {
                     add_to_run(i, w);
                     w = 0;
                 });
        }
        __syncthreads();
    }
    // Draws, given the runs' sums, among the logits of order >= cut.
    __device__ __forceinline__ void draw_from_runs(uint64_t cut)
    {
        constexpr int EACH = kBins / kFThreads;
        uint64_t w[EACH], sum = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            w[i] = sh.w[tid * EACH + i];
            sum += w[i];
        }
        const uint64_t before = before_me(sum);
        const uint64_t S = scanned();
        const uint64_t goal = point(S);
        find_weight(w, before, goal + 1, 0);
        __syncthreads();
        if (wave > 0)
            return;
        int t = (sh.found[0] << shift) * PER - lead; // the run's first token
        const int end = t + (PER << shift) < a.V ? t + (PER << shift) : a.V;
        t = t > 0 ? t : 0;
        for (uint64_t c = sh.value[0]; t < end; t += 64) {
            uint64_t x = 0;
            if (t + lane < end) {
                const float y = at(t + lane);
                x = order(y, t + lane) >= cut ? weigh(y) : 0;
                x = x >= least ? x : 0;
            }
            const uint64_t upto = c + scan_up(x);
            const uint64_t hit = __ballot(upto > goal);
            if (hit) {
                if (lane == __ffsll((unsigned long long)hit) - 1) {
                    a.out_token[row] = t + lane;
                    a.out_logprob[row] = (float)log((double)x / (double)S);
                }
                return;
            }
            c = of_lane(upto, 63);
        }
    }
    // The first token of its pieces that has the largest logit (~0: none), for thread 0.
    __device__ __forceinline__ uint32_t first_of_top()
    {
        uint32_t first = ~0u;
        each(from, to, tid, kFThreads, [&](int t, float x) { first = x == top && (uint32_t)t < first ? (uint32_t)t : first; });
        first = ~group_max<64>(~first);
        __syncthreads();
        if (lane == 0)
            sh.part32[wave] = first;
        __syncthreads();
        for (int w = 0; w < kFWaves; ++w)
            first = sh.part32[w] < first ? sh.part32[w] : first;
        return first;
    }
    __device__ __forceinline__ void put(int token, float logprob)
    {
        if (tid == 0) {
            a.out_token[row] = token;
            a.out_logprob[row] = logprob;
        }
    }

    // ---- the cut of a row with many equal or nearly equal logits around a border: the border's value by
    // its bits, 11 of them at a time, and then its tokens
    static __device__ __forceinline__ uint32_t key(float x) { return (uint32_t)(order(x, 0) >> 32); }
    // The value at which the count (or the weight) of the logits from the largest on reaches `want`, and what lies
    // above it.
    __device__ __forceinline__ float search(bool weights, uint64_t want, uint64_t &above)
    {
        constexpr int EACH = kBins / kFThreads;
        uint32_t hi = key(top), lo = key(-INFINITY); // the border's key lies in [lo, hi]
        above = 0;
        int down = 32;
        while (hi > lo && down > 0) { // at most three times: the range falls below 2^down
            down = 0;
            while ((hi - lo) >> down >= kBins)
                ++down;
            clear_bins();
            each(0, pieces, tid, kFThreads, [&](int, float x) {
                const uint32_t u = key(x);
                if (u <= hi && u >= lo)
                    atomicAdd((unsigned long long *)&sh.w[(hi - u) >> down], weights ? (unsigned long long)weigh(x) : 1ull);
            });
            __syncthreads();
            uint64_t w[EACH], sum = 0;
#pragma unroll
            for (int i = 0; i < EACH; ++i) {
                w[i] = sh.w[tid * EACH + i];
                sum += w[i];
            }
            find_weight(w, above + before_me(sum), want, 0);
            __syncthreads();
            above = sh.value[0];
            hi -= (uint32_t)sh.found[0] << down;
            const uint32_t least_key = hi - ((1u << down) - 1);
            lo = least_key > lo && least_key <= hi ? least_key : lo;
        }
        return value_of((uint64_t)hi << 32);
    }
    // The order of the last logit that top-k and top-p leave.
    __device__ __forceinline__ uint64_t by_values()
    {
        float v = 0.f;
        uint64_t ties = 0, above;
        if (by_k) {
            v = search(false, (uint64_t)k, above);
            ties = (uint64_t)k - above;
        }
        if (by_p) {
            uint64_t w = 0; // of what top-k leaves
            each(0, pieces, tid, kFThreads, [&](int, float x) { w += !by_k || x > v ? weigh(x) : 0; });
            const uint64_t goal = goal_of(all_sum(w) + (by_k ? ties * weigh(v) : 0));
            v = search(true, goal, above);
            const uint64_t one = weigh(v);
            ties = (goal - above + one - 1) / one; // above 0: the border lies there
        }
        // the token of the last tie that is kept
        const int per = (pieces + kFWaves - 1) / kFWaves, p0 = wave * per, p1 = p0 + per < pieces ? p0 + per : pieces;
        uint32_t n = 0;
        each(p0, p1, lane, 64, [&](int, float x) { n += x == v; });
        n = wave_sum(n);
        __syncthreads();
        if (lane == 0)
            sh.scan[wave] = n;
        __syncthreads();
        uint64_t before = 0;
        for (int i = 0; i < wave; ++i)
            before += sh.scan[i];
        if (before < ties && ties <= before + n) {
            for (int j = p0; j < p1; j += 64) {
                const int i = j + lane;
                f_u32x4 q = {0, 0, 0, 0};
                if (i < p1)
                    q = piece(i);
                uint32_t own = 0;
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    own += i < p1 && value(q, e) == v;
                const uint32_t upto = scan_up(own);
                uint64_t at = before + upto - own; // ties in front
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    if (i < p1 && value(q, e) == v && ++at == ties)
                        sh.value[3] = order(v, i * PER + e - lead);
                before += of_lane(upto, 63);
            }
        }
        __syncthreads();
        return sh.value[3];
    }
};

// A workgroup per row. Every pass but the first reads the row from L2.
//   1. The largest logit.
//   2. Where the filters' borders lie, to 1/64 of a factor of two of weight: logits are counted (top-k, min-p) or
//      weighed (top-p) by bins that are linear in the logit.
//   3. Where few logits lie above the borders, as usual, a list is made of them, and what follows reads
//      it instead of the row.
//   4. The logits of the bins in which the borders lie are ordered one by one, which gives the cut. A row
//      with too many equal or nearly equal ones finds it by the bits of the logits.
//   5. Kept weights are summed by runs of the row, and the run that the draw falls in is read again.
// 512 rows of 40000, float16, 54 us, two rows to a CU. Bound by the rows that have top-p alone and
// keep more than a list holds: two passes of 25 to 30 vector instructions per logit, 13 us of issue for two rows by
// their number, and 17 to 23 by stamps; alone on its CU a row's passes take 12 and 17, and half of all wave time is
// waiting. Such a row takes 52 us, one with top-k 23 (its count, 6, waits for LDS). A list of twice the length would save nothing: making and reading it
// takes 15 us, a whole pass 17. Loads three pieces ahead spill (63 us), and 1024 threads leave one row to a CU (69 us;
// with 200 rows 40 against 41).
template <int DT> __global__ __launch_bounds__(kFThreads, 4) void filter_row(const FilterArgs a)
{
    __shared__ Shared sh;
    RowFilter<DT, false> f(a, sh, blockIdx.x);
    float hi, lo;
    f.range(hi, lo);
    if (hi == -INFINITY) {
        f.put(-1, -INFINITY);
        return;
    }
    f.ask(hi, lo);
    if (f.greedy) {
        f.put((int)f.first_of_top(), 0.f);
        return;
    }
    __syncthreads(); // the table
    Borders b = kNoBorders;
    const int low = f.lowest_bin();
    for (int stage = 0; stage < 2; ++stage) {
        int last = kBins; // the last bin of the list, if it can hold all
        if (stage == 0) {
            if (!f.by_k && (f.m == 0.f || f.by_p))
                continue;
            f.count_bins();
            if (f.border_of_count(b, low) <= kList)
                last = f.by_k ? b.kb : low;
        } else {
            if (!f.by_p)
                continue;
            f.weigh_bins();
            f.border_of_weight(b);
            if (!f.by_k && f.number_through(b.p1) <= kList)
                last = low < b.p1 ? low : b.p1;
        }
        if (last < kBins && f.mine < 0)
            f.collect(f.floor_of(last));
    }
    b.sure = f.by_p ? b.p0 : f.by_k ? b.kb : kBins;
    f.weigh_kept(b);
    f.finish(b);
}

// ---- few rows: each cut into `chunks` of whole runs, a workgroup each, in three launches that pass
// histograms, sums and zones through the workspace. 8 rows of 250000, bfloat16, 33 us: 3, 9 and 19 of the launches and
// their gaps; 32 rows of 32000, float32, 25.6. Bound by a chain of short steps that wait for each other, 0.5 to 4 us each
// by stamps: in the last launch ends and histograms 2.3, borders 2.1 and 2.4, weights 3.4, runs, ticket and their reading
// 2.3, the zone's order 4.4, the drawn run 2.0. Instruction fetches miss in 1 to 2 of 100.
struct alignas(256) SplitRow {
    uint64_t w[kBins], runs[kBins], zone[kZone];
    uint32_t n[kBins];
    float2 ends[kFilterChunks];
    uint32_t count, ticket, first;
};
static_assert(sizeof(SplitRow) == kFilterRowBytes, "rtopk_filter.h");

// What one workgroup writes and another reads within a launch goes through the device's coherence point.
__device__ __forceinline__ void put64(uint64_t *p, uint64_t x) { __hip_atomic_store(p, x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ uint64_t get64(const uint64_t *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// The chunk of a workgroup. Few rows wait for memory more than for anything else: what a launch reads is on
// its way together, its first pieces among it.
template <int DT> __device__ __forceinline__ void take_chunk(RowFilter<DT, true> &f, int chunk, int chunks)
{
    const int runs = ((f.pieces - 1) >> f.shift) + 1, per = (runs + chunks - 1) / chunks;
    f.from = (chunk * per) << f.shift;
    f.from = f.from < f.pieces ? f.from : f.pieces;
    f.to = ((chunk + 1) * per) << f.shift;
    f.to = f.to < f.pieces ? f.to : f.pieces;
    f.ready_at = f.from + f.tid < f.pieces ? f.from + f.tid : f.pieces - 1;
    f.ready = f.base[f.ready_at];
}

template <int DT> __global__ __launch_bounds__(kFThreads, 4) void filter_range(const FilterArgs a, SplitRow *rows, int chunks)
{
    __shared__ Shared sh;
    const int row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks;
    RowFilter<DT, true> f(a, sh, row);
    take_chunk(f, chunk, chunks);
    SplitRow &s = rows[row];
    for (int i = chunk * kFThreads + f.tid; i < kBins; i += chunks * kFThreads) {
        s.w[i] = 0;
        s.n[i] = 0;
    }
    if (chunk == 0 && f.tid == 0) {
        s.count = s.ticket = 0;
        s.first = ~0u;
    }
    float hi, lo;
    f.range(hi, lo);
    if (f.tid == 0)
        s.ends[chunk] = make_float2(hi, lo);
}

// The ends of the row from those of its chunks.
template <int DT> __device__ __forceinline__ void row_range(RowFilter<DT, true> &f, const SplitRow &s, int chunks, float &hi, float &lo)
{
    hi = -INFINITY;
    lo = INFINITY;
    if (f.tid < chunks) {
        hi = s.ends[f.tid].x;
        lo = s.ends[f.tid].y;
    }
    f.all_range(hi, lo);
}

template <int DT> __global__ __launch_bounds__(kFThreads, 4) void filter_bins(const FilterArgs a, SplitRow *rows, int chunks)
{
    __shared__ Shared sh;
    const int row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks;
    RowFilter<DT, true> f(a, sh, row);
    take_chunk(f, chunk, chunks);
    SplitRow &s = rows[row];
    float hi, lo;
    row_range(f, s, chunks, hi, lo);
    if (hi == -INFINITY)
        return;
    f.ask(hi, lo);
    if (f.by_k) {
        f.count_bins();
        for (int i = f.tid; i < kBins; i += kFThreads)
            if (sh.n[i])
                atomicAdd(&s.n[i], sh.n[i]);
    }
    if (f.by_p) {
        __syncthreads(); // the table
        f.weigh_bins();
        for (int i = f.tid; i < kBins; i += kFThreads)
            if (sh.w[i])
                atomicAdd((unsigned long long *)&s.w[i], (unsigned long long)sh.w[i]);
    }
}

template <int DT> __global__ __launch_bounds__(kFThreads, 4) void filter_draw(const FilterArgs a, SplitRow *rows, int chunks)
{
    __shared__ Shared sh;
    const int row = blockIdx.x / chunks, chunk = blockIdx.x - row * chunks;
    RowFilter<DT, true> f(a, sh, row);
    take_chunk(f, chunk, chunks);
    SplitRow &s = rows[row];
    constexpr int EACH = kBins / kFThreads;
    uint32_t counts[EACH];
    uint64_t weights[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        counts[i] = s.n[f.tid + i * kFThreads];
        weights[i] = s.w[f.tid + i * kFThreads];
    }
    float hi, lo;
    row_range(f, s, chunks, hi, lo);
    if (hi == -INFINITY) {
        if (chunk == 0)
            f.put(-1, -INFINITY);
        return;
    }
    f.ask(hi, lo);
    Borders b = kNoBorders;
    if (f.greedy) {
        const uint32_t first = f.first_of_top();
        if (f.tid == 0 && first != ~0u)
            atomicMin(&s.first, first);
    } else {
        __syncthreads(); // the table
        if (f.by_k) {
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                sh.n[f.tid + i * kFThreads] = counts[i];
            __syncthreads();
            f.border_of_count(b, 0);
        }
        if (f.by_p) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                sh.w[f.tid + i * kFThreads] = weights[i];
            __syncthreads();
            f.border_of_weight(b);
        }
        b.sure = f.by_p ? b.p0 : f.by_k ? b.kb : kBins;
        f.weigh_kept(b);
        // its runs and its part of the zones (a chunk behind the row's end has no run: the row's last may end early)
        const int r0 = f.from >> f.shift, r1 = f.from < f.to ? (f.to + (1 << f.shift) - 1) >> f.shift : r0;
        for (int i = r0 + f.tid; i < r1; i += kFThreads)
            put64(&s.runs[i], sh.w[i]);
        const uint32_t n = sh.count;
        if (n > 0) {
            if (f.tid == 0)
                sh.found[0] = (int)__hip_atomic_fetch_add(&s.count, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            const uint32_t at = (uint32_t)sh.found[0];
            for (uint32_t i = f.tid; i < n && i < kZone; i += kFThreads)
                if (at + i < kZone)
                    put64(&s.zone[at + i], sh.zone[i]);
        }
    }
    // the last workgroup of the row to arrive draws
    __builtin_amdgcn_s_waitcnt(0x0f70); // this wave's stores are done
    __syncthreads();
    if (f.tid == 0)
        sh.found[1] = __hip_atomic_fetch_add(&s.ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)chunks - 1;
    __syncthreads();
    if (!sh.found[1])
        return;
    if (f.greedy) {
        f.put((int)__hip_atomic_load(&s.first, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), 0.f);
        return;
    }
    const int runs = ((f.pieces - 1) >> f.shift) + 1;
    uint64_t zone[kZone / kFThreads];
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        weights[i] = get64(&s.runs[f.tid + i * kFThreads]);
#pragma unroll
    for (int i = 0; i < kZone / kFThreads; ++i) // (what lies behind the zone's logits is not used)
        zone[i] = get64(&s.zone[f.tid + i * kFThreads]);
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        sh.w[f.tid + i * kFThreads] = f.tid + i * kFThreads < runs ? weights[i] : 0;
#pragma unroll
    for (int i = 0; i < kZone / kFThreads; ++i)
        sh.zone[f.tid + i * kFThreads] = zone[i];
    if (f.tid == 0)
        sh.count = __hip_atomic_load(&s.count, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    f.from = 0;
    f.to = f.pieces;
    __syncthreads();
    f.finish(b);
}

template <int DT> hipError_t launch_type(const FilterArgs &a, int chunks, void *ws, hipStream_t s)
{
    const dim3 block(kFThreads);
    if (chunks == 1) {
        hipLaunchKernelGGL(filter_row<DT>, dim3((unsigned)a.R), block, 0, s, a);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)(a.R * chunks));
    SplitRow *rows = static_cast<SplitRow *>(ws);
    hipLaunchKernelGGL(filter_range<DT>, grid, block, 0, s, a, rows, chunks);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    if (a.top_k || a.top_p) {
        hipLaunchKernelGGL(filter_bins<DT>, grid, block, 0, s, a, rows, chunks);
        if ((e = hipGetLastError()) != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(filter_draw<DT>, grid, block, 0, s, a, rows, chunks);
    return hipGetLastError();
}

} // namespace

hipError_t launch_filter(const FilterArgs &a, int dtype, int chunks, void *ws, hipStream_t s)
{
    return dtype == 0   ? launch_type<0>(a, chunks, ws, s)
           : dtype == 1 ? launch_type<1>(a, chunks, ws, s)
                        : launch_type<2>(a, chunks, ws, s);
}

} // namespace rtopk
