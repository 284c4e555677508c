// gfx950 attention kernels of a decode step: cross attention of every beam's
// rows to the encoder states that the beams share, and attention of a tree of
// drafted tokens over a paged key/value cache.
//
//     x_ij = scale * (q_i . k_j) for the keys j that row i may see,
//     o_i = sum_j exp(x_ij - lse_i) v_j,  lse_i = log sum_j exp(x_ij);
// a row that may see no key gives o = 0 and lse = -inf.
#include <hip/hip_runtime.h>

#include "rtopk_attn.h"

namespace rtopk {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <int DT> struct Elem;
template <> struct Elem<1> {
    typedef _Float16 T;
};
template <> struct Elem<2> {
    typedef __bf16 T;
};

// One wave per query row and head: the lanes share the keys for the scores and
// the head's elements for the outputs.
template <int DT, bool TREE> __global__ __launch_bounds__(64) void attn_rows(const AttnArgs a)
{
    typedef typename Elem<DT>::T T;
    __shared__ float sq[kMaxHeadDim], sp[64];
    __shared__ int64_t sv[64];
    const int lane = threadIdx.x;
    const int h = blockIdx.x % a.Hq, n = (blockIdx.x / a.Hq) % a.N, b = blockIdx.x / a.Hq / a.N;
    const int hk = h / a.G;
    int L = a.S, tree0 = 0x7fffffff;
    uint64_t up[kMaxTree / 64] = {};
    if (TREE) {
        int sz = a.sizes ? a.sizes[b] : a.N;
        sz = sz < 0 ? 0 : sz > a.N ? a.N : sz;
        if (n >= sz)
            return;
        L = a.lens[b];
        L = L < 0 ? 0 : L > a.S ? a.S : L;
        tree0 = L;
        L = L + sz < a.S ? L + sz : a.S;
        for (int i = n; i >= 0; i = a.parents ? parent_of(a.parents[(int64_t)b * a.N + i], i) : i - 1)
            for (int w = 0; w < kMaxTree / 64; ++w)
                up[w] |= (i >> 6) == w ? 1ull << (i & 63) : 0;
    } else if (a.lens) {
        L = a.lens[b];
        L = L < 0 ? 0 : L > a.S ? a.S : L;
    }
    const T *q = static_cast<const T *>(a.q) + b * a.qs[0] + n * a.qs[1] + h * a.qs[2];
    for (int d = lane; d < a.D; d += 64)
        sq[d] = (float)q[d];
    __syncthreads();
    float m = -INFINITY, l = 0.f, o[kMaxHeadDim / 64] = {};
    for (int j0 = 0; j0 < L; j0 += 64) {
        const int j = j0 + lane;
        bool ok = j < L;
        int64_t ko = 0, vo = 0;
        if (TREE) {
            if (ok && j >= tree0) {
                const int t = j - tree0;
                bool in = false;
                for (int w = 0; w < kMaxTree / 64; ++w)
                    in |= (t >> 6) == w && (up[w] >> (t & 63) & 1);
                ok = in;
            }
            if (ok) {
                const int pg = (int)page_of(a.page, (uint32_t)j);
                const int id = checked_page(a.table[(int64_t)b * a.ld + pg], a.num_pages);
                ok = id >= 0;
                ko = vo = id * a.ks[0] + (int64_t)(j - pg * (int)a.page.d) * a.ks[1] + hk * a.ks[2];
            }
        } else {
            if (ok && a.key_mask)
                ok = a.key_mask[(int64_t)b * a.S + j] == 0;
            ko = b * a.ks[0] + j * a.ks[1] + hk * a.ks[2];
            vo = b * a.vs[0] + j * a.vs[1] + hk * a.vs[2];
        }
        float x = -INFINITY;
        if (ok) {
            const T *k = static_cast<const T *>(a.k) + ko;
            float s = 0.f;
            for (int d = 0; d < a.D; ++d)
                s += sq[d] * (float)k[d];
            x = s * (a.scale * kLog2e);
        }
        float mt = x;
        for (int w = 1; w < 64; w <<= 1)
            mt = fmaxf(mt, __shfl_xor(mt, w));
        const float mn = fmaxf(m, mt);
        const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
        const float p = ok && x != -INFINITY ? exp2f(x - mn) : 0.f;
        m = mn;
        float ps = p;
        for (int w = 1; w < 64; w <<= 1)
            ps += __shfl_xor(ps, w);
        l = l * f + ps;
        __syncthreads();
        sp[lane] = p;
        sv[lane] = ok ? vo : -1;
        __syncthreads();
        for (int c = 0; c < kMaxHeadDim / 64; ++c) {
            const int d = c * 64 + lane;
            float acc = o[c] * f;
            if (d < a.D)
                for (int i = 0; i < 64; ++i)
                    if (sv[i] >= 0)
                        acc += sp[i] * (float)(static_cast<const T *>(a.v) + sv[i])[d];
            o[c] = acc;
        }
    }
    T *out = static_cast<T *>(a.out) + (((int64_t)b * a.N + n) * a.Hq + h) * a.D;
    for (int c = 0; c < kMaxHeadDim / 64; ++c) {
        const int d = c * 64 + lane;
        if (d < a.D)
            out[d] = (T)(l == 0.f ? 0.f : o[c] / l);
    }
    if (a.lse && lane == 0)
        a.lse[((int64_t)b * a.N + n) * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

} // namespace

hipError_t launch_attention(const AttnArgs &a, int dtype, bool tree, hipStream_t s)
{
    const dim3 grid((unsigned)((int64_t)a.B * a.N * a.Hq)), block(64);
    if (dtype == 1 && tree)
        hipLaunchKernelGGL((attn_rows<1, true>), grid, block, 0, s, a);
    else if (dtype == 1)
        hipLaunchKernelGGL((attn_rows<1, false>), grid, block, 0, s, a);
    else if (tree)
        hipLaunchKernelGGL((attn_rows<2, true>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((attn_rows<2, false>), grid, block, 0, s, a);
    return hipGetLastError();
}

} // namespace rtopk
