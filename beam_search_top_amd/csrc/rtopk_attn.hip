// gfx950 attention kernels of a decode step: cross attention of every beam's
// rows to the encoder states that the beams share, and attention of a tree of
// drafted tokens over a paged key/value cache.
//
//     x_ij = scale * (q_i . k_j) for the keys j that row i may see,
//     o_i = sum_j exp(x_ij - lse_i) v_j,  lse_i = log sum_j exp(x_ij);
// a row that may see no key gives o = 0 and lse = -inf.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "rtopk_attn.h"
#include "rtopk_cache8.h"

namespace rtopk {
namespace {

// This source is compiled twice: for caches of the type of q, and (RTOPK_ATTN_F8)
// for caches of e4m3 codes with a power of two per token and head (rtopk_cache8.h), whose
// elements become numbers of the type of q on their way into LDS or into operands.
#ifdef RTOPK_ATTN_F8
constexpr bool kF8 = true;
typedef AttnArgs8 Args;
#else
constexpr bool kF8 = false;
typedef AttnArgs Args;
#endif
__device__ __forceinline__ const uint8_t *k_scales(const AttnArgs8 &a) { return a.ksc; }
__device__ __forceinline__ const uint8_t *v_scales(const AttnArgs8 &a) { return a.vsc; }
__device__ __forceinline__ const uint8_t *k_scales(const AttnArgs &) { return nullptr; }
__device__ __forceinline__ const uint8_t *v_scales(const AttnArgs &) { return nullptr; }
constexpr int kElemBytes = kF8 ? 1 : 2; // of a cache's element

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) void glb_void;
// Global memory by its address space: a pointer that may be one of two others'
// would else be loaded from as a generic one, which LDS waits wait for too.
typedef const __attribute__((address_space(1))) char gchar;
typedef const __attribute__((address_space(1))) u32x4 gu32x4;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef const __attribute__((address_space(1))) u32x2 gu32x2;

// The 16-bit types: 1 float16, 2 bfloat16.
template <int DT> struct Elem;
template <> struct Elem<1> {
    typedef _Float16 T;
    static constexpr uint32_t kExp = 0x7c00u; // exponent bits: all set in infinities and NaN
    static constexpr float kBelow = 11.f, kTop = 15.9f; // see raised()
    typedef T V8 __attribute__((ext_vector_type(8)));
    typedef T V2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ f32x16 mfma(V8 a, V8 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
    // two of four codes times a power of two (HI: the upper two)
    template <bool HI> static __device__ __forceinline__ uint32_t decoded(uint32_t codes, float by)
    {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)codes, by, HI));
    }
};
template <> struct Elem<2> {
    typedef __bf16 T;
    static constexpr uint32_t kExp = 0x7f80u;
    static constexpr float kBelow = 0.f, kTop = 8.f;
    typedef T V8 __attribute__((ext_vector_type(8)));
    typedef T V2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ f32x16 mfma(V8 a, V8 b, f32x16 c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
    template <bool HI> static __device__ __forceinline__ uint32_t decoded(uint32_t codes, float by)
    {
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)codes, by, HI));
    }
};

// Row swizzles of tiles whose rows are CH 16-byte chunks: chunk c of row r is at
// slot c ^ f(r). LDS serves 256 bytes at a time: of keys 16 rows at one chunk
// (fk), of values four rows at four neighbouring chunks (fv); both fall on
// different banks then.
template <int CH> __device__ __forceinline__ constexpr int fk(int r) { return CH == 8 ? (r >> 1) & 7 : r & 15; }
template <int CH> __device__ __forceinline__ constexpr int fv(int r)
{
    return CH == 8 ? (r & 2) << 1 | (r >> 1 & 2) : (r & 3) << 2 | (r >> 1 & 2);
}

// The same for the keys of attn_few, whose chunks are 16 bytes: of codes 16 elements. 16 rows at
// one chunk fall on different banks.
template <int CH> __device__ __forceinline__ constexpr int ff(int r)
{
    return !kF8 ? fk<CH>(r) : CH == 8 ? (r >> 1) & 7 : (r >> 2) & 3;
}

// What attn_tiles loads in the place of a key that does not count.
__device__ __align__(16) const uint32_t g_zeros[4] = {0, 0, 0, 0};

// Keys of batch element b that any of its rows may see: [0, end), and where its
// tree begins (tree: the nodes are at tree0 ... tree0 + size - 1).
struct KeyRange {
    int end, tree0, size;
};

template <bool TREE> __device__ __forceinline__ KeyRange key_range(const AttnArgs &a, int b)
{
    KeyRange r;
    if (TREE) {
        const int sz = a.sizes ? a.sizes[b] : a.N, L = a.lens[b];
        r.size = sz < 0 ? 0 : sz > a.N ? a.N : sz;
        r.tree0 = L < 0 ? 0 : L > a.S ? a.S : L;
        r.end = r.tree0 + r.size < a.S ? r.tree0 + r.size : a.S;
    } else {
        const int L = a.lens ? a.lens[b] : a.S;
        r.size = a.N;
        r.end = r.tree0 = L < 0 ? 0 : L > a.S ? a.S : L;
    }
    return r;
}

// A batch element's keys are tiles of `bn`; split s takes tiles [s * per, ...).
__device__ __forceinline__ int tiles_per_split(int tiles, const AttnArgs &a)
{
    const int per = (tiles + a.nsplit - 1) / a.nsplit;
    return per > a.min_tiles ? per : a.min_tiles;
}

// The tile kernel. A workgroup of WR waves takes 32 * WR query rows of one key
// head (rows = nodes or beams x the query heads of the group, which all read
// the same keys) and walks over a range of keys, BN at a time.
//
// Scores are computed transposed, X^T = K Q^T, by v_mfma_f32_32x32x16: a lane
// then holds 16 keys of one query row per 32 x 32 block (row l mod 32, keys
// 8 (i / 4) + 4 (l / 32) + i mod 4), so that maxima and sums over keys stay in
// the lane and end in one exchange between the lane halves, and the weights
// are already the B operand of O^T = V^T P^T: a contraction may go over the
// keys in any order, and lane l's eight keys of step c are registers 8c ... 8c+7.
// The A operand V^T, four keys of one column per load, comes from the
// row-major tile by transposing LDS reads.
//
// Keys and values come by direct-to-LDS loads into rings of ST tiles: ST - 1 tiles
// are in flight while one is multiplied, and the wait for the oldest leaves the
// others in flight. The chunks of a row are permuted (fk, fv): no bank conflicts.
// A key that no row may see (past the end, masked out, on a page that does not
// exist) is loaded from a line of zeros: 0 * infinity would spread to every row.
//
// Bound by the matrix cores and the vector unit together: per 64 keys a wave has
// 1024 cycles of products and about 1100 of exponentials, maxima, sums and
// conversions, which overlap only in part. 8 x 2048 rows over 1000-2000 keys, 16
// heads of 128, bf16: 246 us, 818 TFLOP/s (timing copies: without the softmax
// 222 us of then 264, without loads 231, products and barriers alone 122). A
// wave of 64 rows halves the LDS reads but leaves one wave per SIMD: 318 us.
// 32 requests x 64 nodes x 4 heads over 1500-4000 keys: 158 us, of which the
// longest requests take 1.45 times the mean (one workgroup per CU).
//
// Weights are 2^(x - m), with the reference m of raised(). They are rounded to the
// inputs' type, because the matrix instructions take nothing else next to it:
// half a step per weight, as much as the output's own rounding (float16: down to
// 2^-25 of the row's largest). Their sum is of the unrounded ones, in float32.

// A row's reference after a tile whose largest score (base 2) is mx: as before,
// or kBelow under mx. It moves only when a tile exceeds it by more than kTop, so
// that the accumulators are rarely rescaled; weights stay below 2^kTop. bfloat16
// has float32's exponents, and all its bits for any weight. float16 has all of its
// from 2^-14 to 2^15.99 only, so m lies 11 below the largest score and weights
// use that whole range: those down to 2^-25 of the row's largest keep their
// bits, and those below 2^-36 become zero. (With m at the largest score the bounds
// are 2^-14 and 2^-25: 6000 keys 17 nats under one whose own value is zero gave an
// output 44 % off.) The room of 2^4.9 above is what random scores need not to move m
// again: with 13 below, 8 x 2048 rows over 1000-2000 keys take 261.5 us, with 11 259.2,
// at the largest score 260.2. Sums and outputs carry the same factor, which o / l and
// m + log2(l) take back.
template <typename E> __device__ __forceinline__ float raised(float m, float mx)
{
    float to = mx - E::kBelow;
    to = mx - to > E::kTop ? mx : to; // where mx has no bits left for kBelow
    return to > m ? to : m;
}

// Whether a reference is so large that the exponent's argument has to be taken from
// the rounded score x cs, as m was, and not from x cs in full (one instruction
// less): the two differ by half a step of m, which from 2^28 on is a factor of 2^16
// and more, so that the largest weight overflows or vanishes.
__device__ __forceinline__ bool far_off(float m) { return fabsf(m) >= 1048576.f && m != -INFINITY; }

// A row's lse from its reference and sum. kBelow is taken off both first, where
// that is exact: log2(l) near 11 would round a small lse to a multiple of 2^-20.
template <typename E> __device__ __forceinline__ float row_lse(float m, float l)
{
    return l == 0.f ? -INFINITY : (m + E::kBelow + __builtin_log2f(E::kBelow == 0.f ? l : l * (1.f / (1 << (int)E::kBelow)))) * kLn2;
}

// 2^(s - 127) of a scale byte
__device__ __forceinline__ float power_of(uint32_t s) { return __uint_as_float(scale_bits(held_scale(s))); }

// One element of an 8-bit cache in the type of q
template <typename E> __device__ __forceinline__ typename E::T element8(uint8_t code, uint8_t scale)
{
    return __builtin_bit_cast(typename E::V2, E::template decoded<false>(code, power_of(scale)))[0];
}

// Tiles in each ring: as many as the LDS of a CU holds for one workgroup of
// eight waves, or two for each of two workgroups of four.
constexpr int ring_tiles(int wr) { return wr == 8 ? 4 : 2; }

// Wait until at most N of this wave's loads are in flight (none, where fewer
// than those were started) and its LDS reads are done, then meet the other
// waves: what the older loads brought can be read, and what was read can be
// overwritten. A direct-to-LDS load counts as done once its data is in LDS.
// (__syncthreads would wait for every load.)
template <int N> __device__ __forceinline__ void ring_wait(bool full)
{
    static_assert(N >= 0 && N < 64, "vmcnt field");
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    if (full)
        __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14)); // vmcnt(N) lgkmcnt(0)
    else
        __builtin_amdgcn_s_waitcnt(0x0070); // vmcnt(0) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// Wait until this wave's LDS reads and writes are done, then meet the other waves
// (loads to registers stay in flight).
__device__ __forceinline__ void lds_wait()
{
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(0xc07f); // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// The A operands V^T of keys ROW ... ROW + 15 for DB blocks of 32 columns: per block
// two transposing reads of four keys each. In one asm statement with its
// wait: around the builtin the compiler waits for every direct-to-LDS load in
// flight too, the next tile's among them, although the loop's barrier has
// ordered the ones that matter.
template <typename V8, int DB, int ROWB, int ROW>
__device__ __forceinline__ void values_operand(V8 (&v)[DB], const int (&at)[DB], uint32_t base)
{
    constexpr int A = ROW * ROWB, B = (ROW + 8) * ROWB;
#pragma unroll
    for (int d = 0; d < DB; d += 2) {
        u32x2 x0, x1, y0, y1;
        asm volatile("ds_read_b64_tr_b16 %0, %4 offset:%6\n\t"
                     "ds_read_b64_tr_b16 %1, %4 offset:%7\n\t"
                     "ds_read_b64_tr_b16 %2, %5 offset:%6\n\t"
                     "ds_read_b64_tr_b16 %3, %5 offset:%7\n\t"
                     "s_waitcnt lgkmcnt(0)"
                     : "=&v"(x0), "=&v"(x1), "=&v"(y0), "=&v"(y1)
                     : "v"(at[d] + base), "v"(at[d + 1] + base), "i"(A), "i"(B)
                     : "memory");
        v[d] = __builtin_bit_cast(V8, __builtin_shufflevector(x0, x1, 0, 1, 2, 3));
        v[d + 1] = __builtin_bit_cast(V8, __builtin_shufflevector(y0, y1, 0, 1, 2, 3));
    }
}

template <int DT, int DP, int WR, bool TREE>
__global__ __launch_bounds__(64 * WR, DP > 128 || (WR < 4 && DP > 64) ? 1 : 2) void attn_tiles(const Args a)
{
    typedef Elem<DT> E;
    typedef typename E::T T;
    typedef typename E::V8 V8;
    typedef typename E::V2 V2;
    constexpr int BN = DP > 128 ? 32 : 64; // keys per tile
    constexpr int KB = BN / 32, DB = DP / 32, DC = DP / 16, CH = DP / 8;
    constexpr int ROWB = DP * 2, TILEB = BN * ROWB;   // bytes of a row and of a tile
    constexpr int RPL = 1024 / ROWB;                  // rows of one 1 KiB load of a wave
    constexpr int NI = BN / RPL / WR > 0 ? BN / RPL / WR : 1; // loads per wave and tensor
    static_assert(BN % (RPL * WR) == 0, "a tile is whole loads of every wave");
    constexpr int ST = kF8 ? 2 : ring_tiles(WR);
    constexpr int AHEAD = kF8 ? ST + 1 : ST; // tiles from this one to the last whose keys are on their way
    constexpr int kWords = kMaxTree / 64;
    __shared__ __align__(1024) uint8_t smem[2 * ST * TILEB]; // a ring of K tiles, a ring of V tiles
    __shared__ uint64_t s_up[TREE ? kMaxTree * kWords : 1]; // ancestors of every node
    __shared__ int s_jump[TREE ? kMaxTree : 1];
    // keys with infinities or NaN in their values, a word per tile from the first that meets the tree on
    constexpr int kOddTiles = kMaxTree / BN + 1;
    __shared__ uint64_t s_odd[TREE ? kOddTiles : 1];

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5, col = lane & 31;
    // workgroup w runs on XCD w mod 8: the row tiles of one key head and split, which
    // read the same keys, go to one XCD, the groups of them around all XCDs
    // (their lengths differ)
    const int xi = (int)blockIdx.x / 8, rt = xi % a.row_tiles;
    int w = xi / a.row_tiles * 8 + (int)blockIdx.x % 8;
    if (w >= a.B * a.Hkv * a.nsplit)
        return;
    const int hk = w % a.Hkv;
    w /= a.Hkv;
    const int split = w % a.nsplit;
    int b = w / a.nsplit;
    if (a.longest_first) {
        // workgroups start in rounds: the batch element with the b-th most keys comes b-th, so
        // that the last rounds are short ones (B <= 64: a lane per batch element)
        int keys = -1;
        if (lane < a.B) {
            const KeyRange r = key_range<TREE>(a, lane);
            keys = r.size > 0 ? r.end : 0;
        }
        int rank = lane < a.B ? 0 : 64;
        for (int i = 0; i < a.B; ++i) {
            const int other = __builtin_amdgcn_readlane(keys, i);
            rank += other > keys || (other == keys && i < lane);
        }
        b = __ffsll((unsigned long long)__ballot(rank == b)) - 1;
    }

    const KeyRange kr = key_range<TREE>(a, b);
    const int R = kr.size * a.G, r0 = rt * 32 * WR;
    if (r0 >= R)
        return;
    const int tiles = (kr.end + BN - 1) / BN, per = tiles_per_split(tiles, a);
    const int t_begin = split * per;
    if (split > 0 && t_begin >= tiles)
        return;
    const int t_end = t_begin + per < tiles ? t_begin + per : tiles;
    const bool whole = per >= tiles; // the only split: it writes the outputs itself

    // this lane's query row
    const int row = r0 + wave * 32 + col;
    const bool live = row < R;
    const int node = live ? row / a.G : 0, head = hk * a.G + (live ? row - node * a.G : 0);
    V8 q[DC];
    {
        // the sign is applied here, before the rings start: a wait for the rows later
        // would be one for the rings too
        const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u; // scores by |scale|: the maximum stays a maximum
        const T *qp = static_cast<const T *>(a.q) + b * a.qs[0] + node * a.qs[1] + head * a.qs[2];
#pragma unroll
        for (int c = 0; c < DC; ++c) {
            const int d = 16 * c + 8 * half;
            u32x4 x = {0, 0, 0, 0};
            if (live && d < a.D)
                x = *reinterpret_cast<const u32x4 *>(qp + d);
            x ^= flip;
            q[c] = __builtin_bit_cast(V8, x);
        }
    }
    const float cs = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(fabsf(a.scale) * kLog2e)));

    // ---- ancestors, by pointer doubling: after round r, s_up[i] holds the
    // nearest 2^r nodes above i (i among them) and s_jump[i] the next one
    const bool walk = TREE && kr.size > 1 && t_end * BN > kr.tree0; // this split meets the tree
    if (TREE && walk && a.parents) {
        constexpr int PER = (kMaxTree + 64 * WR - 1) / (64 * WR);
#pragma unroll
        for (int q0 = 0; q0 < PER; ++q0) {
            const int i = tid + q0 * 64 * WR;
            if (i < kr.size) {
                s_jump[i] = parent_of(a.parents[(int64_t)b * a.N + i], i);
#pragma unroll
                for (int x = 0; x < kWords; ++x)
                    s_up[i * kWords + x] = (i >> 6) == x ? 1ull << (i & 63) : 0;
            }
        }
        __syncthreads();
        for (int span = 1; span < kr.size; span <<= 1) {
            uint64_t up[PER][kWords];
            int jump[PER];
#pragma unroll
            for (int q0 = 0; q0 < PER; ++q0) {
                const int i = tid + q0 * 64 * WR;
                jump[q0] = -1;
                const int j = i < kr.size ? s_jump[i] : -1;
                if (j >= 0) {
                    jump[q0] = s_jump[j];
#pragma unroll
                    for (int x = 0; x < kWords; ++x)
                        up[q0][x] = s_up[i * kWords + x] | s_up[j * kWords + x];
                }
            }
            __syncthreads();
#pragma unroll
            for (int q0 = 0; q0 < PER; ++q0) {
                const int i = tid + q0 * 64 * WR;
                if (i < kr.size && s_jump[i] >= 0) {
#pragma unroll
                    for (int x = 0; x < kWords; ++x)
                        s_up[i * kWords + x] = up[q0][x];
                    s_jump[i] = jump[q0];
                }
            }
            __syncthreads();
        }
    }
    const int tree_tile = kr.tree0 / BN;
    if (TREE && walk) {
        if (tid < kOddTiles)
            s_odd[tid] = 0;
        __syncthreads();
    }
    // whether this row's node sees key j of the tile at t0, one bit per key
    auto window = [&](int t0) -> uint64_t {
        const int off = t0 - kr.tree0; // node of the tile's first key
        auto word = [&](int x) -> uint64_t {
            if (x < 0 || x >= kWords || node >= kr.size)
                return 0;
            if (a.parents)
                return s_up[node * kWords + x];
            const int n = node - 64 * x + 1; // a chain: nodes 0 ... node
            return n >= 64 ? ~0ull : n > 0 ? (1ull << n) - 1 : 0;
        };
        if (off <= -64)
            return ~0ull;
        if (off < 0)
            return (word(0) << -off) | ((1ull << -off) - 1);
        const int x = off >> 6, sh = off & 63;
        return sh ? (word(x) >> sh) | (word(x + 1) << (64 - sh)) : word(x);
    };

    // ---- loads. Lane l of a wave's load i brings slot l mod CH of row
    // (wave * NI + i) * RPL + l / CH
    const char *kbase = static_cast<const char *>(a.k) + kElemBytes * (TREE ? hk * a.ks[2] : b * a.ks[0] + hk * a.ks[2]);
    const char *vbase = static_cast<const char *>(a.v) + kElemBytes * (TREE ? hk * a.vs[2] : b * a.vs[0] + hk * a.vs[2]);
    const int lrow = lane / CH, lslot = lane % CH;
    // What decides about a key, its page or its mask, for a window of keys that
    // is read ahead now and then: lane l holds the page id of page win + l, or
    // the masks of keys win + 8 l ... + 7. The wait for it stays in the branch: a
    // wait at the use would drain the loads in flight for every tile.
    int win = 0, held = 0;
    bool loaded = false;
    auto refill = [&](int t) {
        if (!TREE && !a.key_mask)
            return;
        const int j0 = t * BN, j1 = j0 + BN - 1 < kr.end - 1 ? j0 + BN - 1 : kr.end - 1;
        if (TREE) {
            const int pg = (int)page_of(a.page, (uint32_t)j1);
            if (loaded && pg < win + 64)
                return;
            win = (int)page_of(a.page, (uint32_t)j0);
            held = win + lane < a.ld ? a.table[(int64_t)b * a.ld + win + lane] : -1;
        } else {
            if (loaded && j1 < win + 512)
                return;
            win = j0;
            const uint8_t *mp = a.key_mask + (int64_t)b * a.S + win + 8 * lane;
            held = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                held |= (win + 8 * lane + e < a.S && mp[e] != 0) << e;
        }
        loaded = true;
        asm volatile("" : "+v"(held));
    };
    struct Tile {
        uint64_t oks; // the keys that count, one bit each
        int64_t off;  // tree: byte offset of this lane's key, -1: does not count
        int slot;     // 8 bits: its slot
    };
    auto place = [&](int t) -> Tile {
        Tile p{0, -1, 0};
        if (t >= t_end)
            return p;
        refill(t);
        const int j = t * BN + lane;
        bool ok = lane < BN && j < kr.end;
        if (TREE) {
            const int pg = (int)page_of(a.page, (uint32_t)(ok ? j : t * BN));
            const int id = checked_page(__shfl(held, pg - win), a.num_pages);
            ok = ok && id >= 0;
            p.off = ok ? kElemBytes * (id * a.ks[0] + (int64_t)(j - pg * (int)a.page.d) * a.ks[1]) : -1;
            p.slot = ok ? id * (int)a.page.d + (j - pg * (int)a.page.d) : 0;
        } else if (a.key_mask) {
            const int w = t * BN + lane - win, out = __shfl(held, (w >> 3) & 63) >> (w & 7) & 1; // for every lane: none may be idle
            ok = ok && !out;
        }
        p.oks = __ballot(ok);
        return p;
    };
    // starts the loads of tile t's keys (or values) into the buffer at `to`. Where
    // every key counts and rows lie evenly (a load's on one page; 32-bit offsets), the wave
    // computes a load's address once and the lanes only hold an offset.
    const bool even = (!TREE || a.page.d % 8 == 0) && a.ks[1] < (1 << 25) && a.vs[1] < (1 << 25);
    auto load_tile = [&](const Tile &p, int t, const char *base, int64_t stride, bool values, uint8_t *to) {
        if (even && p.oks == (BN == 64 ? ~0ull : (1ull << BN) - 1)) {
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int lr = (wave * NI + i) * RPL, r = lr + lrow;
                const int c = lslot ^ (values ? fv<CH>(r) : fk<CH>(r));
                const uint32_t off = lrow * (uint32_t)(2 * stride) + c * 16;
                gchar *from = (gchar *)base;
                if (TREE)
                    from += (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(p.off >> 32), lr) << 32 |
                                      (uint32_t)__builtin_amdgcn_readlane((int)p.off, lr));
                else
                    from += 2 * (int64_t)(t * BN + lr) * stride;
                from += off;
                if (a.D < DP)
                    from = c * 8 < a.D ? from : (gchar *)g_zeros;
                __builtin_amdgcn_global_load_lds((glb_void *)from, (lds_void *)(to + lr * ROWB), 16, 0, 0);
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int lr = (wave * NI + i) * RPL, r = lr + lrow;
            const int c = lslot ^ (values ? fv<CH>(r) : fk<CH>(r));
            const char *from;
            bool in;
            if (TREE) {
                const int64_t o = ((int64_t)__shfl((int)(p.off >> 32), r) << 32) | (uint32_t)__shfl((int)p.off, r);
                in = o >= 0;
                from = base + o;
            } else {
                in = p.oks >> r & 1;
                from = base + 2 * (int64_t)(t * BN + r) * stride;
            }
            from = in && c * 8 < a.D ? from + c * 16 : reinterpret_cast<const char *>(g_zeros);
            __builtin_amdgcn_global_load_lds((glb_void *)from, (lds_void *)(to + lr * ROWB), 16, 0, 0);
        }
    };

    // ---- loads of an 8-bit cache: to registers, a lane 16 codes of one key, a wave 1 KiB
    // a load; a step later they go to LDS as numbers of the type of q, 2 chunks each. So the
    // products and their operands are those of a 16-bit cache, and a tile is decoded once for all rows. 32 requests
    // of 64 nodes over 1500-4000 keys, 32/8 heads of 128: 165 us (a 16-bit cache: 157), of equal lengths
    // 126: the longest request's workgroup decides. Four waves, two workgroups to a CU, decode every tile twice: 189 us.
    constexpr int CH8 = DP / 16, RPL8 = 64 / CH8, NI8 = BN / RPL8 / WR > 0 ? BN / RPL8 / WR : 1;
    struct Codes {
        u32x4 c[NI8];
        uint32_t s; // the scale of this lane's key
    };
    const int lrow8 = lane / CH8, lch8 = lane % CH8;
    // rows of a load lie evenly on one page
    const bool even8 = a.page.d % RPL8 == 0 && a.ks[1] < (1 << 25);
    auto fetch8 = [&](const Tile &p, const char *base, const uint8_t *scales, Codes &to) {
        to.s = scales[(int64_t)p.slot * a.Hkv + hk]; // of a key that does not count: of slot 0
        const bool whole8 = even8 && p.oks == (BN == 64 ? ~0ull : (1ull << BN) - 1);
#pragma unroll
        for (int i = 0; i < NI8; ++i) {
            const int lr = (wave * NI8 + i) * RPL8, r = (lr + lrow8) & (BN - 1);
            int64_t at;
            if (whole8) {
                const int from = lr & (BN - 1);
                at = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(p.off >> 32), from) << 32 |
                               (uint32_t)__builtin_amdgcn_readlane((int)p.off, from)) + lrow8 * (uint32_t)a.ks[1];
            } else {
                at = ((int64_t)__shfl((int)(p.off >> 32), r) << 32) | (uint32_t)__shfl((int)p.off, r);
                at = at < 0 ? 0 : at; // some place that can be read; not used
            }
            to.c[i] = *(gu32x4 *)(base + at + (lch8 * 16 < a.D ? lch8 * 16 : 0));
        }
    };
    auto put8 = [&](const Codes &from, uint64_t counts, bool values, uint8_t *to) {
#pragma unroll
        for (int i = 0; i < NI8; ++i) {
            const int lr = (wave * NI8 + i) * RPL8, r = (lr + lrow8) & (BN - 1);
            const float by = power_of((uint32_t)__shfl((int)from.s, r));
            const bool in = (counts >> r & 1) && lch8 * 16 < a.D;
            u32x4 y[2];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t lo = E::template decoded<false>(from.c[i][x], by), hi = E::template decoded<true>(from.c[i][x], by);
                y[x / 2][x % 2 * 2] = in ? lo : 0u;
                y[x / 2][x % 2 * 2 + 1] = in ? hi : 0u;
            }
            const int f = values ? fv<CH>(r) : fk<CH>(r);
            if (lr < BN) { // the same for the wave: with eight waves and heads of 64, half of them bring a tile
                *reinterpret_cast<u32x4 *>(to + r * ROWB + ((2 * lch8) ^ f) * 16) = y[0];
                *reinterpret_cast<u32x4 *>(to + r * ROWB + ((2 * lch8 + 1) ^ f) * 16) = y[1];
            }
        }
    };

    f32x16 o[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
        o[d] = f32x16{};
    float m = -INFINITY, l = 0.f;
    bool far = false; // a row of the wave has a reference far off: then scores are multiplied by cs on their own
    float by = 1.f, ce = cs; // (by), and in the exponent's argument by 1 (ce)

    // this lane's operand addresses: K row `col`, and the V rows of its 16-lane group
    const int kaddr = col * ROWB;
    const int vrow = 4 * half + ((lane & 15) >> 2), vchunk = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    int vaddr[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d)
        vaddr[d] = vrow * ROWB + ((4 * d + vchunk) ^ fv<CH>(vrow)) * 16 + (lane & 1) * 8;

    // X^T block k of the tile at ks
    auto scores = [&](const uint8_t *ks, int k) -> f32x16 {
        f32x16 x = {};
#pragma unroll
        for (int c = 0; c < DC; ++c) {
            const V8 kf = *reinterpret_cast<const V8 *>(ks + k * 32 * ROWB + kaddr + ((2 * c + half) ^ fk<CH>(col)) * 16);
            x = E::mfma(kf, q[c], x);
        }
        return x;
    };
    uint8_t *kbuf = smem, *vbuf = smem + ST * TILEB;

    // Keys run one tile ahead of values: the scores of tile t + 1 are multiplied
    // while the weights of tile t are computed, so that a wave keeps the matrix
    // cores and the vector unit busy at once.
    f32x16 x0[KB], x1[KB]; // scores of this tile and the next, in turn
    uint64_t oks[AHEAD + 1]; // of tiles t, t + 1, ...
    Tile last{0, -1, 0};     // the last tile whose keys are on their way
#pragma unroll
    for (int i = 0; i <= AHEAD; ++i)
        oks[i] = 0;
    Codes kq, vq; // 8 bits: of keys t + 2 and values t + 1
    if constexpr (kF8) {
        const Tile p0 = place(t_begin), p1 = place(t_begin + 1);
        last = place(t_begin + 2);
        oks[0] = p0.oks;
        oks[1] = p1.oks;
        oks[2] = last.oks;
        if (t_begin < t_end) {
            Codes k1, v0;
            fetch8(p0, kbase, k_scales(a), kq);
            fetch8(p1, kbase, k_scales(a), k1);
            fetch8(p0, vbase, v_scales(a), v0);
            put8(kq, oks[0], false, kbuf);
            fetch8(last, kbase, k_scales(a), kq);
            put8(k1, oks[1], false, kbuf + TILEB);
            fetch8(p1, vbase, v_scales(a), vq);
            put8(v0, oks[0], true, vbuf);
        }
    } else {
#pragma unroll
        for (int i = 0; i < ST; ++i) { // keys 0; keys 1, values 0; keys 2, values 1; ...
            const Tile p = place(t_begin + i);
            oks[i] = p.oks;
            if (t_begin + i < t_end)
                load_tile(p, t_begin + i, kbase, a.ks[1], false, kbuf + i * TILEB);
            if (i > 0 && t_begin + i - 1 < t_end)
                load_tile(last, t_begin + i - 1, vbase, a.vs[1], true, vbuf + (i - 1) * TILEB);
            last = p;
        }
    }
    if (t_begin < t_end) {
        if constexpr (kF8)
            lds_wait();
        else
            ring_wait<2 * (ST - 1) * NI>(t_begin + ST <= t_end);
#pragma unroll
        for (int k = 0; k < KB; ++k)
            x0[k] = scores(kbuf, k);
    }
    auto step = [&](int t, f32x16 (&x)[KB], f32x16 (&y)[KB]) {
        // keys t + 1 and values t are in LDS; every wave is done with keys t and values t - 1
        const int at = (t - t_begin) & (ST - 1);
        if constexpr (kF8) {
            // what was loaded a step ago goes to LDS, and the next loads start
            lds_wait();
            put8(vq, oks[1], true, vbuf + (at ^ 1) * TILEB);
            fetch8(last, vbase, v_scales(a), vq);
            put8(kq, oks[2], false, kbuf + at * TILEB);
            last = place(t + AHEAD);
            fetch8(last, kbase, k_scales(a), kq);
        } else {
            ring_wait<2 * (ST - 2) * NI>(t + ST <= t_end);
            if (t + ST - 1 < t_end)
                load_tile(last, t + ST - 1, vbase, a.vs[1], true, vbuf + ((at + ST - 1) & (ST - 1)) * TILEB);
            last = place(t + ST);
            if (t + ST < t_end)
                load_tile(last, t + ST, kbase, a.ks[1], false, kbuf + at * TILEB);
        }
        oks[AHEAD] = last.oks;
        const uint8_t *ks = kbuf + ((at + 1) & (ST - 1)) * TILEB, *vs = vbuf + at * TILEB;

        const bool in_tree = walk && (t + 1) * BN > kr.tree0;
        const uint64_t all = BN == 64 ? ~0ull : (1ull << BN) - 1;
        uint64_t see = oks[0];
        const bool masked = see != all || in_tree;
        if (masked || far) {
            if (in_tree)
                see &= window(t * BN);
            const uint64_t bits = see >> (4 * half);
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    x[k][i] = bits >> (32 * k + 8 * (i / 4) + i % 4) & 1 ? x[k][i] * by : -INFINITY;
        }
        // ---- the running reference; scores of the next tile (the last tile's are of whatever
        // lies there, and not used)
        if constexpr (KB > 1)
            y[0] = scores(ks, 0);
        float mx = fmaxf(x[0][0], x[0][1]);
#pragma unroll
        for (int k = 0; k < KB; ++k)
#pragma unroll
            for (int i = 0; i < 16; i += 2)
                mx = fmaxf(fmaxf(mx, x[k][i]), x[k][i + 1]);
        {
            const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(mx), __float_as_uint(mx), false, false);
            mx = fmaxf(__uint_as_float(sw[0]), __uint_as_float(sw[1]));
        }
        mx *= ce;
        if (__any(mx - m > E::kTop)) {
            const float mn = raised<E>(m, mx);
            const float f = m == mn ? 1.f : __builtin_amdgcn_exp2f(m - mn); // from -inf: 0
            m = mn;
            if (!far && __any(far_off(m))) {
                far = true;
                by = cs;
                ce = 1.f;
#pragma unroll
                for (int k = 0; k < KB; ++k)
                    x[k] *= cs;
            }
            l *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
                o[d] *= f;
        }
        // ---- weights
        const float mu = m == -INFINITY ? 0.f : m;
        V8 p[KB][2];
        y[KB - 1] = scores(ks, KB - 1);
#pragma unroll
        for (int k = 0; k < KB; ++k)
#pragma unroll
            for (int i = 0; i < 16; ++i)
                x[k][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[k][i], ce, -mu));
        if (masked && cs == 0.f) { // 0 * -inf is not -inf
            const uint64_t bits = see >> (4 * half);
#pragma unroll
            for (int k = 0; k < KB; ++k)
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    x[k][i] = bits >> (32 * k + 8 * (i / 4) + i % 4) & 1 ? x[k][i] : 0.f;
        }
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KB; ++k)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                part[i % 4] += x[k][i];
                p[k][i / 8][i % 8] = (T)x[k][i];
            }
        l += (part[0] + part[1]) + (part[2] + part[3]);
        // ---- a node's infinities and NaN must not reach the rows that do not
        // see it: they leave the tile, and are added afterwards where they belong
        if (TREE && in_tree) {
            uint8_t *vw = vbuf + at * TILEB;
            for (int u = tid; u < TILEB / 16; u += 64 * WR) {
                u32x4 *place = reinterpret_cast<u32x4 *>(vw + u * 16);
                u32x4 y = *place;
                bool any = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool lo = (y[e] & E::kExp) == E::kExp, hi = (y[e] >> 16 & E::kExp) == E::kExp;
                    any = any || lo || hi;
                    y[e] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u);
                }
                if (any) {
                    *place = y;
                    atomicOr((unsigned long long *)&s_odd[t - tree_tile], 1ull << (u / CH));
                }
            }
            __syncthreads();
        }
        // ---- outputs. The next product's operands are read before this one is
        // multiplied, which hides most of the wait for them
        const uint32_t vb = (uint32_t)(uintptr_t)(lds_void *)vs;
        V8 vf[2][DB];
        values_operand<V8, DB, ROWB, 0>(vf[0], vaddr, vb);
#pragma unroll
        for (int n = 0; n < 2 * KB; ++n) { // 16 keys each
            if (n == 0)
                values_operand<V8, DB, ROWB, 16>(vf[1], vaddr, vb);
            if constexpr (KB > 1) {
                if (n == 1)
                    values_operand<V8, DB, ROWB, 32>(vf[0], vaddr, vb);
                if (n == 2)
                    values_operand<V8, DB, ROWB, 48>(vf[1], vaddr, vb);
            }
#pragma unroll
            for (int d = 0; d < DB; ++d)
                o[d] = E::mfma(vf[n % 2][d], p[n / 2][n % 2], o[d]);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            oks[i] = oks[i + 1];
    };
    int t = t_begin;
    for (; t + 1 < t_end; t += 2) {
        step(t, x0, x1);
        step(t + 1, x1, x0);
    }
    if (t < t_end)
        step(t, x0, x1);
    // what left the tiles, for the rows that see it: the sum is infinite or NaN whatever the weight
    if (TREE && walk) {
        __syncthreads();
        for (int w = 0; w < kOddTiles; ++w) {
            uint64_t odd = s_odd[w];
            const uint64_t see = odd ? window((tree_tile + w) * BN) : 0;
            while (odd) {
                const int j = __ffsll((unsigned long long)odd) - 1;
                odd &= odd - 1;
                if (!(see >> j & 1))
                    continue;
                const int pos = (tree_tile + w) * BN + j, pg = (int)page_of(a.page, (uint32_t)pos);
                const int id = a.table[(int64_t)b * a.ld + pg]; // a page of the cache: the key counts
                // (8 bits: the codes' row and its scale)
                typedef std::conditional_t<kF8, uint8_t, T> C;
                const C *vr = reinterpret_cast<const C *>(vbase) + id * a.ks[0] + (int64_t)(pos - pg * (int)a.page.d) * a.ks[1];
                uint8_t scale = 0;
                if constexpr (kF8)
                    scale = v_scales(a)[((int64_t)id * (int)a.page.d + (pos - pg * (int)a.page.d)) * a.Hkv + hk];
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int e = 32 * d + 8 * (i / 4) + 4 * half + i % 4;
                        if (e < a.D) {
                            if constexpr (kF8) {
                                const T x = element8<E>(vr[e], scale);
                                if ((__builtin_bit_cast(uint16_t, x) & E::kExp) == E::kExp)
                                    o[d][i] += (float)x;
                            } else {
                                const uint16_t raw = reinterpret_cast<const uint16_t *>(vr)[e];
                                if ((raw & E::kExp) == E::kExp)
                                    o[d][i] += (float)vr[e];
                            }
                        }
                    }
            }
        }
    }
    {
        const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
        l = __uint_as_float(sw[0]) + __uint_as_float(sw[1]);
    }
    if (!live)
        return;
    if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t at = ((int64_t)b * a.N + node) * a.Hq + head;
        T *out = static_cast<T *>(a.out) + at * a.D;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int e = 32 * d + 8 * g + 4 * half;
                if (e < a.D) {
                    T y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        y[i] = (T)(l == 0.f ? 0.f : o[d][4 * g + i] * inv);
                    *reinterpret_cast<uint64_t *>(out + e) = __builtin_bit_cast(uint64_t, y);
                }
            }
        if (a.lse && half == 0)
            a.lse[at] = row_lse<E>(m, l);
    } else {
        const int64_t at = ((((int64_t)b * a.Hkv + hk) * a.nsplit + split) * a.N * a.G + row);
        float *po = a.part + at * DP;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4 *>(po + 32 * d + 8 * g + 4 * half) =
                    f32x4{o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
        if (half == 0) {
            a.ml[2 * at] = m;
            a.ml[2 * at + 1] = l;
        }
    }
}

// The kernel of few rows (at most 16 NB per key head): a step of decoding, a
// small tree. It is bound by reading keys and values once, so what counts is
// bytes in flight, whole lines per load and even shares: every wave takes
// steps of 32 keys (few_step) of its own, loads whole rows to registers, and refills the
// key registers as soon as the keys are in LDS and the value registers as soon
// as the outputs are made, without a barrier in the loop (the LDS that turns
// key rows into operands is the wave's own). Loads are non-temporal, for
// nobody reads the data again, but where a row is half a line (fetch_row). One row over 90000 and 131000 keys, 8 key heads
// of 128, bf16 (0.9 GB): 156 us, 5.8 TB/s, where a plain read reaches 7.0; in
// pieces of 64 bytes, as the operands want the keys, and without equal shares
// 200 us. 128 x 4 rows over 130-512 keys, 16 heads of 64 (0.17 GB): 33 us.
//
// v_mfma_f32_16x16x32 takes eight consecutive elements per lane of both
// operands. X^T = K Q^T: the A operand's row r is key 16 k + 4 (r mod 4) + r / 4
// of block k, so that lane l, which holds rows 4 (l / 16) + i of the result,
// holds keys 4 i + l / 16 of each block: the B operand of O^T = V^T P^T when the
// contraction goes over the keys in the order (l / 16, block, i). The A operand
// there needs eight keys of one column per lane, while a load brings VE
// consecutive columns of one key: lane l loads columns VE (l mod 16) ... of its
// eight keys (so that load j of a wave is the four whole rows 4 j ... 4 j + 3), and
// the VE products take column VE r + m as row r of product m, each assembled
// by byte permutes (half an instruction per element).
template <int DT> struct Small;
template <> struct Small<1> {
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
    {
        typedef Elem<1>::V8 V8;
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V8, a), __builtin_bit_cast(V8, b), c, 0, 0, 0);
    }
};
template <> struct Small<2> {
    static __device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c)
    {
        typedef Elem<2>::V8 V8;
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V8, a), __builtin_bit_cast(V8, b), c, 0, 0, 0);
    }
};

// Maximum and sum over the four 16-lane rows of a wave.
__device__ __forceinline__ float rows_max(float x)
{
    auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
    s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float rows_sum(float x)
{
    auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(s[0]) + __uint_as_float(s[1]);
    s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// Data that another workgroup reads within the launch goes through the
// device's coherence point (agent-scope accesses).
__device__ __forceinline__ void put64(void *p, float x, float y)
{
    const uint64_t v = (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
    __hip_atomic_store(static_cast<uint64_t *>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t get64(const void *p)
{
    return __hip_atomic_load(static_cast<const uint64_t *>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

constexpr int kFewWaves = 4;
// Workgroups per CU that the registers of attn_few have to leave room for. 8 bits, one row: with heads of 64 three
// (2 requests of 90000 and 131000 keys of 16 heads, steps of 32 keys: 134 us, with four, which spill, 153), but two where every lane has an offset of
// its own (pages of 24: 129 us, with three, which spill, 133); with heads of 128 two (8 heads: 98 us, 4.7 TB/s; three, which
// spill, 103).
constexpr int few_waves(int dp, int nb, int mode) { return kF8 && nb == 1 && dp == 64 && mode != 2 ? 3 : 2; }
// Keys per step of a wave. 64 of 64 codes: half as many bytes on their way were too few (2 x 440000 keys of 16
// heads: 414 us, with 32 500 us; with 128 codes 64 make no difference, and two blocks of rows spill).
constexpr int few_step(int dp) { return kF8 && dp == 64 ? 64 : 32; }

// A workgroup's share: steps [begin, end) of batch element b, one of `parts`
// shares of it; `unit` numbers the shares of all batch elements, `unit0` is
// that of b's first.
struct Share {
    int b, begin, end, parts, unit, unit0;
};

// Cuts the steps of all batch elements into shares of equal size, `units` of
// them at most: long and short batch elements load the GPU evenly, which the host
// cannot do without knowing the lengths. Every wave sums the lengths by itself
// (B <= 256). A batch element with rows has at least one share.
template <bool TREE, int kFewStep> __device__ __forceinline__ Share find_share(const AttnArgs &a, int unit, int lane)
{
    Share s{-1, 0, 0, 0, unit, 0};
    int tiles[4], total = 0, longest = 0;
    const int chunks = (a.B + 63) / 64;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        tiles[i] = -1; // no rows: no share
        if (i >= chunks)
            continue;
        const int b = 64 * i + lane;
        if (b < a.B) {
            const KeyRange kr = key_range<TREE>(a, b);
            if (kr.size > 0)
                tiles[i] = (kr.end + kFewStep - 1) / kFewStep;
        }
        total += tiles[i] > 0 ? tiles[i] : 0; // of all together at most 2^30: the host cuts no call of more
        longest = tiles[i] > longest ? tiles[i] : longest;
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        total += __shfl_xor(total, o);
        const int x = __shfl_xor(longest, o);
        longest = x > longest ? x : longest;
    }
    const int room = a.units - a.B; // shares besides each batch element's last, partial one
    int quota = (total + room - 1) / room;
    quota = quota > a.min_tiles ? quota : a.min_tiles;
    const int most = (longest + kMaxParts - 1) / kMaxParts;
    quota = quota > most ? quota : most;
    int before = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= chunks)
            break;
        const int n = tiles[i] < 0 ? 0 : tiles[i] <= quota ? 1 : (tiles[i] + quota - 1) / quota;
        int pre = n;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int x = __shfl_up(pre, o);
            pre += lane >= o ? x : 0;
        }
        pre += before;
        const uint64_t hit = __ballot(unit < pre && unit >= pre - n);
        if (hit) {
            const int src = __ffsll((unsigned long long)hit) - 1;
            const int t = __builtin_amdgcn_readlane(tiles[i], src);
            s.b = 64 * i + src;
            s.parts = __builtin_amdgcn_readlane(n, src);
            s.unit0 = __builtin_amdgcn_readlane(pre, src) - s.parts;
            s.begin = (unit - s.unit0) * quota;
            s.end = s.begin + quota < t ? s.begin + quota : t;
            return s;
        }
        before = __builtin_amdgcn_readlane(pre, 63);
    }
    return s;
}

// MODE 0: cross attention; 1: a tree, pages of a multiple of the rows of one load (8; of 64 codes 16) in
// tokens; 2: a tree, other pages. (Modes of one kernel, not branches in it: the counts by which a wave waits for
// its older loads only must be the same on every path.)
template <int DT, int DP, int NB, int MODE>
__global__ __launch_bounds__(64 * kFewWaves, few_waves(DP, NB, MODE)) void attn_few(const Args a)
{
    constexpr bool TREE = MODE != 0;
    constexpr int kFewStep = few_step(DP), GROUPS = kFewStep / 32; // keys of a step, products with the values over them
    typedef std::conditional_t<kFewStep == 64, uint64_t, uint32_t> Mask;
    typedef Elem<DT> E;
    typedef typename E::T T;
    constexpr int VE = DP / 16, DC = DP / 32, VW = VE / 2; // columns per lane, products per score, value dwords
    constexpr int ROWB = DP * kElemBytes, CH = ROWB / 16, RPL = 1024 / ROWB, NK = kFewStep / RPL; // a 1 KiB load is RPL rows
    constexpr int VL = kF8 ? VE / 4 : VW; // value dwords as they are loaded
    constexpr int PITCH = DP + 4;
    constexpr int KEYS = kFewWaves * kFewStep * ROWB, OUTS = kFewWaves * 16 * PITCH * 4;
    // the waves' keys; after the loop their outputs, a block of 16 rows at a time
    __shared__ __align__(1024) uint8_t smem[KEYS > OUTS ? KEYS : OUTS];
    __shared__ float s_m[kFewWaves][16 * NB], s_l[kFewWaves][16 * NB];
    __shared__ int32_t s_parent[TREE ? 16 * NB : 1];
    __shared__ uint32_t s_last;

    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, grp = lane >> 4;
    // workgroup w runs on XCD w mod 8: shares go around the XCDs, and all key
    // heads of a share, which lie side by side in memory, to the same one
    const int xi = (int)blockIdx.x / 8, hk = xi % a.Hkv, unit = xi / a.Hkv * 8 + (int)blockIdx.x % 8;
    Share sh;
    if (a.units > 0) {
        sh = find_share<TREE, kFewStep>(a, unit, lane);
        if (sh.b < 0)
            return;
    } else {
        if (unit >= a.B)
            return;
        sh = Share{unit, 0, 0, 1, unit, unit};
    }
    // the same for every lane, which the compiler does not see through the search
    sh.begin = __builtin_amdgcn_readfirstlane(sh.begin);
    sh.end = __builtin_amdgcn_readfirstlane(sh.end);
    sh.parts = __builtin_amdgcn_readfirstlane(sh.parts);
    sh.unit0 = __builtin_amdgcn_readfirstlane(sh.unit0);
    const int b = __builtin_amdgcn_readfirstlane(sh.b);
    const KeyRange kr = key_range<TREE>(a, b);
    const int R = kr.size * a.G;
    if (R == 0)
        return;
    const int t_begin = sh.begin, t_end = a.units > 0 ? sh.end : (kr.end + kFewStep - 1) / kFewStep, parts = sh.parts;

    // ---- loads
    gchar *kbase = (gchar *)a.k + kElemBytes * (TREE ? hk * a.ks[2] : b * a.ks[0] + hk * a.ks[2]);
    gchar *vbase = (gchar *)a.v + kElemBytes * (TREE ? hk * a.vs[2] : b * a.vs[0] + hk * a.vs[2]);
    uint8_t *mine = smem + wave * kFewStep * ROWB;
    // Step t is kFewStep rows from first(t) on. Past the last row that can be read (cross, steps of
    // 32: S >= 32) it begins earlier and leaves out the keys of the step before.
    auto first = [&](int t) -> int {
        if (TREE)
            return t * kFewStep;
        const int f = (t < t_end ? t : t_begin) * kFewStep;
        return f < a.S - kFewStep ? f : a.S - kFewStep;
    };
    // what decides about key first(t) + lane mod kFewStep, read ahead: its page, or its mask
    auto fetch = [&](int t) -> int {
        const int j = first(t) + (lane & (kFewStep - 1));
        if (t >= t_end || j >= kr.end)
            return -1;
        if (TREE)
            return a.table[(int64_t)b * a.ld + page_of(a.page, (uint32_t)j)];
        return a.key_mask ? a.key_mask[(int64_t)b * a.S + j] : 0;
    };
    // Keys that do not count are loaded all the same, from some place that can
    // be read (tree: the cache's first rows); their scores are replaced and their
    // values zeroed where they are used.
    struct Step {
        Mask oks;     // the keys that count
        int64_t off;  // tree: byte offset of this lane's key
        int slot;     // 8 bits: its slot
    };
    auto place = [&](int t, int info) -> Step {
        const int j = first(t) + (lane & (kFewStep - 1));
        bool ok = t < t_end && j >= t * kFewStep && j < kr.end;
        Step s{0, 0, 0};
        if (TREE) {
            const int id = checked_page(info, a.num_pages);
            ok = ok && id >= 0;
            const int pg = (int)page_of(a.page, (uint32_t)(ok ? j : 0));
            s.off = ok ? kElemBytes * (id * a.ks[0] + (int64_t)(j - pg * (int)a.page.d) * a.ks[1]) : 0;
            s.slot = ok ? id * (int)a.page.d + (j - pg * (int)a.page.d) : 0;
        } else {
            ok = ok && info == 0;
        }
        s.oks = (Mask)__ballot(ok);
        return s;
    };
    // Row u + lane_r of a step (u the same for the wave) lies at a base of the wave's and a
    // 32-bit offset of the lane's: cross attention's rows are evenly spaced (the
    // host sees to it that 32 of them span less than 2^32 bytes), the rows of one load of a tree (8; of
    // 64 codes 16) lie on one page where pages allow it. Else every lane has a 64-bit offset of its own.
    const int lrow = lane / CH, lchunk = lane % CH;
    constexpr int CE = 16 / kElemBytes; // elements of a chunk
    const uint32_t kstep = kElemBytes * (uint32_t)a.ks[1], vstep = kElemBytes * (uint32_t)a.vs[1];
    const uint32_t kcol = lchunk * CE < a.D ? lchunk * 16 : 0, vcol = VE * col < a.D ? kElemBytes * VE * col : 0;
    const uint32_t klane = lrow * kstep + kcol, vlane = grp * vstep + vcol;
    auto row = [&](gchar *base, const Step &s, int t, int u, int lane_r, uint32_t step, uint32_t lane_off, uint32_t lane_col) -> gchar * {
        // behind the last step, every lane reads the same line
        if constexpr (MODE == 0)
            return base + (t < t_end ? (int64_t)(first(t) + u) * step : 0) + (t < t_end ? lane_off : 0);
        else if constexpr (MODE == 1)
            return base + (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(s.off >> 32), u) << 32 |
                                    (uint32_t)__builtin_amdgcn_readlane((int)s.off, u)) + (t < t_end ? lane_off : 0);
        else
            return base + (int64_t)((uint64_t)(uint32_t)__shfl((int)(s.off >> 32), u + lane_r) << 32 |
                                    (uint32_t)__shfl((int)s.off, u + lane_r)) + (t < t_end ? lane_col : 0);
    };
    // 64-byte rows are half lines: the next head's workgroup reads the other half soon after (and fetches the line
    // again if the first load has marked it as read once: 137 against 115 us)
    auto fetch_row = [](auto *p) {
        if constexpr (ROWB < 128)
            return *p;
        else
            return __builtin_nontemporal_load(p);
    };
    u32x4 kq[NK];
    auto load_keys = [&](const Step &s, int t) {
#pragma unroll
        for (int i = 0; i < NK; ++i)
            kq[i] = fetch_row((gu32x4 *)row(kbase, s, t, i * RPL, lrow, kstep, klane, kcol));
    };
    // 8 bits: the scales of key and value `lane` of the step
    auto load_scale = [&](const Step &s) -> uint32_t {
        if constexpr (kF8) {
            const int64_t at = (int64_t)s.slot * a.Hkv + hk;
            return k_scales(a)[at] | (uint32_t)v_scales(a)[at] << 16;
        }
        return 0;
    };
    uint32_t vq[8 * GROUPS][VL];
    auto load_values = [&](const Step &s, int t) {
#pragma unroll
        for (int j = 0; j < 8 * GROUPS; ++j) {
            gchar *p = row(vbase, s, t, 4 * j, grp, vstep, vlane, vcol);
            if constexpr (VL == 1) {
                vq[j][0] = fetch_row((const __attribute__((address_space(1))) uint32_t *)p);
            } else if constexpr (VL == 4) {
                const u32x4 y = __builtin_nontemporal_load((gu32x4 *)p);
#pragma unroll
                for (int x = 0; x < VL; ++x)
                    vq[j][x] = y[x];
            } else {
                const u32x2 y = __builtin_nontemporal_load((gu32x2 *)p);
                vq[j][0] = y[0];
                vq[j][1] = y[1];
            }
        }
    };
    // ---- this lane's query rows
    u32x4 q[NB][DC];
    int node[NB], head[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        const int row = 16 * n + col;
        const bool live = row < R;
        node[n] = live ? row / a.G : 0;
        head[n] = hk * a.G + (live ? row - node[n] * a.G : 0);
        gchar *qp = (gchar *)a.q + 2 * (b * a.qs[0] + node[n] * a.qs[1] + head[n] * a.qs[2]);
#pragma unroll
        for (int c = 0; c < DC; ++c) {
            const int e = 32 * c + 8 * grp;
            u32x4 x = {0, 0, 0, 0};
            if (live && e < a.D)
                x = *(gu32x4 *)(qp + 2 * e);
            q[n][c] = x;
        }
    }
    int t = t_begin + wave;
    Step now = place(t, fetch(t));
    load_keys(now, t);
    uint32_t scale = load_scale(now);
    int info = fetch(t + kFewWaves);
    load_values(now, t);

    if (a.scale < 0.f) { // scores by |scale|: the maximum stays a maximum
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int c = 0; c < DC; ++c)
                q[n][c] ^= 0x80008000u;
    }
    const float cs = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(fabsf(a.scale) * kLog2e)));
    // the nodes that each of its rows sees (at most 32 nodes: R <= 16 NB)
    const bool walk = TREE && kr.size > 1 && t_end * kFewStep > kr.tree0;
    uint32_t up[NB] = {};
    if (TREE && walk) {
        if (a.parents) {
            if (tid < kr.size)
                s_parent[tid] = parent_of(a.parents[(int64_t)b * a.N + tid], tid);
            __syncthreads();
        }
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            if (a.parents)
                for (int i = node[n]; i >= 0; i = s_parent[i])
                    up[n] |= 1u << i;
            else
                up[n] = node[n] >= 31 ? ~0u : (1u << (node[n] + 1)) - 1;
        }
    }
    // this lane's key in each block, as the A operand's row col
    const int kr0 = 4 * (col & 3) + (col >> 2);

    f32x4 o[NB][VE];
    float m[NB], l[NB], ce[NB];
    bool far[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        far[n] = false;
        ce[n] = cs;
        m[n] = -INFINITY;
        l[n] = 0.f;
#pragma unroll
        for (int x = 0; x < VE; ++x)
            o[n][x] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    for (; t < t_end; t += kFewWaves) {
        const bool in_tree = walk && (t + 1) * kFewStep > kr.tree0;
        const bool masked = now.oks != (Mask)~(Mask)0 || in_tree;
        // ---- scores
        if (a.D < DP) { // elements past the head's are zeros in both operands
#pragma unroll
            for (int i = 0; i < NK; ++i)
                kq[i] = lchunk * CE < a.D ? kq[i] : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int r = i * RPL + lrow;
            *reinterpret_cast<u32x4 *>(mine + r * ROWB + (lchunk ^ ff<CH>(r)) * 16) = kq[i];
        }
        // of key and value `lane`
        const uint32_t kby = kF8 ? scale_bits(held_scale(scale & 0xffu)) : 0, vby = kF8 ? scale_bits(held_scale(scale >> 16)) : 0;
        const Step next = place(t + kFewWaves, info);
        load_keys(next, t + kFewWaves);
        scale = load_scale(next);
        info = fetch(t + 2 * kFewWaves);
        // this wave's own LDS, which serves it in order: no other wave to wait for
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        f32x4 x[NB][2 * GROUPS];
#pragma unroll
        for (int k = 0; k < 2 * GROUPS; ++k) {
            const int r = 16 * k + kr0;
            u32x4 kf[DC];
            if constexpr (kF8) {
                const float f = __uint_as_float((uint32_t)__shfl((int)kby, r));
#pragma unroll
                for (int c = 0; c < DC; ++c) {
                    const u32x2 y = *reinterpret_cast<const u32x2 *>(mine + r * ROWB + ((2 * c + grp / 2) ^ ff<CH>(r)) * 16 + grp % 2 * 8);
                    kf[c] = u32x4{E::template decoded<false>(y[0], f), E::template decoded<true>(y[0], f),
                                  E::template decoded<false>(y[1], f), E::template decoded<true>(y[1], f)};
                }
            } else {
#pragma unroll
                for (int c = 0; c < DC; ++c)
                    kf[c] = *reinterpret_cast<const u32x4 *>(mine + r * ROWB + ((4 * c + grp) ^ ff<CH>(r)) * 16);
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                x[n][k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < DC; ++c)
                    x[n][k] = Small<DT>::mfma(kf[c], q[n][c], x[n][k]);
            }
        }
        // ---- weights
        Mask see[NB];
        u32x4 p[NB][GROUPS];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            see[n] = now.oks;
            if (in_tree) {
                const int off = t * kFewStep - kr.tree0; // node of the step's first key: above -kFewStep
                see[n] &= off < 0 ? ((Mask)up[n] << -off) | (((Mask)1 << -off) - 1) : off < 32 ? up[n] >> off : 0;
            }
            const Mask bits = see[n] >> grp;
            if (masked || far[n]) {
                if (far[n]) {
#pragma unroll
                    for (int k = 0; k < 2 * GROUPS; ++k)
                        x[n][k] *= cs;
                }
#pragma unroll
                for (int k = 0; k < 2 * GROUPS; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[n][k][i] = bits >> (16 * k + 4 * i) & 1 ? x[n][k][i] : -INFINITY;
            }
            float mx = x[n][0][0];
#pragma unroll
            for (int k = 0; k < 2 * GROUPS; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mx = fmaxf(mx, x[n][k][i]);
            mx = rows_max(mx) * ce[n];
            if (__any(mx - m[n] > E::kTop)) {
                const float mn = raised<E>(m[n], mx);
                const float f = m[n] == mn ? 1.f : __builtin_amdgcn_exp2f(m[n] - mn);
                m[n] = mn;
                if (!far[n] && __any(far_off(mn))) {
                    far[n] = true;
                    ce[n] = 1.f;
#pragma unroll
                    for (int k = 0; k < 2 * GROUPS; ++k)
                        x[n][k] *= cs;
                }
                l[n] *= f;
#pragma unroll
                for (int y = 0; y < VE; ++y)
                    o[n][y] *= f;
            }
            const float mu = m[n] == -INFINITY ? 0.f : m[n];
            T y[GROUPS][8];
#pragma unroll
            for (int k = 0; k < 2 * GROUPS; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float e = __builtin_amdgcn_exp2f(__builtin_fmaf(x[n][k][i], ce[n], -mu));
                    if (masked && cs == 0.f) // 0 * -inf is not -inf
                        e = bits >> (16 * k + 4 * i) & 1 ? e : 0.f;
                    l[n] += e;
                    y[k / 2][4 * (k % 2) + i] = (T)e;
                }
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
                p[n][g] = __builtin_bit_cast(u32x4, y[g]);
        }
        bool odd = false;
        if constexpr (kF8) {
            // two columns at a time as numbers of the type of q; what is done about places that do not count and about
            // a node's NaN is as below
            if (now.oks != (Mask)~(Mask)0) { // (code 0 is 0)
#pragma unroll
                for (int j = 0; j < 8 * GROUPS; ++j)
#pragma unroll
                    for (int e = 0; e < VL; ++e)
                        vq[j][e] = now.oks >> (4 * j + grp) & 1 ? vq[j][e] : 0u;
                asm volatile("" ::: "memory"); // a branch, not a selection in every step
            }
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                float vf[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    vf[j] = __uint_as_float((uint32_t)__shfl((int)vby, 32 * g + 4 * j + grp));
#pragma unroll
                for (int y = 0; y < VE; y += 2) {
                    uint32_t d[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        d[j] = y % 4 ? E::template decoded<true>(vq[8 * g + j][y / 4], vf[j])
                                     : E::template decoded<false>(vq[8 * g + j][y / 4], vf[j]);
                    if (in_tree) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const bool lo = (d[j] & E::kExp) == E::kExp, hi = (d[j] >> 16 & E::kExp) == E::kExp;
                            odd = odd || lo || hi;
                            d[j] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u);
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        u32x4 v;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            v[j] = __builtin_amdgcn_perm(d[2 * j + 1], d[2 * j], h ? 0x07060302u : 0x05040100u);
#pragma unroll
                        for (int n = 0; n < NB; ++n)
                            o[n][y + h] = Small<DT>::mfma(v, p[n][g], o[n][y + h]);
                    }
                }
            }
            odd = in_tree && __any(odd);
        } else {
            if (now.oks != ~0u) { // 0 * infinity: a value that does not count must be finite
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < VW; ++e)
                        vq[j][e] = now.oks >> (4 * j + grp) & 1 ? vq[j][e] : 0u;
            }
            // ---- a node's infinities and NaN, as in attn_tiles
            if (TREE && in_tree) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int e = 0; e < VW; ++e) {
                        const bool lo = (vq[j][e] & E::kExp) == E::kExp, hi = (vq[j][e] >> 16 & E::kExp) == E::kExp;
                        odd = odd || lo || hi;
                        vq[j][e] &= (lo ? 0xffff0000u : ~0u) & (hi ? 0x0000ffffu : ~0u);
                    }
                odd = __any(odd);
            }
            // ---- outputs
#pragma unroll
            for (int y = 0; y < VE; ++y) {
                u32x4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = __builtin_amdgcn_perm(vq[2 * j + 1][y / 2], vq[2 * j][y / 2], y % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    o[n][y] = Small<DT>::mfma(v, p[n][0], o[n][y]);
            }
        }
        load_values(next, t + kFewWaves);
        if (TREE && odd) {
            for (int j = 0; j < kFewStep; ++j) {
                if (!(now.oks >> j & 1))
                    continue;
                const int pos = t * kFewStep + j, pg = (int)page_of(a.page, (uint32_t)pos);
                const int id = a.table[(int64_t)b * a.ld + pg]; // a page of the cache: the key counts
                typedef std::conditional_t<kF8, uint8_t, T> C;
                const C *vr = static_cast<const C *>(a.v) + hk * a.vs[2] + id * a.ks[0] + (int64_t)(pos - pg * (int)a.page.d) * a.ks[1];
                uint8_t its = 0; // scale
                if constexpr (kF8)
                    its = v_scales(a)[((int64_t)id * (int)a.page.d + (pos - pg * (int)a.page.d)) * a.Hkv + hk];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int y = 0; y < VE; ++y) {
                        const int e = VE * (4 * grp + i) + y;
                        if (e >= a.D)
                            continue;
                        if constexpr (kF8) {
                            const T x = element8<E>(vr[e], its);
                            if ((__builtin_bit_cast(uint16_t, x) & E::kExp) != E::kExp)
                                continue;
#pragma unroll
                            for (int n = 0; n < NB; ++n)
                                if (see[n] >> j & 1)
                                    o[n][y][i] += (float)x;
                            continue;
                        }
                        const uint16_t raw = reinterpret_cast<const uint16_t *>(vr)[e];
                        if ((raw & E::kExp) != E::kExp)
                            continue;
#pragma unroll
                        for (int n = 0; n < NB; ++n)
                            if (see[n] >> j & 1)
                                o[n][y][i] += (float)vr[e];
                    }
            }
        }
        now = next;
    }

    // ---- the waves' parts, joined in their order
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        l[n] = rows_sum(l[n]);
        if (grp == 0) {
            s_m[wave][16 * n + col] = m[n];
            s_l[wave][16 * n + col] = l[n];
        }
    }
    float *s_o = reinterpret_cast<float *>(smem);
    const int64_t step = (int64_t)a.Hkv * a.N * a.G; // rows of a unit
    float *part = a.part + (sh.unit0 * step + (int64_t)hk * a.N * a.G) * DP;
    float *ml = a.ml + (sh.unit0 * step + (int64_t)hk * a.N * a.G) * 2;
    const int split = sh.unit - sh.unit0;
    auto finish = [&](int row, int e, f32x4 y, float M, float L) {
        const int nd = row / a.G, hd = hk * a.G + row - nd * a.G;
        const int64_t at = ((int64_t)b * a.N + nd) * a.Hq + hd;
        if (e < a.D) {
            const float inv = 1.f / L;
            T z[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                z[i] = (T)(L == 0.f ? 0.f : y[i] * inv);
            *reinterpret_cast<uint64_t *>(static_cast<T *>(a.out) + at * a.D + e) = __builtin_bit_cast(uint64_t, z);
        }
        if (a.lse && e == 0)
            a.lse[at] = row_lse<E>(M, L);
    };
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        __syncthreads();
        float *to = s_o + (wave * 16 + col) * PITCH + 4 * VE * grp;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int y = 0; y < VE; y += 4)
                *reinterpret_cast<f32x4 *>(to + VE * i + y) = f32x4{o[n][y][i], o[n][y + 1][i], o[n][y + 2][i], o[n][y + 3][i]};
        __syncthreads();
        for (int u = tid; u < 16 * DP / 4; u += 64 * kFewWaves) {
            const int r = u / (DP / 4), e = u % (DP / 4) * 4, row = 16 * n + r;
            if (row >= R)
                continue;
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int x = 0; x < kFewWaves; ++x)
                M = fmaxf(M, s_m[x][row]);
            const float mu = M == -INFINITY ? 0.f : M;
            f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < kFewWaves; ++x) {
                const float f = __builtin_amdgcn_exp2f(s_m[x][row] - mu);
                L += f * s_l[x][row];
                y += f * *reinterpret_cast<const f32x4 *>(s_o + (x * 16 + r) * PITCH + e);
            }
            if (parts == 1) {
                finish(row, e, y, M, L);
            } else {
                float *to = part + (split * step + row) * DP + e;
                put64(to, y[0], y[1]);
                put64(to + 2, y[2], y[3]);
                if (e == 0)
                    put64(ml + 2 * (split * step + row), M, L);
            }
        }
    }
    if (parts == 1)
        return;
    // ---- the last workgroup of the group to arrive joins the splits, in their
    // order whichever arrives last; the ticket is zero again afterwards
    __builtin_amdgcn_s_waitcnt(0x0f70); // this wave's stores are done
    __syncthreads();
    uint32_t *ticket = a.ticket + b * a.Hkv + hk;
    if (tid == 0) {
        s_last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)parts - 1;
        if (s_last)
            __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (!s_last)
        return;
    for (int u = tid; u < R * (DP / 4); u += 64 * kFewWaves) {
        const int row = u / (DP / 4), e = u % (DP / 4) * 4;
        float M = -INFINITY, L = 0.f;
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
        constexpr int AT = 8; // splits whose loads are in flight together
        for (int s0 = 0; s0 < parts; s0 += AT) {
            uint64_t h[AT], y0[AT], y1[AT];
#pragma unroll
            for (int x = 0; x < AT; ++x) {
                const int sp = s0 + x < parts ? s0 + x : parts - 1;
                h[x] = get64(ml + 2 * (sp * step + row));
                y0[x] = get64(part + (sp * step + row) * DP + e);
                y1[x] = get64(part + (sp * step + row) * DP + e + 2);
            }
            float Mn = M;
#pragma unroll
            for (int x = 0; x < AT; ++x)
                Mn = fmaxf(Mn, __uint_as_float((uint32_t)h[x]));
            const float mu = Mn == -INFINITY ? 0.f : Mn, f0 = __builtin_amdgcn_exp2f(M - mu);
            L *= f0;
            y *= f0;
            M = Mn;
#pragma unroll
            for (int x = 0; x < AT; ++x) {
                if (s0 + x >= parts)
                    break;
                const float f = __builtin_amdgcn_exp2f(__uint_as_float((uint32_t)h[x]) - mu);
                L += f * __uint_as_float((uint32_t)(h[x] >> 32));
                y[0] += f * __uint_as_float((uint32_t)y0[x]);
                y[1] += f * __uint_as_float((uint32_t)(y0[x] >> 32));
                y[2] += f * __uint_as_float((uint32_t)y1[x]);
                y[3] += f * __uint_as_float((uint32_t)(y1[x] >> 32));
            }
        }
        finish(row, e, y, M, L);
    }
}

// Joins the splits of attn_tiles, in their order: a wave per row, eight parts'
// loads in flight (4060 rows of 80, nine parts: 6.8 us; one part at a time 11.6).
template <int DT, int DP, bool TREE> __global__ __launch_bounds__(256) void attn_join(const Args a, int bn)
{
    typedef typename Elem<DT>::T T;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (id >= (int64_t)a.B * a.Hkv * a.N * a.G)
        return;
    const int row = (int)(id % (a.N * a.G));
    const int hk = (int)(id / (a.N * a.G) % a.Hkv), b = (int)(id / (a.N * a.G) / a.Hkv);
    const KeyRange kr = key_range<TREE>(a, b);
    const int tiles = (kr.end + bn - 1) / bn, per = tiles_per_split(tiles, a);
    if (row >= kr.size * a.G || per >= tiles)
        return;
    const int n = (tiles + per - 1) / per; // splits with keys
    const int64_t at0 = ((int64_t)b * a.Hkv + hk) * a.nsplit * a.N * a.G + row, step = (int64_t)a.N * a.G;
    float M = -INFINITY, L = 0.f;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    constexpr int AT = 8; // splits whose loads are in flight together
    for (int s0 = 0; s0 < n; s0 += AT) {
        float2 h[AT];
        f32x4 y[AT];
#pragma unroll
        for (int x = 0; x < AT; ++x) {
            const int64_t at = at0 + (s0 + x < n ? s0 + x : n - 1) * step;
            h[x] = *reinterpret_cast<const float2 *>(a.ml + 2 * at);
            y[x] = *reinterpret_cast<const f32x4 *>(a.part + at * DP + (4 * lane < DP ? 4 * lane : 0));
        }
        float Mn = M;
#pragma unroll
        for (int x = 0; x < AT; ++x)
            Mn = fmaxf(Mn, h[x].x);
        const float mu = Mn == -INFINITY ? 0.f : Mn, f0 = __builtin_amdgcn_exp2f(M - mu);
        L *= f0;
        acc *= f0;
        M = Mn;
#pragma unroll
        for (int x = 0; x < AT; ++x) {
            if (s0 + x >= n)
                break;
            const float f = __builtin_amdgcn_exp2f(h[x].x - mu);
            L += f * h[x].y;
            acc += f * y[x];
        }
    }
    const int node = row / a.G, head = hk * a.G + row - node * a.G;
    const int64_t at = ((int64_t)b * a.N + node) * a.Hq + head;
    if (4 * lane < a.D) {
        T y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            y[i] = (T)(L == 0.f ? 0.f : acc[i] / L);
        *reinterpret_cast<uint64_t *>(static_cast<T *>(a.out) + at * a.D + 4 * lane) = __builtin_bit_cast(uint64_t, y);
    }
    if (a.lse && lane == 0)
        a.lse[at] = row_lse<Elem<DT>>(M, L);
}

template <int DT, int DP, bool TREE> hipError_t launch_dims(const Args &a, const AttnPlan &p, hipStream_t s)
{
    const dim3 grid((unsigned)p.grid);
    if constexpr (DP <= 128) {
        if (p.few) {
            const dim3 block(64 * kFewWaves);
            if constexpr (TREE) {
                const bool even = a.page.d % (kF8 && DP == 64 ? 16 : 8) == 0;
                if (p.few == 1 && even)
                    hipLaunchKernelGGL((attn_few<DT, DP, 1, 1>), grid, block, 0, s, a);
                else if (p.few == 1)
                    hipLaunchKernelGGL((attn_few<DT, DP, 1, 2>), grid, block, 0, s, a);
                else if (even)
                    hipLaunchKernelGGL((attn_few<DT, DP, 2, 1>), grid, block, 0, s, a);
                else
                    hipLaunchKernelGGL((attn_few<DT, DP, 2, 2>), grid, block, 0, s, a);
            } else if (p.few == 1) {
                hipLaunchKernelGGL((attn_few<DT, DP, 1, 0>), grid, block, 0, s, a);
            } else {
                hipLaunchKernelGGL((attn_few<DT, DP, 2, 0>), grid, block, 0, s, a);
            }
            return hipGetLastError();
        }
    }
    if (p.waves == 1)
        hipLaunchKernelGGL((attn_tiles<DT, DP, 1, TREE>), grid, dim3(64), 0, s, a);
    else if (p.waves == 2)
        hipLaunchKernelGGL((attn_tiles<DT, DP, 2, TREE>), grid, dim3(128), 0, s, a);
    else if (p.waves == 4 || DP > 128)
        hipLaunchKernelGGL((attn_tiles<DT, DP, 4, TREE>), grid, dim3(256), 0, s, a);
    else if constexpr (DP <= 128)
        hipLaunchKernelGGL((attn_tiles<DT, DP, 8, TREE>), grid, dim3(512), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.nsplit > 1) {
        const int64_t rows = (int64_t)a.B * a.N * a.Hq;
        hipLaunchKernelGGL((attn_join<DT, DP, TREE>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, s, a, p.bn);
        e = hipGetLastError();
    }
    return e;
}

template <int DT, bool TREE> hipError_t launch_type(const Args &a, const AttnPlan &p, hipStream_t s)
{
    if (p.dp == 64)
        return launch_dims<DT, 64, TREE>(a, p, s);
    if (p.dp == 128)
        return launch_dims<DT, 128, TREE>(a, p, s);
    return launch_dims<DT, 256, TREE>(a, p, s);
}

} // namespace

#ifdef RTOPK_ATTN_F8
hipError_t launch_attention_fp8(const Args &a, const AttnPlan &p, int dtype, hipStream_t s)
{
    return dtype == 1 ? launch_type<1, true>(a, p, s) : launch_type<2, true>(a, p, s);
}
#else
hipError_t launch_attention(const Args &a, const AttnPlan &p, int dtype, bool tree, hipStream_t s)
{
    if (dtype == 1)
        return tree ? launch_type<1, true>(a, p, s) : launch_type<1, false>(a, p, s);
    return tree ? launch_type<2, true>(a, p, s) : launch_type<2, false>(a, p, s);
}
#endif

} // namespace rtopk
