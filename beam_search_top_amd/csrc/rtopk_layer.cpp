// Host side of the paged-cache and attention entry points: argument checks,
// the split of an attention call over workgroups, launches. As elsewhere, a
// rejected call touches neither the GPU nor its outputs.
#include "rtopk.h"
#include "rtopk_attn.h"

#include <hip/hip_runtime_api.h>

#include <climits>
#include <cmath>
#include <exception>

using rtopk::set_error;

namespace {

// An exception must not leave a C entry point.
template <typename F> int guarded(const char *what, F f)
{
    try {
        return f();
    } catch (const std::exception &e) {
        return set_error(RTOPK_ENOMEM, "%s: %s", what, e.what());
    }
}

bool mul_fits(long long a, long long b, long long most) { return a == 0 || b <= most / a; }

// The largest element offset of a [n0][n1][n2][D] view stays far from 2^63.
bool strides_fit(const int64_t st[3], long long n0, long long n1, long long n2)
{
    const long long most = 1ll << 58;
    const long long n[3] = {n0, n1, n2};
    long long sum = 0;
    for (int i = 0; i < 3; ++i) {
        if (st[i] < 0 || !mul_fits(n[i], st[i], most))
            return false;
        sum += (n[i] - 1) * st[i];
    }
    return sum <= most;
}

// A [n0][n1][n2][D] view that is read 16 bytes at a time. The stride of a
// dimension of one entry says nothing and is dropped.
int check_view(const char *what, const char *name, const void *p, int64_t st[3], long long n0, long long n1, long long n2)
{
    const long long n[3] = {n0, n1, n2};
    for (int i = 0; i < 3; ++i)
        st[i] = n[i] == 1 ? 0 : st[i];
    if ((uintptr_t)p % 16)
        return set_error(RTOPK_EINVAL, "%s: %s is not 16-byte aligned", what, name);
    for (int i = 0; i < 3; ++i)
        if (st[i] % 8)
            return set_error(RTOPK_EINVAL, "%s: %s stride %lld is not a multiple of 8 elements", what, name,
                             (long long)st[i]);
    if (!strides_fit(st, n0, n1, n2))
        return set_error(RTOPK_EINVAL, "%s: %s strides are negative or overflow", what, name);
    return RTOPK_OK;
}

void set_strides(int64_t to[3], const int64_t *given, long long n1, long long n2, long long D)
{
    to[0] = given ? given[0] : n1 * n2 * D;
    to[1] = given ? given[1] : n2 * D;
    to[2] = given ? given[2] : D;
}

// What both attention entry points ask of their sizes.
int check_attention(const char *what, int dtype, int B, int N, int Hq, int Hkv, int D, float scale)
{
    if (dtype != RTOPK_F32 && dtype != RTOPK_F16 && dtype != RTOPK_BF16)
        return set_error(RTOPK_EINVAL, "%s: unknown dtype %d", what, dtype);
    if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || D < 1)
        return set_error(RTOPK_EINVAL, "%s: sizes must be >= 1 (B=%d N=%d Hq=%d Hkv=%d D=%d)", what, B, N, Hq, Hkv, D);
    if (Hq % Hkv)
        return set_error(RTOPK_EINVAL, "%s: Hq=%d is not a multiple of Hkv=%d", what, Hq, Hkv);
    if (!std::isfinite(scale) || std::fabs(scale) > 0x1p127f) // so that scale * log2(e) is finite too
        return set_error(RTOPK_EINVAL, "%s: scale must be finite, at most 2^127", what);
    if (dtype == RTOPK_F32)
        return set_error(RTOPK_ENOTSUP, "%s: float32 is not supported, only float16 and bfloat16", what);
    if (D % 8 || D > rtopk::kMaxHeadDim)
        return set_error(RTOPK_ENOTSUP, "%s: D=%d is not a multiple of 8 up to %d", what, D, rtopk::kMaxHeadDim);
    if (!mul_fits((long long)B * N, Hq, INT_MAX / D))
        return set_error(RTOPK_ENOTSUP, "%s: B*N*Hq*D exceeds 2^31-1", what);
    return RTOPK_OK;
}

// Workspace of a call whatever its strides.
size_t attention_bytes(int B, int N, int Hq, int Hkv, int D, int S)
{
    const size_t x = rtopk::plan_attention(B, N, Hq, Hkv, D, S, false).ws_bytes;
    const size_t y = rtopk::plan_attention(B, N, Hq, Hkv, D, S, true).ws_bytes;
    return x > y ? x : y;
}

int enqueue_attention(const char *what, rtopk::AttnArgs &a, int dtype, bool tree, void *workspace, size_t ws_bytes,
                      hipStream_t stream)
{
    // attn_few holds the offsets of 32 rows in 32 bits, and needs 32 rows to read
    const bool wide = a.ks[1] >= (1 << 25) || a.vs[1] >= (1 << 25) || (!tree && a.S < 32);
    const rtopk::AttnPlan p = rtopk::plan_attention(a.B, a.N, a.Hq, a.Hkv, a.D, a.S, wide);
    if (workspace && (uintptr_t)workspace % 256)
        return set_error(RTOPK_EINVAL, "%s: workspace is not 256-byte aligned", what);
    if (workspace && ws_bytes < p.ws_bytes)
        return set_error(RTOPK_ENOMEM, "%s: workspace of %zu bytes is smaller than the %zu needed", what, ws_bytes,
                         p.ws_bytes);
    if (p.grid > (int64_t)UINT32_MAX / (64 * p.waves)) // a launch counts its threads in 32 bits
        return set_error(RTOPK_ENOTSUP, "%s: %lld workgroups of %d threads exceed one launch", what, (long long)p.grid,
                         64 * p.waves);
    a.row_tiles = p.row_tiles;
    a.nsplit = p.nsplit;
    a.min_tiles = p.min_tiles;
    a.units = p.units;
    a.longest_first = p.longest_first && a.lens;
    const auto go = [&](void *ws) {
        a.ml = ws ? (float *)((uint8_t *)ws + p.ml_off) : nullptr;
        a.part = ws ? (float *)((uint8_t *)ws + p.part_off) : nullptr;
        a.ticket = ws ? (uint32_t *)((uint8_t *)ws + rtopk::kWsTicketOff) : nullptr;
        const hipError_t e = rtopk::launch_attention(a, p, dtype, tree, stream);
        if (e != hipSuccess)
            return set_error(RTOPK_EHIP, "%s launch: %s", what, hipGetErrorString(e));
        return (int)RTOPK_OK;
    };
    if (p.ws_bytes == rtopk::kWsFixedBytes || workspace)
        return go(workspace);
    return rtopk::with_workspace(p.ws_bytes, stream, go);
}

} // namespace

namespace rtopk {

AttnPlan plan_attention(int B, int N, int Hq, int Hkv, int D, int S, bool wide)
{
    AttnPlan p{};
    p.dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
    const int64_t R = (int64_t)N * (Hq / Hkv); // query rows that read the same keys
    const auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    p.nsplit = 1;
    p.ml_off = up(kWsFixedBytes);
    size_t rows = 0; // rows of partial outputs
    // Up to 32 rows the call is bound by reading, which attn_few is made for; with
    // more, attn_tiles shares each key among 32 rows of every wave (8 rows x 4 heads
    // over 4 x 30001 keys: attn_tiles 120 us, attn_few 90 us).
    p.few = p.dp <= 128 && R <= 32 && !wide ? (R <= 16 ? 1 : 2) : 0;
    if (p.few) {
        // The keys are cut when the batch elements' key heads alone do not fill the
        // GPU (2 workgroups per CU hold enough loads in flight at D = 128, 4 at D = 64:
        // with 3 and 8 the call above takes 107 and 110 us). 128 x 16 of them are not
        // cut: 34 us, cut in two or more 44 us, for the ends of every share cost more
        // than the balance gains.
        p.bn = 32;
        p.waves = 4;
        p.row_tiles = 1;
        p.min_tiles = 4;
        const int64_t places = p.dp == 64 ? 1024 : 512, tiles = ((int64_t)S + p.bn - 1) / p.bn;
        int64_t units = (places + Hkv - 1) / Hkv;
        units = units > 2 * (int64_t)B ? units : 2 * (int64_t)B;
        const bool cut = tiles > p.min_tiles && (int64_t)B * Hkv < places && B <= kMaxShareBatch &&
                         (int64_t)B * tiles <= (1 << 30);
        p.units = cut ? (int)units : 0;
        p.grid = ((cut ? units : B) + 7) / 8 * 8 * Hkv;
        rows = cut ? (size_t)units * Hkv * R : 0;
    } else {
        // 32 rows per wave; from 129 rows on a workgroup of eight waves, whose rings fill a CU's
        // LDS, else two workgroups of up to four per CU. Keys are cut, evenly per batch
        // element, until every place has a workgroup.
        p.waves = R <= 32 ? 1 : R <= 64 ? 2 : R <= 128 || p.dp > 128 ? 4 : 8;
        p.bn = p.dp > 128 ? 32 : 64;
        p.row_tiles = (int)((R + 32 * p.waves - 1) / (32 * p.waves));
        p.min_tiles = 4;
        const int64_t groups = (int64_t)B * Hkv * p.row_tiles, places = p.waves == 8 ? 256 : 512;
        const int64_t tiles = ((int64_t)S + p.bn - 1) / p.bn, most = (tiles + p.min_tiles - 1) / p.min_tiles;
        int64_t want = (places + groups - 1) / groups;
        want = want < most ? want : most;
        p.nsplit = (int)(want > 1 ? want : 1);
        p.grid = ((int64_t)B * Hkv * p.nsplit + 7) / 8 * 8 * p.row_tiles;
        rows = p.nsplit > 1 ? (size_t)B * Hkv * p.nsplit * R : 0;
        p.longest_first = B > 1 && B <= 64 && groups > places;
    }
    p.part_off = up(p.ml_off + 8 * rows);
    p.ws_bytes = rows ? up(p.part_off + 4 * rows * p.dp) : kWsFixedBytes;
    return p;
}

} // namespace rtopk

extern "C" {

int rtopk_page_tables(const int32_t *cache_lens, const int32_t *new_lens, int B, int page, const int32_t *free_pages,
                      int nfree, const int32_t *free_head, int num_pages, int32_t *table, int table_ld, int32_t *slots,
                      int32_t *positions, int T, int rows, int32_t *cu_new, int32_t *free_next, void *stream)
{
    const char *what = "page tables";
    if (!cache_lens || !new_lens || !table || !slots || !cu_new || (!free_pages && nfree > 0))
        return set_error(RTOPK_EINVAL, "%s: NULL pointer", what);
    if (B < 1 || page < 1 || num_pages < 1 || table_ld < 1 || T < 1 || nfree < 0 || rows < 0)
        return set_error(RTOPK_EINVAL, "%s: sizes must be >= 1 (B=%d page=%d num_pages=%d table_ld=%d T=%d nfree=%d rows=%d)",
                         what, B, page, num_pages, table_ld, T, nfree, rows);
    if (B > rtopk::kTicketCap)
        return set_error(RTOPK_ENOTSUP, "%s: B=%d exceeds the implementation limit %d", what, B, rtopk::kTicketCap);
    if (!mul_fits(num_pages, page, INT_MAX) || !mul_fits(table_ld, page, INT_MAX))
        return set_error(RTOPK_EINVAL, "%s: num_pages*page or table_ld*page exceeds 2^31-1", what);
    if (rows > 0 && (long long)B * rows != T)
        return set_error(RTOPK_EINVAL, "%s: T=%d is not B*rows=%lld", what, T, (long long)B * rows);
    if (free_head && free_head == free_next)
        return set_error(RTOPK_EINVAL, "%s: free_head and free_next must be different buffers", what);
    rtopk::TableArgs a{};
    a.lens = cache_lens;
    a.news = new_lens;
    a.B = B;
    a.ld = table_ld;
    a.rows = rows;
    a.num_pages = num_pages;
    a.page = rtopk::make_page_div((uint32_t)page);
    a.free = free_pages;
    a.nfree = nfree;
    a.head = free_head;
    a.table = table;
    a.slots = slots;
    a.positions = positions;
    a.cap = T;
    a.cu = cu_new;
    a.next = free_next;
    const hipError_t e = rtopk::launch_page_tables(a, (hipStream_t)stream);
    if (e != hipSuccess)
        return set_error(RTOPK_EHIP, "%s launch: %s", what, hipGetErrorString(e));
    return RTOPK_OK;
}

int rtopk_cache_store(const void *k, const int64_t *k_strides, const void *v, const int64_t *v_strides, int dtype,
                      const int32_t *slots, int T, int Hkv, int D, void *k_cache, void *v_cache,
                      const int64_t *cache_strides, int num_pages, int page, void *stream)
{
    const char *what = "cache store";
    if (!k || !v || !slots || !k_cache || !v_cache)
        return set_error(RTOPK_EINVAL, "%s: NULL pointer", what);
    if (dtype != RTOPK_F32 && dtype != RTOPK_F16 && dtype != RTOPK_BF16)
        return set_error(RTOPK_EINVAL, "%s: unknown dtype %d", what, dtype);
    if (T < 1 || Hkv < 1 || D < 1 || num_pages < 1 || page < 1)
        return set_error(RTOPK_EINVAL, "%s: sizes must be >= 1 (T=%d Hkv=%d D=%d num_pages=%d page=%d)", what, T, Hkv, D,
                         num_pages, page);
    if (!mul_fits(num_pages, page, INT_MAX))
        return set_error(RTOPK_EINVAL, "%s: num_pages*page exceeds 2^31-1", what);
    if (!mul_fits(Hkv, D, 1 << 20))
        return set_error(RTOPK_ENOTSUP, "%s: rows of more than 2^20 elements (Hkv=%d D=%d)", what, Hkv, D);
    const int esz = dtype == RTOPK_F32 ? 4 : 2;
    rtopk::StoreArgs a{};
    a.k = k;
    a.v = v;
    a.kc = k_cache;
    a.vc = v_cache;
    a.slots = slots;
    a.T = T;
    int64_t ks[2] = {k_strides ? k_strides[0] : (int64_t)Hkv * D, k_strides ? k_strides[1] : D};
    int64_t vs[2] = {v_strides ? v_strides[0] : (int64_t)Hkv * D, v_strides ? v_strides[1] : D};
    int64_t cs[3];
    set_strides(cs, cache_strides, page, Hkv, D);
    const int64_t k3[3] = {0, ks[0], ks[1]}, v3[3] = {0, vs[0], vs[1]};
    if (!strides_fit(k3, 1, T, Hkv) || !strides_fit(v3, 1, T, Hkv) || !strides_fit(cs, num_pages, page, Hkv))
        return set_error(RTOPK_EINVAL, "%s: strides are negative or overflow", what);
    for (const void *p : {k, v, (const void *)k_cache, (const void *)v_cache})
        if ((uintptr_t)p % esz)
            return set_error(RTOPK_EINVAL, "%s: a pointer is not aligned to its element size", what);
    // 16 bytes at a time where every row allows it, else one element
    bool wide = D * esz % 16 == 0;
    for (const void *p : {k, v, (const void *)k_cache, (const void *)v_cache})
        wide = wide && (uintptr_t)p % 16 == 0;
    for (int64_t st : {ks[0], ks[1], vs[0], vs[1], cs[0], cs[1], cs[2]})
        wide = wide && st * esz % 16 == 0;
    const int unit = wide ? 16 / esz : 1; // elements
    for (int i = 0; i < 2; ++i) {
        a.ks[i] = ks[i] / unit;
        a.vs[i] = vs[i] / unit;
    }
    for (int i = 0; i < 3; ++i)
        a.cs[i] = cs[i] / unit;
    a.row = rtopk::make_page_div((uint32_t)(Hkv * (D / unit)));
    a.head = rtopk::make_page_div((uint32_t)(D / unit));
    a.page = rtopk::make_page_div((uint32_t)page);
    a.nslots = num_pages * page;
    const hipError_t e = rtopk::launch_cache_store(a, wide ? 16 : esz, (hipStream_t)stream);
    if (e != hipSuccess)
        return set_error(RTOPK_EHIP, "%s launch: %s", what, hipGetErrorString(e));
    return RTOPK_OK;
}

int rtopk_tree_attention(const void *q, const int64_t *q_strides, const void *k_cache, const void *v_cache,
                         const int64_t *cache_strides, int dtype, const int32_t *table, int table_ld, int num_pages,
                         int page, const int32_t *cache_lens, const int32_t *parents, const int32_t *sizes, int B, int N,
                         int Hq, int Hkv, int D, float scale, void *out, float *lse, void *workspace, size_t ws_bytes,
                         void *stream)
{
    const char *what = "tree attention";
    if (!q || !k_cache || !v_cache || !table || !cache_lens || !out)
        return set_error(RTOPK_EINVAL, "%s: NULL pointer", what);
    int st = check_attention(what, dtype, B, N, Hq, Hkv, D, scale);
    if (st != RTOPK_OK)
        return st;
    if (table_ld < 1 || num_pages < 1 || page < 1)
        return set_error(RTOPK_EINVAL, "%s: sizes must be >= 1 (table_ld=%d num_pages=%d page=%d)", what, table_ld,
                         num_pages, page);
    if (!mul_fits(num_pages, page, INT_MAX) || !mul_fits(table_ld, page, INT_MAX - 4096))
        return set_error(RTOPK_EINVAL, "%s: num_pages*page or table_ld*page exceeds 2^31-4097", what);
    if (N > rtopk::kMaxTree)
        return set_error(RTOPK_ENOTSUP, "%s: N=%d exceeds the implementation limit %d", what, N, rtopk::kMaxTree);
    rtopk::AttnArgs a{};
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    set_strides(a.qs, q_strides, N, Hq, D);
    set_strides(a.ks, cache_strides, page, Hkv, D);
    set_strides(a.vs, cache_strides, page, Hkv, D);
    if ((st = check_view(what, "q", q, a.qs, B, N, Hq)) != RTOPK_OK ||
        (st = check_view(what, "k_cache", k_cache, a.ks, num_pages, page, Hkv)) != RTOPK_OK ||
        (st = check_view(what, "v_cache", v_cache, a.vs, num_pages, page, Hkv)) != RTOPK_OK)
        return st;
    if ((uintptr_t)out % 16)
        return set_error(RTOPK_EINVAL, "%s: out is not 16-byte aligned", what);
    a.B = B;
    a.N = N;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.D = D;
    a.S = table_ld * page;
    a.scale = scale;
    a.lens = cache_lens;
    a.table = table;
    a.ld = table_ld;
    a.num_pages = num_pages;
    a.page = rtopk::make_page_div((uint32_t)page);
    a.parents = parents;
    a.sizes = sizes;
    a.out = out;
    a.lse = lse;
    return guarded(what, [&] { return enqueue_attention(what, a, dtype, true, workspace, ws_bytes, (hipStream_t)stream); });
}

size_t rtopk_tree_attention_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int table_ld, int page)
{
    if (check_attention("tree attention", RTOPK_F16, B, N, Hq, Hkv, D, 1.f) != RTOPK_OK || N > rtopk::kMaxTree ||
        table_ld < 1 || page < 1 || !mul_fits(table_ld, page, INT_MAX - 4096))
        return 0;
    return attention_bytes(B, N, Hq, Hkv, D, table_ld * page);
}

size_t rtopk_cross_attention_workspace_bytes(int B, int N, int S, int Hq, int Hkv, int D)
{
    if (check_attention("cross attention", RTOPK_F16, B, N, Hq, Hkv, D, 1.f) != RTOPK_OK || S < 1 || S > INT_MAX - 4096)
        return 0;
    return attention_bytes(B, N, Hq, Hkv, D, S);
}

int rtopk_cross_attention(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides, const void *v,
                          const int64_t *v_strides, int dtype, const int32_t *lens, const uint8_t *key_mask, int B, int N,
                          int S, int Hq, int Hkv, int D, float scale, void *out, float *lse, void *workspace,
                          size_t ws_bytes, void *stream)
{
    const char *what = "cross attention";
    if (!q || !k || !v || !out)
        return set_error(RTOPK_EINVAL, "%s: NULL pointer", what);
    int st = check_attention(what, dtype, B, N, Hq, Hkv, D, scale);
    if (st != RTOPK_OK)
        return st;
    if (S < 1)
        return set_error(RTOPK_EINVAL, "%s: S=%d must be >= 1", what, S);
    if (S > INT_MAX - 4096)
        return set_error(RTOPK_ENOTSUP, "%s: S=%d exceeds 2^31-4097", what, S);
    rtopk::AttnArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    set_strides(a.qs, q_strides, N, Hq, D);
    set_strides(a.ks, k_strides, S, Hkv, D);
    set_strides(a.vs, v_strides, S, Hkv, D);
    if ((st = check_view(what, "q", q, a.qs, B, N, Hq)) != RTOPK_OK ||
        (st = check_view(what, "k", k, a.ks, B, S, Hkv)) != RTOPK_OK ||
        (st = check_view(what, "v", v, a.vs, B, S, Hkv)) != RTOPK_OK)
        return st;
    if ((uintptr_t)out % 16)
        return set_error(RTOPK_EINVAL, "%s: out is not 16-byte aligned", what);
    a.B = B;
    a.N = N;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = Hq / Hkv;
    a.D = D;
    a.S = S;
    a.scale = scale;
    a.lens = lens;
    a.key_mask = key_mask;
    a.page = rtopk::make_page_div(1);
    a.out = out;
    a.lse = lse;
    return guarded(what, [&] { return enqueue_attention(what, a, dtype, false, workspace, ws_bytes, (hipStream_t)stream); });
}

} // extern "C"
