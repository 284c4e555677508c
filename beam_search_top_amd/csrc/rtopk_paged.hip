// gfx950 kernels of the paged key/value cache: page tables and slot maps built
// from request lengths, and the store of new tokens' keys and values.
#include <hip/hip_runtime.h>

#include "rtopk_attn.h"

namespace rtopk {
namespace {

constexpr int kTabThreads = 256;
constexpr int kTabTile = 2048;     // slots a workgroup fills
constexpr int kTabReq = 8;         // requests a thread takes per scan step
constexpr int kTabStep = kTabThreads * kTabReq;

// Sum over the lower threads of the workgroup (exclusive) and the whole sum,
// of two 64-bit values at once. Two barriers; `sm` holds one pair per wave.
struct Pair {
    int64_t n, need;
};

__device__ __forceinline__ Pair wave_scan(Pair v, int lane)
{
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) {
        const int64_t a = __shfl_up(v.n, o), b = __shfl_up(v.need, o);
        if (lane >= o) {
            v.n += a;
            v.need += b;
        }
    }
    return v;
}

// Slots of a request with n new tokens: a row of the map holds no more than `rows`.
__device__ __forceinline__ int own_slots(const TableArgs &a, int n) { return a.rows && n > a.rows ? a.rows : n; }

// Workgroup w fills slots [w * kTabTile, ...) of the slot map, and the table
// entries of the pages that begin in them. Every workgroup sums the requests
// before its own by itself, kTabStep of them per step: the lengths are a few
// KB that every L2 holds, and a launch more to share the sums would cost more
// than reading them again. The last workgroup, which passes over all
// requests anyway, writes the offsets and the new head of the free list.
//
// Every new page holds exactly one token at offset 0 of the page among the
// new tokens, so the thread that maps that token writes the table entry, and
// entries of pages that a request already has are only read.
__global__ __launch_bounds__(kTabThreads) void page_tables(const TableArgs a)
{
    // the requests that own this workgroup's slots, in order
    __shared__ int32_t s_start[kTabTile + 1], s_req[kTabTile], s_len[kTabTile], s_have[kTabTile];
    __shared__ int32_t s_taken[kTabTile]; // place of the first new page, -1: refused
    __shared__ Pair s_wave[kTabThreads / kLanes];
    __shared__ int s_cnt[kTabThreads / kLanes];
    const int tid = threadIdx.x, lane = tid & (kLanes - 1), wave = tid / kLanes;
    const int64_t i0 = (int64_t)blockIdx.x * kTabTile;
    const int64_t i1 = i0 + kTabTile < a.cap ? i0 + kTabTile : a.cap;
    const bool last = blockIdx.x == gridDim.x - 1;
    int64_t head = a.head ? a.head[0] : 0;
    head = head < 0 ? 0 : head;
    int64_t base_n = 0, base_need = 0, granted = 0;
    int found = 0;
    for (int b0 = 0; b0 < a.B; b0 += kTabStep) {
        // a thread takes kTabReq consecutive requests
        PageNeed r[kTabReq];
        Pair sum{0, 0};
#pragma unroll
        for (int q = 0; q < kTabReq; ++q) {
            const int b = b0 + tid * kTabReq + q;
            r[q] = b < a.B ? page_need(a.page, a.lens[b], a.news[b], a.ld, a.rows) : PageNeed{0, 0, 0, 0, false};
            sum.n += r[q].n;
            sum.need += r[q].need;
        }
        Pair inc = wave_scan(sum, lane);
        if (lane == kLanes - 1)
            s_wave[wave] = inc;
        __syncthreads();
        Pair ex{base_n + inc.n - sum.n, base_need + inc.need - sum.need};
        Pair all{0, 0};
#pragma unroll
        for (int w = 0; w < kTabThreads / kLanes; ++w) {
            if (w < wave) {
                ex.n += s_wave[w].n;
                ex.need += s_wave[w].need;
            }
            all.n += s_wave[w].n;
            all.need += s_wave[w].need;
        }
        // which of them own slots here
        int mine = 0;
        int64_t first = ex.n;
#pragma unroll
        for (int q = 0; q < kTabReq; ++q) {
            const int64_t at = a.rows ? (int64_t)(b0 + tid * kTabReq + q) * a.rows : first;
            mine += r[q].n > 0 && at < i1 && at + own_slots(a, r[q].n) > i0;
            first += r[q].n;
        }
        int pre = mine;
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) {
            const int v = __shfl_up(pre, o);
            pre += lane >= o ? v : 0;
        }
        if (lane == kLanes - 1)
            s_cnt[wave] = pre;
        __syncthreads();
        int at_req = found + pre - mine;
#pragma unroll
        for (int w = 0; w < kTabThreads / kLanes; ++w) {
            at_req += w < wave ? s_cnt[w] : 0;
            found += s_cnt[w];
        }
#pragma unroll
        for (int q = 0; q < kTabReq; ++q) {
            const int b = b0 + tid * kTabReq + q;
            if (b >= a.B)
                break;
            const int64_t taken = head + ex.need;
            const bool ok = page_granted(r[q], taken, ex.n, a.nfree, a.cap, a.rows);
            const int64_t at = a.rows ? (int64_t)b * a.rows : ex.n;
            if (r[q].n > 0 && at < i1 && at + own_slots(a, r[q].n) > i0) {
                s_start[at_req] = (int32_t)(at - i0); // may be negative: it began before this tile
                s_req[at_req] = b;
                s_len[at_req] = r[q].c;
                s_have[at_req] = r[q].have;
                s_taken[at_req] = ok ? (int32_t)(taken < a.nfree ? taken : a.nfree) : -1;
                ++at_req;
            }
            if (last) {
                a.cu[b] = (int32_t)(ex.n < INT32_MAX ? ex.n : INT32_MAX);
                granted += ok ? r[q].need : 0;
            }
            ex.n += r[q].n;
            ex.need += r[q].need;
        }
        base_n += all.n;
        base_need += all.need;
        if (!last && !a.rows && base_n >= i1)
            break;
        if (!last && a.rows && (int64_t)(b0 + kTabStep) * a.rows >= i1)
            break;
    }
    if (last) {
        const Pair g = wave_scan(Pair{granted, 0}, lane);
        __syncthreads();
        if (lane == kLanes - 1)
            s_wave[wave] = g;
        __syncthreads();
        if (tid == 0) {
            int64_t t = 0;
#pragma unroll
            for (int w = 0; w < kTabThreads / kLanes; ++w)
                t += s_wave[w].n;
            a.cu[a.B] = (int32_t)(base_n < INT32_MAX ? base_n : INT32_MAX);
            if (a.next)
                a.next[0] = (int32_t)(head + t < INT32_MAX ? head + t : INT32_MAX);
        }
    }
    __syncthreads(); // the owners are in LDS
    for (int q0 = tid; q0 < kTabTile; q0 += kTabThreads) {
        const int64_t i = i0 + q0;
        if (i >= i1)
            break;
        // the last owner that starts at or before this slot
        int lo = 0, hi = found;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (s_start[mid] <= q0)
                lo = mid + 1;
            else
                hi = mid;
        }
        int32_t slot = -1, pos = -1;
        if (lo > 0) {
            const int e = lo - 1;
            const int b = s_req[e], t = q0 - s_start[e];
            if (s_taken[e] >= 0 && t < (a.news[b] > 0 ? a.news[b] : 0)) {
                pos = s_len[e] + t; // below ld * page < 2^31
                const int pg = (int)page_of(a.page, (uint32_t)pos), off = pos - pg * (int)a.page.d;
                int32_t id;
                int32_t *row = a.table + (int64_t)b * a.ld;
                if (pg < s_have[e]) {
                    id = row[pg];
                } else {
                    id = a.free[s_taken[e] + (pg - s_have[e])];
                    if (off == 0)
                        row[pg] = id;
                }
                slot = slot_of(id, a.num_pages, (int)a.page.d, off);
            }
        }
        a.slots[i] = slot;
        if (a.positions)
            a.positions[i] = pos;
    }
}

// ---------------------------------------------------------------- store
constexpr int kStoreThreads = 256;
constexpr int kStoreVecs = 4; // units per lane and tensor

// Workgroup w copies tokens [w * tpw, ...): every lane takes one unit (16
// bytes, or one element where alignment does not allow that) of a key row and
// the same unit of a value row at a time, kStoreVecs of them in flight. A pure
// copy: bound by HBM, so no LDS.
template <typename U> __global__ __launch_bounds__(kStoreThreads) void cache_store(const StoreArgs a)
{
    const int64_t t0 = (int64_t)blockIdx.x * a.tpw;
    const int nt = (int)(t0 + a.tpw < a.T ? a.tpw : a.T - t0);
    const uint32_t units = (uint32_t)nt * a.row.d;
    for (uint32_t u0 = threadIdx.x; u0 < units; u0 += kStoreThreads * kStoreVecs) {
        U kv[kStoreVecs] = {}, vv[kStoreVecs] = {};
        int64_t to[kStoreVecs];
#pragma unroll
        for (int q = 0; q < kStoreVecs; ++q) {
            const uint32_t u = u0 + q * kStoreThreads;
            to[q] = -1;
            if (u >= units)
                continue;
            const uint32_t t = page_of(a.row, u), w = u - t * a.row.d; // token of the workgroup, unit of its row
            const uint32_t h = page_of(a.head, w), x = w - h * a.head.d;
            const int32_t slot = a.slots[t0 + t];
            if (slot < 0 || slot >= a.nslots)
                continue;
            const int64_t pg = page_of(a.page, (uint32_t)slot), off = slot - pg * a.page.d;
            to[q] = pg * a.cs[0] + off * a.cs[1] + h * a.cs[2] + x;
            kv[q] = static_cast<const U *>(a.k)[(t0 + t) * a.ks[0] + h * a.ks[1] + x];
            vv[q] = static_cast<const U *>(a.v)[(t0 + t) * a.vs[0] + h * a.vs[1] + x];
        }
#pragma unroll
        for (int q = 0; q < kStoreVecs; ++q) {
            if (to[q] < 0)
                continue;
            static_cast<U *>(a.kc)[to[q]] = kv[q];
            static_cast<U *>(a.vc)[to[q]] = vv[q];
        }
    }
}

} // namespace

hipError_t launch_page_tables(const TableArgs &a, hipStream_t s)
{
    const int64_t blocks = a.cap > 0 ? (a.cap + kTabTile - 1) / kTabTile : 1;
    hipLaunchKernelGGL(page_tables, dim3((unsigned)blocks), dim3(kTabThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_cache_store(StoreArgs a, int unit_bytes, hipStream_t s)
{
    // tokens per workgroup: one round of its lanes, and at least one token
    const int per = kStoreThreads * kStoreVecs;
    a.tpw = (int)a.row.d >= per ? 1 : per / (int)a.row.d;
    const int64_t blocks = (a.T + a.tpw - 1) / a.tpw;
    if (unit_bytes == 16)
        hipLaunchKernelGGL(cache_store<uint4>, dim3((unsigned)blocks), dim3(kStoreThreads), 0, s, a);
    else if (unit_bytes == 4)
        hipLaunchKernelGGL(cache_store<uint32_t>, dim3((unsigned)blocks), dim3(kStoreThreads), 0, s, a);
    else
        hipLaunchKernelGGL(cache_store<uint16_t>, dim3((unsigned)blocks), dim3(kStoreThreads), 0, s, a);
    return hipGetLastError();
}

int64_t page_tables_blocks(int64_t cap) { return cap > 0 ? (cap + kTabTile - 1) / kTabTile : 1; }

} // namespace rtopk
