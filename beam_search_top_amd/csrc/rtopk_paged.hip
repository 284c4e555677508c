// gfx950 kernels of the paged key/value cache: page tables and slot maps built
// from request lengths, and the store of new tokens' keys and values.
#include <hip/hip_runtime.h>

#include "rtopk_attn.h"

namespace rtopk {
namespace {

constexpr int kTabThreads = 256;
constexpr int kTabWaves = kTabThreads / kLanes;

__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// Inclusive scan over a wave by saturating addition (sums past 2^32 - 1 stay
// there, so huge lengths cannot wrap around into small ones): four DPP
// shifts within the 16-lane rows, then each row's last value to the rows
// behind it.
__device__ __forceinline__ uint32_t scan_sat(uint32_t x)
{
    x = add_sat(x, __builtin_amdgcn_update_dpp(0u, x, 0x111, 0xf, 0xf, false)); // row_shr:1
    x = add_sat(x, __builtin_amdgcn_update_dpp(0u, x, 0x112, 0xf, 0xf, false)); // row_shr:2
    x = add_sat(x, __builtin_amdgcn_update_dpp(0u, x, 0x114, 0xf, 0xf, false)); // row_shr:4
    x = add_sat(x, __builtin_amdgcn_update_dpp(0u, x, 0x118, 0xf, 0xf, false)); // row_shr:8
    x = add_sat(x, __builtin_amdgcn_update_dpp(0u, x, 0x142, 0xa, 0xf, false)); // row_bcast:15
    x = add_sat(x, __builtin_amdgcn_update_dpp(0u, x, 0x143, 0xc, 0xf, false)); // row_bcast:31
    return x;
}
// The same, without the lane's own value.
__device__ __forceinline__ uint32_t before_me(uint32_t incl, int lane)
{
    const uint32_t x = __shfl_up(incl, 1);
    return lane ? x : 0u;
}

// Slots of a request with n new tokens: a row of the map holds no more than `rows`.
__device__ __forceinline__ int own_slots(const TableArgs &a, int n) { return a.rows && n > a.rows ? a.rows : n; }

// Workgroup w fills slots [w * TILE, ...) of the slot map, SPT per lane, and
// the table entries of the pages that begin in them. Every workgroup sums the
// requests before its own by itself, REQ of them per lane and step: the
// lengths are a few KB that every L2 holds, and a launch more to share the
// sums would cost more than reading them again. The last workgroup, which
// passes over all requests anyway, writes the offsets and the new head of the
// free list. Latency decides here (a chain of dependent loads, scans and
// searches), so every stage runs for all of a lane's slots before the next.
//
// Every new page holds exactly one token at offset 0 of the page among the
// new tokens, so the lane that maps that token writes the table entry, and
// entries of pages that a request already has are only read.
template <int REQ, int SPT> __global__ __launch_bounds__(kTabThreads) void page_tables(const TableArgs a)
{
    constexpr int TILE = kTabThreads * SPT, STEP = kTabThreads * REQ;
    // the requests that own this workgroup's slots, in order: first slot (relative, may
    // be negative), row, tokens held and new, pages held, place of the first new page (-1: refused)
    __shared__ int32_t s_start[TILE], s_req[TILE], s_len[TILE], s_new[TILE], s_have[TILE], s_taken[TILE];
    __shared__ uint32_t s_n[kTabWaves], s_need[kTabWaves], s_cnt[kTabWaves];
    const int tid = threadIdx.x, lane = tid & (kLanes - 1), wave = tid / kLanes;
    const int64_t i0 = (int64_t)blockIdx.x * TILE;
    const int64_t i1 = i0 + TILE < a.cap ? i0 + TILE : a.cap;
    const bool last = blockIdx.x == gridDim.x - 1;
    int64_t head = a.head ? a.head[0] : 0;
    head = head < 0 ? 0 : head;
    uint32_t base_n = 0, base_need = 0, granted = 0;
    int found = 0;
    for (int b0 = 0; b0 < a.B; b0 += STEP) {
        PageNeed r[REQ]; // consecutive requests
        uint32_t sum_n = 0, sum_need = 0;
#pragma unroll
        for (int q = 0; q < REQ; ++q) {
            const int b = b0 + tid * REQ + q;
            r[q] = b < a.B ? page_need(a.page, a.lens[b], a.news[b], a.ld, a.rows) : PageNeed{0, 0, 0, 0, false};
            sum_n = add_sat(sum_n, r[q].n);
            sum_need = add_sat(sum_need, r[q].need);
        }
        const uint32_t in = scan_sat(sum_n), ip = scan_sat(sum_need);
        if (lane == kLanes - 1) {
            s_n[wave] = in;
            s_need[wave] = ip;
        }
        __syncthreads();
        uint32_t ex_n = base_n, ex_need = base_need;
#pragma unroll
        for (int w = 0; w < kTabWaves; ++w) {
            if (w < wave) {
                ex_n = add_sat(ex_n, s_n[w]);
                ex_need = add_sat(ex_need, s_need[w]);
            }
            base_n = add_sat(base_n, s_n[w]);
            base_need = add_sat(base_need, s_need[w]);
        }
        ex_n = add_sat(ex_n, before_me(in, lane));
        ex_need = add_sat(ex_need, before_me(ip, lane));
        // which of them own slots here
        auto owns = [&](int b, const PageNeed &p, int64_t first) {
            const int64_t at = a.rows ? (int64_t)b * a.rows : first;
            return p.n > 0 && at < i1 && at + own_slots(a, p.n) > i0;
        };
        uint32_t mine = 0, first = ex_n;
#pragma unroll
        for (int q = 0; q < REQ; ++q) {
            mine += owns(b0 + tid * REQ + q, r[q], first);
            first = add_sat(first, r[q].n);
        }
        const uint32_t ic = scan_sat(mine);
        if (lane == kLanes - 1)
            s_cnt[wave] = ic;
        __syncthreads();
        int at_req = found + (int)before_me(ic, lane);
#pragma unroll
        for (int w = 0; w < kTabWaves; ++w) {
            at_req += w < wave ? (int)s_cnt[w] : 0;
            found += (int)s_cnt[w];
        }
#pragma unroll
        for (int q = 0; q < REQ; ++q) {
            const int b = b0 + tid * REQ + q;
            if (b < a.B) {
                const int64_t taken = head + ex_need;
                const bool ok = page_granted(r[q], taken, ex_n, a.nfree, a.cap, a.rows);
                if (owns(b, r[q], ex_n)) {
                    s_start[at_req] = (int32_t)((a.rows ? (int64_t)b * a.rows : (int64_t)ex_n) - i0);
                    s_req[at_req] = b;
                    s_len[at_req] = r[q].c;
                    s_new[at_req] = r[q].n;
                    s_have[at_req] = r[q].have;
                    s_taken[at_req] = ok ? (int32_t)(taken < a.nfree ? taken : a.nfree) : -1;
                    ++at_req;
                }
                if (last) {
                    a.cu[b] = (int32_t)(ex_n < INT32_MAX ? ex_n : INT32_MAX);
                    granted = add_sat(granted, ok ? r[q].need : 0);
                }
                ex_n = add_sat(ex_n, r[q].n);
                ex_need = add_sat(ex_need, r[q].need);
            }
        }
        if (!last && (a.rows ? (int64_t)(b0 + STEP) * a.rows >= i1 : (int64_t)base_n >= i1))
            break;
    }
    if (last) {
        const uint32_t g = scan_sat(granted);
        __syncthreads(); // the sums of the last step have been read
        if (lane == kLanes - 1)
            s_n[wave] = g;
        __syncthreads();
        if (tid == 0) {
            uint32_t t = 0;
#pragma unroll
            for (int w = 0; w < kTabWaves; ++w)
                t = add_sat(t, s_n[w]);
            a.cu[a.B] = (int32_t)(base_n < INT32_MAX ? base_n : INT32_MAX);
            if (a.next)
                a.next[0] = (int32_t)(head + t < INT32_MAX ? head + t : INT32_MAX);
        }
    }
    __syncthreads(); // the owners are in LDS
    // each slot's owner: the last that starts at or before it
    int lo[SPT], hi[SPT];
#pragma unroll
    for (int q = 0; q < SPT; ++q) {
        lo[q] = 0;
        hi[q] = found;
    }
    for (int n = found; n > 0; n >>= 1) { // found + 1 answers, halved every time
#pragma unroll
        for (int q = 0; q < SPT; ++q) {
            if (lo[q] < hi[q]) {
                const int mid = (lo[q] + hi[q]) >> 1;
                const bool at = s_start[mid] <= tid + q * kTabThreads;
                lo[q] = at ? mid + 1 : lo[q];
                hi[q] = at ? hi[q] : mid;
            }
        }
    }
    int32_t pos[SPT], off[SPT], id[SPT];
    int32_t *to[SPT]; // the table entry to write
#pragma unroll
    for (int q = 0; q < SPT; ++q) {
        pos[q] = off[q] = id[q] = -1;
        to[q] = nullptr;
        if (lo[q] > 0) {
            const int e = lo[q] - 1, t = tid + q * kTabThreads - s_start[e];
            if (s_taken[e] >= 0 && t < s_new[e]) {
                pos[q] = s_len[e] + t; // below ld * page < 2^31
                const int pg = (int)page_of(a.page, (uint32_t)pos[q]), have = s_have[e];
                off[q] = pos[q] - pg * (int)a.page.d;
                int32_t *entry = a.table + (int64_t)s_req[e] * a.ld + pg;
                const int32_t *from = pg < have ? entry : a.free + (s_taken[e] + (pg - have));
                id[q] = *from;
                to[q] = pg >= have && off[q] == 0 ? entry : nullptr;
            }
        }
    }
#pragma unroll
    for (int q = 0; q < SPT; ++q) {
        const int64_t i = i0 + tid + q * kTabThreads;
        if (i >= i1)
            continue;
        if (to[q])
            *to[q] = id[q];
        a.slots[i] = pos[q] < 0 ? -1 : slot_of(id[q], a.num_pages, (int)a.page.d, off[q]);
        if (a.positions)
            a.positions[i] = pos[q];
    }
}

// ---------------------------------------------------------------- store
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
constexpr int kStoreThreads = 256;
constexpr int kStoreVecs = 4; // units per lane and tensor

// Workgroup w copies tokens [w * tpw, ...): every lane takes one unit (16
// bytes, or one element where alignment does not allow that) of a key row and
// the same unit of a value row at a time, kStoreVecs of them in flight. A pure
// copy: bound by HBM, so no LDS. 129001 tokens of 8 heads of 128, bf16 (1.06 GB
// read and written): 212 us, 5.0 TB/s, the rate of a large device copy.
template <typename U> __global__ __launch_bounds__(kStoreThreads) void cache_store(const StoreArgs a)
{
    const int64_t t0 = (int64_t)blockIdx.x * a.tpw;
    const int nt = (int)(t0 + a.tpw < a.T ? a.tpw : a.T - t0);
    const uint32_t units = (uint32_t)nt * a.row.d;
    const U *k = static_cast<const U *>(a.k), *v = static_cast<const U *>(a.v);
    U *kc = static_cast<U *>(a.kc), *vc = static_cast<U *>(a.vc);
    for (uint32_t u0 = threadIdx.x; u0 < units; u0 += kStoreThreads * kStoreVecs) {
        U kv[kStoreVecs], vv[kStoreVecs];
        int64_t to[kStoreVecs];
#pragma unroll
        for (int q = 0; q < kStoreVecs; ++q) {
            // past the last unit: the last one again, not stored
            const uint32_t u = u0 + q * kStoreThreads < units ? u0 + q * kStoreThreads : units - 1;
            const uint32_t t = page_of(a.row, u), w = u - t * a.row.d; // token of the workgroup, unit of its row
            const uint32_t h = page_of(a.head, w), x = w - h * a.head.d;
            const int32_t slot = a.slots[t0 + t];
            const uint32_t s = (uint32_t)slot < (uint32_t)a.nslots ? (uint32_t)slot : 0u;
            const uint32_t pg = page_of(a.page, s), off = s - pg * a.page.d;
            const int64_t at = (int64_t)pg * a.cs[0] + (int64_t)off * a.cs[1] + (int64_t)h * a.cs[2] + x;
            to[q] = (uint32_t)slot < (uint32_t)a.nslots && u0 + q * kStoreThreads < units ? at : -1;
            kv[q] = __builtin_nontemporal_load(k + (t0 + t) * a.ks[0] + h * a.ks[1] + x);
            vv[q] = __builtin_nontemporal_load(v + (t0 + t) * a.vs[0] + h * a.vs[1] + x);
        }
#pragma unroll
        for (int q = 0; q < kStoreVecs; ++q) {
            if (to[q] >= 0) {
                kc[to[q]] = kv[q];
                vc[to[q]] = vv[q];
            }
        }
    }
}

template <int REQ> hipError_t launch_tables(const TableArgs &a, int spt, hipStream_t s)
{
    const dim3 grid((unsigned)((a.cap + kTabThreads * spt - 1) / (kTabThreads * spt))), block(kTabThreads);
    if (spt == 1)
        hipLaunchKernelGGL((page_tables<REQ, 1>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((page_tables<REQ, 4>), grid, block, 0, s, a);
    return hipGetLastError();
}

} // namespace

// Small tiles while they leave the grid within one workgroup per CU, else four
// slots per lane; one request per lane and step up to 1024 requests (600
// requests, 1.2 M slots: 9.2 us; with 8 slots 9.9, 2 slots 10.6, 8 requests 13.9).
hipError_t launch_page_tables(const TableArgs &a, hipStream_t s)
{
    const int spt = a.cap <= 256 * kTabThreads ? 1 : 4;
    return a.B <= 1024 ? launch_tables<1>(a, spt, s) : launch_tables<8>(a, spt, s);
}

hipError_t launch_cache_store(StoreArgs a, int unit_bytes, hipStream_t s)
{
    static_assert(kStoreThreads == 256, "store_tokens");
    a.tpw = (int)store_tokens(a.T, a.row.d, kStoreThreads * kStoreVecs);
    const int64_t blocks = (a.T + a.tpw - 1) / a.tpw;
    if (unit_bytes == 16)
        hipLaunchKernelGGL(cache_store<u32x4>, dim3((unsigned)blocks), dim3(kStoreThreads), 0, s, a);
    else if (unit_bytes == 4)
        hipLaunchKernelGGL(cache_store<uint32_t>, dim3((unsigned)blocks), dim3(kStoreThreads), 0, s, a);
    else
        hipLaunchKernelGGL(cache_store<uint16_t>, dim3((unsigned)blocks), dim3(kStoreThreads), 0, s, a);
    return hipGetLastError();
}

} // namespace rtopk
