// Arithmetic of the paged key/value cache, shared by the kernels and the host
// (it compiles with a plain C++ compiler, so tests run it on the CPU).
//
// A cache is num_pages pages of `page` tokens; slot s is token s mod page of
// page s / page. Request b's tokens lie in the pages of its table row: token
// at position p is token p mod page of page table[b][p / page].
#pragma once

#include <stddef.h>
#include <stdint.h>

#if defined(__HIP__)
#define RTOPK_HD __host__ __device__ __forceinline__
#else
#define RTOPK_HD inline
#endif

namespace rtopk {

// floor(n / d) for n < 2^31 by a multiplication and a shift (the constants of
// make_magic in rtopk_internal.h).
struct PageDiv {
    uint32_t mul, shr, d;
};

inline PageDiv make_page_div(uint32_t d)
{
    uint32_t l = 0;
    while ((1ull << l) < d)
        ++l;
    const uint32_t shr = 31 + l;
    return PageDiv{(uint32_t)((1ull << shr) / d + 1), shr, d};
}

RTOPK_HD uint32_t page_of(PageDiv p, uint32_t pos) { return (uint32_t)(((uint64_t)pos * p.mul) >> p.shr); }

// A page id as read from a table: -1 unless it names a page of the cache.
RTOPK_HD int32_t checked_page(int32_t id, int num_pages) { return (uint32_t)id < (uint32_t)num_pages ? id : -1; }

// What one request asks of the free list.
struct PageNeed {
    int32_t c, n;       // tokens it holds, tokens it takes (negative counts as 0)
    int32_t have, need; // pages it has, pages it takes
    bool fits;          // whether its table row and its row of slots hold it
};

// rows: slots of its row (0: the slots are packed, and `cap` bounds them elsewhere)
RTOPK_HD PageNeed page_need(PageDiv p, int32_t len, int32_t add, int ld, int rows)
{
    PageNeed r;
    r.c = len > 0 ? len : 0;
    r.n = add > 0 ? add : 0;
    const int64_t total = (int64_t)r.c + r.n;
    r.fits = total <= (int64_t)ld * (int64_t)p.d && (rows == 0 || r.n <= rows);
    r.have = 0;
    r.need = 0;
    if (r.fits) { // total <= ld * page < 2^31
        r.have = r.c ? (int32_t)page_of(p, (uint32_t)r.c - 1) + 1 : 0;
        r.need = (total ? (int32_t)page_of(p, (uint32_t)total - 1) + 1 : 0) - r.have;
    }
    return r;
}

// Whether a request that fits gets what it asks: `taken` is the place of its
// first page in the free list, `first` that of its first token among packed slots.
RTOPK_HD bool page_granted(const PageNeed &r, int64_t taken, int64_t first, int64_t nfree, int64_t cap, int rows)
{
    return r.fits && (r.need == 0 || taken + r.need <= nfree) && (rows != 0 || first + r.n <= cap);
}

// The slot of token `off` of page `id`, or -1.
RTOPK_HD int32_t slot_of(int32_t id, int num_pages, int page, int off)
{
    return checked_page(id, num_pages) < 0 ? -1 : id * page + off; // num_pages * page < 2^31
}

// Tokens per workgroup of the store: as many rows of `row` units as one round of its
// lanes moves (`round` units), at least one, and more where T tokens would take 2^24
// workgroups of 256 threads: a launch counts its threads in 32 bits.
inline int64_t store_tokens(int64_t T, int64_t row, int64_t round)
{
    const int64_t most = (1 << 24) - 1, least = (T + most - 1) / most, per = row >= round ? 1 : round / row;
    return per > least ? per : least;
}

// Node i's parent: a value outside [0, i) is no parent.
RTOPK_HD int parent_of(int32_t p, int i) { return p >= 0 && p < i ? p : -1; }

} // namespace rtopk
