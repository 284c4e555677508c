// Internal interface between the host side (rtopk_layer.cpp) of the paged
// cache and attention entry points and their kernels. Not part of the ABI.
#pragma once

#include "rtopk_internal.h"
#include "rtopk_pages.h"

#include <functional>

namespace rtopk {

// Page tables and slot maps (rtopk_paged.hip).
struct TableArgs {
    const int32_t *lens, *news; // [B] tokens held, tokens to add
    int B, ld, rows, num_pages;
    PageDiv page;
    const int32_t *free;        // [nfree] page ids
    int64_t nfree;
    const int32_t *head;        // place of the first unused id, or null (0)
    int32_t *table;             // [B][ld]
    int32_t *slots, *positions; // [cap]
    int64_t cap;                // slots: T, or B * rows
    int32_t *cu;                // [B + 1]
    int32_t *next;              // [1] or null
};
hipError_t launch_page_tables(const TableArgs &a, hipStream_t s);

// Store of new keys and values; strides and counts in units of a load.
struct StoreArgs {
    const void *k, *v;
    void *kc, *vc;
    const int32_t *slots;
    int64_t T;
    int64_t ks[2], vs[2]; // token, head
    int64_t cs[3];        // page, token, head
    PageDiv row, head, page; // units per row, units per head, tokens per page
    int32_t nslots;
    int tpw;
};
hipError_t launch_cache_store(StoreArgs a, int unit_bytes, hipStream_t s);

constexpr int kMaxTree = 256;   // nodes of a tree
constexpr int kMaxHeadDim = 256;
constexpr int kMaxParts = 64;   // shares of a batch element in attn_few
constexpr int kMaxShareBatch = 256; // batch elements whose lengths a wave of attn_few sums

// Attention of N query rows per batch element over its keys (rtopk_attn.hip).
struct AttnArgs {
    const void *q, *k, *v;
    int64_t qs[3];             // batch, row, head strides in elements
    int64_t ks[3], vs[3];      // cross: batch, token, head; tree: page, token, head (ks == vs)
    int B, N, Hq, Hkv, G, D;   // G = Hq / Hkv
    int S;                     // cross: keys per batch element at most; tree: ld * page
    float scale;
    const int32_t *lens;       // [B]: cross: keys (null: S); tree: tokens before the tree
    const uint8_t *key_mask;   // cross: [B][S], nonzero = left out, or null
    const int32_t *table;      // tree: [B][ld]
    int ld, num_pages;
    PageDiv page;
    const int32_t *parents;    // tree: [B][N] or null (a chain)
    const int32_t *sizes;      // tree: [B] nodes, or null (N)
    void *out;                 // [B][N][Hq][D]
    float *lse;                // [B][N][Hq] or null
    // the split over workgroups (plan_attention)
    int row_tiles, nsplit, min_tiles;
    int longest_first;         // attn_tiles: batch elements in the order of their lengths (B <= 64)
    int units;                 // attn_few: shares of all batch elements at most, 0 = one each
    float *part;               // [B][Hkv][nsplit][N * G][dp] (attn_few: [units][Hkv][N * G][dp]) unnormalised outputs
    float *ml;                 // the same with [2] for [dp]: their maxima (base 2) and sums
    uint32_t *ticket;          // [B * Hkv] arrivals of attn_few's shares, zero between calls
};

// How a call is cut: workgroups of `waves` x 32 rows (few: of 16 or 32 rows,
// by attn_few), tiles of `bn` keys, heads padded to `dp` elements, keys in at
// most `nsplit` parts of at least min_tiles tiles (attn_few: in `units` shares).
struct AttnPlan {
    int few, dp, bn, waves, row_tiles, nsplit, min_tiles, units, longest_first;
    int64_t grid;
    size_t ml_off, part_off, ws_bytes; // workspace behind the fixed region
};
// wide: rows of keys or values lie 2^25 elements or more apart (not for attn_few)
AttnPlan plan_attention(int B, int N, int Hq, int Hkv, int D, int S, bool wide);
hipError_t launch_attention(const AttnArgs &a, const AttnPlan &p, int dtype, bool tree, hipStream_t s);

// Calls `launch` with a library-owned workspace of `need` bytes for `stream`
// (rtopk_host.cpp), held until it returns; a status code.
int with_workspace(size_t need, hipStream_t stream, const std::function<int(void *)> &launch);

} // namespace rtopk
