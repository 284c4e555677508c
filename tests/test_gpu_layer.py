"""Paged cache and attention operators on the GPU against plain 64-bit
references (layer_ref.py, which derives the tolerances)."""
import math

import numpy as np
import pytest
import torch

from beam_search_top_amd import rtopk
from layer_ref import check_cross, check_tree, tables
from libutil import ensure_built

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_built()


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rnd(g, *shape, dt=F16):
    return torch.randn(*shape, generator=g, device=DEV).to(dt)


# ------------------------------------------------------------------ page tables
def _tables_case(B, page, ld, most, new_most, rows, seed, nfree=None, head=0, T=None, num_pages=None):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, most + 1, B).astype(np.int32)
    new = rng.integers(0, new_most + 1, B).astype(np.int32)
    need = int(sum(-(-(int(c) + int(n)) // page) - -(-int(c) // page) for c, n in zip(lens, new)))
    nfree = need + head + 3 if nfree is None else nfree
    ids = rng.permutation(B * ld + nfree).astype(np.int32)
    table, free = ids[:B * ld].reshape(B, ld).copy(), ids[B * ld:].copy()
    T = (B * rows if rows else max(1, int(new.sum()) + 3)) if T is None else T
    return lens, new, page, free, head, (B * ld + nfree if num_pages is None else num_pages), table, T, rows


def _run_tables(lens, new, page, free, head, num_pages, table, T, rows):
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
    tab = d(table)
    got = rtopk.page_tables(d(lens), d(new), page, d(free), tab, num_pages,
                            free_head=torch.tensor([head], dtype=torch.int32, device=DEV),
                            tokens=None if rows else T, rows=rows or None)
    want = tables(lens, new, page, free, head, num_pages, table, T, rows)
    torch.cuda.synchronize()
    for name, g, w in zip(("table", "slots", "positions", "cu_new", "free_next"), (tab,) + got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name
    return got


@pytest.mark.parametrize("B,page,ld,most,new_most,rows", [
    (1, 16, 4, 30, 1, 0), (1, 1, 9, 4, 5, 0), (5, 16, 40, 100, 500, 0), (7, 24, 10, 100, 64, 64), (3, 7, 400, 10, 2500, 0),
    (300, 16, 20, 200, 1, 0), (300, 16, 20, 200, 9, 9), (2049, 8, 9, 40, 3, 0), (4100, 16, 4, 50, 2, 2), (9, 16, 300, 0, 4300, 4300),
    (64, 3, 60, 90, 60, 0), (2, 1, 70, 1, 0, 0),
])
def test_page_tables(B, page, ld, most, new_most, rows):
    print(f"[tables] B={B} page={page} new={new_most} rows={rows}", flush=True)
    _run_tables(*_tables_case(B, page, ld, most, new_most, rows, seed=B + page))


def test_page_tables_refuse_requests():
    # table rows and slot rows that are too short, a list that ends, slots that end, a head inside and past the list
    _run_tables(*_tables_case(40, 16, 3, 60, 30, 0, seed=1))
    _run_tables(*_tables_case(40, 16, 9, 60, 30, 8, seed=2))
    _run_tables(*_tables_case(40, 4, 30, 60, 30, 0, seed=3, nfree=37))
    _run_tables(*_tables_case(40, 4, 30, 60, 30, 0, seed=4, T=211))
    _run_tables(*_tables_case(40, 4, 30, 60, 30, 30, seed=5, nfree=50, head=21))
    _run_tables(*_tables_case(40, 4, 30, 60, 30, 0, seed=6, nfree=5, head=900))
    _run_tables(*_tables_case(40, 4, 30, 60, 30, 0, seed=7, num_pages=600))  # page ids past the cache
    c = list(_tables_case(2600, 4, 6, 10, 9, 4, seed=8))  # many rows over their slots in every tile
    c[1][:2500] = 2 ** 31 - 1
    c[0][5:50] = -7
    _run_tables(*c)


def test_page_tables_free_next_feeds_the_next_call():
    lens, new, page, free, _, num_pages, table, T, _ = _tables_case(20, 8, 40, 30, 20, 0, seed=9, nfree=400)
    got = _run_tables(lens, new, page, free, 0, num_pages, table, T, 0)
    head = int(got[3][0])
    t1 = tables(lens, new, page, free, 0, num_pages, table, T, 0)[0]
    _run_tables(lens + new, new[::-1].copy(), page, free, head, num_pages, t1, T, 0)


# ------------------------------------------------------------------ cache store
@pytest.mark.parametrize("T,Hkv,D,page,dt,layout", [
    (1, 1, 64, 16, F16, "nhd"), (37, 3, 80, 24, BF16, "nhd"), (500, 8, 128, 16, BF16, "hnd"), (65, 2, 7, 5, F16, "nhd"),
    (33, 4, 16, 1, torch.float32, "hnd"), (20, 1, 3, 4, torch.float32, "nhd"), (1025, 16, 64, 64, F16, "nhd"), (3, 64, 256, 16, F16, "nhd"),
])
def test_cache_store(T, Hkv, D, page, dt, layout):
    print(f"[store] T={T} Hkv={Hkv} D={D} page={page} {dt} {layout}", flush=True)
    g = _gen(T + D)
    pages = T // page + 3
    shape = (pages, page, Hkv, D) if layout == "nhd" else (pages, Hkv, page, D)
    kc, vc = _rnd(g, *shape, dt=dt), _rnd(g, *shape, dt=dt)
    if layout == "hnd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    kv = _rnd(g, T, 2, Hkv, D, dt=dt)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:T].to(torch.int32)
    slots[T // 2::7] = -1
    if T > 8:
        slots[1], slots[2] = pages * page, 2 ** 31 - 1
    wk, wv = kc.clone(), vc.clone()
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            wk[s // page, s % page], wv[s // page, s % page] = kv[t, 0], kv[t, 1]
    rtopk.cache_store(kv[:, 0], kv[:, 1], slots, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_cache_store_unaligned_and_padded_rows():
    g = _gen(3)
    B, N, Hkv, D, page, pages = 3, 5, 2, 32, 8, 9
    base = _rnd(g, B * N * Hkv * D + 1)
    k = base[1:].view(B, N, Hkv, D)  # two bytes off a 16-byte boundary: one element at a time
    v = _rnd(g, B, N, Hkv, D)
    kc, vc = _rnd(g, pages, page, Hkv, D), _rnd(g, pages, page, Hkv, D)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:B * N].to(torch.int32).view(B, N)
    slots[1, 3:] = -1
    wk, wv = kc.clone(), vc.clone()
    for b in range(B):
        for n in range(N):
            s = int(slots[b, n])
            if s >= 0:
                wk[s // page, s % page], wv[s // page, s % page] = k[b, n], v[b, n]
    rtopk.cache_store(k, v, slots, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


# ------------------------------------------------------------------ cross attention
def _cross(B, N, S, Hq, Hkv, D, dt, seed, lens=None, mask=None, scale=None, q=None, k=None, v=None):
    g = _gen(seed)
    q = _rnd(g, B, N, Hq, D, dt=dt) * 1.5 if q is None else q
    k = _rnd(g, B, S, Hkv, D, dt=dt) if k is None else k
    v = _rnd(g, B, S, Hkv, D, dt=dt) if v is None else v
    lse = torch.full((B, N, Hq), 7.0, device=DEV)
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, _ = rtopk.cross_attention(q, k, v, lens=lt, key_mask=mask, scale=scale, lse=lse)
    torch.cuda.synchronize()
    check_cross(q, k, v, lens, mask, D ** -0.5 if scale is None else scale, out, lse, f"cross {B} {N} {S} {Hq} {Hkv} {D}")
    return out, lse


@pytest.mark.parametrize("B,N,S,Hq,Hkv,D,dt", [
    (1, 1, 1, 1, 1, 64, F16), (2, 4, 63, 4, 4, 64, F16), (2, 4, 64, 4, 4, 64, BF16), (3, 4, 65, 8, 2, 64, F16),
    (1, 31, 100, 2, 2, 64, BF16), (2, 32, 129, 2, 2, 128, F16), (1, 33, 257, 4, 2, 128, BF16), (1, 130, 200, 2, 2, 64, F16),
    (1, 129, 513, 2, 1, 128, BF16), (2, 300, 333, 2, 2, 64, BF16), (1, 5, 70, 10, 2, 80, F16), (2, 3, 90, 3, 3, 40, BF16),
    (1, 2, 40, 2, 1, 8, F16), (1, 7, 300, 4, 4, 96, BF16), (1, 9, 150, 4, 2, 256, F16), (1, 70, 200, 2, 1, 192, BF16),
    (2, 1, 5000, 4, 1, 128, BF16), (1, 8, 9001, 8, 2, 64, F16), (5, 12, 31, 16, 16, 64, F16), (1, 17, 4097, 2, 2, 256, BF16),
    (1, 16, 700, 2, 2, 128, F16), (1, 600, 70, 1, 1, 32, F16), (2, 260, 1100, 3, 1, 128, F16),
])
def test_cross_attention(B, N, S, Hq, Hkv, D, dt):
    print(f"[cross] B={B} N={N} S={S} Hq={Hq} Hkv={Hkv} D={D} {dt}", flush=True)
    _cross(B, N, S, Hq, Hkv, D, dt, seed=S + D)


@pytest.mark.parametrize("N,D,dt", [(4, 64, F16), (4, 128, BF16), (40, 64, BF16), (150, 128, F16), (3, 256, BF16)])
def test_cross_lengths_and_masks(N, D, dt):
    S, B = 777, 6
    g = _gen(N)
    lens = [0, 1, 64, 500, 777, 100000]
    print(f"[cross lens] N={N} D={D}", flush=True)
    _cross(B, N, S, 4, 2, D, dt, seed=1, lens=lens)
    mask = (torch.rand(B, S, generator=g, device=DEV) < 0.3).to(torch.uint8)
    mask[3] = 1  # nothing is left of it
    mask[4, :700] = 255
    mask[5, 64:] = 1
    _cross(B, N, S, 4, 2, D, dt, seed=2, lens=lens, mask=mask)
    _cross(B, N, S, 4, 2, D, dt, seed=3, lens=[-5, 777, 30, 2, 3, 129], mask=mask.bool())


@pytest.mark.parametrize("N,dt", [(4, F16), (50, BF16), (200, F16)])
def test_cross_masked_places_hold_anything(N, dt):
    B, S, Hkv, D = 3, 400, 2, 64
    g = _gen(N)
    k, v = _rnd(g, B, S, Hkv, D, dt=dt), _rnd(g, B, S, Hkv, D, dt=dt)
    mask = (torch.rand(B, S, generator=g, device=DEV) < 0.2).to(torch.uint8)
    lens = [400, 333, 50]
    for b, L in enumerate(lens):
        for t, bad in ((k, math.nan), (v, math.inf)):
            t[b, L:] = bad
        k[b][mask[b] != 0] = math.inf
        v[b][mask[b] != 0] = math.nan
    out, lse = _cross(B, N, S, 4, Hkv, D, dt, seed=4, lens=lens, mask=mask, k=k, v=v)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()


def test_cross_infinite_values_that_count():
    # a value that rows do see reaches them
    g = _gen(8)
    for N in (4, 80):
        k, v = _rnd(g, 1, 100, 1, 64), _rnd(g, 1, 100, 1, 64)
        v[0, 70, 0, 5] = math.inf
        v[0, 71, 0, 9] = math.nan
        q = _rnd(g, 1, N, 2, 64)
        out, _ = rtopk.cross_attention(q, k, v)
        torch.cuda.synchronize()
        assert (out[..., 5] == math.inf).all() and torch.isnan(out[..., 9]).all()
        keep = [d for d in range(64) if d not in (5, 9)]
        assert torch.isfinite(out[..., keep].float()).all()


@pytest.mark.parametrize("N", [4, 70])
def test_cross_strides(N):
    g = _gen(11)
    B, S, H, D = 3, 150, 4, 64
    qkv = _rnd(g, N, B, 3, H, D, dt=BF16)  # tokens first, fused
    kv = _rnd(g, B, 2, H, S, D, dt=BF16)   # heads before tokens
    q = qkv[:, :, 1].transpose(0, 1)
    k, v = kv[:, 0].transpose(1, 2), kv[:, 1].transpose(1, 2)
    assert not q.is_contiguous() and not k.is_contiguous()
    _cross(B, N, S, H, H, D, BF16, seed=0, q=q, k=k, v=v)
    one = _rnd(g, 1, S, H, D, dt=BF16).expand(B, S, H, D)  # one encoder for every batch element
    _cross(B, N, S, H, H, D, BF16, seed=0, q=q, k=one, v=v)
    _cross(B, N, S, H, 1, D, BF16, seed=0, q=q, k=k[:, :, :1], v=v[:, :, :1], scale=0.3)


def test_cross_large_scores_and_signs():
    # sums that would overflow without the running maximum; negative and zero scale
    g = _gen(12)
    for N in (4, 64):
        q, k, v = _rnd(g, 1, N, 2, 64, dt=BF16) * 30, _rnd(g, 1, 300, 2, 64, dt=BF16) * 30, _rnd(g, 1, 300, 2, 64, dt=BF16)
        _cross(1, N, 300, 2, 2, 64, BF16, seed=0, q=q, k=k, v=v, scale=1.0)
        _cross(1, N, 300, 2, 2, 64, BF16, seed=0, q=q, k=k, v=v, scale=-0.125)
        _cross(1, N, 300, 2, 2, 64, BF16, seed=0, q=q, k=k, v=v, scale=0.0)
        # keys whose scores rise along the sequence: the maximum moves in every tile
        k = torch.linspace(-4, 4, 300, device=DEV)[None, :, None, None].expand(1, 300, 2, 64).to(BF16).contiguous()
        q = torch.ones(1, N, 2, 64, device=DEV, dtype=BF16) * 3
        _cross(1, N, 300, 2, 2, 64, BF16, seed=0, q=q, k=k, v=v)


# ------------------------------------------------------------------ tree attention
def _tree_inputs(B, N, Hq, Hkv, D, page, lens, dt, seed, sizes=None, tree=True, layout="nhd", spare=2):
    g = _gen(seed)
    ld = max(1, -(-(max(lens) + N) // page))
    pages = B * ld + spare
    shape = (pages, page, Hkv, D) if layout == "nhd" else (pages, Hkv, page, D)
    kc, vc = _rnd(g, *shape, dt=dt), _rnd(g, *shape, dt=dt)
    if layout == "hnd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    q = _rnd(g, B, N, Hq, D, dt=dt) * 1.5
    table = torch.randperm(pages, generator=g, device=DEV)[:B * ld].to(torch.int32).view(B, ld)
    i = torch.arange(N, device=DEV)
    parents = (i - torch.randint(1, 6, (B, N), generator=g, device=DEV)).clamp(min=-1).to(torch.int32) if tree else None
    t = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(q=q, kc=kc, vc=vc, table=table, lens=t(lens), parents=parents, sizes=t(sizes))


def _tree(c, what, scale=None, workspace=None):
    B, N, Hq, D = c["q"].shape
    out = torch.full_like(c["q"], 3.0)
    lse = torch.full((B, N, Hq), 5.0, device=DEV)
    rtopk.tree_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], parents=c["parents"], sizes=c["sizes"], scale=scale,
                         out=out, lse=lse, workspace=workspace)
    torch.cuda.synchronize()
    lens = c["lens"].tolist()
    sizes = None if c["sizes"] is None else c["sizes"].tolist()
    check_tree(c["q"], c["kc"], c["vc"], c["table"], lens, c["parents"], sizes, D ** -0.5 if scale is None else scale, out, lse, what)
    if sizes is not None:  # rows behind the last node stay
        for b, n in enumerate(sizes):
            n = max(0, min(N, n))
            assert (out[b, n:] == 3.0).all() and (lse[b, n:] == 5.0).all(), what
    return out, lse


@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,lens,dt,tree", [
    (1, 1, 1, 1, 64, 16, [0], F16, False), (2, 1, 4, 4, 64, 16, [63, 64], F16, False), (3, 1, 8, 2, 128, 16, [5, 300, 1000], BF16, False),
    (2, 2, 4, 4, 64, 1, [100, 7], BF16, True), (2, 29, 10, 2, 80, 24, [0, 331], F16, True), (2, 64, 8, 2, 128, 16, [500, 130], BF16, True),
    (1, 64, 4, 4, 64, 64, [64], F16, True), (1, 65, 2, 2, 64, 100, [63], BF16, True), (2, 256, 2, 1, 64, 16, [10, 90], F16, True),
    (1, 200, 2, 1, 128, 8, [40], BF16, False), (1, 17, 8, 1, 128, 32, [4000], BF16, True), (1, 1, 16, 1, 64, 128, [9000], F16, False),
    (1, 3, 4, 2, 256, 16, [700], BF16, True), (1, 40, 4, 1, 192, 24, [129], F16, True), (1, 12, 2, 2, 32, 7, [200], F16, True),
    (4, 16, 4, 4, 8, 16, [1, 2, 3, 4], BF16, True), (1, 100, 8, 2, 64, 16, [0], F16, True),
])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_tree_attention(B, N, Hq, Hkv, D, page, lens, dt, tree, layout):
    what = f"tree B={B} N={N} Hq={Hq} Hkv={Hkv} D={D} page={page} {dt} {layout}"
    print(f"[{what}]", flush=True)
    _tree(_tree_inputs(B, N, Hq, Hkv, D, page, lens, dt, seed=N + D, tree=tree, layout=layout), what)


@pytest.mark.parametrize("N,G", [(1, 4), (9, 4), (70, 4), (256, 1)])
def test_tree_sizes_and_lengths(N, G):
    lens = [0, 0, 5, 64, 200, -3]
    sizes = [0, N, 1, N // 2, N + 50, -1]
    print(f"[tree sizes] N={N}", flush=True)
    _tree(_tree_inputs(6, N, 2 * G, 2, 64, 16, lens, F16, seed=N, sizes=sizes), f"sizes N={N}")


@pytest.mark.parametrize("N,dt", [(1, F16), (8, BF16), (66, F16)])
def test_tree_places_that_no_row_sees(N, dt):
    # pages of nobody, the rest of a last page, table entries behind the last token: anything may stand there
    c = _tree_inputs(3, N, 4, 2, 64, 16, [37, 0, 130], dt, seed=N, sizes=[N, N, max(1, N - 1)])
    used = torch.zeros(c["kc"].shape[0] * 16, dtype=torch.bool, device=DEV)
    for b in range(3):
        n = int(c["lens"][b]) + int(c["sizes"][b])
        at = torch.arange(n, device=DEV)
        used[(c["table"][b, at // 16] * 16 + at % 16).long()] = True
        c["table"][b, -(-n // 16):] = torch.tensor([-1, 2 ** 31 - 1, 10 ** 6, -2 ** 31] * 9, dtype=torch.int32, device=DEV)[:c["table"].shape[1] - -(-n // 16)]
    used = used.view(-1, 16)
    c["kc"][~used] = math.nan
    c["vc"][~used] = math.inf
    out, lse = _tree(c, "unseen")
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("N,dt,G", [(8, F16, 1), (8, BF16, 4), (70, F16, 2)])
def test_tree_nodes_that_a_row_does_not_see(N, dt, G):
    # a node's infinities and NaN reach its own descendants and nobody else
    c = _tree_inputs(2, N, 2 * G, 2, 64, 16, [40, 61], dt, seed=N + 1)
    c["parents"][:, 1:] = torch.where(torch.arange(1, N, device=DEV) % 2 == 0, torch.arange(1, N, device=DEV) - 2, -1).to(torch.int32)
    bad = [1, 5]  # two branches: even nodes below node 0, odd ones alone
    for b, L in ((0, 40), (1, 61)):
        for j, val in zip(bad, (math.inf, math.nan)):
            s = L + j
            p = int(c["table"][b, s // 16])
            c["vc"][p, s % 16, :, 3] = val
            c["vc"][p, s % 16, :, 40] = -val
    out, _ = _tree(c, "unseen nodes")
    even = out[:, 0::2].float()
    assert torch.isfinite(even).all() and not torch.isfinite(out[:, 1, :, 3].float()).any()
    for b, L in ((0, 40), (1, 61)):  # and so do a node's keys
        s = L + 3
        c["kc"][int(c["table"][b, s // 16]), s % 16] = math.nan
    out, _ = _tree(c, "unseen keys") if N < 0 else rtopk.tree_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], parents=c["parents"])
    torch.cuda.synchronize()
    assert torch.isfinite(out[:, 0::2].float()).all() and torch.isnan(out[:, 3].float()).all()


@pytest.mark.parametrize("N", [1, 40])
def test_tree_bad_pages_and_short_tables(N):
    c = _tree_inputs(3, N, 4, 2, 64, 16, [100, 120, 90], F16, seed=5)
    c["table"][0, 2] = -1
    c["table"][0, 4] = c["kc"].shape[0]
    c["table"][1] = 2 ** 31 - 1  # nothing is left
    out, lse = _tree(c, "bad pages")
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    c = _tree_inputs(2, N, 4, 2, 64, 16, [40, 20], F16, seed=6)
    c["table"] = c["table"][:, :3].contiguous()  # 48 tokens: nodes past them are left out
    _tree(c, "short table")
    c["lens"] = torch.tensor([10 ** 9, 48], dtype=torch.int32, device=DEV)
    _tree(c, "lengths past the table")


def test_tree_odd_parents():
    # parents at or behind a node, far away, negative: no parent
    c = _tree_inputs(2, 20, 4, 2, 64, 16, [3, 30], F16, seed=7)
    c["parents"][0] = torch.arange(20, device=DEV).to(torch.int32)  # every node its own parent
    c["parents"][1] = torch.tensor([5, 0, 1, -2 ** 31, 2 ** 31 - 1, 4, 5, 6, 19, 8, 9, 10, 3, 3, 3, 14, 15, 100, -7, 18],
                                   dtype=torch.int32, device=DEV)
    _tree(c, "odd parents")


def test_tree_far_offsets():
    # a cache of more than 2^32 bytes with the pages at its end
    page, Hkv, D = 64, 8, 128
    pages = (1 << 32) // (page * Hkv * D * 2) + 40  # 4 GiB and 40 pages more
    kc = torch.empty(pages, page, Hkv, D, dtype=BF16, device=DEV)
    vc = torch.empty_like(kc)
    c = _tree_inputs(2, 6, 16, 8, 128, page, [700, 1200], BF16, seed=8, spare=0)
    n = c["kc"].shape[0]
    kc[-n:], vc[-n:] = c["kc"], c["vc"]
    lse = torch.empty(2, 6, 16, device=DEV)
    a, _ = rtopk.tree_attention(c["q"], kc, vc, c["table"] + (pages - n), c["lens"], parents=c["parents"], lse=lse)
    b, _ = _tree(c, "near")
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    far = torch.arange(700, 706, device=DEV).to(torch.int32) + (pages - n) * page
    k = _rnd(_gen(1), 6, Hkv, D, dt=BF16)
    rtopk.cache_store(k, k, far, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc.view(-1, Hkv, D)[far.long()], k) and torch.equal(vc.view(-1, Hkv, D)[far.long()], k)


# ------------------------------------------------------------------ many batch elements, long and far keys
@pytest.mark.parametrize("B,N,S,Hkv,D", [(70, 2, 700, 1, 64), (256, 1, 300, 2, 128), (257, 1, 300, 1, 64), (130, 20, 400, 1, 128)])
def test_cross_many_batch_elements(B, N, S, Hkv, D):
    # shares of keys across up to 256 lengths, empty and full ones among them; more than that one share each
    rng = np.random.default_rng(B)
    lens = rng.integers(0, S + 1, B)
    lens[::9] = 0
    lens[3::17] = S
    print(f"[cross many] B={B} N={N} S={S}", flush=True)
    _cross(B, N, S, Hkv, Hkv, D, F16, seed=B, lens=lens.tolist())


def test_more_workgroups_than_places():
    # they start longest first; equal, empty and full lengths among them
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 131, 40)
    lens[::8] = 0
    lens[1::8] = 130
    lens[2::8] = 77
    _cross(40, 260, 130, 4, 4, 64, F16, seed=4, lens=lens.tolist())
    sizes = rng.integers(0, 71, 64)
    c = _tree_inputs(64, 70, 24, 12, 64, 16, rng.integers(0, 90, 64).tolist(), BF16, seed=5, sizes=sizes.tolist())
    _tree(c, "longest first")


@pytest.mark.parametrize("B,N", [(65, 1), (200, 2), (40, 60)])
def test_tree_many_requests(B, N):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 900, B)
    sizes = rng.integers(0, N + 1, B)
    lens[::7] = 0
    print(f"[tree many] B={B} N={N}", flush=True)
    _tree(_tree_inputs(B, N, 2, 1, 64, 16, lens.tolist(), BF16, seed=B, sizes=sizes.tolist()), f"many B={B}")


@pytest.mark.parametrize("N,D", [(1, 64), (20, 128), (70, 64)])
def test_cross_long(N, D):
    # more shares than one batch element may have
    print(f"[cross long] N={N} D={D}", flush=True)
    _cross(1, N, 70001, 1, 1, D, BF16, seed=N, lens=[69990])


@pytest.mark.parametrize("N", [2, 40])
def test_cross_rows_far_apart(N):
    # rows of keys 2^25 elements apart, in a buffer of more than 2^31 bytes
    S, D, far = 35, 64, 1 << 25
    g = _gen(N)
    buf = torch.zeros(far * S, dtype=F16, device=DEV)
    k = torch.as_strided(buf, (1, S, 1, D), (0, far, D, 1), 0)
    v = torch.as_strided(buf, (1, S, 1, D), (0, far, D, 1), 128)
    k.copy_(_rnd(g, 1, S, 1, D))
    v.copy_(_rnd(g, 1, S, 1, D))
    _cross(1, N, S, 2, 1, D, F16, seed=1, k=k, v=v)


# ------------------------------------------------------------------ calls as programs make them
def test_same_bits_every_time():
    c = _tree_inputs(2, 6, 8, 2, 128, 16, [3000, 41], BF16, seed=1)
    a = [rtopk.tree_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], parents=c["parents"])[0] for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(a[0], x) for x in a)
    g = _gen(2)
    q, k = _rnd(g, 2, 4, 4, 64), _rnd(g, 2, 3000, 4, 64)
    a = [rtopk.cross_attention(q, k, k)[0] for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(a[0], x) for x in a)


def _ws(n):
    return torch.zeros(n, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("N", [1, 40])
def test_graph_replays(N):
    # both attentions and the cache calls in one graph, on workspaces of the caller's; new inputs between replays
    c = _tree_inputs(3, N, 8, 2, 64, 16, [1500, 40, 700], F16, seed=N)
    B, _, Hq, D = c["q"].shape
    pages, page, Hkv, _ = c["kc"].shape
    g = _gen(N)
    S = 1300
    ek, ev = _rnd(g, B, S, Hkv, D), _rnd(g, B, S, Hkv, D)
    new = torch.full((B,), N, dtype=torch.int32, device=DEV)
    free = torch.arange(4, dtype=torch.int32, device=DEV)
    nk, nv = _rnd(g, B, N, Hkv, D), _rnd(g, B, N, Hkv, D)
    ld = c["table"].shape[1]
    w1 = _ws(rtopk.rtopk_tree_attention_workspace_bytes(B, N, Hq, Hkv, D, ld, page))
    w2 = _ws(rtopk.rtopk_cross_attention_workspace_bytes(B, N, S, Hq, Hkv, D))
    outs = [torch.zeros_like(c["q"]) for _ in range(2)]
    tabs = (torch.zeros(B, N, dtype=torch.int32, device=DEV), torch.zeros(B, N, dtype=torch.int32, device=DEV),
            torch.zeros(B + 1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV))
    lens0 = c["lens"].clone()

    def step():
        rtopk.page_tables(c["lens"], new, page, free, c["table"], pages, out=tabs)
        rtopk.cache_store(nk, nv, tabs[0], c["kc"], c["vc"])
        rtopk.tree_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], parents=c["parents"], out=outs[0], workspace=w1)
        rtopk.cross_attention(outs[0], ek, ev, out=outs[1], workspace=w2)

    # enough tokens are in every row's own pages already, so that the free list stays unused
    c["lens"].copy_(((lens0 + N + page - 1) // page) * page - N)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        step()
    for rep in range(4):
        c["q"].copy_(torch.roll(c["q"], rep + 1, 3))
        nk.copy_(torch.roll(nk, rep + 1, 0))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs)), rep
        check_tree(c["q"], c["kc"], c["vc"], c["table"], c["lens"].tolist(), c["parents"], None, D ** -0.5, got[0], None, "graph")


def test_capture_without_a_workspace_is_refused():
    g = _gen(1)
    q, k = _rnd(g, 1, 1, 2, 64), _rnd(g, 1, 20000, 2, 64)  # few rows, many keys: split
    out = torch.zeros_like(q)
    rtopk.cross_attention(q, k, k, out=out)
    torch.cuda.synchronize()
    want = out.clone()
    need = rtopk.rtopk_cross_attention_workspace_bytes(1, 1, 20000, 2, 2, 64)
    if need == rtopk.RTOPK_WS_FIXED_BYTES:
        pytest.skip("nothing is split here")
    graph = torch.cuda.CUDAGraph()
    err = None
    w = _ws(need)
    with torch.cuda.graph(graph):
        try:
            rtopk.cross_attention(q, k, k, out=out)
        except rtopk.RtopkError as e:
            err = e
        rtopk.cross_attention(q, k, k, out=out, workspace=w)
    assert err is not None and err.status == rtopk.RTOPK_EINVAL and "captured" in str(err)
    out.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_two_streams_at_once():
    g = _gen(5)
    q, k, v = _rnd(g, 2, 4, 4, 128, dt=BF16), _rnd(g, 2, 9000, 4, 128, dt=BF16), _rnd(g, 2, 9000, 4, 128, dt=BF16)
    want = rtopk.cross_attention(q, k, v)[0]
    q2 = q.flip(1).contiguous()
    want2 = rtopk.cross_attention(q2, k, v)[0]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    o1, o2 = [torch.zeros_like(q) for _ in range(8)], [torch.zeros_like(q) for _ in range(8)]
    torch.cuda.synchronize()
    for i in range(8):
        with torch.cuda.stream(s1):
            rtopk.cross_attention(q, k, v, out=o1[i])
        with torch.cuda.stream(s2):
            rtopk.cross_attention(q2, k, v, out=o2[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in o1) and all(torch.equal(o, want2) for o in o2)


def test_a_workspace_serves_selection_and_attention():
    # one caller workspace for beam_step_ws and both attentions, in turn on one stream
    from beam_search_top_amd import synth
    from gpu_util import to_device
    s = synth.make_custom(8, 4, 4, 4000, synth.F16, seed=90, n_finished=3)
    x, a, f = to_device(s)
    want = [o.clone() for o in rtopk.beam_step(x, a, f, k=4, eos_id=s.eos_id)]
    g = _gen(6)
    q, k = _rnd(g, 1, 4, 4, 64), _rnd(g, 1, 9000, 4, 64)
    wa = rtopk.cross_attention(q, k, k)[0]
    n = max(rtopk.rtopk_workspace_bytes(8, 4, 4000, 4, synth.F16), rtopk.rtopk_cross_attention_workspace_bytes(1, 4, 9000, 4, 4, 64))
    w = _ws(n)
    for _ in range(3):
        got = rtopk.beam_step(x, a, f, k=4, eos_id=s.eos_id, workspace=w)
        ga = rtopk.cross_attention(q, k, k, workspace=w)[0]
        torch.cuda.synchronize()
        assert all(torch.equal(p, r) for p, r in zip(got, want)) and torch.equal(ga, wa)
    assert (w[:rtopk.RTOPK_WS_FIXED_BYTES] == 0).all()


def test_a_decoder_step_with_beams_as_a_tree():
    """Three decode steps in which the hypotheses stay a tree of nodes over the
    shared prefix: page tables, store, tree attention, cross attention, LM head
    and selection; the selection's beam ids become the next level's parents.
    Each level's attention is checked against the 64-bit reference, and the
    selection against the library's own on the same hidden states."""
    g = _gen(77)
    B, beam, H, Hkv, D, page, V, S = 3, 4, 4, 2, 64, 16, 500, 90
    E, levels = H * D, 3
    N = beam * levels
    lens = torch.tensor([35, 0, 61], dtype=torch.int32, device=DEV)
    ld = -(-(61 + N) // page)
    pages = B * ld + 4
    kc, vc = _rnd(g, pages, page, Hkv, D, dt=BF16), _rnd(g, pages, page, Hkv, D, dt=BF16)
    table = torch.full((B, ld), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    # the prefix's pages and tokens
    _, _, _, head = rtopk.page_tables(torch.zeros_like(lens), lens, page, free, table, pages, tokens=100)
    emb = _rnd(g, V, E, dt=BF16)
    wq, wk, wv = _rnd(g, E, H * D, dt=BF16) / 16, _rnd(g, E, Hkv * D, dt=BF16) / 16, _rnd(g, E, Hkv * D, dt=BF16) / 16
    head_w = _rnd(g, V, E, dt=BF16) / 4
    ek, ev = _rnd(g, B, S, Hkv, D, dt=BF16), _rnd(g, B, S, Hkv, D, dt=BF16)
    elens = torch.tensor([90, 17, 0], dtype=torch.int32, device=DEV)
    parents = torch.full((B, N), -1, dtype=torch.int32, device=DEV)
    alive = torch.zeros(B, beam, device=DEV)
    alive[:, 1:] = -50.0  # one start
    tok = torch.full((B, beam), 1, dtype=torch.int32, device=DEV)
    x_all = torch.zeros(B, N, E, dtype=BF16, device=DEV)
    held = lens.clone()
    for lv in range(levels):
        lo, n = lv * beam, (lv + 1) * beam
        x_all[:, lo:n] = emb[tok.long()]
        slots, pos, _, nxt = rtopk.page_tables(held, torch.full_like(held, beam), page, free, table, pages, free_head=head, rows=beam)
        head = nxt
        x = x_all[:, lo:n].reshape(B * beam, E)
        rtopk.cache_store((x @ wk).view(B, beam, Hkv, D), (x @ wv).view(B, beam, Hkv, D), slots, kc, vc)
        held = held + beam
        # all nodes so far are the tree; the last level's rows are used
        q = (x_all[:, :n].reshape(B * n, E) @ wq).view(B, n, H, D)
        par = parents[:, :n].contiguous()
        o, _ = rtopk.tree_attention(q, kc, vc, table, lens, parents=par)
        torch.cuda.synchronize()
        check_tree(q, kc, vc, table, lens.tolist(), par, None, D ** -0.5, o, None, f"level {lv}")
        h = o[:, lo:].contiguous()
        c, _ = rtopk.cross_attention(h, ek, ev, lens=elens)
        torch.cuda.synchronize()
        check_cross(h, ek, ev, elens.tolist(), None, D ** -0.5, c, None, f"cross level {lv}")
        hid = (c + h).reshape(B * beam, E).contiguous()
        bi, ti, sc = rtopk.lmhead_step(hid, head_w, alive, None, k=beam)
        li, lt, ls = rtopk.beam_step((hid.float() @ head_w.float().T).view(B, beam, V), alive, None, k=beam)
        torch.cuda.synchronize()
        assert torch.equal(bi, li) and torch.equal(ti, lt)
        assert (bi >= 0).all() and torch.equal(pos, held[:, None] - beam + torch.arange(beam, device=DEV, dtype=torch.int32)[None])
        if lv + 1 < levels:
            parents[:, n:n + beam] = bi + lo
        alive, tok = sc, ti
