"""Tree attention over a cache in 8 bits on the GPU against the plain 64-bit
reference of tree attention (layer_ref.py, which derives the tolerances) on
what the codes and scales stand for: those values are numbers of the queries' type,
so that the kernel rounds what it rounds over a cache of that type and nothing more."""
import math
import threading

import numpy as np
import pytest
import torch

from beam_search_top_amd import rtopk
from layer_ref import check_tree
from libutil import ensure_built
from serve_ref import CODES, rope, sample

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


def _decode(codes, scales):
    return torch.from_numpy(CODES).to(DEV)[codes.view(torch.uint8).int()] * torch.exp2(scales.double().clamp(1, 254) - 127)[..., None]


def _codes(g, *shape):
    return (torch.randn(*shape, generator=g, device=DEV) * 80).clamp(-448, 448).to(torch.float8_e4m3fn)


def _inputs(B, N, Hq, Hkv, D, page, lens, dt, seed, sizes=None, tree=True, layout="nhd", spare=2):
    g = _gen(seed)
    ld = max(1, -(-(max(lens) + N) // page))
    pages = B * ld + spare
    shape = (pages, page, Hkv, D) if layout == "nhd" else (pages, Hkv, page, D)
    kc, vc = _codes(g, *shape), _codes(g, *shape)
    if layout == "hnd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    ks, vs = (torch.randint(119, 123, (pages, page, Hkv), generator=g, device=DEV).to(torch.uint8) for _ in range(2))
    q = torch.randn(B, N, Hq, D, generator=g, device=DEV).to(dt) * 1.5
    table = torch.randperm(pages, generator=g, device=DEV)[:B * ld].to(torch.int32).view(B, ld)
    i = torch.arange(N, device=DEV)
    parents = (i - torch.randint(1, 6, (B, N), generator=g, device=DEV)).clamp(min=-1).to(torch.int32) if tree else None
    t = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=t(lens), parents=parents, sizes=t(sizes))


def _call(c, **kw):
    return rtopk.tree_attention_fp8(c["q"], c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["lens"], parents=c["parents"],
                                    sizes=c["sizes"], **kw)


def _tree(c, what, scale=None, workspace=None):
    B, N, Hq, D = c["q"].shape
    out = torch.full_like(c["q"], 3.0)
    lse = torch.full((B, N, Hq), 5.0, device=DEV)
    _call(c, scale=scale, out=out, lse=lse, workspace=workspace)
    torch.cuda.synchronize()
    lens = c["lens"].tolist()
    sizes = None if c["sizes"] is None else c["sizes"].tolist()
    check_tree(c["q"], _decode(c["kc"], c["ks"]), _decode(c["vc"], c["vs"]), c["table"], lens, c["parents"], sizes,
               D ** -0.5 if scale is None else scale, out, lse, what)
    if sizes is not None:  # rows behind the last node stay
        for b, n in enumerate(sizes):
            n = max(0, min(N, n))
            assert (out[b, n:] == 3.0).all() and (lse[b, n:] == 5.0).all(), what
    return out, lse


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("B,N,Hq,Hkv,D,page,lens,dt,tree", [
    (1, 1, 1, 1, 64, 16, [0], F16, False), (1, 1, 1, 1, 16, 16, [1], BF16, False), (3, 1, 8, 2, 64, 16, [5, 100, 333], F16, False),
    (2, 1, 16, 2, 128, 64, [1000, 4097], BF16, False), (2, 1, 20, 1, 128, 24, [63, 300], F16, False), (4, 1, 4, 4, 80, 1, [7, 31, 32, 33], BF16, True),
    (2, 1, 8, 8, 32, 3, [64, 65], F16, False), (2, 5, 8, 2, 48, 8, [100, 0], F16, True), (2, 16, 4, 2, 96, 16, [31, 200], BF16, True),
    (2, 7, 10, 2, 128, 16, [129, 1500], F16, True), (1, 32, 2, 2, 64, 8, [77], BF16, True), (2, 33, 2, 1, 128, 16, [50, 64], BF16, True),
    (2, 29, 20, 4, 80, 24, [0, 301], F16, True), (2, 64, 8, 2, 128, 16, [150, 400], BF16, True), (1, 200, 4, 1, 64, 100, [500], F16, True),
    (2, 100, 4, 2, 112, 12, [33, 65], BF16, False), (2, 1, 4, 2, 256, 16, [10, 700], F16, False), (2, 1, 2, 2, 192, 5, [64, 31], BF16, True),
    (2, 20, 4, 1, 256, 8, [40, 90], BF16, True), (1, 256, 2, 1, 192, 16, [100], F16, True), (1, 150, 8, 8, 64, 1, [70], BF16, False),
])
def test_tree_attention(B, N, Hq, Hkv, D, page, lens, dt, tree, layout):
    print(f"[tree8] B={B} N={N} {Hq}/{Hkv} x {D} page={page} {dt} {layout}", flush=True)
    _tree(_inputs(B, N, Hq, Hkv, D, page, lens, dt, seed=B + N + D, tree=tree, layout=layout), "tree")


@pytest.mark.parametrize("N,G", [(1, 4), (9, 4), (70, 4), (256, 1)])
def test_sizes_and_lengths(N, G):
    c = _inputs(6, N, 2 * G, 2, 64, 16, [0, 1, 15, 16, 17, 200], F16, seed=N, sizes=[N, 0, 1, N // 2, -3, 10 ** 6])
    _tree(c, "sizes")


@pytest.mark.parametrize("N,D", [(1, 64), (20, 128), (70, 64), (3, 256), (1, 128)])
def test_long(N, D):
    print(f"[tree8 long] N={N} D={D}", flush=True)
    _tree(_inputs(2, N, 4, 2, D, 16, [9001, 20000], BF16, seed=N, sizes=[N, max(1, N - 1)]), "long")


@pytest.mark.parametrize("N,dt,D", [(1, F16, 64), (8, BF16, 64), (66, F16, 64), (4, BF16, 128), (2, F16, 256)])
def test_places_that_no_row_sees(N, dt, D):
    # pages of nobody, the rest of a last page, table entries behind the last token: any codes and scales may stand there
    c = _inputs(3, N, 4, 2, D, 16, [37, 0, 130], dt, seed=N, sizes=[N, N, max(1, N - 1)])
    used = torch.zeros(c["kc"].shape[0] * 16, dtype=torch.bool, device=DEV)
    for b in range(3):
        n = int(c["lens"][b]) + int(c["sizes"][b])
        at = torch.arange(n, device=DEV)
        used[(c["table"][b, at // 16] * 16 + at % 16).long()] = True
        c["table"][b, -(-n // 16):] = torch.tensor([-1, 2 ** 31 - 1, 10 ** 6, -2 ** 31] * 9, dtype=torch.int32, device=DEV)[:c["table"].shape[1] - -(-n // 16)]
    used = used.view(-1, 16)
    c["kc"].view(torch.uint8)[~used] = 0x7f
    c["vc"].view(torch.uint8)[~used] = 0xff
    c["ks"][~used] = 255
    c["vs"][~used] = 254
    out, lse = _tree(c, "unseen")
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("N,dt,G,D", [(8, F16, 1, 64), (8, BF16, 4, 64), (70, F16, 2, 64), (9, BF16, 2, 128), (40, F16, 1, 256)])
def test_nodes_that_a_row_does_not_see(N, dt, G, D):
    # a node's NaN reach its own descendants and nobody else
    c = _inputs(2, N, 2 * G, 2, D, 16, [40, 61], dt, seed=N + 1)
    c["parents"][:, 1:] = torch.where(torch.arange(1, N, device=DEV) % 2 == 0, torch.arange(1, N, device=DEV) - 2, -1).to(torch.int32)
    for b, L in ((0, 40), (1, 61)):
        for j in (1, 5):  # two branches: even nodes below node 0, odd ones alone
            s = L + j
            row = c["vc"].view(torch.uint8)[int(c["table"][b, s // 16]), s % 16]
            row[:, 3] = 0x7f
            row[:, 40] = 0xff
    out, _ = _tree(c, "unseen nodes")
    assert torch.isfinite(out[:, 0::2].float()).all() and torch.isnan(out[:, 1, :, 3].float()).all() and torch.isnan(out[:, 5, :, 40].float()).all()
    for b, L in ((0, 40), (1, 61)):  # and so do a node's keys
        s = L + 3
        c["kc"].view(torch.uint8)[int(c["table"][b, s // 16]), s % 16] = 0x7f
    out, _ = _call(c)
    torch.cuda.synchronize()
    assert torch.isfinite(out[:, 0::2].float()).all() and torch.isnan(out[:, 3].float()).all()


@pytest.mark.parametrize("N,D", [(1, 64), (40, 64), (2, 128), (1, 256)])
def test_bad_pages_and_short_tables(N, D):
    c = _inputs(3, N, 4, 2, D, 16, [100, 120, 90], F16, seed=5)
    c["table"][0, 2] = -1
    c["table"][0, 4] = c["kc"].shape[0]
    c["table"][1] = 2 ** 31 - 1  # nothing is left
    out, lse = _tree(c, "bad pages")
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    c = _inputs(2, N, 4, 2, D, 16, [40, 20], F16, seed=6)
    c["table"] = c["table"][:, :3].contiguous()  # 48 tokens: nodes past them are left out
    _tree(c, "short table")
    c["lens"] = torch.tensor([10 ** 9, 48], dtype=torch.int32, device=DEV)
    _tree(c, "lengths past the table")


@pytest.mark.parametrize("N", [1, 50])
def test_scales_of_every_size(N):
    # scales that differ by powers of 2^10 between tokens and heads; the smallest and largest of a type
    for dt, lo, hi in ((F16, 127 - 15, 127 + 6), (BF16, 127 - 60, 127 + 20)):
        c = _inputs(2, N, 4, 2, 64, 16, [200, 77], dt, seed=N)
        g = _gen(9)
        c["ks"] = torch.randint(127 - 12, 127 - 5, c["ks"].shape, generator=g, device=DEV).to(torch.uint8)
        c["vs"] = torch.randint(lo, hi, c["vs"].shape, generator=g, device=DEV).to(torch.uint8)
        _tree(c, "scales")
    c = _inputs(1, N, 2, 1, 64, 16, [0], BF16, seed=3, tree=True)
    c["parents"][:] = -1  # every row sees its own key alone: its value comes out as it is
    c["ks"][:] = 100
    for s in (0, 1, 2, 40, 200, 246):
        c["vs"][:] = s
        out, _ = _call(c)
        torch.cuda.synchronize()
        at = torch.arange(N, device=DEV)
        v = _decode(c["vc"], c["vs"])[c["table"][0, at // 16].long(), at % 16, 0].float()
        # subnormal codes at the smallest scales are below bfloat16's normal numbers: they may become zero
        near = (out[0, :, 0].float() - v).abs() <= (2.0 ** -126 if s < 9 else 0.0)
        assert near.all() and torch.equal(out[:, :, 0], out[:, :, 1]), s


def test_a_value_beyond_the_type_is_infinite():
    c = _inputs(1, 3, 1, 1, 64, 16, [0], F16, seed=4)
    c["parents"][:] = -1
    c["ks"][:] = 100
    c["vs"][:] = 127 + 14
    out, _ = _call(c)
    torch.cuda.synchronize()
    at = torch.arange(3, device=DEV)
    v = _decode(c["vc"], c["vs"])[c["table"][0, at // 16].long(), at % 16, 0]
    big = v.abs() >= 65520
    assert big.any() and torch.equal(out[0, :, 0].double()[big], torch.sign(v[big]) * math.inf)
    assert torch.equal(out[0, :, 0].double()[~big], v[~big])


def test_scale_and_sign():
    c = _inputs(2, 3, 4, 2, 128, 16, [200, 30], BF16, seed=2)
    _tree(c, "negative", scale=-0.2)
    _tree(c, "zero", scale=0.0)
    _tree(c, "large", scale=3.0)
    c = _inputs(2, 40, 4, 2, 64, 16, [200, 30], F16, seed=2)
    _tree(c, "negative, tiles", scale=-0.2)
    _tree(c, "zero, tiles", scale=0.0)


def test_agrees_with_the_16_bit_cache():
    # the same values in both caches: the same attention up to the order of sums
    for N, D in ((1, 128), (50, 128), (6, 64)):
        c = _inputs(3, N, 8, 2, D, 16, [700, 33, 1200], BF16, seed=N)
        k, v = _decode(c["kc"], c["ks"]).to(BF16), _decode(c["vc"], c["vs"]).to(BF16)
        a, _ = _call(c)
        b, _ = rtopk.tree_attention(c["q"], k, v, c["table"], c["lens"], parents=c["parents"])
        torch.cuda.synchronize()
        d = (a.float() - b.float()).abs()
        # weights are rounded in both, each by half a step at most: 2^-8 of the largest value there is, twice
        assert d.max() <= 2 * 2.0 ** -8 * float(v.float().abs().max())


@pytest.mark.parametrize("B,N", [(65, 1), (200, 2), (40, 60), (300, 1)])
def test_many_requests(B, N):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 900, B)
    sizes = rng.integers(0, N + 1, B)
    lens[::7] = 0
    print(f"[tree8 many] B={B} N={N}", flush=True)
    _tree(_inputs(B, N, 2, 1, 64, 16, lens.tolist(), BF16, seed=B, sizes=sizes.tolist()), f"many B={B}")


@pytest.mark.parametrize("N", [1, 40])
def test_far_offsets(N):
    # a cache of more than 2^32 bytes with the pages at its end
    page, Hkv, D = 64, 8, 128
    pages = (1 << 32) // (page * Hkv * D) + 40
    kc, vc = (torch.zeros(pages, page, Hkv, D, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(pages, page, Hkv, dtype=torch.uint8, device=DEV) for _ in range(2))
    c = _inputs(2, N, 16, 8, D, page, [700, 1200], BF16, seed=8, spare=0)
    n = c["kc"].shape[0]
    for big, t in ((kc, "kc"), (vc, "vc"), (ks, "ks"), (vs, "vs")):
        big[-n:] = c[t].view(torch.uint8)
    a, _ = rtopk.tree_attention_fp8(c["q"], kc, vc, ks, vs, c["table"] + (pages - n), c["lens"], parents=c["parents"])
    b, _ = _tree(c, "near")
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_same_bits_every_time_and_on_two_streams():
    c = _inputs(2, 6, 8, 2, 128, 16, [3000, 41], BF16, seed=1)
    want = _call(c)[0].clone()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(want) for _ in range(8)]
    torch.cuda.synchronize()
    for i in range(8):
        with torch.cuda.stream(s1 if i % 2 else s2):
            _call(c, out=outs[i])
    torch.cuda.synchronize()
    assert all(torch.equal(want, o) for o in outs)


@pytest.mark.parametrize("N", [1, 40])
def test_graph_replays(N):
    """A step's cache calls in one graph: rotation, store, attention, read back, draw; new inputs between replays."""
    c = _inputs(3, N, 8, 2, 64, 16, [1500, 40, 700], F16, seed=N)
    B, _, Hq, D = c["q"].shape
    pages, page, Hkv, _ = c["kc"].shape
    g = _gen(N)
    ld = c["table"].shape[1]
    ws = torch.zeros(rtopk.rtopk_tree_attention_fp8_workspace_bytes(B, N, Hq, Hkv, D, ld, page), dtype=torch.uint8, device=DEV)
    x = torch.randn(B, N, Hq + 2 * Hkv, D, generator=g, device=DEV).to(F16)
    freqs = (10000.0 ** (-torch.arange(0, D, 2, device=DEV) / D)).float()
    pos = c["lens"][:, None] + torch.arange(N, device=DEV, dtype=torch.int32)
    slots = (torch.gather(c["table"], 1, (pos // page).long()) * page + pos % page).to(torch.int32)
    qo, ko = torch.zeros(B, N, Hq, D, dtype=F16, device=DEV), torch.zeros(B, N, Hkv, D, dtype=F16, device=DEV)
    out = torch.zeros_like(qo)
    back = (torch.zeros_like(ko), torch.zeros_like(ko))
    u = torch.rand(B * N, generator=g, device=DEV)
    p = torch.full((B * N,), 0.9, device=DEV)
    drawn = (torch.zeros(B * N, dtype=torch.int32, device=DEV), torch.zeros(B * N, device=DEV))

    def step():
        rtopk.qk_norm_rope(x[:, :, :Hq].reshape(B * N, Hq, D), x[:, :, Hq:Hq + Hkv].reshape(B * N, Hkv, D), pos.view(-1), freqs,
                           q_out=qo.view(B * N, Hq, D), k_out=ko.view(B * N, Hkv, D))
        rtopk.cache_store_fp8(ko, x[:, :, Hq + Hkv:].contiguous(), slots, c["kc"], c["vc"], c["ks"], c["vs"])
        rtopk.tree_attention_fp8(qo, c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["lens"], parents=c["parents"], out=out, workspace=ws)
        rtopk.cache_load_fp8(c["kc"], c["vc"], c["ks"], c["vs"], slots, out=back)
        rtopk.sample_filtered(out.view(B * N, Hq * D), u, top_p=p, out=drawn)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        step()
    for rep in range(4):
        x.copy_(torch.roll(x, rep + 1, 3))
        u.copy_(torch.rand(B * N, generator=g, device=DEV))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in (out, *back, *drawn)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (out, *back, *drawn))), rep
        check_tree(qo, _decode(c["kc"], c["ks"]), _decode(c["vc"], c["vs"]), c["table"], c["lens"].tolist(), c["parents"], None,
                   D ** -0.5, got[0], None, "graph")


def test_capture_without_a_workspace_is_refused():
    c = _inputs(1, 1, 2, 2, 64, 16, [20000], F16, seed=1)  # few rows, many keys: split
    want = _call(c)[0].clone()
    out = torch.zeros_like(want)
    ws = torch.zeros(rtopk.rtopk_tree_attention_fp8_workspace_bytes(1, 1, 2, 2, 64, c["table"].shape[1], 16), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    err = None
    with torch.cuda.graph(graph):
        try:
            _call(c, out=out)
        except rtopk.RtopkError as e:
            err = e
        _call(c, out=out, workspace=ws)
    assert err is not None and err.status == rtopk.RTOPK_EINVAL and "captured" in str(err)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_decode_steps_that_sample():
    """Prompts and three decode steps as a server makes them: page tables, rotation of
    queries and keys at their positions, the store into the 8-bit cache,
    attention, a projection to logits, the filtered draw; each step against the references."""
    g = _gen(78)
    B, H, Hkv, D, page, V = 4, 4, 2, 64, 16, 5000
    E = H * D
    prompts = torch.tensor([35, 1, 61, 16], dtype=torch.int32, device=DEV)
    ld = 6
    pages = B * ld + 3
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    kc, vc = (torch.zeros(pages, page, Hkv, D, dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(pages, page, Hkv, dtype=torch.uint8, device=DEV) for _ in range(2))
    table = torch.full((B, ld), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    emb, wqkv, wo = rnd(V, E).to(BF16), (rnd(E, (H + 2 * Hkv) * D) / 16).to(BF16), (rnd(E, V) / 4).to(BF16)
    qw, kw = (1 + 0.2 * rnd(D)).to(BF16), (1 + 0.2 * rnd(D)).to(BF16)
    freqs = (10000.0 ** (-torch.arange(0, D, 2, device=DEV) / D)).float()
    kinds = dict(temperature=torch.tensor([1.0, 0.7, 0.0, 1.2], device=DEV), top_k=torch.tensor([50, 0, 0, 5], dtype=torch.int32, device=DEV),
                 top_p=torch.tensor([0.9, 0.8, 1.0, 1.0], device=DEV), min_p=torch.tensor([0.0, 0.05, 0.0, 0.0], device=DEV))
    head, held = None, torch.zeros_like(prompts)
    new, rows = prompts, 64
    tokens = torch.randint(0, V, (B, rows), generator=g, device=DEV)
    for step in range(4):
        slots, pos, _, head = rtopk.page_tables(held, new, page, free, table, pages, free_head=head, rows=rows)
        x = (emb[tokens] @ wqkv).view(B, rows, H + 2 * Hkv, D)
        q, k, v = x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:]
        qo, ko = rtopk.qk_norm_rope(q, k, pos, freqs, q_weight=qw, k_weight=kw)
        rtopk.cache_store_fp8(ko, v, slots, kc, vc, ks, vs)
        o, _ = rtopk.tree_attention_fp8(qo, kc, vc, ks, vs, table, held, sizes=new, out=torch.zeros_like(qo))
        last = o[torch.arange(B, device=DEV), (new - 1).long()].reshape(B, E)
        logits = last @ wo
        u = torch.rand(B, generator=g, device=DEV)
        tok, lp = rtopk.sample_filtered(logits, u, **kinds)
        torch.cuda.synchronize()
        live = (pos >= 0).cpu()
        for got, want, w in ((qo, q, qw), (ko, k, kw)):
            y, tol = rope(want.reshape(B * rows, -1, D).cpu(), w.cpu(), pos.view(-1).cpu(), freqs.cpu(), 1e-6, False)
            near = (got.reshape(B * rows, -1, D).cpu().double() - y).abs() <= tol
            assert near[live.view(-1)].all(), step
        check_tree(qo, _decode(kc, ks), _decode(vc, vs), table, held.tolist(), None, new.tolist(), D ** -0.5, o, None, f"step {step}")
        for b in range(B):
            f = [float(kinds["temperature"][b]), int(kinds["top_k"][b]), float(kinds["top_p"][b]), float(kinds["min_p"][b])]
            want, wlp = sample(logits[b].double().cpu().numpy(), float(u[b]), *f)
            assert int(tok[b]) == want and abs(float(lp[b]) - wlp) < 1e-5, (step, b)
        # the cache holds what was stored, to half a step
        kb, vb = rtopk.cache_load_fp8(kc, vc, ks, vs, slots)
        for got, want in ((kb, ko), (vb, v)):
            d = (got.float() - want.float()).abs()
            assert (d <= torch.maximum(want.float().abs() * 2.0 ** -4, want.float().abs().amax(-1, keepdim=True) * 2.0 ** -17))[pos >= 0].all()
        held = held + new
        new, rows = torch.ones_like(prompts), 1
        tokens = tok[:, None].long()


def test_two_threads_with_a_stream_each():
    # library-owned workspaces are one per stream: calls of two host threads do not meet
    cases = [_inputs(2, 3, 8, 2, 128, 16, [5000, 300], BF16, seed=s) for s in (81, 82)]
    logits = [torch.randn(3, 60000, generator=_gen(s), device=DEV).to(BF16) * 2 for s in (83, 84)]
    u, p = torch.tensor([0.2, 0.5, 0.9], device=DEV), torch.full((3,), 0.9, device=DEV)

    def both(i):
        return [_call(cases[i])[0], *rtopk.sample_filtered(logits[i], u, top_p=p)]

    want = [both(i) for i in range(2)]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(30):
                got[i].append(both(i))
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in range(2):
        assert len(got[i]) == 30 and all(torch.equal(a, b) for one in got[i] for a, b in zip(one, want[i])), i
