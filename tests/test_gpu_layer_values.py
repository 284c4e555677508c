"""Attention outputs where a wrong value, a lost weight or an extreme score shows:
weights far below the largest, every key counted once, rows that pick one key
out of many, NaN keys, scores near the largest floats; a store of more tokens
than a launch has workgroups. References in 64 bits."""
import math

import pytest
import torch

from beam_search_top_amd import rtopk
from layer_ref import check_tree
from test_gpu_layer import DEV, _gen, _rnd, _tree, _tree_inputs, lib  # noqa: F401

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
HALF = {F16: 2.0 ** -11, BF16: 2.0 ** -8}  # half a step, relative
F = 2.0 ** -24


def _cross(q, k, v, **kw):
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    out, _ = rtopk.cross_attention(q, k, v, lse=lse, **kw)
    torch.cuda.synchronize()
    return out.cpu().double(), lse.cpu().double()


def _paged(k, v, page, seed, spare=3):
    """k, v [S, Hkv, D] in pages in random order: (k_cache, v_cache, table [1, ld])."""
    S, Hkv, D = k.shape
    ld = -(-S // page)
    g = _gen(seed)
    kc, vc = (torch.full((ld + spare, page, Hkv, D), math.nan, dtype=k.dtype, device=DEV) for _ in range(2))
    table = torch.randperm(ld + spare, generator=g, device=DEV)[:ld]
    at = torch.arange(S, device=DEV)
    kc[table[at // page], at % page] = k
    vc[table[at // page], at % page] = v
    return kc, vc, table.to(torch.int32)[None]


def _tree1(q, k, v, page, seed):
    """One request whose last q.shape[1] keys are its chain of nodes."""
    kc, vc, table = _paged(k[0], v[0], page, seed)
    lens = torch.tensor([k.shape[1] - q.shape[1]], dtype=torch.int32, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    out, _ = rtopk.tree_attention(q, kc, vc, table, lens, lse=lse)
    torch.cuda.synchronize()
    return out.cpu().double(), lse.cpu().double()


# ------------------------------------------------------------------ weights far below the largest
def _leads(S, N):
    return (10, 0, 0), (14, 0, S // 2), (15.5, 0.5, 3), (17, 0, 0), (17, 0.5, S - N - 1), (18, 0, 1000)


def _lead_keys(S, D, lead, spread, at, dt, g):
    k = torch.zeros(1, S, 1, D, device=DEV, dtype=dt)
    k[..., 0] = (torch.randn(1, S, 1, generator=g, device=DEV) * spread * D ** 0.5).to(dt)
    k[0, at, 0, 0] = lead * D ** 0.5
    v = (2 + 4 * torch.rand(1, S, 1, D, generator=g, device=DEV)).to(dt)
    v[0, at] = 0.0
    return k, v


def _check_leads(out, lse, k, v, N, lead, dt, chain):
    """out [N, D], lse [N]. One key stands out by `lead` nats and its value is zero, so
    that the output is what all the others add up to.

    Tolerance, with A = sum_j w_j |v_j| = |o| here (values are positive): the
    output's and a weight's rounding, u (|o| + A); scores (exact but for the scale
    and the exponent's argument), float32: e = f (12 lead + 4), 2.1 e A; sums of S
    weights and S products, 2 S f A; float16 weights below 2^-25 of the largest
    are subnormal (2^11 is the largest), half a step of which is 2^-25 / 2^11 of the
    largest: 2^-36 sum |v| / sum of the weights; a float16 output below 2^-14, 2^-25.
    """
    S, D = k.shape[1], k.shape[3]
    x = (k[0, :, 0, 0].cpu().double() * D ** -0.5)[None].expand(N, S)
    if chain:
        x = torch.where(torch.arange(S)[None] <= S - N + torch.arange(N)[:, None], x, -math.inf)
    want_lse = torch.logsumexp(x, 1)
    w = torch.exp(x - want_lse[:, None])
    vd = v[0, :, 0].cpu().double()
    o = w @ vd
    e = F * (12 * lead + 4)
    sub = 2.0 ** -36 * w.amax(1)[:, None] * vd.sum(0) + 2.0 ** -25 if dt is F16 else 0.0
    bound = 2 * HALF[dt] * o * 1.01 + (2.1 * e + 2 * S * F) * o + sub
    off = ((out - o).abs() / bound).max()
    assert off <= 1, f"lead {lead}: {off:.3f} of the tolerance"
    assert ((lse - want_lse).abs() <= e + S * F + 4 * F * want_lse.abs()).all()


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("N,D,tree", [(N, D, tree) for N, D in ((1, 64), (20, 128), (40, 64), (70, 128), (40, 256))
                                      for tree in (False, True)] + [(300, 64, False)])
def test_small_weights(N, D, tree, dt):
    # one batch element: its keys are cut, and only the part with the heavy key has small weights
    S = 20001
    g = _gen(N + D)
    for lead, spread, at in _leads(S, N):
        print(f"[small weights] N={N} D={D} {dt} tree={tree} lead={lead} spread={spread} at={at}", flush=True)
        q = torch.zeros(1, N, 1, D, device=DEV, dtype=dt)
        q[..., 0] = 1.0
        k, v = _lead_keys(S, D, lead, spread, at, dt, g)
        out, lse = _tree1(q, k, v, 16, N) if tree else _cross(q, k, v)
        _check_leads(out[0, :, 0], lse[0, :, 0], k, v, N, lead, dt, tree)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("B,N,D", [(1040, 1, 64), (530, 20, 128), (520, 40, 64), (520, 70, 128), (140, 300, 64), (270, 5, 128)])
def test_small_weights_of_many_batch_elements(B, N, D, dt):
    # enough of them that their keys are not cut (the last: a share each, or cut); all read one encoder's states
    S = 6001
    g = _gen(N + D)
    for lead, spread, at in _leads(S, N):
        print(f"[small weights, many] B={B} N={N} D={D} {dt} lead={lead} spread={spread} at={at}", flush=True)
        q = torch.zeros(B, N, 1, D, device=DEV, dtype=dt)
        q[..., 0] = 1.0
        k, v = _lead_keys(S, D, lead, spread, at, dt, g)
        out, lse = _cross(q, k.expand(B, S, 1, D), v.expand(B, S, 1, D))
        for b in (0, B // 2, B - 1):
            _check_leads(out[b, :, 0], lse[b, :, 0], k, v, N, lead, dt, False)


def test_seen_infinities_spoil_their_column_only():
    """An infinite value that a row sees gives an infinity, or NaN where its weight
    rounds to zero; the other columns are as if it were not there."""
    for N in (1, 70):
        g = _gen(N)
        q = torch.zeros(1, N, 1, 64, device=DEV, dtype=F16)
        q[..., 0] = 1.0
        k, v = _rnd(g, 1, 500, 1, 64), _rnd(g, 1, 500, 1, 64)
        k[0, 7, 0, 0] = 40 * 8.0
        v[0, 100, 0, 3] = math.inf
        out, _ = _cross(q, k, v)
        keep = [d for d in range(64) if d != 3]
        assert not torch.isfinite(out[..., 3]).any()
        want = v[0, 7, 0].cpu().double()[keep]
        assert ((out[0, :, 0][:, keep] - want).abs() <= 2.02 * HALF[F16] * want.abs() + 1e-12).all()


# ------------------------------------------------------------------ every key counted once
def _whole(shape, seed, dt):
    return torch.randint(-8, 9, shape, generator=_gen(seed), device=DEV).to(dt)


def _check_means(out, lse, total, count, dt, what):
    """All scores are zero, so that weights are equal, and values are whole: the sums
    are exact, and an output is rounded by the reciprocal, the product, an
    exponential (together 4 f) and once to its type."""
    want = torch.where(count > 0, total / count.clamp(min=1), 0.0)
    assert ((out - want).abs() <= (HALF[dt] * 1.01 + 4 * F) * want.abs()).all(), what
    full = (count[..., 0] > 0).expand(lse.shape)
    wl = torch.log(count[..., 0].clamp(min=1)).expand(lse.shape)
    assert torch.equal(lse == -math.inf, ~full) and ((lse - wl).abs() <= 4 * F * wl + F)[full].all(), what


@pytest.mark.parametrize("N,D,dt", [(1, 64, F16), (1, 128, BF16), (20, 128, F16), (20, 64, BF16), (40, 64, F16), (70, 128, BF16),
                                    (300, 128, F16), (300, 64, BF16), (40, 256, BF16), (7, 80, F16)])
@pytest.mark.parametrize("masked", [False, True])
def test_cross_every_key_counts_once(N, D, dt, masked):
    B, S, H = 3, 40007, 1
    lens = [40007, 12345, 33]
    print(f"[cross counts] N={N} D={D} {dt} masked={masked}", flush=True)
    g = _gen(N)
    q, k, v = _rnd(g, B, N, H, D, dt=dt), _rnd(g, B, S, H, D, dt=dt), _whole((B, S, H, D), N + D, dt)
    mask = (torch.rand(B, S, generator=g, device=DEV) < 0.3) if masked else None
    out, lse = _cross(q, k, v, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), key_mask=mask, scale=0.0)
    ok = torch.arange(S)[None] < torch.tensor(lens)[:, None]
    if masked:
        ok &= ~mask.cpu()
    vd = torch.where(ok[:, :, None, None], v.cpu().double(), 0.0)
    _check_means(out, lse, vd.sum(1)[:, None], ok.sum(1).double()[:, None, None, None], dt, "cross")


@pytest.mark.parametrize("N,Hq,D,page,dt", [(1, 2, 64, 16, F16), (1, 16, 128, 64, BF16), (6, 4, 128, 16, F16), (1, 2, 64, 24, BF16),
                                            (1, 4, 128, 7, F16), (40, 2, 64, 16, F16), (70, 2, 128, 24, BF16), (33, 8, 128, 16, F16),
                                            (64, 8, 64, 5, BF16), (40, 2, 256, 16, F16)])
def test_tree_every_key_counts_once(N, Hq, D, page, dt):
    B, Hkv = 3, 2
    lens = [20011, 0, 7000]
    print(f"[tree counts] N={N} Hq={Hq} D={D} page={page} {dt}", flush=True)
    c = _tree_inputs(B, N, Hq, Hkv, D, page, lens, dt, seed=N + D, tree=N > 1)
    c["vc"].copy_(_whole(c["vc"].shape, 5, dt))
    lse = torch.full((B, N, Hq), 7.0, device=DEV)
    out, _ = rtopk.tree_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], parents=c["parents"], scale=0.0, lse=lse)
    torch.cuda.synchronize()
    out, lse, vd, tab = out.cpu().double(), lse.cpu().double(), c["vc"].cpu().double(), c["table"].cpu().long()
    for b, L in enumerate(lens):
        at = torch.arange(L + N)
        v = vd[tab[b, at // page], at % page]  # [L + N, Hkv, D]
        total, count = torch.zeros(N, Hkv, D, dtype=torch.float64), torch.zeros(N, dtype=torch.float64)
        for i in range(N):
            p = -1 if c["parents"] is None else int(c["parents"][b, i])
            total[i] = (total[p] if p >= 0 else v[:L].sum(0)) + v[L + i]
            count[i] = (count[p] if p >= 0 else L) + 1
        _check_means(out[b], lse[b], total.repeat_interleave(Hq // Hkv, 1), count[:, None, None], dt, f"tree b={b}")


# ------------------------------------------------------------------ rows that pick one key out of many
def _pick(S, n, seed):
    """n positions: the ends of the keys, ends of pieces of 8, 24, 32 and 64, any others."""
    g = torch.Generator().manual_seed(seed)
    edge = torch.randint(0, S // 64, (n,), generator=g) * 64
    off = torch.tensor([0, -1, 8, 23, 24, 31, 32, 63])[torch.randint(0, 8, (n,), generator=g)]
    p = torch.where(torch.rand(n, generator=g) < 0.7, edge + off, torch.randint(0, S, (n,), generator=g)).clamp(0, S - 1)
    p[0], p[-1] = S - 1, 0
    return p


def _signs(shape, seed, dt):
    return (torch.randint(0, 2, shape, generator=_gen(seed), device=DEV) * 2 - 1).to(dt)


def _check_picks(out, lse, v, at, D, dt, what):
    """A row is 8 times the signs of its key: that key's score is 8 sqrt(D), another's
    8 times a normal variable. The weights of the others sum up to less than 2^-13
    (asserted on the scores by the caller), which moves an output by less than 2^-13 of
    two values (at most 6 each); the rest is rounding: twice half a step."""
    want = v[at]
    assert ((out - want).abs() <= 2.02 * HALF[dt] * want.abs() + 2.0 ** -13 * 12).all(), what
    assert ((lse - 8 * D ** 0.5).abs() <= 2.0 ** -13 + F * 8 * D ** 0.5 * (D + 8)).all(), what


@pytest.mark.parametrize("N,D,dt", [(1, 64, F16), (32, 64, F16), (32, 128, BF16), (16, 128, F16), (64, 128, BF16), (100, 64, F16),
                                    (500, 64, BF16), (500, 128, F16), (60, 256, BF16)])
def test_cross_rows_pick_a_key(N, D, dt):
    S = 50021
    k, v = _signs((1, S, 1, D), D, dt), _rnd(_gen(D), 1, S, 1, D, dt=dt)
    kd, vd = k[0, :, 0].cpu().float(), v[0, :, 0].cpu().double()
    for rep in range(6 if N < 100 else 2):
        print(f"[cross picks] N={N} D={D} {dt} rep={rep}", flush=True)
        at = _pick(S, N, 100 * rep + D)
        q = (8 * k[0, at.to(DEV)])[None].contiguous()
        x = (8 * D ** -0.5) * (kd[at] @ kd.T)
        x[torch.arange(N), at] = -math.inf
        assert torch.logsumexp(x.double(), 1).max() < 8 * D ** 0.5 - math.log(2 ** 13)
        out, lse = _cross(q, k, v)
        _check_picks(out[0, :, 0], lse[0, :, 0], vd, at, D, dt, f"rep {rep}")


@pytest.mark.parametrize("N,G,D,page,dt", [(1, 32, 64, 16, F16), (1, 16, 128, 64, BF16), (2, 16, 128, 24, F16), (1, 32, 64, 5, BF16),
                                           (16, 4, 128, 16, BF16), (29, 4, 64, 24, F16), (64, 4, 128, 16, F16), (20, 2, 256, 16, F16)])
def test_tree_rows_pick_a_key(N, G, D, page, dt):
    S = 30011
    k, v = _signs((1, S, 1, D), D, dt), _rnd(_gen(D), 1, S, 1, D, dt=dt)
    kd, vd = k[0, :, 0].cpu().float(), v[0, :, 0].cpu().double()
    for rep in range(4):
        print(f"[tree picks] N={N} G={G} D={D} page={page} {dt} rep={rep}", flush=True)
        at = _pick(S - N, N * G, 100 * rep + D)  # before the tree
        x = (8 * D ** -0.5) * (kd[at] @ kd.T)
        x[torch.arange(N * G), at] = -math.inf
        assert torch.logsumexp(x.double(), 1).max() < 8 * D ** 0.5 - math.log(2 ** 13)
        q = (8 * k[0, at.to(DEV), 0]).view(1, N, G, D)
        out, lse = _tree1(q, k, v, page, rep)
        _check_picks(out[0].reshape(N * G, D), lse[0].reshape(-1), vd, at, D, dt, f"rep {rep}")


# ------------------------------------------------------------------ keys with NaN that some rows see
@pytest.mark.parametrize("N,dt,G", [(8, F16, 1), (8, BF16, 4), (70, F16, 2), (200, BF16, 1)])
def test_tree_nan_keys_reach_the_rows_that_see_them(N, dt, G):
    c = _tree_inputs(2, N, 2 * G, 2, 64, 16, [40, 61], dt, seed=N + 1)
    i = torch.arange(1, N, device=DEV)
    c["parents"][:, 1:] = torch.where(i % 2 == 0, i - 2, -1).to(torch.int32)  # even nodes below node 0, odd ones alone
    node3 = [(int(c["table"][b, (L + 3) // 16]), (L + 3) % 16) for b, L in ((0, 40), (1, 61))]
    clean, clean_lse = _tree(c, "without NaN")
    kept = c["kc"].clone()
    for at in node3:
        c["kc"][at] = math.nan
    out, lse = torch.full_like(c["q"], 3.0), torch.full((2, N, 2 * G), 5.0, device=DEV)
    rtopk.tree_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], parents=c["parents"], out=out, lse=lse)
    torch.cuda.synchronize()
    assert torch.isnan(out[:, 3].float()).all() and torch.isnan(lse[:, 3]).all()
    out[:, 3], lse[:, 3] = clean[:, 3], clean_lse[:, 3]  # every other row as if the key were any
    check_tree(c["q"], kept, c["vc"], c["table"], [40, 61], c["parents"], None, 64 ** -0.5, out, lse, "NaN keys")


# ------------------------------------------------------------------ scores near the largest floats
@pytest.mark.parametrize("dt,top", [(F16, 2.0 ** 15), (BF16, 2.0 ** 15), (BF16, 2.0 ** 20), (BF16, 2.0 ** 55)])
@pytest.mark.parametrize("N", [1, 20, 40, 70, 300])
def test_far_scores(dt, top, N):
    """Scores from 2^30 to beyond 2^110, where a float32 has no bits left for
    differences of a few nats: one key wins by a large factor (two share it where
    they are equal), and the output is its value, rounded as a weight and once."""
    D, S = 64, 300
    print(f"[far scores] {dt} top={top} N={N}", flush=True)
    g = _gen(N)
    v = _rnd(g, 1, S, 1, D, dt=dt)
    vd = v[0, :, 0].cpu().double()
    for sign in (1.0, -1.0):
        for scale in (0.125, 0.1, -0.3):
            for first in (5, 250):
                # the winner's size times 1.5 where the score is positive, times 1/4 where negative
                wins = sign * scale > 0
                size = torch.full((S,), 0.75, device=DEV) - 0.25 * torch.rand(S, generator=g, device=DEV)
                size[first] = 1.5 if wins else 0.25
                size[first + 1] = size[first] if first == 250 else size[first + 1]
                k = (sign * size * top)[None, :, None, None].expand(1, S, 1, D).to(dt).contiguous()
                q = torch.full((1, N, 1, D), top, device=DEV).to(dt)
                out, lse = _cross(q, k, v, scale=scale)
                x = k[0, :, 0, 0].cpu().double() * q[0, 0, 0, 0].item() * D * scale
                want = vd[[first, first + 1]].mean(0) if first == 250 else vd[first]
                mag = vd[[first, first + 1]].abs().mean(0) if first == 250 else vd[first].abs()
                what = f"sign {sign} scale {scale} first {first}"
                assert int(x.argmax()) in (first, first + 1), what
                assert ((out[0, :, 0] - want).abs() <= 2.02 * HALF[dt] * mag).all(), what
                assert ((lse[0, :, 0] - x.max()).abs() <= F * (D + 8) * x.max().abs()).all(), what


# ------------------------------------------------------------------ more tokens than a launch has workgroups
def test_store_of_2_to_the_24_tokens():
    # overlapping rows of 4 x 257 elements, so that every token differs; few of them have a slot
    T, H, D, page, pages = (1 << 24) + 5, 4, 257, 16, 6
    g = _gen(3)
    buf = _rnd(g, T + H * D + 7)
    k = torch.as_strided(buf, (T, H, D), (1, D, 1))
    v = torch.as_strided(buf, (T, H, D), (1, D, 1), 7)
    slots = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    at = torch.cat([torch.tensor([0, 1, T - 1, T - 2, T // 2, (1 << 24) - 1, 1 << 24], device=DEV),
                    torch.randint(2, T // 2, (60,), generator=g, device=DEV).unique()])
    slots[at] = torch.randperm(pages * page, generator=g, device=DEV)[:at.numel()].to(torch.int32)
    kc, vc = torch.full((pages, page, H, D), 3.0, dtype=F16, device=DEV), torch.full((pages, page, H, D), 4.0, dtype=F16, device=DEV)
    wk, wv = kc.clone().view(-1, H, D), vc.clone().view(-1, H, D)
    wk[slots[at].long()], wv[slots[at].long()] = k[at], v[at]
    print("[store] 2^24 tokens", flush=True)
    rtopk.cache_store(k, v, slots, kc, vc)
    torch.cuda.synchronize()
    assert torch.equal(kc.view(-1, H, D), wk) and torch.equal(vc.view(-1, H, D), wv)


# ------------------------------------------------------------------ library workspaces
def test_a_captured_step_keeps_its_library_workspace():
    """A selection step captured on its stream's library-owned workspace, then
    attention calls on that stream which need ever more workspace, memory that is
    allocated and overwritten between replays: every replay as the eager step."""
    g = _gen(9)
    B, beam, V, H = 16, 4, 6000, 256
    hid, w = _rnd(g, B * beam, H, dt=BF16), _rnd(g, V, H, dt=BF16)
    alive = torch.randn(B, beam, generator=g, device=DEV)
    want = [o.clone() for o in rtopk.lmhead_step(hid, w, alive, None, k=4)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        rtopk.lmhead_step(hid, w, alive, None, k=4)  # the workspace exists before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = rtopk.lmhead_step(hid, w, alive, None, k=4)
    q, k = _rnd(g, 2, 32, 8, 128), _rnd(g, 2, 40000, 8, 128)
    first = rtopk.cross_attention(q, k, k)[0]
    torch.cuda.synchronize()
    for rep in range(4):
        n = 8 * (rep + 1)
        with torch.cuda.stream(s):
            out = rtopk.cross_attention(q[:, :n].contiguous(), k, k)[0]
            junk = torch.full((1 << 24,), math.nan, device=DEV)
        for o in got:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), rep
        del junk
    assert torch.equal(out, first)
