"""Attention outputs where a lost weight or an extreme score shows. References in
64 bits."""
import math

import pytest
import torch

from beam_search_top_amd import rtopk
from test_gpu_layer import DEV, _gen, _rnd, lib  # noqa: F401

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
