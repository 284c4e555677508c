"""Norms and rotation of queries and keys on the GPU against a plain 64-bit
reference (serve_ref.py, which derives the tolerances)."""
import pytest
import torch

from beam_search_top_amd import rtopk
from libutil import ensure_built
from serve_ref import rope

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_built()


def _inputs(T, Hq, Hkv, D, rot, dt, norm, seed, far=5000):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV).to(dt)
    pos = torch.randint(0, far, (T,), generator=g, device=DEV).to(torch.int32)
    freqs = (10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / max(rot, 1))).float()
    w = (1 + 0.3 * torch.randn(2, D, generator=g, device=DEV)).to(dt) if norm else (None, None)
    return x[:, :Hq], x[:, Hq:Hq + Hkv], pos, freqs, w[0], w[1]


def _check(got, x, w, pos, freqs, pairs, what, eps=1e-6):
    y, tol = rope(x.cpu(), None if w is None else w.cpu(), pos.cpu(), freqs.cpu(), eps, pairs)
    off = (got.cpu().double() - y).abs() / tol
    live = pos.cpu() >= 0
    assert off[live].numel() == 0 or off[live].max() <= 1, f"{what}: {off[live].max():.3f} of the tolerance"


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,dt,norm", [
    (1, 1, 1, 64, 64, F16, True), (37, 16, 16, 64, 64, F16, True), (5, 32, 8, 128, 128, BF16, True), (9, 20, 4, 80, 80, BF16, False),
    (3, 5, 1, 96, 32, F16, True), (300, 4, 2, 256, 128, BF16, True), (7, 3, 3, 192, 192, F32, True), (4, 2, 1, 256, 256, F32, True),
    (6, 4, 2, 32, 16, F32, True), (11, 3, 1, 40, 20, F16, True), (11, 2, 2, 7, 6, BF16, True), (5, 1, 1, 1, 0, F32, True),
    (5, 2, 1, 64, 0, F16, True), (8, 2, 1, 250, 250, F32, False), (13, 1, 2, 2, 2, F16, True), (1025, 2, 1, 16, 16, BF16, True),
])
def test_rope(T, Hq, Hkv, D, rot, dt, norm, pairs):
    print(f"[rope] T={T} {Hq}/{Hkv} x {D}, rot {rot} {dt} norm={norm} pairs={pairs}", flush=True)
    q, k, pos, freqs, qw, kw = _inputs(T, Hq, Hkv, D, rot, dt, norm, seed=T + D)
    qo, ko = rtopk.qk_norm_rope(q, k, pos, freqs, q_weight=qw, k_weight=kw, interleaved=pairs)
    torch.cuda.synchronize()
    _check(qo, q, qw, pos, freqs, pairs, "q")
    _check(ko, k, kw, pos, freqs, pairs, "k")


def test_far_positions():
    q, k, pos, freqs, _, _ = _inputs(64, 2, 1, 64, 64, F32, False, seed=1, far=2 ** 31 - 1)
    pos[0], pos[1] = 2 ** 31 - 1, 0
    qo, ko = rtopk.qk_norm_rope(q, k, pos, freqs)
    torch.cuda.synchronize()
    _check(qo, q, None, pos, freqs, False, "q")
    assert torch.equal(ko[1], k[1])  # position 0 turns nothing


@pytest.mark.parametrize("D,dt", [(64, F16), (20, BF16)])
def test_skipped_tokens_keep_their_rows(D, dt):
    q, k, pos, freqs, qw, kw = _inputs(50, 4, 2, D, D, dt, True, seed=2)
    pos[::3] = -1
    pos[4] = -2 ** 31
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 9.0)
    got = rtopk.qk_norm_rope(q, k, pos, freqs, q_weight=qw, k_weight=kw, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    assert got[0] is qo and got[1] is ko
    skip = pos < 0
    assert (qo[skip] == 7).all() and (ko[skip] == 9).all()
    _check(qo, q, qw, pos, freqs, False, "q")
    _check(ko, k, kw, pos, freqs, False, "k")
    fresh = rtopk.qk_norm_rope(q, k, pos, freqs, q_weight=qw, k_weight=kw)
    assert (fresh[0][skip] == 0).all() and torch.equal(fresh[0][~skip], qo[~skip])


@pytest.mark.parametrize("D,dt,pairs", [(128, BF16, False), (64, F16, True), (6, F32, False)])
def test_in_place_in_a_packed_projection(D, dt, pairs):
    q, k, pos, freqs, qw, kw = _inputs(33, 6, 2, D, D, dt, True, seed=3)
    whole = q._base if q._base is not None else q
    before = whole.clone()
    want = rtopk.qk_norm_rope(q.clone(), k.clone(), pos, freqs, q_weight=qw, k_weight=kw, interleaved=pairs)
    got = rtopk.qk_norm_rope(q, k, pos, freqs, q_weight=qw, k_weight=kw, interleaved=pairs, q_out=q, k_out=k)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(whole[:, 8:], before[:, 8:])  # the values beside them


def test_layouts_and_alignments_agree():
    # heads before tokens, rows two bytes off a boundary, [B, N] tokens, a broadcast key
    q, k, pos, freqs, qw, kw = _inputs(24, 4, 2, 64, 64, F16, True, seed=4)
    q, k = q.contiguous(), k.contiguous()
    want = rtopk.qk_norm_rope(q, k, pos, freqs, q_weight=qw, k_weight=kw)
    qt, kt = q.transpose(0, 1).contiguous().transpose(0, 1), k.transpose(0, 1).contiguous().transpose(0, 1)
    ot = torch.empty(4, 24, 64, dtype=F16, device=DEV).transpose(0, 1)
    got = rtopk.qk_norm_rope(qt, kt, pos, freqs, q_weight=qw, k_weight=kw, q_out=ot)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    off = torch.empty(24 * 4 * 64 + 1, dtype=F16, device=DEV)[1:].view(24, 4, 64)
    off.copy_(q)
    got = rtopk.qk_norm_rope(off, k, pos, freqs, q_weight=qw, k_weight=kw)
    tol = rope(q.cpu(), qw.cpu(), pos.cpu(), freqs.cpu(), 1e-6, False)[1]
    assert ((got[0] - want[0]).cpu().double().abs() <= 2 * tol).all()  # sums in another order
    got = rtopk.qk_norm_rope(q.view(3, 8, 4, 64), k.view(3, 8, 2, 64), pos.view(3, 8), freqs, q_weight=qw, k_weight=kw)
    assert got[0].shape == (3, 8, 4, 64) and torch.equal(got[0].view(24, 4, 64), want[0])
    kb = k[:1].expand(24, 2, 64)
    got = rtopk.qk_norm_rope(q, kb, pos, freqs, q_weight=qw, k_weight=kw)
    torch.cuda.synchronize()
    _check(got[1], kb, kw, pos, freqs, False, "broadcast k")


def test_norm_of_one_alone_zeros_and_infinities():
    q, k, pos, freqs, qw, kw = _inputs(8, 2, 2, 64, 64, BF16, True, seed=5)
    q, k = q.clone(), k.clone()
    q[0] = 0
    k[1, 0, 3] = float("inf")
    k[2, 1, 5] = float("nan")
    qo, ko = rtopk.qk_norm_rope(q, k, pos, freqs, q_weight=qw, eps=0.5)
    torch.cuda.synchronize()
    assert (qo[0] == 0).all()
    _check(qo, q, qw, pos, freqs, False, "q", eps=0.5)
    # without a norm a bad element stays with its pair, and with its head
    bad = ~torch.isfinite(ko)
    assert set(bad[1, 0].nonzero().flatten().tolist()) <= {3, 35} and bad[1, 0].any() and not bad[1, 1].any()
    assert bad[2, 1].nonzero().flatten().tolist() == [5, 37] and not bad[2, 0].any() and not bad[3:].any()


def test_two_streams_and_a_graph():
    q, k, pos, freqs, qw, kw = _inputs(64, 8, 2, 128, 128, BF16, True, seed=6)
    want = rtopk.qk_norm_rope(q, k, pos, freqs, q_weight=qw, k_weight=kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = rtopk.qk_norm_rope(q, k, pos, freqs, q_weight=qw, k_weight=kw)
    torch.cuda.synchronize()
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    qo, ko = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rtopk.qk_norm_rope(q, k, pos, freqs, q_weight=qw, k_weight=kw, q_out=qo, k_out=ko)
    for i in range(3):
        qo.zero_(), ko.zero_()
        pos.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        eager = rtopk.qk_norm_rope(q, k, pos, freqs, q_weight=qw, k_weight=kw)
        assert torch.equal(qo, eager[0]) and torch.equal(ko, eager[1]), i
