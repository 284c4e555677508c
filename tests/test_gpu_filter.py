"""Filtered sampling on the GPU against its definition in 64 bits
(serve_ref.sample): the same tokens, and their log-probabilities.

A token may differ where a running sum comes within the sums' error of a border: the
kernel's weights are off by 2^-44 of the largest at V = 250000 (2^-48 below 4096), a
sum of n of them by 2^-44 sqrt(n), which is under 2^-35 of the sum; with a border every
2^-18 of it that is one row in 2^17 for flat rows and far fewer for others. The inputs are
fixed. Log-probabilities are rounded once, and log(w / S) is off by at most 2^-24 in absolute terms for
weights over 2^-20 of the largest: tolerance 2^-24 (|log p| + 1) for the rounding, 2^-20 besides.
"""
import math

import numpy as np
import pytest
import torch

from beam_search_top_amd import rtopk
from libutil import ensure_built
from serve_ref import sample

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_built()


def _check(x, u, what, **f):
    d = lambda a, dt: None if a is None else torch.tensor(a, dtype=dt, device=DEV)  # noqa: E731
    R = x.shape[0]
    for n in f:
        if np.isscalar(f[n]):
            f[n] = [f[n]] * R
    u = np.asarray(u, dtype=np.float32)
    tok, lp = rtopk.sample_filtered(x, d(u, F32), temperature=d(f.get("t"), F32), top_k=d(f.get("k"), torch.int32),
                                    top_p=d(f.get("p"), F32), min_p=d(f.get("m"), F32))
    torch.cuda.synchronize()
    xs, tok, lp = x.double().cpu().numpy(), tok.tolist(), lp.tolist()
    f32 = lambda n, r, other: float(np.float32(f[n][r])) if n in f else other  # noqa: E731
    for r in range(R):
        want, wlp = sample(xs[r], float(u[r]), f32("t", r, 1.0), f["k"][r] if "k" in f else 0, f32("p", r, 1.0), f32("m", r, 0.0))
        assert tok[r] == want, f"{what} row {r}: token {tok[r]}, not {want}"
        assert lp[r] == wlp or abs(lp[r] - wlp) <= 2.0 ** -24 * (abs(wlp) + 1) + 2.0 ** -20, (what, r, lp[r], wlp)
    return tok, lp


def _rows(R, V, dt, seed, sigma=3.0, ld=None):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(R, ld or V, generator=g, device=DEV) * sigma).to(dt)[:, :V], np.random.default_rng(seed)


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("R,V,ld", [(1, 1, 1), (3, 2, 2), (5, 7, 9), (4, 63, 63), (4, 64, 64), (3, 65, 65), (2, 1000, 1001), (6, 8191, 8191),
                                    (3, 32000, 32000), (2, 40000, 40064), (1, 250000, 250000), (33, 129, 131)])
def test_sizes(R, V, ld, dt):
    print(f"[filter] R={R} V={V} ld={ld} {dt}", flush=True)
    x, rng = _rows(R, V, dt, seed=V + R, ld=ld)
    u = rng.random(R)
    _check(x, u, "none")
    _check(x, u, "temperature", t=[0.7, 1.3, 0.0, 1.0, 2.5][:R] + [0.9] * (R - 5))
    _check(x, u, "k", k=list(rng.integers(0, min(V, 300) + 2, R)))
    _check(x, u, "p", p=list(rng.choice([0.1, 0.5, 0.9, 0.99, 1.0], R)))
    _check(x, u, "m", m=list(rng.choice([0.0, 0.02, 0.3, 1.0], R)))
    _check(x, u, "all", t=list(rng.choice([0.6, 1.0, 1.4], R)), k=list(rng.integers(1, V + 1, R)), p=list(rng.choice([0.5, 0.9, 0.95], R)),
           m=list(rng.choice([0.0, 0.05], R)))


@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_many_draws_of_one_row(dt):
    # the whole distribution: equal steps of u meet every kept token in its order
    x, _ = _rows(1, 500, dt, seed=3, sigma=1.0)
    n = 256
    u = (np.arange(n) + 0.5) / n
    rows = x.expand(n, 500).contiguous()
    for kw in (dict(), dict(k=40), dict(p=0.7), dict(m=0.2), dict(k=100, p=0.8, m=0.05, t=0.8)):
        tok, _ = _check(rows, u, str(kw), **kw)
        assert tok == sorted(tok)  # in the order of tokens


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("V", [10, 4096, 40000])
def test_ties(V, dt):
    # equal logits: the lower tokens are kept; sums of equal weights are exact
    x = torch.zeros(8, V, dtype=dt, device=DEV)
    u = [0.0, 0.25, 0.5, 0.75, 0.999, 0.1, 0.3, 0.6]
    _check(x, u, "flat")
    tok, lp = _check(x, u, "flat k", k=5)
    assert max(tok) <= 4 and abs(lp[0] + math.log(5)) < 1e-6
    tok, _ = _check(x, u, "flat p", p=0.5)
    assert max(tok) < V // 2
    x[:, V // 2:] = 1.0
    _check(x, u, "two values, k in the lower", k=V // 2 + 3)
    _check(x, u, "two values, k in the upper", k=2)
    _check(x, u, "two values, p", p=0.75)
    x[:, 0::2] = -0.0
    x[:, 1::2] = 0.0
    tok, _ = _check(x, u, "signed zeros", k=3)  # one value
    assert max(tok) <= 2


@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_infinities_and_nan(dt):
    x, rng = _rows(8, 3001, dt, seed=5)
    u = rng.random(8)
    inf, nan = float("inf"), float("nan")
    x[0] = -inf
    x[1, ::2] = -inf
    x[2, 5:] = -inf
    x[3] = -inf
    x[3, 1234] = -7.0
    x[4] = nan
    x[5, ::3] = nan
    x[6, 17] = x[6, 2000] = inf
    x[7] = torch.finfo(dt).min
    for kw in (dict(), dict(k=50), dict(p=0.9), dict(m=0.1), dict(k=20, p=0.5, m=0.01), dict(t=0.0), dict(k=2000, p=0.99)):
        tok, lp = _check(x, u, str(kw), **dict(kw))
        assert tok[0] == tok[4] == -1 and lp[0] == lp[4] == -inf and tok[3] == 1234 and lp[3] == 0


def test_values_of_the_filters():
    x, rng = _rows(12, 5000, F32, seed=6, sigma=2.0)
    u = rng.random(12)
    inf, nan = float("inf"), float("nan")
    _check(x, u, "p", p=[0.0, -1.0, 1.0, 2.0, nan, inf, 1e-30, 0.999999, 0.5, 0.25, 1 - 2.0 ** -24, 0.9])
    _check(x, u, "m", m=[0.0, -1.0, 1.0, 2.0, nan, inf, 1e-30, 0.999, 0.5, 0.25, 1e-6, 0.9])
    _check(x, u, "k", k=[0, -1, 1, 2, 4999, 5000, 5001, 2 ** 31 - 1, -2 ** 31, 64, 65, 2048])
    _check(x, u, "t", t=[0.0, -1.0, nan, -inf, 1e-30, 1e-6, 0.01, 100.0, 1e6, 1e30, 0.5, 1.0])
    tok, _ = _check(x, [0.0, -1.0, 1.0, 2.0, nan, inf, 1 - 2.0 ** -24, 1e-30, -inf, 0.5, 0.1, 0.9], "u", k=30)
    far = torch.cat((x[:6], x[:6] * 1e4, x[:6] - 1e30, x[:6] * 1e37)).contiguous()
    _check(far, rng.random(24), "large", k=100)
    _check(far, rng.random(24), "large", p=0.8, t=3.0)


def test_unaligned_rows_and_out():
    x, rng = _rows(5, 777, BF16, seed=7)
    u = torch.tensor(rng.random(5), dtype=F32, device=DEV)
    p = torch.full((5,), 0.8, device=DEV)
    want = rtopk.sample_filtered(x, u, top_p=p)
    for shift in range(1, 8):
        y = torch.full((5 * 779 + 16,), float("inf"), dtype=BF16, device=DEV)  # what lies around the rows is not read as logits
        z = torch.as_strided(y, (5, 777), (779, 1), shift)
        z.copy_(x)
        out = (torch.zeros(5, dtype=torch.int32, device=DEV), torch.zeros(5, device=DEV))
        got = rtopk.sample_filtered(z, u, top_p=p, out=out)
        torch.cuda.synchronize()
        assert got[0] is out[0] and torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), shift


def test_repeats_streams_and_a_graph():
    x, rng = _rows(40, 20000, F16, seed=8)
    u = torch.tensor(rng.random(40), dtype=F32, device=DEV)
    kw = dict(top_k=torch.full((40,), 900, dtype=torch.int32, device=DEV), top_p=torch.full((40,), 0.93, device=DEV))
    want = rtopk.sample_filtered(x, u, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            b = rtopk.sample_filtered(x, u, **kw)
        a = rtopk.sample_filtered(x, u, **kw)  # both at once
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for got in (a, b) for g, w in zip(got, want))
    out = (torch.zeros(40, dtype=torch.int32, device=DEV), torch.zeros(40, device=DEV))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rtopk.sample_filtered(x, u, out=out, **kw)
    for i in range(3):
        u.copy_(torch.tensor(rng.random(40)))
        x.neg_()
        graph.replay()
        torch.cuda.synchronize()
        eager = rtopk.sample_filtered(x, u, **kw)
        assert torch.equal(out[0], eager[0]) and torch.equal(out[1], eager[1]), i


def test_agrees_with_the_top_k_step():
    # the same distribution as rtopk_sample_step's: log-probabilities of tokens that both can draw
    x, rng = _rows(64, 40000, F16, seed=9)
    lists = rtopk.beam_step(x.view(64, 1, 40000), torch.zeros(64, 1, device=DEV), k=40)
    u = torch.tensor(rng.random(64), dtype=F32, device=DEV)
    tok, lp = rtopk.sample_filtered(x, u, top_k=torch.full((64,), 40, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    p = torch.log_softmax(lists[2], 1)
    for r in range(64):
        at = (lists[1][r] == tok[r]).nonzero()
        assert at.numel() == 1 and abs(float(p[r, at[0, 0]]) - float(lp[r])) < 1e-4


def _both_forms(x, u, what, oracle=True, **f):
    """Few long rows are cut over workgroups, but not in a captured call without a workspace: all give the same."""
    R = x.shape[0]
    d = lambda a, dt: None if a is None else torch.tensor([a] * R if np.isscalar(a) else a, dtype=dt, device=DEV)  # noqa: E731
    ud = torch.tensor(np.asarray(u, dtype=np.float32), device=DEV)
    kw = dict(temperature=d(f.get("t"), F32), top_k=d(f.get("k"), torch.int32), top_p=d(f.get("p"), F32), min_p=d(f.get("m"), F32))
    out = (torch.zeros(R, dtype=torch.int32, device=DEV), torch.zeros(R, device=DEV))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rtopk.sample_filtered(x, ud, out=out, **kw)
    cut = (torch.zeros(R, dtype=torch.int32, device=DEV), torch.zeros(R, device=DEV))
    ws = torch.full((rtopk.rtopk_sample_filtered_workspace_bytes(*x.shape),), 0xa5, dtype=torch.uint8, device=DEV)
    given = torch.cuda.CUDAGraph()
    with torch.cuda.graph(given):
        rtopk.sample_filtered(x, ud, out=cut, workspace=ws, **kw)
    eager = rtopk.sample_filtered(x, ud, **kw)
    graph.replay()
    given.replay()
    torch.cuda.synchronize()
    one, other, third = [[t.tolist() for t in pair] for pair in (out, eager, cut)]
    assert one == other == third, what
    return _check(x, u, what, **f) if oracle else tuple(other)


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("R,V,ld,shift", [(1, 28672, 28672, 0), (1, 28671, 28671, 0), (3, 40001, 40003, 3), (2, 100003, 100004, 1), (2, 250000, 250000, 0),
                                          (1, 270007, 270007, 7)])
def test_rows_cut_over_workgroups(R, V, ld, shift, dt):
    print(f"[filter cut] R={R} V={V} ld={ld} {dt}", flush=True)
    y, rng = _rows(1, (R - 1) * ld + V + shift, dt, seed=V + R, sigma=2.0)
    x = torch.as_strided(y, (R, V), (ld, 1), shift)
    for what, kw in dict(none={}, t=dict(t=0.8), k=dict(k=64), m=dict(m=0.01), p=dict(p=0.95), wide=dict(p=0.999), all=dict(t=0.9, k=900, p=0.9, m=0.001),
                         many=dict(k=V - 5, p=0.9999), greedy=dict(t=0.0)).items():
        _both_forms(x, rng.random(R), what, **kw)
    # equal logits: a draw lands on token floor(u V), in the first and the last run of the row too
    flat = torch.as_strided(torch.zeros_like(y), (R, V), (ld, 1), shift)
    for n in (0, 1, V // 2, V - 40, V - 9, V - 2, V - 1):
        tok, _ = _both_forms(flat, [(n + 0.5) / V] * R, f"flat {n}", oracle=False)
        assert tok == [n] * R  # u is rounded by 2^-25 at most, V 2^-25 of a token


@pytest.mark.parametrize("R,V", [(128, 28672), (129, 28672), (64, 33000), (300, 1000)])
def test_numbers_of_rows(R, V):
    x, rng = _rows(R, V, BF16, seed=R)
    u = rng.random(R)
    for kw in (dict(p=0.9), dict(k=50, p=0.95, m=0.02, t=0.9), dict()):
        tok, lp = _both_forms(x, u, str(kw), oracle=False, **kw)
        some = [0, 1, R // 2, R - 1]
        assert _check(x[some].contiguous(), u[some], str(kw), **kw) == ([tok[r] for r in some], [lp[r] for r in some])


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("V", [9000, 40000])
def test_many_equal_and_many_kept(V, dt):
    # borders among more equal logits, and kept sets of more, than a workgroup holds
    rng = np.random.default_rng(V)
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5], device=DEV)
    at = torch.tensor(rng.integers(0, 4, (6, V)), device=DEV)
    x = levels[at].to(dt)
    u = rng.random(6)
    n = int((at[0] == 3).sum())
    for kw in (dict(k=n - 1), dict(k=n), dict(k=n + 1), dict(k=V - 7), dict(p=0.3), dict(p=0.77), dict(k=2 * n, p=0.8), dict(k=n // 2, p=0.5, m=0.3),
               dict(m=0.5), dict(p=1e-6), dict(p=0.999999)):
        _both_forms(x, u, str(kw), **kw)
    near = (torch.tensor(rng.random((6, V)), device=DEV) * 0.01).to(dt)
    for kw in (dict(p=0.9), dict(k=V // 2), dict(k=V // 2, p=0.9), dict(m=0.995), dict(p=0.9, m=0.995)):
        _both_forms(near, u, "near " + str(kw), **kw)
    x[:, 1:] = float("-inf")
    for kw in (dict(p=0.5), dict(k=3), dict(k=3, p=0.1, m=0.2)):
        tok, lp = _both_forms(x, u, "one " + str(kw), **kw)
        assert tok == [0] * 6 and lp == [0.0] * 6


def test_long_rows_on_two_streams():
    x, rng = _rows(4, 150000, F16, seed=21)
    y, _ = _rows(6, 90000, F16, seed=22)
    u = torch.tensor(rng.random(6), dtype=F32, device=DEV)
    p = torch.full((6,), 0.97, device=DEV)
    call = lambda z: rtopk.sample_filtered(z, u[:z.shape[0]], top_p=p[:z.shape[0]])  # noqa: E731
    want = call(x), call(y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = []
        for s, z in zip(streams, (x, y)):
            with torch.cuda.stream(s):
                got.append([call(z) for _ in range(5)])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for one in g for a, b in zip(one, w))


def test_odd_temperatures():
    x, rng = _rows(6, 31000, F32, seed=23, sigma=2.0)
    u = rng.random(6)
    inf = float("inf")
    _both_forms(x, u, "t", t=[inf, 1e-40, 1e38, 2.0 ** -126, 3e-39, 0.3])
    _both_forms(x, u, "t p", t=[1e-40, 1e-20, 1e38, 5.0, 1e-3, 0.3], p=0.9)
    _both_forms(x, u, "t k", t=[inf, 1e-20, 1e38, 5.0, 1e-3, 0.3], k=700)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_the_longest_row(dt):
    # equal logits, u a whole number of 1 / V: exactly token u V, and of the lower half with p = 1/2
    V = 1 << 24
    x = torch.zeros(1, V, dtype=dt, device=DEV)
    for n in (0, 1, 12345679, V - 2, V - 1):
        assert _both_forms(x, [n / V], str(n), oracle=False)[0] == [n]
        tok, lp = _both_forms(x, [n / V], str(n), oracle=False, p=0.5)
        assert tok == [n // 2] and abs(lp[0] + 23 * math.log(2)) < 1e-5
    assert _both_forms(x, [0.75], "k", oracle=False, k=V - 4)[0] == [V // 4 * 3 - 3]
    x[0, V - 3] = 1.0
    assert _both_forms(x, [0.99], "greedy", oracle=False, t=0.0)[0] == [V - 3]


def test_the_most_rows_and_far_ones():
    R = 1 << 20
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    u = torch.rand(R, generator=g, device=DEV)
    tok, lp = rtopk.sample_filtered(torch.zeros(R, 2, dtype=F16, device=DEV), u)
    torch.cuda.synchronize()
    assert torch.equal(tok, (u >= 0.5).int()) and ((lp + math.log(2)).abs() < 1e-6).all()
    far = torch.zeros((1 << 31) + 30008, dtype=F16, device=DEV)  # the second row's offset passes 32 bits
    x = torch.as_strided(far, (2, 30000), (1 << 31, 1))
    x.copy_(_rows(2, 30000, F16, seed=31)[0])
    for kw in (dict(k=30, p=0.9), dict(p=0.99), dict()):
        assert _both_forms(x, [0.3, 0.8], "far", oracle=False, **kw) == _check(x.contiguous(), [0.3, 0.8], "near", **kw)


@pytest.mark.parametrize("n", [2, 63, 64, 65, 130, 511, 512, 513, 700, 1023, 1024, 1025, 1500])
def test_borders_in_a_cluster(n):
    # n distinct logits in one of the bins that a row is cut into: their order decides
    rng = np.random.default_rng(n)
    for V in (6000, 30000):
        x = (-5 - 15 * rng.random((3, V))).astype(np.float32)
        for r in range(3):
            at = rng.permutation(V)[:n + 2]
            x[r, at] = 1 + np.arange(n + 2, dtype=np.float32) * np.float32(2.0 ** -22)
            x[r, at[0]], x[r, at[1]] = 3.0, -40.0
        x = torch.tensor(x, device=DEV)
        u = rng.random(3)
        for kw in (dict(k=1 + n // 3), dict(k=n), dict(k=1 + n), dict(p=0.31), dict(p=0.9), dict(k=1 + n // 2, p=0.77), dict(k=n, p=0.5, m=0.1)):
            _both_forms(x, u, f"{V} {kw}", **kw)


def test_replays_with_a_workspace():
    # two captured calls that share one workspace, in order, over inputs that change
    x, rng = _rows(5, 60000, BF16, seed=41)
    y, _ = _rows(3, 100000, F16, seed=42)
    u = torch.tensor(rng.random(5), dtype=F32, device=DEV)
    p = torch.full((5,), 0.9, device=DEV)
    n = max(rtopk.rtopk_sample_filtered_workspace_bytes(*z.shape) for z in (x, y))
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    outs = [(torch.zeros(len(z), dtype=torch.int32, device=DEV), torch.zeros(len(z), device=DEV)) for z in (x, y)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for z, o in zip((x, y), outs):
            rtopk.sample_filtered(z, u[:len(z)], top_p=p[:len(z)], out=o, workspace=ws)
    for i in range(4):
        u.copy_(torch.tensor(rng.random(5)))
        x.neg_()
        y.mul_(0.8)
        graph.replay()
        torch.cuda.synchronize()
        for z, o in zip((x, y), outs):
            want = rtopk.sample_filtered(z, u[:len(z)], top_p=p[:len(z)])
            assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1]), i
    with pytest.raises(rtopk.RtopkError):
        rtopk.sample_filtered(x, u, workspace=ws[:1000])
    with pytest.raises(ValueError):
        rtopk.sample_filtered(x, u, workspace=ws.view(torch.int8))
    with pytest.raises(ValueError):
        rtopk.sample_filtered(x, u, workspace=torch.empty(n, dtype=torch.uint8))
