"""Values at the ends of what the rotation, the 8-bit cache and filtered sampling
accept, on the GPU: against their definitions in 64 bits (serve_ref.py), in every form of their kernels."""
import math

import numpy as np
import pytest
import torch

from beam_search_top_amd import rtopk
from libutil import ensure_built
from serve_ref import CODES, rope
from test_gpu_filter import _both_forms, _check, _rows

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_built()


# ------------------------------------------------------------------ filtered sampling
@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("V", [2, 3001, 31000])
def test_infinite_logits_whatever_the_temperature(V, dt):
    # an infinite logit weighs 1 and the others 0, also where (x - max) / T is small: the kernel's
    # stand-in for infinity is a number
    x, rng = _rows(6, V, dt, seed=V, sigma=2.0)
    x[:, V - 1] = INF
    x[1::2, 0] = INF
    x[2] = torch.finfo(dt).max / 2
    x[2, V // 2] = INF
    call = _both_forms if V > 28672 else _check
    t = [INF, 1e38, 3e37, 1e37, 1e36, INF]
    for u in ([0.75] * 6, [0.999] * 6, rng.random(6)):
        for kw in (dict(), dict(p=0.9), dict(m=0.2), dict(k=V - 1), dict(k=V - 1, p=0.6, m=0.1)):
            tok, lp = call(x, u, f"{V} {kw}", t=t, **kw)
            assert lp[0] == lp[2] == 0 and tok[0] == V - 1 and tok[2] == V // 2 and tok[1] in (0, V - 1)
    # all infinite, and a row of two numbers far apart
    x[:] = INF
    call(x, [0.1, 0.3, 0.5, 0.7, 0.9, 0.99], "all", t=t)
    x[:] = -torch.finfo(dt).max
    x[:, 1] = torch.finfo(BF16).max if dt is F32 else torch.finfo(dt).max
    call(x, [0.1, 0.3, 0.5, 0.7, 0.9, 0.99], "far apart", t=t)


# ------------------------------------------------------------------ norms
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("D,rot", [(16, 16), (64, 64), (128, 64), (256, 256), (20, 20), (250, 0)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_norms_of_rows_whose_squares_leave_float32(dt, D, rot, pairs):
    # every row at a size of its own, so that lanes of one wave go both ways
    g = torch.Generator(device=DEV)
    g.manual_seed(D)
    size = [1e38, 1.0, 1e25, 1e-25, 1e-38, 3e19, 1e-19, 1e18, 1e-15, 2.0 ** -133]
    T, Hq, Hkv = len(size), 5, 3
    x = torch.randn(T, Hq + Hkv, D, generator=g, device=DEV).clamp(-3, 3) * torch.tensor(size, device=DEV)[:, None, None]
    x = x.to(dt)
    x[1, ::2] *= 1e30
    x[2, 1::2] *= 1e-24
    q, k = x[:, :Hq], x[:, Hq:]
    w = (1 + 0.3 * torch.randn(2, D, generator=g, device=DEV)).to(dt)
    pos = torch.randint(0, 1000, (T,), generator=g, device=DEV).to(torch.int32)
    freqs = (10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / max(rot, 1))).float()
    for eps in (0.0, 1e-30, 1e-6, 1e30):
        e = float(np.float32(eps))
        qo, ko = rtopk.qk_norm_rope(q, k, pos, freqs, q_weight=w[0], k_weight=w[1], eps=eps, interleaved=pairs)
        torch.cuda.synchronize()
        for got, y, z in ((qo, q, w[0]), (ko, k, w[1])):
            want, tol = rope(y.cpu(), z.cpu(), pos.cpu(), freqs.cpu(), e, pairs)
            # (the reference's floor is for a float32 output below its normal numbers)
            off = (got.cpu().double() - want).abs() / tol
            assert off.max() <= 1, (dt, D, eps, float(off.max()))
    # a row of zeros divides nothing by nothing; an infinite element leaves the others nothing
    x[0] = 0
    x[3, :, D // 2] = INF
    qo, ko = rtopk.qk_norm_rope(q, k, pos.zero_(), freqs, q_weight=w[0], k_weight=w[1], eps=0.0, interleaved=pairs)
    torch.cuda.synchronize()
    assert torch.isnan(qo[0].float()).all() and torch.isnan(ko[0].float()).all()
    assert torch.isnan(qo[3].float()).any() and torch.isfinite(qo[1:3].float()).all()


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("R,V", [(10, 40000), (3, 270007)])
def test_special_rows_cut_over_workgroups(R, V, dt):
    # what a chunk of a row does not see of the others: ends, ties of the largest, nothing at all
    x, rng = _rows(10, V, dt, seed=V, sigma=2.0)
    x[0] = -INF
    x[1] = NAN
    x[2] = -INF
    x[2, V - 1] = -7.0  # in the last chunk alone
    x[3, 17] = x[3, V - 100] = INF  # in two chunks
    x[4, ::3] = NAN
    x[5, : V // 2] = -INF  # whole chunks
    x[5, V // 2 + 9000 // 8 :: 2] = NAN
    x[6] = torch.finfo(dt).min
    x[7, 100] = x[7, V // 2] = x[7, V - 1] = 60.0  # the largest in several chunks
    x[8, V // 3:] = -INF
    x[9, ::2] = -INF
    # each row once, whatever R
    for first in range(0, 10, R):
        y, n = x[first:first + R].contiguous(), min(R, 10 - first)
        u = rng.random(n)
        for kw in (dict(), dict(k=50), dict(p=0.9), dict(m=0.1), dict(k=20, p=0.5, m=0.01), dict(t=0.0), dict(k=V // 2, p=0.99), dict(t=INF, p=0.4)):
            tok, lp = _both_forms(y, u, f"{first} {kw}", **kw)
            for r in range(n):
                if first + r in (0, 1):
                    assert tok[r] == -1 and lp[r] == -INF
                if first + r == 2:
                    assert tok[r] == V - 1 and lp[r] == 0
                if first + r == 7 and kw == dict(t=0.0):
                    assert tok[r] == 100


# ------------------------------------------------------------------ what 8 bits stand for
def _exact(codes, scales, dt):
    """The values of codes and scale bytes, rounded to a type (four bits each: exact but beyond the type's ends)."""
    return (torch.from_numpy(CODES).to(DEV)[codes.long()] * torch.exp2(scales.double().clamp(1, 254) - 127)).to(dt)


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("N,D", [(1, 64), (9, 64), (32, 64), (64, 64), (1, 128), (32, 128), (64, 128), (1, 256), (32, 256)])
def test_every_code_and_scale_as_a_value(N, D, dt):
    # every row sees its own key alone, so that its output is that key's value: a tree's nodes have all
    # scales in turn and the heads all codes; subnormal numbers of the type are numbers like others
    Hkv, pages = 256 // D, 256
    at = torch.arange(256, device=DEV)
    codes = at.to(torch.uint8).view(1, 1, Hkv, D).expand(pages, 1, Hkv, D).contiguous()
    scales = at.to(torch.uint8).view(pages, 1, 1).expand(pages, 1, Hkv).contiguous()
    B = 256 // N + (256 % N > 0)
    table = (torch.arange(B * N, device=DEV) % 256).to(torch.int32).view(B, N)
    q = torch.randn(B, N, Hkv, D, device=DEV).to(dt)
    out, lse = rtopk.tree_attention_fp8(q, torch.zeros_like(codes), codes, torch.full_like(scales, 100), scales, table,
                                        torch.zeros(B, dtype=torch.int32, device=DEV),
                                        parents=torch.full((B, N), -1, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    want = _exact(codes.view(256, 256), scales.view(256, Hkv)[:, :1], dt)[table.view(-1).long()]
    got = out.view(B * N, 256)
    same = (got == want) | (got.isnan() & want.isnan())
    assert same.all(), [(int(table.view(-1)[i]), int(c), float(got[i, c]), float(want[i, c])) for i, c in (~same).nonzero()[:5].tolist()]


@pytest.mark.parametrize("dt", [F16, BF16])
@pytest.mark.parametrize("N,D", [(1, 64), (32, 64), (64, 64), (1, 128), (32, 128), (64, 128), (1, 256), (64, 256)])
def test_every_code_and_scale_as_a_key(N, D, dt):
    # one key per row again, and one element of the query: the score is that element times the key's, and lse is the score
    Hkv = 4
    B = 65536 // (N * Hkv)
    at = torch.arange(65536, device=DEV).view(B, N, Hkv)
    code, scales = (at % 256).to(torch.uint8), (at // 256).to(torch.uint8)
    d = (at * 7 % D)[..., None]
    codes = torch.zeros(B, N, Hkv, D, dtype=torch.uint8, device=DEV).scatter_(3, d, code[..., None])
    # the types' ranges over several calls: scores of 2^-10 to 2^20, which are not rounded but by float32
    for e in (range(0, 60, 30) if dt is F16 else range(-100, 150, 30)):
        a = min(e, 120) if dt is BF16 else min(e, 14)  # query 2^a, scale 2^(e - a)
        q = torch.zeros(B, N, Hkv, D, dtype=dt, device=DEV).scatter_(3, d, torch.full((B, N, Hkv, 1), 2.0 ** a, dtype=dt, device=DEV))
        out, lse = torch.empty_like(q), torch.zeros(B, N, Hkv, device=DEV)
        rtopk.tree_attention_fp8(q, codes, torch.zeros_like(codes), scales, torch.full_like(scales, 127), torch.arange(B, dtype=torch.int32, device=DEV).view(B, 1),
                                 torch.zeros(B, dtype=torch.int32, device=DEV), parents=torch.full((B, N), -1, dtype=torch.int32, device=DEV),
                                 scale=2.0 ** (e - a), out=out, lse=lse)
        torch.cuda.synchronize()
        want = _exact(code, scales, dt).double() * 2.0 ** e
        see = (want.abs() >= 2.0 ** -10) & (want.abs() < 2.0 ** 20)
        assert see.sum() > 1000
        # the score in base 2 and back: four roundings of it, and one of a number up to 11 above it (lse's reference)
        off = (lse.double() - want).abs() <= 4 * 2.0 ** -24 * want.abs() + 2 * 2.0 ** -24 * (want.abs() + 16)
        assert off[see].all(), (e, float((lse.double() - want).abs()[see].max()))


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("R,V", [(129, 65536), (170, 70001), (171, 70001), (66, 100352), (67, 100352), (3, 35839), (3, 35840)])
def test_rows_at_the_limits_of_the_cut(R, V, dt):
    x, rng = _rows(R, V, dt, seed=R, sigma=2.0)
    u = rng.random(R)
    for kw in (dict(k=50), dict(k=3000, m=0.01), dict(p=0.9), dict(k=50, p=0.95, m=0.02, t=0.9), dict()):
        tok, lp = _both_forms(x, u, str(kw), oracle=False, **kw)
        some = [0, R // 2, R - 1]
        assert _check(x[some].contiguous(), u[some], str(kw), **kw) == ([tok[r] for r in some], [lp[r] for r in some])
