"""Values at the ends of what the rotation, the 8-bit cache and filtered sampling
accept, on the GPU: against their definitions in 64 bits (serve_ref.py), in every form of their kernels."""
import math

import numpy as np
import pytest
import torch

from beam_search_top_amd import rtopk
from libutil import ensure_built
from serve_ref import rope
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
