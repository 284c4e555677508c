"""Values at the ends of what the rotation, the 8-bit cache and filtered sampling
accept, on the GPU: against their definitions in 64 bits (serve_ref.py), in every form of their kernels."""
import math

import numpy as np
import pytest
import torch

from beam_search_top_amd import rtopk
from libutil import ensure_built
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
