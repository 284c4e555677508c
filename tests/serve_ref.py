"""Plain 64-bit references of the rotation, the 8-bit cache and filtered
sampling, on the CPU, and the tolerances their outputs are held to."""
import math

import numpy as np
import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


# ------------------------------------------------------------------ norms and rotation
def rope(x, w, positions, freqs, eps, pairs):
    """x [T, H, D] (any type): float64 outputs and their tolerance.

    What the kernel rounds, f = 2**-24: the sum of D squares, its mean, the root, the
    quotient and two products, at most (D / 2 + 8) f of the normalised value; an angle in turns, taken off
    whole turns in 64 bits (|turns| 2**-51) and rounded to float32 (2**-26), times 2 pi; a sine or
    cosine by 4 f (the library's 2 ulp); two products and a sum, 2 f of |a| + |b|; the output once.
    """
    T, H, D = x.shape
    y = x.double().clone()
    if w is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * w.double()
    rot = 2 * freqs.numel()
    t = positions.double()[:, None] * freqs.double()
    cos, sin = t.cos()[:, None], t.sin()[:, None]
    i = torch.arange(rot // 2)
    ia, ib = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
    a, b = y[..., ia].clone(), y[..., ib].clone()
    size = y.abs()
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    y[..., ia], y[..., ib] = a * cos - b * sin, b * cos + a * sin
    f = 2.0 ** -24
    turns = (t.abs() / (2 * math.pi)).amax(-1) if rot else torch.zeros(T, dtype=torch.float64)
    angle = 2 * math.pi * (turns * 2.0 ** -51 + 2.0 ** -26) + 4 * f
    tol = size * ((D / 2 + 10) * f + angle[:, None, None]) + y.abs() * HALF_STEP[x.dtype] * 1.01
    return y, tol + (2.0 ** -25 if x.dtype is torch.float16 else 1e-37)


# ------------------------------------------------------------------ the 8-bit format
def code_values():
    """The value of each of the 256 codes."""
    v = np.empty(256)
    for c in range(256):
        e, m = c >> 3 & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = math.nan if c & 127 == 127 else -x if c >> 7 else x
    return v


CODES = code_values()


def quantise(x):
    """x [..., D] tensor: codes (0 .. 255) and scale bytes, by search among the values that there are."""
    limit = 61440.0 if x.dtype is torch.float16 else 240 * 2.0 ** 120
    y = x.double().cpu().numpy()
    shape = y.shape
    y = y.reshape(-1, shape[-1])
    codes = np.zeros(y.shape, np.uint8)
    scales = np.zeros(len(y), np.uint8)
    up = CODES[:127]  # ascending
    for r, row in enumerate(y):
        fine = np.isfinite(row)
        amax = np.abs(row[fine]).max() if fine.any() else 0.0
        e = -126
        if amax > 448 * 2.0 ** -126:
            e = int(math.floor(math.log2(amax / 448))) - 1
            while amax > 448 * 2.0 ** e:
                e += 1
        scales[r] = e + 127
        z = np.minimum(np.abs(np.where(fine, row, 0.0)), limit) / 2.0 ** e
        hi = np.clip(np.searchsorted(up, z, side="left"), 0, 126)  # the first value not below z
        lo = np.maximum(hi - 1, 0)
        low = (z - up[lo] < up[hi] - z) | ((z - up[lo] == up[hi] - z) & (lo % 2 == 0))  # ties to the even code
        c = np.where(low, lo, hi)
        codes[r] = np.where(fine, c | np.where(np.signbit(row), 128, 0), 127)
    return codes.reshape(shape), scales.reshape(shape[:-1])


def values(codes, scales):
    """What codes and scale bytes stand for, in 64 bits (numpy uint8 arrays)."""
    return CODES[codes] * 2.0 ** (np.clip(scales.astype(np.int64), 1, 254) - 127.0)[..., None]


# ------------------------------------------------------------------ filtered sampling
def sample(row, u, temperature=1.0, k=0, p=1.0, m=0.0):
    """(token, log-probability) of one row of float64 logits, from the definition."""
    row = np.where(np.isnan(row), -math.inf, row)
    order = np.argsort(-row, kind="stable")
    top = row[order[0]]
    if top == -math.inf:
        return -1, -math.inf
    if not temperature > 0:
        return int(order[0]), 0.0
    w = np.array([1.0 if x == top else 0.0 if top == math.inf or x == -math.inf else math.exp((x - top) / temperature)
                  for x in row[order]])
    n = min(len(w), k) if k > 0 else len(w)
    if p < 1:
        n = min(n, 1 + int(np.searchsorted(np.cumsum(w[:n]), max(p, 0.0) * w[:n].sum(), side="left")))
    m = min(1.0, m) if m > 0 else 0.0
    n = max(1, min(n, int((w >= m).sum())))
    at = np.argsort(order[:n])
    kept, w = order[:n][at], w[:n][at]
    upto = np.cumsum(w)
    u = u if u > 0 else 0.0
    i = int(np.searchsorted(upto, u * upto[-1], side="right")) if u < 1 else n
    i = min(i, int(np.flatnonzero(w)[-1]))
    return int(kept[i]), math.log(w[i] / upto[-1])
