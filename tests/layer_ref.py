"""Plain 64-bit references of the paged cache and the attention operators, on
the CPU, and the tolerances their outputs are held to."""
import math

import numpy as np
import torch


def ancestors(parents, n):
    """[n, n] truth values: j is i or above i (a parent outside [0, i) is none)."""
    up = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while j >= 0:
            up[i, j] = True
            p = int(parents[j])
            j = p if 0 <= p < j else -1
    return up


def attend(q, k, v, allowed, scale):
    """q [R, D], k, v [S, D] float64, allowed [R, S]: out, lse, tolerances of both.

    The tolerance of an output follows from what a kernel rounds, with
    u = half a step of the type t of the inputs, f = 2**-24 and, per row,
    A_d = sum_j w_j |v_jd| (w the softmax weights):
      * the output once: u |o|; a weight once: u A;
      * a score: D products and sums, the scale and the exponent's argument, all
        float32: at most e = f ((D + 8) max_j scale sum_d |q_d k_jd| + 4 max_j |x_j - max x| + 4),
        which moves every weight by a factor of exp(+-2e): 2.1 e A for e < 0.01;
      * the sums of S weights and of S products: 2 S f A;
      * float16 weights below 2**-14 are subnormal: 2**-25 sum_j |v_j|.
    An lse moves by e + S f + 4 f |lse|.
    """
    D, S = q.shape[1], k.shape[0]
    u = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
    f = 2.0 ** -24
    x = (q @ k.T) * scale
    x = torch.where(allowed, x, -math.inf)
    m = x.amax(1, keepdim=True)
    safe = torch.where(m == -math.inf, 0.0, m)
    p = torch.where(allowed, torch.exp(x - safe), 0.0)
    total = p.sum(1, keepdim=True)
    w = torch.where(total > 0, p / total, 0.0)
    # a key that no row of this call may see must not be touched: its value may be anything
    vz = torch.where(allowed.any(0)[:, None], v, 0.0)
    o = torch.where(w[:, :, None] != 0, w[:, :, None] * vz[None], 0.0).sum(1) if not torch.isfinite(vz).all() else w @ vz
    lse = (safe + total.log())[:, 0]
    kz = torch.where(allowed.any(0)[:, None], k, 0.0)
    mag = torch.where(allowed, q.abs() @ kz.abs().T, 0.0).amax(1, keepdim=True) * abs(scale)
    spread = torch.where(allowed, (safe - x).abs(), 0.0).amax(1, keepdim=True)
    e = f * ((D + 8) * mag + 4 * spread + 4)
    vf = torch.where(torch.isfinite(vz), vz, 0.0).abs()  # for the outputs that are finite
    A = w @ vf

    def tol(t):
        sub = 2.0 ** -25 * vf.sum(0)[None] if t is torch.float16 else 0.0
        return u[t] * (o.abs() + A) * 1.01 + (2.1 * e + 2 * S * f) * A + sub + 1e-30

    return o, lse, tol, e[:, 0] + S * f + 4 * f * lse.abs()


def check_rows(got, glse, o, lse, tol, ltol, what):
    """got, glse as computed; the rest of attend()."""
    got, t = got.cpu(), got.dtype
    bound = tol(t)
    fine = torch.isfinite(o)
    g = got.double()
    assert torch.equal(torch.isnan(g), torch.isnan(o)) and torch.equal(g[~fine & ~torch.isnan(o)], o[~fine & ~torch.isnan(o)]), what
    off = ((g - o).abs() / bound)[fine]
    assert off.numel() == 0 or off.max() <= 1, f"{what}: {off.max():.3f} of the tolerance"
    if glse is not None:
        glse = glse.cpu().double()
        empty = lse == -math.inf
        assert torch.equal(glse == -math.inf, empty), what
        d = ((glse - lse).abs() / ltol)[~empty & torch.isfinite(lse)]
        assert d.numel() == 0 or d.max() <= 1, f"{what}: lse {d.max():.3f} of the tolerance"


def check_cross(q, k, v, lens, mask, scale, out, lse, what):
    """Every batch element and key head of cross attention (CPU or device tensors)."""
    B, N, Hq, D = q.shape
    S, Hkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    qc, kc, vc = q.cpu().double(), k.cpu().double(), v.cpu().double()
    for b in range(B):
        L = S if lens is None else max(0, min(S, int(lens[b])))
        ok = torch.arange(S) < L
        if mask is not None:
            ok &= mask[b].cpu() == 0
        for h in range(Hkv):
            rows = qc[b, :, h * G:(h + 1) * G].reshape(N * G, D)
            o, l, tol, ltol = attend(rows, kc[b, :, h], vc[b, :, h], ok[None].expand(N * G, S), scale)
            check_rows(out[b, :, h * G:(h + 1) * G].reshape(N * G, D),
                       None if lse is None else lse[b, :, h * G:(h + 1) * G].reshape(-1), o, l, tol, ltol, f"{what} b={b} h={h}")


def check_tree(q, kc, vc, table, lens, parents, sizes, scale, out, lse, what):
    """Every request and key head of tree attention. Checks live rows only."""
    B, N, Hq, D = q.shape
    pages, page, Hkv, _ = kc.shape
    G = Hq // Hkv
    ld = table.shape[1]
    qc, kd, vd = q.cpu().double(), kc.cpu().double(), vc.cpu().double()
    tab = table.cpu().numpy()
    for b in range(B):
        n = N if sizes is None else max(0, min(N, int(sizes[b])))
        if n == 0:
            continue
        L = max(0, min(ld * page, int(lens[b])))
        par = np.arange(-1, N - 1) if parents is None else parents[b].cpu().numpy()
        S = min(L + n, ld * page)
        allowed = np.zeros((n, S), dtype=bool)
        allowed[:, :L] = True
        allowed[:, L:] = ancestors(par, n)[:, :S - L]
        at = np.arange(S)
        ids = tab[b, at // page].astype(np.int64)
        good = (ids >= 0) & (ids < pages)
        allowed &= good[None]
        ids = np.where(good, ids, 0)
        k, v = kd[ids, at % page], vd[ids, at % page]
        ok = torch.from_numpy(allowed).repeat_interleave(G, 0)
        for h in range(Hkv):
            rows = qc[b, :n, h * G:(h + 1) * G].reshape(n * G, D)
            o, l, tol, ltol = attend(rows, k[:, h], v[:, h], ok, scale)
            check_rows(out[b, :n, h * G:(h + 1) * G].reshape(n * G, D),
                       None if lse is None else lse[b, :n, h * G:(h + 1) * G].reshape(-1), o, l, tol, ltol, f"{what} b={b} h={h}")


def tables(lens, new, page, free, head, num_pages, table, T, rows):
    """page_tables in plain Python: (table, slots, positions, cu_new, free_next)."""
    B, ld = table.shape
    table = table.copy()
    slots = np.full(T, -1, np.int64)
    pos = np.full(T, -1, np.int64)
    cu, first, taken, granted = [0], 0, max(0, head), 0
    for b in range(B):
        c, n = max(0, int(lens[b])), max(0, int(new[b]))
        fits = c + n <= ld * page and (rows == 0 or n <= rows)
        have = -(-c // page)
        need = -(-(c + n) // page) - have if fits else 0
        ok = fits and (need == 0 or taken + need <= len(free)) and (rows > 0 or first + n <= T)
        if ok:
            for i in range(need):
                table[b, have + i] = free[taken + i]
            granted += need
            for t in range(n):
                p = c + t
                i = (b * rows if rows else first) + t
                page_id = int(table[b, p // page])
                pos[i] = p
                slots[i] = page_id * page + p % page if 0 <= page_id < num_pages else -1
        taken += need
        first += n
        cu.append(min(first, 2 ** 31 - 1))
    return table, slots, pos, np.array(cu), min(max(0, head) + granted, 2 ** 31 - 1)
