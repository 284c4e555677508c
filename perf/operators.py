"""The cache and attention operators of a decode step, as they are timed and compared.

Four operators stand between the projections of a decoder layer and the
selection step: the page tables of a paged key/value cache, the store that
fills it, the attention of a tree of drafted tokens over it (a single token is
the tree of one node, parents a beam step's beam ids), and the cross attention
of every beam's rows to the encoder states that the beams of a sentence share.

With `own` false, run() computes them in their plain form, elementary torch
operations in 32 bits rounded once at the end; with `own` true it calls the
library (beam_search_top_amd.rtopk).
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of a small translation batch: 8 sentences x 4 beams, short sources; latency counts
        dict(name="cross_small", op="cross", dtype="f16", B=8, N=4, S=64, Hq=16, Hkv=16, D=64, least=9, mask=False),
        # the 128 x 4 batch of the default benchmark, 16 heads of 64, sources of up to 512 tokens
        dict(name="cross_beams", op="cross", dtype="f16", B=128, N=4, S=512, Hq=16, Hkv=16, D=64, least=130, mask=False),
        # four long documents as sources, 8 beams, grouped heads, holes in the sources (masked sections)
        dict(name="cross_long", op="cross", dtype="bf16", B=4, N=8, S=30001, Hq=32, Hkv=8, D=128, least=20000, mask=True),
        # whole hypotheses rescored against their sources: many rows, bound by the matrix cores
        dict(name="cross_rescore", op="cross", dtype="bf16", B=8, N=2048, S=2000, Hq=16, Hkv=16, D=128, least=1000, mask=False),
        # one new token for 8 short requests; latency counts
        dict(name="tree_token", op="tree", dtype="f16", B=8, N=1, Hq=16, Hkv=16, D=64, page=16, least=100, most=500, tree=False),
        # one new token for two very long requests
        dict(name="tree_token_long", op="tree", dtype="bf16", B=2, N=1, Hq=32, Hkv=8, D=128, page=64, least=90000, most=131000, tree=False),
        # 64 drafted tokens for each of 32 requests, checked in one pass
        dict(name="tree_draft", op="tree", dtype="bf16", B=32, N=64, Hq=32, Hkv=8, D=128, page=16, least=1500, most=4000, tree=True),
        # odd everything: 29 nodes, pages of 24 tokens, 5 query heads per key head, heads of 80
        dict(name="tree_odd", op="tree", dtype="f16", B=7, N=29, Hq=20, Hkv=4, D=80, page=24, least=0, most=3001, tree=True),
        # a step's drafted tokens for 256 requests, rows of 64 slots
        dict(name="tables_draft", op="tables", B=256, page=16, least=0, most=3000, new_least=1, new_most=64, rows=64),
        # prompts of 600 requests laid one behind the other
        dict(name="tables_prompt", op="tables", B=600, page=16, least=0, most=700, new_least=1, new_most=4001, rows=0),
        # the new tokens' keys and values of one layer: one token for each of 200 requests
        dict(name="store_tokens", op="store", dtype="f16", T=200, Hkv=16, D=64, page=16, pages=600, skip=8),
        # the prompts' keys and values of one layer
        dict(name="store_prompt", op="store", dtype="bf16", T=130001, Hkv=8, D=128, page=16, pages=9001, skip=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("cross", "cross", "tree", "tree", "tables", "store"))
    dtype = rng.choice(("f16", "bf16"))
    Hkv = rng.choice((1, 2, 4, 8, 16))
    G = rng.choice((1, 1, 2, 4, 5, 8))
    D = rng.choice((64, 64, 128, 128, 32, 40, 80, 96, 192, 256))
    if op == "cross":
        # as many keys as 400 MB hold, and the rows that a budget of multiply-adds, less than the largest listed case's, leaves
        S = _log(rng, 1, min(30000, int(1e8 // (Hkv * D))))
        B = _log(rng, 1, max(1, min(160, int(1e8 // (S * Hkv * D)))))
        N = _log(rng, 1, max(1, min(2000, int(4.5e10 // (B * S * Hkv * G * D)), int(1e8 // (B * Hkv * G * D)))))
        return dict(op=op, dtype=dtype, B=B, N=N, S=S, Hq=Hkv * G, Hkv=Hkv, D=D, least=rng.randint(0, S),
                    mask=rng.random() < 0.4)
    if op == "tree":
        most = _log(rng, 1, min(120000, int(1e8 // (Hkv * D))))
        N = rng.choice((1, 1, _log(rng, 2, 200), _log(rng, 2, 64)))
        B = _log(rng, 1, max(1, min(100, int(1e8 // ((most + N) * Hkv * D)), int(4.5e10 // ((most + N) * N * Hkv * G * D)))))
        return dict(op=op, dtype=dtype, B=B, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, page=rng.choice((1, 8, 16, 16, 24, 32, 64, 100, 128)),
                    least=rng.randint(0, most), most=most, tree=rng.random() < 0.7)
    if op == "tables":
        new_most = _log(rng, 1, 4000)
        B = _log(rng, 1, max(1, min(3000, 800000 // new_most)))
        return dict(op=op, B=B, page=rng.choice((1, 8, 16, 24, 64)), least=0, most=_log(rng, 1, 3000), new_least=rng.randint(0, 1),
                    new_most=new_most, rows=rng.choice((0, new_most)))
    T = _log(rng, 2, min(500000, int(1.2e8 // (Hkv * D))))
    page = rng.choice((1, 8, 16, 24, 64))
    return dict(op=op, dtype=dtype, T=T, Hkv=Hkv, D=D, page=page, pages=T // page + 1 + _log(rng, 1, 1000), skip=rng.randint(0, T // 2))


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly spread with both ends among them (one length: hi)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


# ------------------------------------------------------------------ what a program has in hand
def _paged(c, g):
    """Lengths, drafted sizes and a table of distinct pages in random order."""
    B, N, page = c["B"], c["N"], c["page"]
    perm = torch.randperm(B, generator=g, device=DEV)
    lens = torch.tensor(_spread(B, c["least"], c["most"]), dtype=torch.int32, device=DEV)[perm]
    sizes = torch.tensor(_spread(B, (N + 1) // 2, N), dtype=torch.int32, device=DEV)[torch.randperm(B, generator=g, device=DEV)]
    ld = (c["most"] + N + page - 1) // page
    pages = B * ld
    table = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).reshape(B, ld)
    return lens, sizes, table, pages


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *shape, dt=torch.float32: torch.randn(*shape, generator=g, device=DEV).to(dt)  # noqa: E731
    s = dict(case=c)
    if c["op"] == "cross":
        dt = DTYPES[c["dtype"]]
        s["q"] = rnd(c["B"], c["N"], c["Hq"], c["D"], dt=dt) * 1.5
        # one projection gives keys and values side by side
        kv = rnd(c["B"], c["S"], 2, c["Hkv"], c["D"], dt=dt)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        perm = torch.randperm(c["B"], generator=g, device=DEV)
        s["lens"] = torch.tensor(_spread(c["B"], c["least"], c["S"]), dtype=torch.int32, device=DEV)[perm]
        s["mask"] = (torch.rand(c["B"], c["S"], generator=g, device=DEV) < 0.1).to(torch.uint8) if c["mask"] else None
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(c["B"], c["N"], c["Hq"], device=DEV)
    elif c["op"] == "tree":
        dt = DTYPES[c["dtype"]]
        B, N = c["B"], c["N"]
        s["lens"], s["sizes"], s["table"], pages = _paged(c, g)
        s["q"] = rnd(B, N, c["Hq"], c["D"], dt=dt) * 1.5
        s["kc"] = rnd(pages, c["page"], c["Hkv"], c["D"], dt=dt)
        s["vc"] = rnd(pages, c["page"], c["Hkv"], c["D"], dt=dt)
        # node i hangs below one of the eight nodes before it, or starts a branch of its own (-1)
        i = torch.arange(N, device=DEV)
        back = torch.randint(1, 9, (B, N), generator=g, device=DEV)
        s["parents"] = torch.clamp(i - back, min=-1).to(torch.int32) if c["tree"] else None
        # rows behind a request's last node stay as they are: zero here
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(B, N, c["Hq"], device=DEV)
    elif c["op"] == "tables":
        B, page = c["B"], c["page"]
        perm = lambda: torch.randperm(B, generator=g, device=DEV)  # noqa: E731
        s["lens"] = torch.tensor(_spread(B, c["least"], c["most"]), dtype=torch.int32, device=DEV)[perm()]
        s["new"] = torch.tensor(_spread(B, c["new_least"], c["new_most"]), dtype=torch.int32, device=DEV)[perm()]
        ld = (c["most"] + c["new_most"] + page - 1) // page
        have = (c["most"] + page - 1) // page
        free = sum((n + page - 1) // page + 1 for n in _spread(B, c["new_least"], c["new_most"]))
        s["pages"] = B * have + free
        ids = torch.randperm(s["pages"], generator=g, device=DEV).to(torch.int32)
        s["table"] = torch.full((B, ld), -1, dtype=torch.int32, device=DEV)
        s["table"][:, :have] = ids[:B * have].reshape(B, have)
        s["free"] = ids[B * have:].contiguous()
        s["head"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["T"] = sum(_spread(B, c["new_least"], c["new_most"])) + 5  # the last five slots belong to nobody
        n = (B, c["rows"]) if c["rows"] else (s["T"],)
        s["out"] = (torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV),
                    torch.zeros(B + 1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV))
    else:
        dt = DTYPES[c["dtype"]]
        T, Hkv, D = c["T"], c["Hkv"], c["D"]
        kv = rnd(T, 2, Hkv, D, dt=dt)  # one projection gives keys and values side by side
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        s["kc"] = rnd(c["pages"], c["page"], Hkv, D, dt=dt)
        s["vc"] = rnd(c["pages"], c["page"], Hkv, D, dt=dt)
        s["slots"] = torch.randperm(c["pages"] * c["page"], generator=g, device=DEV)[:T].to(torch.int32)
        if c["skip"]:  # padding tokens
            s["slots"][torch.randperm(T, generator=g, device=DEV)[:c["skip"]]] = -1
    return s


# ------------------------------------------------------------------ the plain forms
def _attend(q, k, v, allowed, dt):
    """q [B, N, Hq, D], k and v [B, S, Hkv, D], allowed [B, N or 1, S]: outputs and log-sum-exp;
    a row that nothing is allowed for gives zeros and -inf."""
    B, N, Hq, D = q.shape
    Hkv = k.shape[2]
    G = Hq // Hkv
    q = q.float().reshape(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    k = k.float().permute(0, 2, 3, 1).contiguous()
    seen = allowed.any(1)  # [B, S]
    v = torch.where(seen[:, :, None, None], v.float(), 0.0).permute(0, 2, 1, 3).contiguous()
    x = torch.matmul(q, k).reshape(B, Hkv, N, G, -1) / math.sqrt(D)
    x = x.masked_fill_(~allowed[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hkv, N * G, -1), v).reshape(B, Hkv, N, G, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + total.log())[..., 0]
    return o.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(dt), lse.permute(0, 2, 1, 3).reshape(B, N, Hq)


def _ancestors(parents):
    """[B, N, N]: whether j is i or above i; a parent outside [0, i) is none."""
    B, N = parents.shape
    i = torch.arange(N, device=parents.device)
    m = ((parents[:, :, None] == i) & (i[None, :] < i[:, None])[None] | (i[:, None] == i)[None]).float()
    m = torch.matmul(m, m).clamp_(max=1)  # paths of up to 2, 4, ..., 256 steps
    m = torch.matmul(m, m).clamp_(max=1)
    m = torch.matmul(m, m).clamp_(max=1)
    m = torch.matmul(m, m).clamp_(max=1)
    m = torch.matmul(m, m).clamp_(max=1)
    m = torch.matmul(m, m).clamp_(max=1)
    m = torch.matmul(m, m).clamp_(max=1)
    m = torch.matmul(m, m)
    return m > 0


def _plain_cross(s):
    S = s["k"].shape[1]
    allowed = torch.arange(S, device=DEV) < s["lens"][:, None]
    if s["mask"] is not None:
        allowed = allowed & (s["mask"] == 0)
    return _attend(s["q"], s["k"], s["v"], allowed[:, None, :], s["q"].dtype)


def _plain_tree(s):
    B, N, Hq, D = s["q"].shape
    ld, page = s["table"].shape[1], s["kc"].shape[1]
    k = s["kc"][s["table"].long()].reshape(B, ld * page, -1, D)
    v = s["vc"][s["table"].long()].reshape(B, ld * page, -1, D)
    parents = s["parents"]
    if parents is None:
        parents = (torch.arange(N, device=DEV) - 1).to(torch.int32).expand(B, N)
    above = _ancestors(parents)
    j = torch.arange(ld * page, device=DEV)[None, :] - s["lens"][:, None]  # the node at each place, negative in the cache
    drafted = torch.gather(above, 2, j.clamp(0, N - 1)[:, None, :].expand(B, N, -1)) & (j < N)[:, None, :] & (j >= 0)[:, None, :]
    live = torch.arange(N, device=DEV) < s["sizes"][:, None]
    allowed = ((j < 0)[:, None, :] | drafted) & live[:, :, None]
    o, lse = _attend(s["q"], k, v, allowed, s["q"].dtype)
    return torch.where(live[:, :, None, None], o, s["out"]), torch.where(live[:, :, None], lse, s["lse"])


def _plain_tables(s):
    c = s["case"]
    B, page, rows = c["B"], c["page"], c["rows"]
    lens, new, table = s["lens"].long(), s["new"].long(), s["table"].long()
    have, want = (lens + page - 1) // page, (lens + new + page - 1) // page
    need = want - have
    taken = torch.cumsum(need, 0) - need + s["head"].long()  # each request's place in the list of free pages
    ends = torch.cumsum(new, 0)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), ends])
    # a page is the request's own while it has it, and then the next of the list
    p = torch.arange(table.shape[1], device=DEV)[None, :]
    fresh = s["free"].long()[(taken[:, None] + p - have[:, None]).clamp(0, s["free"].numel() - 1)]
    table = torch.where((p >= have[:, None]) & (p < want[:, None]), fresh, table)
    if rows:
        t = torch.arange(rows, device=DEV)[None, :].expand(B, rows)
        b = torch.arange(B, device=DEV)[:, None].expand(B, rows)
        valid = t < new[:, None]
    else:
        i = torch.arange(s["T"], device=DEV)
        b = torch.searchsorted(ends, i, right=True)
        valid = b < B
        b = b.clamp(max=B - 1)
        t = i - cu[b]
    pos = lens[b] + t
    slot = table[b, (pos // page).clamp(max=table.shape[1] - 1)] * page + pos % page
    return (table.to(torch.int32), torch.where(valid, slot, -1).to(torch.int32), torch.where(valid, pos, -1).to(torch.int32),
            cu.to(torch.int32), (s["head"] + need.sum()).to(torch.int32))


def _plain_store(s):
    valid = s["slots"] >= 0
    first = torch.argmax(valid.to(torch.int32))
    # a token without a slot repeats the first token that has one
    to = torch.where(valid, s["slots"], s["slots"][first]).long()
    kc, vc = s["kc"].reshape(-1, *s["kc"].shape[2:]), s["vc"].reshape(-1, *s["vc"].shape[2:])
    kc[to] = torch.where(valid[:, None, None], s["k"], s["k"][first])
    vc[to] = torch.where(valid[:, None, None], s["v"], s["v"][first])
    return s["kc"], s["vc"]


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"cross": _plain_cross, "tree": _plain_tree, "tables": _plain_tables, "store": _plain_store}[op](s)
    from beam_search_top_amd import rtopk
    if op == "cross":
        return rtopk.cross_attention(s["q"], s["k"], s["v"], lens=s["lens"], key_mask=s["mask"], out=s["out"], lse=s["lse"])
    if op == "tree":
        return rtopk.tree_attention(s["q"], s["kc"], s["vc"], s["table"], s["lens"], parents=s["parents"], sizes=s["sizes"],
                                    out=s["out"], lse=s["lse"])
    if op == "tables":
        return (s["table"],) + rtopk.page_tables(s["lens"], s["new"], s["case"]["page"], s["free"], s["table"], s["pages"],
                                                 free_head=s["head"], out=s["out"])
    return rtopk.cache_store(s["k"], s["v"], s["slots"], s["kc"], s["vc"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "cross":
        keys = sum(_spread(c["B"], c["least"], c["S"]))
        rows = c["B"] * c["N"] * c["Hq"]
        return {"bytes": 4 * keys * c["Hkv"] * c["D"] + rows * (4 * c["D"] + 4) + 4 * c["B"] + (keys if c["mask"] else 0),
                "flops": 4 * keys * c["N"] * c["Hq"] * c["D"]}
    if c["op"] == "tree":
        # every request's average number of nodes: which lengths meet which sizes goes by the seed
        n = sum(_spread(c["B"], (c["N"] + 1) // 2, c["N"]))
        keys = sum(_spread(c["B"], c["least"], c["most"])) + n
        return {"bytes": 4 * keys * c["Hkv"] * c["D"] + n * c["Hq"] * (4 * c["D"] + 4) + 4 * (keys // c["page"]) + (4 * n if c["tree"] else 0) + 8 * c["B"],
                "flops": 4 * keys * n // c["B"] * c["Hq"] * c["D"]}
    if c["op"] == "tables":
        n = sum(_spread(c["B"], c["new_least"], c["new_most"]))
        slots = c["B"] * c["rows"] if c["rows"] else n + 5
        return {"bytes": 12 * c["B"] + 8 * (n // c["page"]) + 8 * slots, "flops": 0}
    return {"bytes": 8 * (c["T"] - c["skip"]) * c["Hkv"] * c["D"] + 4 * c["T"], "flops": 0}


# ------------------------------------------------------------------ in 64 bits, from the definition
def _softmax_rows(q, k, v, allowed):
    """One request and one key head in 64 bits: q [R, D], k and v [S, D], allowed [R, S]."""
    x = (q @ k.T) / math.sqrt(q.shape[1])
    x = torch.where(allowed, x, torch.full_like(x, -math.inf))
    lse = torch.logsumexp(x, -1)
    w = torch.where(allowed, torch.exp(x - lse[:, None]), torch.zeros_like(x))
    return w @ v, lse


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "tables":
        return None  # whole numbers only
    if c["op"] == "store":
        kc, vc = s["kc"].double(), s["vc"].double()
        ok = s["slots"] >= 0
        at = s["slots"][ok].long()
        kc[at // c["page"], at % c["page"]] = s["k"][ok].double()
        vc[at // c["page"], at % c["page"]] = s["v"][ok].double()
        return kc, vc
    B, N, Hq, D = s["q"].shape
    G = Hq // c["Hkv"]
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(B, N, Hq, dtype=torch.float64, device=DEV)
    if c["op"] == "tree":
        table, lens, sizes = (s[n].cpu().numpy() for n in ("table", "lens", "sizes"))
        parents = s["parents"].cpu().numpy() if s["parents"] is not None else np.arange(-1, N - 1)[None].repeat(B, 0)
    for b in range(B):
        if c["op"] == "cross":
            n, L = N, int(s["lens"][b])
            k, v = s["k"][b, :L], s["v"][b, :L]
            row = torch.ones(L, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"][b, :L] == 0
            allowed = row[None].expand(n, L)
        else:
            n, L = int(sizes[b]), int(lens[b])
            at = np.arange(L + n)
            places = torch.from_numpy(table[b, at // c["page"]].astype(np.int64) * c["page"] + at % c["page"]).to(DEV)
            k = s["kc"].reshape(-1, c["Hkv"], D)[places]
            v = s["vc"].reshape(-1, c["Hkv"], D)[places]
            up = np.zeros((n, L + n), dtype=bool)
            up[:, :L] = True
            for i in range(n):
                j = i
                while j >= 0:
                    up[i, L + j] = True
                    j = int(parents[b, j]) if parents[b, j] < j else -1
            allowed = torch.from_numpy(up).to(DEV)
        for h in range(c["Hkv"]):
            q = s["q"][b, :n, h * G:(h + 1) * G].double().reshape(n * G, D)
            o, l = _softmax_rows(q, k[:, h].double(), v[:, h].double(), allowed.repeat_interleave(G, 0))
            out[b, :n, h * G:(h + 1) * G] = o.reshape(n, G, D)
            lse[b, :n, h * G:(h + 1) * G] = l.reshape(n, G)
    return out, lse
