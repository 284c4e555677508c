"""The operators of a sampled decode step with a cache in 8 bits, as they are timed and compared.

Five operators join the decoder layer's cache and attention and the sampling
step: the norms of queries and keys with the position rotation in the same
pass; the store that quantises keys and values into a paged cache of 8-bit
floating point with one power of two per token and head; the reading back of
such a cache; the attention of a tree of tokens over it; and sampling with
temperature, top-k, top-p and min-p from given random numbers.

With `own` false, run() computes them in their plain form, elementary torch
operations rounded once at the end; with `own` true it calls the library
(beam_search_top_amd.rtopk).
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token of 200 requests, 16 heads of 64, as a projection leaves them; latency counts
        dict(name="rope_tokens", op="rope", dtype="f16", T=200, Hq=16, Hkv=16, D=64, rot=64, pairs=False, norm=True, far=4000, skip=8),
        # prompts of 60001 tokens, 32/8 heads of 128, positions of long texts
        dict(name="rope_prompt", op="rope", dtype="bf16", T=60001, Hq=32, Hkv=8, D=128, rot=128, pairs=False, norm=True, far=131000, skip=1000),
        # one layer's new keys and values for 200 requests, written and read back
        dict(name="store_tokens", op="store", dtype="f16", T=200, Hkv=16, D=64, page=16, pages=600, skip=8),
        # a layer's keys and values of long prompts, written and read back
        dict(name="store_prompt", op="store", dtype="bf16", T=130001, Hkv=8, D=128, page=16, pages=9001, skip=1000),
        # a short shared beginning taken out of the cache
        dict(name="load_short", op="load", dtype="f16", T=500, Hkv=16, D=64, page=16, pages=600, skip=0),
        # a long shared beginning taken out of the cache, odd pages
        dict(name="load_long", op="load", dtype="bf16", T=100001, Hkv=8, D=128, page=24, pages=6001, skip=0),
        # one new token for 8 short requests; latency counts
        dict(name="token", op="tree", dtype="f16", B=8, N=1, Hq=16, Hkv=16, D=64, page=16, least=100, most=500, tree=False),
        # one new token for two very long requests
        dict(name="token_long", op="tree", dtype="bf16", B=2, N=1, Hq=32, Hkv=8, D=128, page=64, least=90000, most=131000, tree=False),
        # 64 drafted tokens for each of 32 requests, checked in one pass
        dict(name="draft", op="tree", dtype="bf16", B=32, N=64, Hq=32, Hkv=8, D=128, page=16, least=1500, most=4000, tree=True),
        # 8 requests over a vocabulary of 250000, every filter in use; latency counts
        dict(name="sample_few", op="sample", dtype="bf16", R=8, V=250000, pad=0, sigma=3.0, filters="all"),
        # a batch of 32 over a vocabulary of 32000 in float32, top-p alone
        dict(name="sample_32k", op="sample", dtype="f32", R=32, V=32000, pad=0, sigma=2.0, filters="top_p"),
        # 512 requests over a vocabulary of 40000 in rows of 40064, every filter in use
        dict(name="sample_batch", op="sample", dtype="f16", R=512, V=40000, pad=64, sigma=3.0, filters="all"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "store", "load", "tree", "tree", "sample", "sample"))
    dtype = rng.choice(("f16", "bf16", "f16", "bf16", "f32"))
    Hkv = rng.choice((1, 2, 4, 8, 16))
    G = rng.choice((1, 1, 2, 4, 5, 8))
    D = rng.choice((64, 64, 128, 128, 32, 48, 80, 96, 192, 256))
    if op == "rope":
        T = _log(rng, 1, max(1, min(60000, int(3e8 // (Hkv * (G + 1) * D)))))
        return dict(op=op, dtype=dtype, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, rot=rng.choice((D, D, D // 2, D // 4)), pairs=rng.random() < 0.4,
                    norm=rng.random() < 0.7, far=_log(rng, 1, 1000000), skip=rng.randint(0, T // 4))
    if op in ("store", "load"):
        T = _log(rng, 2, min(200000, int(1.3e8 // (Hkv * D))))
        page = rng.choice((1, 8, 16, 24, 64))
        return dict(op=op, dtype=dtype, T=T, Hkv=Hkv, D=D, page=page, pages=T // page + 1 + _log(rng, 1, 1000), skip=rng.randint(0, T // 2))
    if op == "tree":
        most = _log(rng, 1, min(120000, int(1.2e8 // (Hkv * D))))
        N = rng.choice((1, 1, _log(rng, 2, 200), _log(rng, 2, 64)))
        B = _log(rng, 1, max(1, min(100, int(1.2e8 // ((most + N) * Hkv * D)), int(4.5e10 // ((most + N) * N * Hkv * G * D)))))
        return dict(op=op, dtype="f16" if dtype == "f32" else dtype, B=B, N=N, Hq=Hkv * G, Hkv=Hkv, D=D,
                    page=rng.choice((1, 8, 16, 16, 24, 32, 64, 100, 128)), least=rng.randint(0, most), most=most, tree=rng.random() < 0.7)
    V = _log(rng, 100, 260000)
    return dict(op=op, dtype=dtype, R=_log(rng, 1, max(1, min(1000, 20000000 // V))), V=V, pad=rng.choice((0, 0, 1, 64)),
                sigma=rng.choice((1.0, 2.0, 3.0, 5.0)), filters=rng.choice(("all", "all", "top_p", "top_k", "min_p", "none")))


def _spread(n, lo, hi):
    """n lengths from lo to hi, evenly spread with both ends among them (one length: hi)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


# ------------------------------------------------------------------ what a program has in hand
def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *shape: torch.randn(*shape, generator=g, device=DEV)  # noqa: E731
    uni = lambda *shape: torch.rand(*shape, generator=g, device=DEV)  # noqa: E731
    perm = lambda n: torch.randperm(n, generator=g, device=DEV)  # noqa: E731
    s = dict(case=c)
    dt = DTYPES[c["dtype"]]
    if c["op"] == "rope":
        T, Hq, Hkv, D = c["T"], c["Hq"], c["Hkv"], c["D"]
        # one projection gives queries, keys and values side by side; a few channels are large, as in trained models
        x = rnd(T, Hq + 2 * Hkv, D) * torch.exp(0.7 * rnd(D))
        x = x.to(dt)
        s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + Hkv]
        s["positions"] = torch.randint(0, c["far"], (T,), generator=g, device=DEV).to(torch.int32)
        s["positions"][perm(T)[:c["skip"]]] = -1  # padding tokens
        s["freqs"] = (10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])).float()
        s["qw"], s["kw"] = ((1 + 0.2 * rnd(D)).to(dt), (1 + 0.2 * rnd(D)).to(dt)) if c["norm"] else (None, None)
        # rows of padding tokens stay as they are: zero here
        s["q_out"] = torch.zeros(T, Hq, D, dtype=dt, device=DEV)
        s["k_out"] = torch.zeros(T, Hkv, D, dtype=dt, device=DEV)
    elif c["op"] in ("store", "load"):
        T, Hkv, D, page, pages = c["T"], c["Hkv"], c["D"], c["page"], c["pages"]
        s["slots"] = perm(pages * page)[:T].to(torch.int32)
        if c["skip"]:  # padding tokens
            s["slots"][perm(T)[:c["skip"]]] = -1
        _cache8(s, g, pages, page, Hkv, D)
        if c["op"] == "store":
            # one projection gives keys and values side by side; some tokens and heads are much larger than others
            kv = (rnd(T, 2, Hkv, D) * torch.exp(1.5 * rnd(T, 2, Hkv, 1))).to(dt)
            s["k"], s["v"] = kv[:, 0], kv[:, 1]
        s["k_out"] = torch.zeros(T, Hkv, D, dtype=dt, device=DEV)
        s["v_out"] = torch.zeros(T, Hkv, D, dtype=dt, device=DEV)
    elif c["op"] == "tree":
        B, N, page = c["B"], c["N"], c["page"]
        s["lens"] = torch.tensor(_spread(B, c["least"], c["most"]), dtype=torch.int32, device=DEV)[perm(B)]
        s["sizes"] = torch.tensor(_spread(B, (N + 1) // 2, N), dtype=torch.int32, device=DEV)[perm(B)]
        ld = (c["most"] + N + page - 1) // page
        s["table"] = perm(B * ld).to(torch.int32).reshape(B, ld)
        s["q"] = (rnd(B, N, c["Hq"], c["D"]) * 1.5).to(dt)
        _cache8(s, g, B * ld, page, c["Hkv"], c["D"])
        # node i hangs below one of the eight nodes before it, or starts a branch of its own (-1)
        back = torch.randint(1, 9, (B, N), generator=g, device=DEV)
        s["parents"] = torch.clamp(torch.arange(N, device=DEV) - back, min=-1).to(torch.int32) if c["tree"] else None
        # rows behind a request's last node stay as they are: zero here
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(B, N, c["Hq"], device=DEV)
    else:
        R, V = c["R"], c["V"]
        s["logits"] = (rnd(R, V + c["pad"]) * c["sigma"]).to(dt)[:, :V]
        s["u"] = uni(R)
        f = c["filters"]
        pick = lambda values, dtype: torch.tensor(values, dtype=dtype, device=DEV)[torch.randint(0, len(values), (R,), generator=g, device=DEV)]  # noqa: E731
        # temperature 0 is the best token; top_k 0, top_p 1 and min_p 0 ask for nothing
        s["temperature"] = pick([1.0, 0.7, 0.9, 1.3, 0.0 if f == "all" else 1.0], torch.float32)
        s["top_k"] = pick([0, 0, 20, 50, 1, 1000], torch.int32) if f in ("all", "top_k") else None
        s["top_p"] = pick([1.0, 0.9, 0.95, 0.5, 0.99], torch.float32) if f in ("all", "top_p") else None
        s["min_p"] = pick([0.0, 0.0, 0.05, 0.02], torch.float32) if f in ("all", "min_p") else None
        s["tokens"] = torch.zeros(R, dtype=torch.int32, device=DEV)
        s["logprobs"] = torch.zeros(R, device=DEV)
    return s


def _cache8(s, g, pages, page, Hkv, D):
    """A filled cache: codes of normal values near the top of their range, powers of two around one per token and head."""
    for n in ("k", "v"):
        s[n + "c"] = (torch.randn(pages, page, Hkv, D, generator=g, device=DEV) * 80).clamp_(-448, 448).to(F8)
        s[n + "s"] = torch.randint(119, 123, (pages, page, Hkv), generator=g, device=DEV).to(torch.uint8)


# ------------------------------------------------------------------ the plain forms
def _plain_rope(s):
    c = s["case"]
    rot = c["rot"]
    angle = s["positions"].double()[:, None] * s["freqs"].double()  # [T, rot / 2], far positions: in 64 bits
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    live = (s["positions"] >= 0)[:, None, None]
    outs = []
    for x, w, before in ((s["q"], s["qw"], s["q_out"]), (s["k"], s["kw"], s["k_out"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()
        if c["pairs"]:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            z = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            z = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        outs.append(torch.where(live, torch.cat((z, y[..., rot:]), -1).to(x.dtype), before))
    return tuple(outs)


_LIMIT = {"f16": 61440.0, "bf16": 240 * 2.0 ** 120, "f32": 240 * 2.0 ** 120}  # the largest value in 8 bits that each type holds


def _plain_quantise(x, limit):
    """Codes and bytes of the powers of two: the smallest 2^e, e >= -126, with no finite element over 448 2^e."""
    y = x.float()
    fine = torch.isfinite(y)
    a = torch.where(fine, y.abs(), 0.0).amax(-1)
    m, e = torch.frexp(a)  # a = m 2^e, m in [0.5, 1)
    e = (e - 9 + (m > 0.875)).clamp(min=-126)
    y = torch.where(fine, y.clamp(-limit, limit), math.nan)
    half = e // 2  # in two steps: 2^-e need not be a number of 32 bits
    return torch.ldexp(torch.ldexp(y, -half[..., None]), (half - e)[..., None]).to(F8), (e + 127).to(torch.uint8)


def _plain_values(codes, scales, dt):
    return torch.ldexp(codes.float(), scales.int()[..., None].clamp(1, 254) - 127).to(dt)


def _plain_load(s):
    valid = s["slots"] >= 0
    at = torch.where(valid, s["slots"], 0).long()
    outs = []
    for n in ("k", "v"):
        codes, scales = s[n + "c"], s[n + "s"]
        x = _plain_values(codes.reshape(-1, *codes.shape[2:])[at], scales.reshape(-1, scales.shape[2])[at], s["k_out"].dtype)
        outs.append(torch.where(valid[:, None, None], x, 0))
    return tuple(outs)


def _plain_store(s):
    valid = s["slots"] >= 0
    first = torch.argmax(valid.to(torch.int32))
    # a token without a slot repeats the first token that has one
    to = torch.where(valid, s["slots"], s["slots"][first]).long()
    for n in ("k", "v"):
        codes, scales = _plain_quantise(s[n], _LIMIT[s["case"]["dtype"]])
        s[n + "c"].view(torch.uint8).reshape(-1, *codes.shape[1:])[to] = torch.where(valid[:, None, None], codes.view(torch.uint8), codes.view(torch.uint8)[first])
        s[n + "s"].reshape(-1, scales.shape[1])[to] = torch.where(valid[:, None], scales, scales[first])
    return _plain_load(s)


def _ancestors(parents):
    """[B, N, N]: whether j is i or above i; a parent outside [0, i) is none."""
    N = parents.shape[1]
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


def _plain_tree(s):
    B, N, Hq, D = s["q"].shape
    ld, page, Hkv = s["table"].shape[1], s["kc"].shape[1], s["kc"].shape[2]
    G = Hq // Hkv
    parents = s["parents"]
    if parents is None:
        parents = (torch.arange(N, device=DEV) - 1).to(torch.int32).expand(B, N)
    above = _ancestors(parents)
    j = torch.arange(ld * page, device=DEV)[None, :] - s["lens"][:, None]  # the node at each place, negative in the cache
    drafted = torch.gather(above, 2, j.clamp(0, N - 1)[:, None, :].expand(B, N, -1)) & (j < N)[:, None, :] & (j >= 0)[:, None, :]
    live = torch.arange(N, device=DEV) < s["sizes"][:, None]
    allowed = ((j < 0)[:, None, :] | drafted) & live[:, :, None]
    at = s["table"].long()
    codes = s["kc"].view(torch.uint8)[at].view(F8).reshape(B, ld * page, Hkv, D)
    k = _plain_values(codes, s["ks"][at].reshape(B, ld * page, Hkv), torch.float32).permute(0, 2, 3, 1).contiguous()
    codes = s["vc"].view(torch.uint8)[at].view(F8).reshape(B, ld * page, Hkv, D)
    v = _plain_values(codes, s["vs"][at].reshape(B, ld * page, Hkv), torch.float32)
    v = torch.where(allowed.any(1)[:, :, None, None], v, 0.0).permute(0, 2, 1, 3).contiguous()
    q = s["q"].float().reshape(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D)
    x = torch.matmul(q, k).reshape(B, Hkv, N, G, -1) / math.sqrt(D)
    x = x.masked_fill_(~allowed[:, None, :, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hkv, N * G, -1), v).reshape(B, Hkv, N, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(s["q"].dtype)
    lse = (m + total.log())[..., 0].permute(0, 2, 1, 3).reshape(B, N, Hq)
    return torch.where(live[:, :, None, None], o, s["out"]), torch.where(live[:, :, None], lse, s["lse"])


def _plain_sample(s):
    """In 64 bits: a sum at a border decides about a token."""
    x = s["logits"].double()
    R, V = x.shape
    t = s["temperature"].double()[:, None]
    greedy = ~(t > 0)
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.exp((x - x[:, :1]) / torch.where(greedy, 1.0, t))
    rank = torch.arange(V, device=DEV)[None, :]
    keep = (rank < 1) | ~greedy
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep = keep & ((rank < k) | (k <= 0))
    w = torch.where(keep, w, 0.0)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        upto = torch.cumsum(w, 1)
        before = torch.cat((torch.zeros_like(upto[:, :1]), upto[:, :-1]), 1)
        keep = keep & ((before < p * upto[:, -1:]) | (rank < 1) | (p >= 1))
    if s["min_p"] is not None:
        keep = keep & (w >= s["min_p"].double()[:, None].clamp(max=1))
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))  # in the order of tokens again
    upto = torch.cumsum(w, 1)
    over = (upto > s["u"].double()[:, None] * upto[:, -1:]) & (w > 0)
    last = (torch.where(w > 0, rank, -1)).amax(1)
    token = torch.where(over.any(1), torch.argmax(over.to(torch.uint8), 1), last)
    logprob = torch.log(torch.gather(w, 1, token[:, None])[:, 0] / upto[:, -1])
    return token.to(torch.int32), logprob.float()


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"rope": _plain_rope, "store": _plain_store, "load": _plain_load, "tree": _plain_tree, "sample": _plain_sample}[op](s)
    from beam_search_top_amd import rtopk
    if op == "rope":
        return rtopk.qk_norm_rope(s["q"], s["k"], s["positions"], s["freqs"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                                  interleaved=s["case"]["pairs"], q_out=s["q_out"], k_out=s["k_out"])
    if op == "store":
        rtopk.cache_store_fp8(s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"])
    if op in ("store", "load"):
        return rtopk.cache_load_fp8(s["kc"], s["vc"], s["ks"], s["vs"], s["slots"], out=(s["k_out"], s["v_out"]))
    if op == "tree":
        return rtopk.tree_attention_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], parents=s["parents"],
                                        sizes=s["sizes"], out=s["out"], lse=s["lse"])
    return rtopk.sample_filtered(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                 min_p=s["min_p"], out=(s["tokens"], s["logprobs"]))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rope":
        n = (c["T"] - c["skip"]) * (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": 2 * n * size + 4 * c["T"] + 2 * c["rot"] + (2 * c["D"] * size if c["norm"] else 0),
                "flops": n * ((4 if c["norm"] else 0) + 3 * c["rot"] // c["D"])}
    if c["op"] in ("store", "load"):
        n = 2 * (c["T"] - c["skip"]) * c["Hkv"]
        load = n * (c["D"] + 1) + 2 * c["T"] * c["Hkv"] * c["D"] * size + 4 * c["T"]
        return {"bytes": load + (n * c["D"] * (size + 1) + n + 4 * c["T"] if c["op"] == "store" else 0), "flops": 0}
    if c["op"] == "tree":
        # every request's average number of nodes: which lengths meet which sizes goes by the seed
        n = sum(_spread(c["B"], (c["N"] + 1) // 2, c["N"]))
        keys = sum(_spread(c["B"], c["least"], c["most"])) + n
        return {"bytes": 2 * keys * c["Hkv"] * (c["D"] + 1) + n * c["Hq"] * (4 * c["D"] + 4) + 4 * (keys // c["page"]) + (4 * n if c["tree"] else 0) + 8 * c["B"],
                "flops": 4 * keys * n // c["B"] * c["Hq"] * c["D"]}
    # a weight's difference, quotient, exponential and sum
    return {"bytes": c["R"] * (c["V"] * size + 28), "flops": 4 * c["R"] * c["V"]}


# ------------------------------------------------------------------ in 64 bits, from the definition
_CODES = np.array([(-1) ** (i >> 7) * ((i & 7) / 8 * 2.0 ** -6 if (i >> 3 & 15) == 0 else (1 + (i & 7) / 8) * 2.0 ** ((i >> 3 & 15) - 7))
                   for i in range(256)])
_CODES[[127, 255]] = np.nan


def _decoded(codes, scales):
    """What codes and bytes of powers of two stand for, in 64 bits."""
    value = torch.from_numpy(_CODES).to(DEV)[codes.view(torch.uint8).int()]
    return value * torch.exp2(scales.double().clamp(1, 254) - 127)[..., None]


def _stored(x, limit):
    """What a stored tensor reads as, in 64 bits: each row on the grid of three bits below its leading one under its power of two."""
    y = x.double()
    fine = torch.isfinite(y)
    a = torch.where(fine, y.abs(), 0.0).amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(torch.clamp(a, min=2.0 ** -200) / 448)).clamp(min=-126)
    e = torch.where(a > 448 * torch.exp2(e), e + 1, e)
    e = torch.where((a <= 448 * torch.exp2(e - 1)) & (e > -126), e - 1, e)
    z = y.abs().clamp(max=limit)
    z = torch.where(fine, z, 1.0)
    lead = torch.floor(torch.log2(torch.clamp(z, min=2.0 ** -200)))
    lead = torch.where(z < torch.exp2(lead), lead - 1, torch.where(z >= torch.exp2(lead + 1), lead + 1, lead))
    step = torch.exp2(torch.maximum(lead, e - 6) - 3)
    return torch.where(fine, torch.sign(y) * torch.round(z / step) * step, math.nan)


def _exact_rope(s, c):
    outs = []
    angle = s["positions"].double()[:, None, None] * s["freqs"].double()
    turn = torch.polar(torch.ones_like(angle), angle)
    rot = c["rot"]
    for x, w, n in ((s["q"], s["qw"], "q_out"), (s["k"], s["kw"], "k_out")):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / c["D"] + 1e-6) * w.double()
        p = y[..., :rot].unflatten(-1, (rot // 2, 2)) if c["pairs"] else y[..., :rot].unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(p.contiguous()) * turn)
        y[..., :rot] = (z if c["pairs"] else z.transpose(-1, -2)).flatten(-2)
        outs.append(torch.where((s["positions"] >= 0)[:, None, None], y, s[n].double()))
    return tuple(outs)


def _exact_tree(s, c):
    B, N, Hq, D = s["q"].shape
    Hkv, page = c["Hkv"], c["page"]
    G = Hq // Hkv
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(B, N, Hq, dtype=torch.float64, device=DEV)
    table, lens, sizes = (s[n].cpu().numpy() for n in ("table", "lens", "sizes"))
    parents = s["parents"].cpu().numpy() if s["parents"] is not None else np.arange(-1, N - 1)[None].repeat(B, 0)
    for b in range(B):
        n, L = int(sizes[b]), int(lens[b])
        at = np.arange(L + n)
        to = torch.from_numpy(table[b, at // page].astype(np.int64) * page + at % page).to(DEV)
        up = np.zeros((n, L + n), dtype=bool)
        up[:, :L] = True
        for i in range(n):
            j = i
            while j >= 0:
                up[i, L + j] = True
                j = int(parents[b, j]) if parents[b, j] < j else -1
        allowed = torch.from_numpy(up).to(DEV).repeat_interleave(G, 0)
        for h in range(Hkv):
            k = _decoded(s["kc"].view(torch.uint8).reshape(-1, Hkv, D)[to, h], s["ks"].reshape(-1, Hkv)[to, h])
            v = _decoded(s["vc"].view(torch.uint8).reshape(-1, Hkv, D)[to, h], s["vs"].reshape(-1, Hkv)[to, h])
            q = s["q"][b, :n, h * G:(h + 1) * G].double().reshape(n * G, D)
            x = (q @ k.T) / math.sqrt(D)
            x = torch.where(allowed, x, torch.full_like(x, -math.inf))
            l = torch.logsumexp(x, -1)
            w = torch.where(allowed, torch.exp(x - l[:, None]), torch.zeros_like(x))
            out[b, :n, h * G:(h + 1) * G] = (w @ v).reshape(n, G, D)
            lse[b, :n, h * G:(h + 1) * G] = l.reshape(n, G)
    return out, lse


def _exact_sample(s, c):
    x = s["logits"].float().cpu().numpy().astype(np.float64)
    got = {n: None if s[n] is None else s[n].cpu().numpy().astype(np.float64) for n in ("u", "temperature", "top_k", "top_p", "min_p")}
    tokens, logprobs = [], []
    for r, row in enumerate(x):
        order = np.argsort(-row, kind="stable")
        t = got["temperature"][r]
        if not t > 0:
            tokens.append(order[0])
            logprobs.append(0.0)
            continue
        w = np.exp((row[order] - row[order[0]]) / t)
        n = len(w)
        if got["top_k"] is not None and got["top_k"][r] > 0:
            n = min(n, int(got["top_k"][r]))
        if got["top_p"] is not None and got["top_p"][r] < 1:
            n = 1 + int(np.searchsorted(np.cumsum(w[:n]), got["top_p"][r] * w[:n].sum(), side="left"))
        if got["min_p"] is not None and got["min_p"][r] > 0:
            n = min(n, int((w >= min(1.0, got["min_p"][r])).sum()))
        kept = np.sort(order[:n])
        w = np.exp((row[kept] - row[order[0]]) / t)
        upto = np.cumsum(w)
        i = min(int(np.searchsorted(upto, got["u"][r] * upto[-1], side="right")), n - 1)
        tokens.append(kept[i])
        logprobs.append(math.log(w[i] / upto[-1]))
    return np.array(tokens, dtype=np.int32), np.array(logprobs)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rope":
        return _exact_rope(s, c)
    if c["op"] == "store":
        valid = (s["slots"] >= 0)[:, None, None]
        return tuple(torch.where(valid, _stored(s[n], _LIMIT[c["dtype"]]), 0.0) for n in ("k", "v"))
    if c["op"] == "load":
        ok = s["slots"] >= 0
        at = s["slots"].long().clamp(min=0)
        outs = []
        for n in ("k", "v"):
            x = _decoded(s[n + "c"].view(torch.uint8).reshape(-1, c["Hkv"], c["D"])[at], s[n + "s"].reshape(-1, c["Hkv"])[at])
            outs.append(torch.where(ok[:, None, None], x, 0.0))
        return tuple(outs)
    if c["op"] == "tree":
        return _exact_tree(s, c)
    return _exact_sample(s, c)
