"""The paged cache in 8 bits on the GPU: what is stored and read back, bit by
bit, against the format's definition (serve_ref.py)."""
import numpy as np
import pytest
import torch

from beam_search_top_amd import rtopk
from libutil import ensure_built
from serve_ref import CODES, quantise, values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ensure_built()


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _cache(g, pages, page, Hkv, D, layout="nhd"):
    shape = (pages, page, Hkv, D) if layout == "nhd" else (pages, Hkv, page, D)
    c = [torch.randint(0, 256, shape, generator=g, device=DEV).to(torch.uint8) for _ in range(2)]
    if layout != "nhd":
        c = [x.transpose(1, 2) for x in c]
    return c + [torch.randint(0, 256, (pages, page, Hkv), generator=g, device=DEV).to(torch.uint8) for _ in range(2)]


def _same(a, b):
    """Equal values, NaN where NaN."""
    a, b = torch.as_tensor(a).double(), torch.as_tensor(b).double()
    return torch.equal(torch.nan_to_num(a, nan=1e300), torch.nan_to_num(b, nan=1e300))


def _store(k, v, slots, cache):
    """Stores, and holds the whole cache to what it has to be."""
    kc, vc, ks, vs = cache
    nslots = kc.shape[0] * kc.shape[1]
    want = [c.cpu().numpy().reshape(nslots, *c.shape[2:]).copy() for c in (kc, vc, ks, vs)]
    for n, x in enumerate((k, v)):
        codes, scales = quantise(x)
        for t, s in enumerate(slots.reshape(-1).tolist()):
            if 0 <= s < nslots:
                want[n][s] = codes.reshape(-1, *codes.shape[-2:])[t]
                want[n + 2][s] = scales.reshape(-1, scales.shape[-1])[t]
    rtopk.cache_store_fp8(k, v, slots, kc, vc, ks, vs)
    torch.cuda.synchronize()
    for n, (c, name) in enumerate(zip((kc, vc, ks, vs), ("k codes", "v codes", "k scales", "v scales"))):
        got = c.cpu().numpy().reshape(nslots, *c.shape[2:])
        if n < 2:  # a NaN has two codes, and a sign
            got, w = np.where(got & 127 == 127, 127, got), np.where(want[n] & 127 == 127, 127, want[n])
        else:
            w = want[n]
        assert np.array_equal(got, w), name


@pytest.mark.parametrize("T,Hkv,D,page,dt,layout", [
    (1, 1, 64, 16, F16, "nhd"), (37, 3, 80, 24, BF16, "nhd"), (500, 8, 128, 16, BF16, "hnd"), (65, 2, 7, 5, F16, "nhd"),
    (33, 4, 16, 1, F32, "hnd"), (20, 1, 3, 4, F32, "nhd"), (300, 16, 64, 64, F16, "nhd"), (3, 64, 256, 16, F16, "nhd"),
    (9, 2, 192, 8, F32, "nhd"), (5, 1, 1, 3, BF16, "nhd"), (12, 3, 250, 8, BF16, "hnd"),
])
def test_store_and_load(T, Hkv, D, page, dt, layout):
    print(f"[cache8] T={T} Hkv={Hkv} D={D} page={page} {dt} {layout}", flush=True)
    g = _gen(T + D)
    pages = T // page + 3
    cache = _cache(g, pages, page, Hkv, D, layout)
    kv = (torch.randn(T, 2, Hkv, D, generator=g, device=DEV) * torch.exp(3 * torch.randn(T, 2, Hkv, 1, generator=g, device=DEV))).to(dt)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:T].to(torch.int32)
    slots[T // 2::7] = -1
    if T > 8:
        slots[1], slots[2] = pages * page, 2 ** 31 - 1
    _store(kv[:, 0], kv[:, 1], slots, cache)
    for out_dt in (dt, F32):
        k, v = rtopk.cache_load_fp8(*cache, slots, dtype=out_dt)
        torch.cuda.synchronize()
        ok = ((slots >= 0) & (slots < pages * page)).cpu()
        for got, x in ((k, kv[:, 0]), (v, kv[:, 1])):
            want = torch.from_numpy(values(*quantise(x)))
            assert (got.cpu()[~ok] == 0).all()
            assert _same(got.cpu()[ok], want[ok])  # exact in the type that was stored
            # and off by half a step at most, 2^-4 of an element or 2^-17 of its row's largest; infinities, which
            # some of these rows hold in float16, are NaN then
            xd = x.double().cpu()
            fine = torch.isfinite(xd)
            size = torch.where(fine, xd.abs(), 0.0)
            within = (want - xd).abs() <= torch.maximum(size * 2.0 ** -4, size.amax(-1, keepdim=True) * 2.0 ** -17)
            assert torch.equal(torch.isfinite(want), fine) and within[fine].all()


@pytest.mark.parametrize("dt", [F16, BF16, F32])
@pytest.mark.parametrize("D", [64, 6])
def test_values_at_the_edges(dt, D):
    # borders between codes, ties, subnormal codes, the largest of the type, tiny numbers, signed zeros, infinities, NaN
    big = torch.finfo(dt).max
    tiny = {F16: 2.0 ** -24, BF16: 2.0 ** -133, F32: 2.0 ** -149}[dt]
    rows = []
    base = [448, 447, 240, 17, 18, 19, 20, 21, 22, 23, 1.0625, 1.1875, 1.0 / 512, 1.0 / 1024, 3.0 / 1024, 1.5 / 1024, -0.0, 0.0, -7.5]
    for e in (-8, 0, 5):
        rows.append([x * 2.0 ** e for x in base])
    rows += [[449], [464], [465], [-896.0], [big, 1.0, big / 2], [-big, big, 61440.0, 63487.0], [tiny, -tiny, 3 * tiny], [0.0], [-0.0],
             [float("inf"), 1.0, -2.0], [float("-inf")], [float("nan"), 5.0], [float("nan"), float("inf")], [448 * 2.0 ** -14, 449 * 2.0 ** -14]]
    x = torch.zeros(len(rows), 1, D, dtype=torch.float64)
    for i, r in enumerate(rows):
        r = (r * D)[:D]
        x[i, 0, :len(r)] = torch.tensor(r, dtype=torch.float64)
    x = x.to(dt).to(DEV)
    T = len(rows)
    cache = _cache(_gen(1), T, 1, 1, D)
    slots = torch.arange(T, dtype=torch.int32, device=DEV)
    _store(x, x.flip(0), slots, cache)
    k, v = rtopk.cache_load_fp8(*cache, slots, dtype=dt)
    torch.cuda.synchronize()
    assert _same(k.cpu(), values(*quantise(x))) and _same(v.cpu(), values(*quantise(x.flip(0))))
    assert torch.equal(torch.isfinite(k), torch.isfinite(x))


@pytest.mark.parametrize("dt", [F16, BF16, F32])
def test_every_code_and_scale_reads_back(dt):
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).expand(256, 1, 1, 256).contiguous()
    scales = torch.arange(256, dtype=torch.uint8, device=DEV).view(256, 1, 1)
    slots = torch.arange(256, dtype=torch.int32, device=DEV)
    k, v = rtopk.cache_load_fp8(codes.view(F8), codes.flip(3).contiguous().view(F8), scales, scales.flip(0).contiguous(), slots, dtype=dt)
    torch.cuda.synchronize()
    c, s = codes.cpu().numpy().reshape(256, 256), scales.cpu().numpy().reshape(256)
    for got, want in ((k, values(c, s)), (v, values(c[:, ::-1], s[::-1]))):
        with np.errstate(over="ignore"):
            want = torch.from_numpy(want).float().to(dt)  # exact in 32 bits, and rounded once
        assert _same(got.cpu().reshape(256, 256), want)


def test_unaligned_views_and_repeated_slots():
    g = _gen(3)
    B, N, Hkv, D, page, pages = 3, 5, 2, 32, 8, 9
    k = torch.randn(B * N * Hkv * D + 1, generator=g, device=DEV).to(F16)[1:].view(B, N, Hkv, D)  # two bytes off a boundary
    v = torch.randn(B, N, Hkv, D, generator=g, device=DEV).to(F16)
    cache = _cache(g, pages, page, Hkv, D)
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:B * N].to(torch.int32).view(B, N)
    slots[1, 3:] = -1
    _store(k, v, slots, cache)
    again = slots[[0, 0, 2]].contiguous()  # a beginning that two requests share
    got = rtopk.cache_load_fp8(*cache, again, dtype=F16)
    off = torch.empty(2, again.numel() * Hkv * D + 1, dtype=F16, device=DEV)[:, 1:]
    out = tuple(o.view(3, N, Hkv, D) for o in off)
    rtopk.cache_load_fp8(*cache, again, out=out)
    torch.cuda.synchronize()
    assert torch.equal(got[0], out[0]) and torch.equal(got[1], out[1]) and torch.equal(got[0][0], got[0][1])


def test_captured_store_and_load():
    g = _gen(5)
    T, Hkv, D = 40, 4, 64
    cache = _cache(g, 8, 16, Hkv, D)
    k, v = (torch.randn(T, Hkv, D, generator=g, device=DEV).to(BF16) for _ in range(2))
    slots = torch.randperm(128, generator=g, device=DEV)[:T].to(torch.int32)
    out = (torch.zeros_like(k), torch.zeros_like(v))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rtopk.cache_store_fp8(k, v, slots, *cache)
        rtopk.cache_load_fp8(*cache, slots, out=out)
    for i in range(3):
        k.mul_(-1.7), v.add_(0.3)
        slots.copy_(torch.randperm(128, generator=g, device=DEV)[:T])
        graph.replay()
        torch.cuda.synchronize()
        assert _same(out[0].cpu(), values(*quantise(k))) and _same(out[1].cpu(), values(*quantise(v))), i


def test_far_slots():
    # a cache whose bytes pass 2^32: offsets in 64 bits
    Hkv, D, page, pages = 8, 128, 64, 66000
    kc, vc = (torch.zeros(pages, page, Hkv, D, dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros(pages, page, Hkv, dtype=torch.uint8, device=DEV) for _ in range(2))
    assert kc.numel() > 2 ** 32
    slots = torch.tensor([pages * page - 1, 0, 4194304, 4194303, pages * page - 65], dtype=torch.int32, device=DEV)
    k, v = (torch.randn(5, Hkv, D, generator=_gen(6), device=DEV).to(BF16) for _ in range(2))
    rtopk.cache_store_fp8(k, v, slots, kc, vc, ks, vs)
    got = rtopk.cache_load_fp8(kc, vc, ks, vs, slots, dtype=BF16)
    torch.cuda.synchronize()
    assert _same(got[0].cpu(), values(*quantise(k))) and _same(got[1].cpu(), values(*quantise(v)))
    written = sorted((ks.view(-1, Hkv) != 0).any(1).nonzero().flatten().tolist())
    assert written == sorted(slots.tolist())


def test_codes_are_those_of_torch():
    assert _same(torch.arange(256, dtype=torch.uint8).view(F8).double(), CODES)
