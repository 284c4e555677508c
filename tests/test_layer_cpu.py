"""The paged cache's arithmetic (the header the kernels use, compiled for the
CPU) and the refusals of its and the attention entry points. No call here
reaches a launch."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from beam_search_top_amd import rtopk
from libutil import ensure_built

CSRC = os.path.join(os.path.dirname(rtopk.__file__), "csrc")
FAKE = 0x7000_0000  # never dereferenced: every call below fails validation first
E, N = rtopk.RTOPK_EINVAL, rtopk.RTOPK_ENOTSUP


@pytest.fixture(scope="module")
def lib():
    return ensure_built()


@pytest.fixture(scope="module")
def pages(tmp_path_factory):
    d = tmp_path_factory.mktemp("pages")
    src = d / "pages.cpp"
    src.write_text('''#include "rtopk_pages.h"
using namespace rtopk;
extern "C" unsigned div_(unsigned d, unsigned n) { return page_of(make_page_div(d), n); }
extern "C" int slot_(int id, int np, int page, int off) { return slot_of(id, np, page, off); }
extern "C" int parent_(int p, int i) { return parent_of(p, i); }
extern "C" void need_(int page, int c, int n, int ld, int rows, int *out)
{
    const PageNeed r = page_need(make_page_div(page), c, n, ld, rows);
    out[0] = r.c; out[1] = r.n; out[2] = r.have; out[3] = r.need; out[4] = r.fits;
}
''')
    so = d / "pages.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", CSRC, str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so))


def test_page_division(pages):
    pages.div_.restype = ctypes.c_uint
    rng = np.random.default_rng(0)
    for d in [1, 2, 3, 7, 16, 24, 100, 4097, 2 ** 30, 2 ** 31 - 1]:
        for n in [0, 1, d - 1, d, d + 1, 2 ** 31 - 1] + rng.integers(0, 2 ** 31, 200).tolist():
            if n < 2 ** 31:
                assert pages.div_(d, n) == n // d, (n, d)


def test_page_need(pages):
    out = (ctypes.c_int * 5)()
    big = 2 ** 31 - 1
    for page in (1, 5, 16):
        for c in (-3, 0, 1, 15, 16, 17, 100, big):
            for n in (-1, 0, 1, 16, 33, big):
                for ld in (1, 4, 9):
                    for rows in (0, 20):
                        pages.need_(page, c, n, ld, rows, out)
                        cc, nn = max(0, c), max(0, n)
                        fits = cc + nn <= ld * page and (rows == 0 or nn <= rows)
                        have = -(-cc // page) if fits else 0
                        need = -(-(cc + nn) // page) - have if fits else 0
                        assert list(out) == [cc, nn, have, need, int(fits)], (page, c, n, ld, rows)


def test_bad_pages_and_parents(pages):
    assert pages.slot_(-1, 10, 16, 3) == -1 and pages.slot_(10, 10, 16, 3) == -1
    assert pages.slot_(-2 ** 31, 10, 16, 0) == -1 and pages.slot_(2 ** 31 - 1, 10, 16, 0) == -1
    assert pages.slot_(9, 10, 16, 15) == 159 and pages.slot_(0, 10, 16, 0) == 0
    assert [pages.parent_(p, 3) for p in (-5, -1, 0, 2, 3, 4, 1000)] == [-1, -1, 0, 2, -1, -1, -1]
    assert pages.parent_(0, 0) == -1


def _call(fn, order, base, kw):
    a = dict(base)
    a.update(kw)
    st = fn(*[a[n] for n in order])
    return st, rtopk.rtopk_last_error()


def _i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


TABLES = dict(lens=FAKE, new=FAKE, B=4, page=16, free=FAKE, nfree=10, head=None, num_pages=100, table=FAKE, ld=8, slots=FAKE,
              pos=None, T=64, rows=0, cu=FAKE, next=None, stream=None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(lens=None), E, "NULL"), (dict(new=None), E, "NULL"), (dict(table=None), E, "NULL"), (dict(slots=None), E, "NULL"),
    (dict(cu=None), E, "NULL"), (dict(free=None), E, "NULL"),
    (dict(B=0), E, "sizes"), (dict(page=0), E, "sizes"), (dict(num_pages=0), E, "sizes"), (dict(ld=0), E, "sizes"),
    (dict(T=0), E, "sizes"), (dict(nfree=-1), E, "sizes"), (dict(rows=-1), E, "sizes"),
    (dict(B=65537), N, "limit"), (dict(num_pages=2 ** 30), E, "2^31"), (dict(ld=2 ** 28), E, "2^31"),
    (dict(rows=15), E, "B*rows"), (dict(head=FAKE, next=FAKE), E, "different"),
])
def test_page_tables_refusals(lib, kw, status, msg):
    st, err = _call(rtopk.rtopk_page_tables, list(TABLES), TABLES, kw)
    assert st == status and msg in err, err


STORE = dict(k=FAKE, ks=None, v=FAKE, vs=None, dtype=1, slots=FAKE, T=5, Hkv=2, D=64, kc=FAKE, vc=FAKE, cs=None, num_pages=10,
             page=16, stream=None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(k=None), E, "NULL"), (dict(v=None), E, "NULL"), (dict(slots=None), E, "NULL"), (dict(kc=None), E, "NULL"),
    (dict(vc=None), E, "NULL"), (dict(dtype=3), E, "dtype"), (dict(T=0), E, "sizes"), (dict(Hkv=0), E, "sizes"),
    (dict(D=0), E, "sizes"), (dict(num_pages=0), E, "sizes"), (dict(page=-1), E, "sizes"),
    (dict(num_pages=2 ** 28), E, "2^31"), (dict(Hkv=2 ** 15), N, "2^20"), (dict(k=FAKE + 1), E, "aligned"),
    (dict(kc=FAKE + 2, dtype=0), E, "aligned"), (dict(ks=_i64(-64, 64)), E, "strides"),
    (dict(cs=_i64(2 ** 60, 64, 64)), E, "strides"),
])
def test_cache_store_refusals(lib, kw, status, msg):
    st, err = _call(rtopk.rtopk_cache_store, list(STORE), STORE, kw)
    assert st == status and msg in err, err


TREE = dict(q=FAKE, qs=None, kc=FAKE, vc=FAKE, cs=None, dtype=1, table=FAKE, ld=8, num_pages=100, page=16, lens=FAKE,
            parents=None, sizes=None, B=2, N=4, Hq=8, Hkv=2, D=64, scale=0.125, out=FAKE, lse=None, ws=None, nws=0, stream=None)
CROSS = dict(q=FAKE, qs=None, k=FAKE, ks=None, v=FAKE, vs=None, dtype=1, lens=None, mask=None, B=2, N=4, S=100, Hq=8, Hkv=2,
             D=64, scale=0.125, out=FAKE, lse=None, ws=None, nws=0, stream=None)
BOTH = [
    (dict(q=None), E, "NULL"), (dict(out=None), E, "NULL"), (dict(dtype=7), E, "dtype"), (dict(dtype=0), N, "float32"),
    (dict(B=0), E, "sizes"), (dict(N=0), E, "sizes"), (dict(Hq=0), E, "sizes"), (dict(Hkv=0), E, "sizes"), (dict(D=0), E, "sizes"),
    (dict(Hkv=3), E, "multiple of Hkv"), (dict(D=60), N, "D=60"), (dict(D=264), N, "D=264"),
    (dict(scale=float("nan")), E, "scale"), (dict(scale=float("inf")), E, "scale"),
    (dict(q=FAKE + 8), E, "q is not 16"), (dict(out=FAKE + 4), E, "out is not 16"),
    (dict(qs=_i64(2048, 516, 64)), E, "multiple of 8"), (dict(qs=_i64(2048, -512, 64)), E, "negative"),
    (dict(qs=_i64(2 ** 60, 512, 64)), E, "overflow"), (dict(B=2 ** 20, Hq=64, Hkv=2), N, "2^31"),
    (dict(ws=FAKE, nws=256), rtopk.RTOPK_ENOMEM, "workspace"), (dict(ws=FAKE + 16, nws=1 << 30), E, "256-byte"),
]


@pytest.mark.parametrize("kw,status,msg", BOTH + [
    (dict(kc=None), E, "NULL"), (dict(vc=None), E, "NULL"), (dict(table=None), E, "NULL"), (dict(lens=None), E, "NULL"),
    (dict(kc=FAKE + 2), E, "k_cache is not 16"), (dict(vc=FAKE + 2), E, "v_cache is not 16"),
    (dict(cs=_i64(16 * 128, 130, 64)), E, "multiple of 8"), (dict(N=257), N, "N=257"),
    (dict(ld=0), E, "sizes"), (dict(num_pages=0), E, "sizes"), (dict(page=0), E, "sizes"),
    (dict(num_pages=2 ** 28), E, "2^31"), (dict(ld=2 ** 28), E, "2^31"),
])
def test_tree_attention_refusals(lib, kw, status, msg):
    st, err = _call(rtopk.rtopk_tree_attention, list(TREE), TREE, kw)
    assert st == status and msg in err, err


@pytest.mark.parametrize("kw,status,msg", BOTH + [
    (dict(k=None), E, "NULL"), (dict(v=None), E, "NULL"), (dict(S=0), E, "S=0"), (dict(S=2 ** 31 - 1), N, "S="),
    (dict(k=FAKE + 2), E, "k is not 16"), (dict(v=FAKE + 2), E, "v is not 16"),
    (dict(ks=_i64(12800, 132, 64)), E, "multiple of 8"), (dict(vs=_i64(12800, 128, -64)), E, "negative"),
])
def test_cross_attention_refusals(lib, kw, status, msg):
    st, err = _call(rtopk.rtopk_cross_attention, list(CROSS), CROSS, kw)
    assert st == status and msg in err, err


def test_workspace_sizes(lib):
    assert rtopk.rtopk_cross_attention_workspace_bytes(2, 4, 100, 8, 2, 64) >= rtopk.RTOPK_WS_FIXED_BYTES
    assert rtopk.rtopk_tree_attention_workspace_bytes(2, 4, 8, 2, 64, 8, 16) >= rtopk.RTOPK_WS_FIXED_BYTES
    assert rtopk.rtopk_cross_attention_workspace_bytes(2, 4, 0, 8, 2, 64) == 0
    assert rtopk.rtopk_cross_attention_workspace_bytes(2, 4, 100, 8, 3, 64) == 0
    assert rtopk.rtopk_tree_attention_workspace_bytes(2, 300, 8, 2, 64, 8, 16) == 0
    assert rtopk.rtopk_tree_attention_workspace_bytes(2, 4, 8, 2, 64, 0, 16) == 0


def test_binding_rejects_host_tensors(lib):
    q = torch.zeros(1, 1, 2, 64, dtype=torch.float16)
    k = torch.zeros(1, 4, 2, 64, dtype=torch.float16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        rtopk.cross_attention(q, k, k)
    with pytest.raises(ValueError):
        rtopk.tree_attention(q, k, k, i[None], i)
    with pytest.raises(ValueError):
        rtopk.cache_store(k[0], k[0], i, k, k)
    with pytest.raises(ValueError):
        rtopk.page_tables(i, i, 16, i, i[None], 4, tokens=4)
