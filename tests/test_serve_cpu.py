"""The arithmetic of the 8-bit cache's format (the header the kernels use,
compiled for the CPU) and the refusals of the rotation, the 8-bit cache and filtered
sampling. No call here reaches a launch."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from beam_search_top_amd import rtopk
from libutil import ensure_built
from serve_ref import CODES, quantise, sample, values

CSRC = os.path.join(os.path.dirname(rtopk.__file__), "csrc")
FAKE = 0x7000_0000  # never dereferenced: every call below fails validation first
E, N = rtopk.RTOPK_EINVAL, rtopk.RTOPK_ENOTSUP


@pytest.fixture(scope="module")
def lib():
    return ensure_built()


@pytest.fixture(scope="module")
def arith(tmp_path_factory):
    d = tmp_path_factory.mktemp("cache8")
    src = d / "cache8.cpp"
    src.write_text('''#define RTOPK_ARITHMETIC_ONLY
#include "rtopk_cache8.h"
using namespace rtopk;
extern "C" unsigned scale_(float a) { unsigned b; memcpy(&b, &a, 4); return scale_of(b); }
extern "C" float power_(unsigned s) { unsigned b = scale_bits(held_scale(s)); float f; memcpy(&f, &b, 4); return f; }
extern "C" float inverse_(unsigned s) { unsigned b = inverse_bits(s); float f; memcpy(&f, &b, 4); return f; }
extern "C" float limit_(int dt) { return stored_limit(dt); }
extern "C" int tokens_(long long T, long long row) { return rope_tokens(T, row); }
''')
    so = d / "cache8.so"
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I", CSRC, str(src), "-o", str(so)], check=True)
    L = ctypes.CDLL(str(so))
    L.scale_.argtypes = [ctypes.c_float]
    L.tokens_.argtypes = [ctypes.c_longlong] * 2
    for f in (L.power_, L.inverse_, L.limit_):
        f.restype = ctypes.c_float
    return L


def test_scales(arith):
    rng = np.random.default_rng(0)
    xs = [0.0, 2.0 ** -149, 2.0 ** -126, 448 * 2.0 ** -126, 449 * 2.0 ** -126, 1.0, 1.75, 448.0, 448.1, 464.0, 512.0, 65504.0, 3.4e38]
    xs += (2.0 ** rng.uniform(-149, 127.9, 3000)).tolist()
    for x in np.float32(xs):
        s = arith.scale_(float(x))
        assert 1 <= s <= 247
        p = 2.0 ** (s - 127)
        assert float(x) <= 448 * p and (s == 1 or float(x) > 448 * p / 2)
        assert arith.power_(s) == p and arith.inverse_(s) * p == 1
    assert arith.power_(0) == 2.0 ** -126 and arith.power_(255) == 2.0 ** 127
    assert arith.limit_(1) == 61440 and arith.limit_(0) == arith.limit_(2) == 240 * 2.0 ** 120


def test_rope_tokens_fit(arith):
    for T in (1, 200, 10 ** 6, 2 ** 24 + 5, 2 ** 28):
        for row in (1, 7, 128, 4096, 5120, 2 ** 20):
            n = arith.tokens_(T, row)
            assert 1 <= n <= 17 and (T + n - 1) // n < 2 ** 24


def test_the_reference_quantises_as_torch_does():
    x = torch.randn(300, 64, dtype=torch.float64, generator=torch.Generator().manual_seed(1)).float()
    codes, scales = quantise(x)
    y = (x / torch.from_numpy(2.0 ** (scales.astype(np.float64) - 127)).float()[:, None]).to(torch.float8_e4m3fn)
    assert torch.equal(y.double(), torch.from_numpy(CODES[codes]))
    assert np.abs(values(codes, scales) - x.double().numpy()).max() < 2.0 ** -4 * 5


def test_the_reference_samples():
    row = np.array([1.0, 3.0, 3.0, 2.0, -math.inf])
    assert sample(row, 0.0) == (0, pytest.approx(math.log(math.exp(-2) / (2 + math.exp(-2) + math.exp(-1)))))
    assert sample(row, 0.9, k=1) == (1, 0.0) and sample(row, 0.9, k=2) == (2, pytest.approx(math.log(0.5)))
    assert sample(row, 0.5, p=0.5) [0] == 2 and sample(row, 0.4, p=0.3) == (1, 0.0)
    assert sample(row, 0.99, m=0.5)[0] == 2 and sample(row, 1.0)[0] == 3 and sample(row, 0.3, temperature=0)[0] == 1


def _call(fn, base, kw):
    a = dict(base)
    a.update(kw)
    return fn(*a.values()), rtopk.rtopk_last_error()


def _i64(*v):
    return (ctypes.c_int64 * len(v))(*v)


ROPE = dict(q=FAKE, qs=None, k=FAKE + 2 ** 20, ks=None, dtype=1, pos=FAKE, freqs=FAKE, rot=64, pairs=0, qw=None, kw=None, eps=1e-6, T=5, Hq=4,
            Hkv=2, D=64, qo=FAKE + 2 ** 21, qos=None, ko=FAKE + 2 ** 22, kos=None, stream=None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(q=None), E, "NULL"), (dict(k=None), E, "NULL"), (dict(pos=None), E, "NULL"), (dict(freqs=None), E, "NULL"),
    (dict(qo=None), E, "NULL"), (dict(ko=None), E, "NULL"), (dict(dtype=3), E, "dtype"), (dict(dtype=-1), E, "dtype"),
    (dict(T=0), E, "sizes"), (dict(Hq=0), E, "sizes"), (dict(Hkv=-1), E, "sizes"), (dict(D=0), E, "sizes"),
    (dict(rot=-2), E, "rot"), (dict(rot=7), E, "rot"), (dict(rot=66), E, "rot"),
    (dict(eps=-1e-6), E, "eps"), (dict(eps=math.nan), E, "eps"), (dict(eps=-math.nan), E, "eps"), (dict(eps=math.inf), E, "eps"),
    (dict(D=257), N, "256"), (dict(Hq=2 ** 14), N, "2^20"), (dict(Hq=2 ** 31 - 1), N, "2^20"), (dict(T=2 ** 28 + 1), N, "2^28"),
    (dict(q=FAKE + 1), E, "aligned"), (dict(qw=FAKE + 1), E, "aligned"), (dict(ko=FAKE + 2 ** 22 + 2, dtype=0), E, "aligned"),
    (dict(qs=_i64(-64, 64)), E, "strides"), (dict(kos=_i64(2 ** 62, 64)), E, "strides"),
    (dict(qos=_i64(0, 64)), E, "overlap"), (dict(qos=_i64(256, 63)), E, "overlap"), (dict(kos=_i64(127, 64)), E, "overlap"),
    (dict(qos=_i64(64, 64 * 4)), E, "overlap"),
    (dict(qo=FAKE, qs=_i64(512, 64)), E, "in place"), (dict(ko=FAKE + 2 ** 20, kos=_i64(512, 64)), E, "in place"),
    (dict(qo=FAKE + 2 ** 22), E, "own"), (dict(qo=FAKE + 2 ** 20), E, "own"), (dict(ko=FAKE), E, "own"),
])
def test_rope_refusals(lib, kw, status, msg):
    st, err = _call(rtopk.rtopk_qk_norm_rope, ROPE, kw)
    assert st == status and msg in err, err


STORE = dict(k=FAKE, ks=None, v=FAKE, vs=None, dtype=1, slots=FAKE, T=5, Hkv=2, D=64, kc=FAKE, vc=FAKE + 2 ** 20, cs=None, ksc=FAKE,
             vsc=FAKE + 2 ** 20, num_pages=10, page=16, stream=None)
LOAD = dict(kc=FAKE, vc=FAKE, cs=None, ksc=FAKE, vsc=FAKE, num_pages=10, page=16, slots=FAKE, T=5, Hkv=2, D=64, ko=FAKE, vo=FAKE + 2 ** 20,
            dtype=1, stream=None)
BOTH = [
    (dict(kc=None), E, "NULL"), (dict(vc=None), E, "NULL"), (dict(ksc=None), E, "NULL"), (dict(vsc=None), E, "NULL"), (dict(slots=None), E, "NULL"),
    (dict(dtype=3), E, "dtype"), (dict(T=0), E, "sizes"), (dict(Hkv=0), E, "sizes"), (dict(D=0), E, "sizes"), (dict(num_pages=0), E, "sizes"),
    (dict(page=-1), E, "sizes"), (dict(num_pages=2 ** 28), E, "2^31"), (dict(D=257), N, "256"), (dict(Hkv=2 ** 15), N, "2^20"),
    (dict(cs=_i64(2 ** 60, 64, 64)), E, "strides"), (dict(cs=_i64(2048, -1, 64)), E, "strides"),
]


@pytest.mark.parametrize("kw,status,msg", BOTH + [
    (dict(k=None), E, "NULL"), (dict(v=None), E, "NULL"), (dict(k=FAKE + 1), E, "aligned"), (dict(v=FAKE + 2, dtype=0), E, "aligned"),
    (dict(ks=_i64(-64, 64)), E, "strides"), (dict(vc=FAKE), E, "own"), (dict(vsc=FAKE), E, "own"),
])
def test_store_refusals(lib, kw, status, msg):
    st, err = _call(rtopk.rtopk_cache_store_fp8, STORE, kw)
    assert st == status and msg in err, err


@pytest.mark.parametrize("kw,status,msg", BOTH + [
    (dict(ko=None), E, "NULL"), (dict(vo=None), E, "NULL"), (dict(ko=FAKE + 1), E, "aligned"), (dict(vo=FAKE), E, "own"),
])
def test_load_refusals(lib, kw, status, msg):
    st, err = _call(rtopk.rtopk_cache_load_fp8, LOAD, kw)
    assert st == status and msg in err, err


FILTER = dict(logits=FAKE, dtype=1, R=4, V=100, ld=100, t=None, k=None, p=None, m=None, u=FAKE, tok=FAKE, lp=FAKE, ws=None, nws=0, stream=None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(logits=None), E, "NULL"), (dict(u=None), E, "NULL"), (dict(tok=None), E, "NULL"), (dict(lp=None), E, "NULL"),
    (dict(dtype=3), E, "dtype"), (dict(R=0), E, "sizes"), (dict(V=0), E, "sizes"), (dict(ld=99), E, "rows"), (dict(ld=-1, R=1), E, "rows"),
    (dict(ld=2 ** 41), E, "rows"), (dict(logits=FAKE + 1), E, "aligned"), (dict(logits=FAKE + 2, dtype=0), E, "aligned"),
    (dict(V=2 ** 24 + 1, ld=2 ** 25), N, "limit"), (dict(R=2 ** 20 + 1), N, "limit"),
    (dict(ws=FAKE + 16, nws=1 << 30), E, "256-byte"), (dict(ws=FAKE, nws=100), rtopk.RTOPK_ENOMEM, "workspace"),
    (dict(ws=FAKE, nws=49920 * 4, V=50000, ld=50000), rtopk.RTOPK_ENOMEM, "workspace"),
])
def test_filter_refusals(lib, kw, status, msg):
    st, err = _call(rtopk.rtopk_sample_filtered, FILTER, kw)
    assert st == status and msg in err, err


def test_filter_workspace_sizes(lib):
    assert all(rtopk.rtopk_sample_filtered_workspace_bytes(*s) == 0 for s in ((0, 5), (5, 0), (1, 2 ** 24 + 1), (2 ** 20 + 1, 5)))
    few, long, many = (rtopk.rtopk_sample_filtered_workspace_bytes(*s) for s in ((8, 1000), (8, 250000), (2 ** 20, 2 ** 24)))
    assert 0 < few < long and many == few


def test_host_tensors_are_refused(lib):
    x = torch.zeros(4, 2, 64)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        rtopk.qk_norm_rope(x, x, i, torch.zeros(32))
    with pytest.raises(ValueError, match="device tensor"):
        rtopk.cache_store_fp8(x, x, i, None, None, None, None)
    with pytest.raises(ValueError, match="device tensor"):
        rtopk.cache_load_fp8(torch.zeros(2, 4, 2, 64, dtype=torch.uint8), None, None, None, i)
    with pytest.raises(ValueError, match="device tensor"):
        rtopk.sample_filtered(torch.zeros(4, 100), torch.zeros(4))


TREE8 = dict(q=FAKE, qs=None, kc=FAKE, vc=FAKE, cs=None, ksc=FAKE, vsc=FAKE, dtype=1, table=FAKE, ld=8, num_pages=100, page=16, lens=FAKE,
             parents=None, sizes=None, B=2, N=4, Hq=8, Hkv=2, D=64, scale=0.125, out=FAKE, lse=None, ws=None, nws=0, stream=None)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(q=None), E, "NULL"), (dict(out=None), E, "NULL"), (dict(kc=None), E, "NULL"), (dict(vc=None), E, "NULL"), (dict(ksc=None), E, "NULL"),
    (dict(vsc=None), E, "NULL"), (dict(table=None), E, "NULL"), (dict(lens=None), E, "NULL"), (dict(dtype=7), E, "dtype"),
    (dict(dtype=0), N, "float32"), (dict(B=0), E, "sizes"), (dict(N=0), E, "sizes"), (dict(D=0), E, "sizes"), (dict(Hkv=3), E, "multiple of Hkv"),
    (dict(D=72), N, "multiple of 16"), (dict(D=8), N, "multiple of 16"), (dict(D=272), N, "D=272"), (dict(N=257), N, "N=257"),
    (dict(scale=math.nan), E, "scale"), (dict(scale=math.inf), E, "scale"), (dict(q=FAKE + 8), E, "q is not 16"), (dict(out=FAKE + 4), E, "out is not 16"),
    (dict(kc=FAKE + 8), E, "k_cache is not 16"), (dict(vc=FAKE + 4), E, "v_cache is not 16"), (dict(qs=_i64(2048, 516, 64)), E, "multiple of 8"),
    (dict(cs=_i64(2048, 136, 64)), E, "multiple of 16"), (dict(cs=_i64(2048, -128, 64)), E, "negative"), (dict(cs=_i64(2 ** 60, 128, 64)), E, "overflow"),
    (dict(num_pages=2 ** 28), E, "2^31"), (dict(ld=2 ** 28), E, "2^31"), (dict(ld=0), E, "sizes"), (dict(page=0), E, "sizes"),
    (dict(ws=FAKE, nws=256), rtopk.RTOPK_ENOMEM, "workspace"), (dict(ws=FAKE + 16, nws=1 << 30), E, "256-byte"), (dict(B=2 ** 20, Hq=64, Hkv=2), N, "2^31"),
])
def test_tree_attention_refusals(lib, kw, status, msg):
    st, err = _call(rtopk.rtopk_tree_attention_fp8, TREE8, kw)
    assert st == status and msg in err, err
