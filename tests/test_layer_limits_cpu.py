"""Limits of one launch and of the scale, kept before anything reaches the GPU."""
import ctypes
import subprocess

import pytest

from beam_search_top_amd import rtopk
from test_layer_cpu import CROSS, CSRC, TREE, _call, lib  # noqa: F401

E, N = rtopk.RTOPK_EINVAL, rtopk.RTOPK_ENOTSUP


@pytest.mark.parametrize("scale", [2.5e38, -2.5e38, 3.4e38])
def test_scales_whose_base_2_form_overflows_are_refused(lib, scale):  # noqa: F811
    # scale * log2(e) is infinite: 0 * infinity would make a score of zero NaN
    for fn, base in ((rtopk.rtopk_tree_attention, TREE), (rtopk.rtopk_cross_attention, CROSS)):
        st, err = _call(fn, list(base), base, dict(scale=scale))
        assert st == E and "scale" in err, err


@pytest.mark.parametrize("B,Hkv", [(1 << 24, 1), (1 << 23, 2), (1 << 22, 8)])
def test_more_threads_than_one_launch_takes_are_refused(lib, B, Hkv):  # noqa: F811
    # a workgroup of 256 threads per batch element and key head: 2^32 of them, which a launch cannot count
    for fn, base in ((rtopk.rtopk_tree_attention, TREE), (rtopk.rtopk_cross_attention, CROSS)):
        st, err = _call(fn, list(base), base, dict(B=B, N=1, Hq=Hkv, Hkv=Hkv, D=8))
        assert st == N and "one launch" in err, err


@pytest.fixture(scope="module")
def store(tmp_path_factory):
    d = tmp_path_factory.mktemp("store")
    (d / "store.cpp").write_text('''#include "rtopk_pages.h"
extern "C" long long per_(long long T, int row) { return rtopk::store_tokens(T, row, 1024); }
''')
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "store.cpp"), "-o", str(d / "store.so")],
                   check=True)
    fn = ctypes.CDLL(str(d / "store.so")).per_
    fn.argtypes, fn.restype = [ctypes.c_longlong, ctypes.c_int], ctypes.c_longlong
    return fn


def test_the_store_fits_one_launch(store):
    # workgroups of 256 threads: fewer than 2^24 of them; a workgroup's units are counted below 2^31
    for T in (1, 5, 1000, (1 << 24) - 1, 1 << 24, (1 << 24) + 3, 123456789, (1 << 31) - 1):
        for row in (1, 8, 100, 1023, 1024, 1025, 1 << 20):
            per = store(T, row)
            assert per >= 1 and -(-T // per) * 256 < 1 << 32 and per * row < 1 << 31, (T, row, per)
            if T < 1 << 24:
                assert per == max(1, 1024 // row)
