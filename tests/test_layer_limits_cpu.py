"""Limits of one launch and of the scale, checked before anything reaches the GPU."""
import pytest

from beam_search_top_amd import rtopk
from test_layer_cpu import CROSS, TREE, _call, lib  # noqa: F401

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
