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
