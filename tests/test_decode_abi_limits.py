"""Refusals of decode-side calls whose sizes or numbers lie past what the kernels' grids and fp32 hold, without a GPU."""
import ctypes

import pytest

from mla_up_projection_amd import binding as bd
from tests.test_decode_abi import L, attn, w4  # noqa: F401


@pytest.mark.parametrize("heads,code", [(2796202, bd.MLA_EALIAS), (2796203, bd.MLA_EUNSUPPORTED), (5592405, bd.MLA_EUNSUPPORTED),
                                        (5592406, bd.MLA_EINVAL)])
def test_w4_columns(L, heads, code):  # noqa: F811
    """2^29 columns and more have no grid (8 work-items a column, 2^32 in a launch). Below, the call goes on to the check
    of overlaps, which these arguments fail."""
    assert L.mla_qup_fwd_w4(ctypes.byref(w4(H=heads, K=32, out=w4().x)), None) == code


@pytest.mark.parametrize("scale", [3e38, -3e38])
def test_attention_scale(L, scale):  # noqa: F811
    """Scores are in powers of two: the scale times log2 e must be a number in fp32 too."""
    assert L.mla_tree_attention(ctypes.byref(attn(scale=scale)), None) == bd.MLA_EINVAL
    assert L.mla_tree_attention_workspace_size(ctypes.byref(attn(scale=scale))) == 0
    assert L.mla_tree_attention_workspace_size(ctypes.byref(attn(scale=scale / 2))) > 0
