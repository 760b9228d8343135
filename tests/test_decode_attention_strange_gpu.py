"""mla_tree_attention where values that are not finite lie in drafts that some tokens see and others do not, behind
committed rows of several blocks of the path that takes such rows; the bound is that of test_decode_attention_gpu."""
import math

import pytest
import torch

from tests.test_decode_attention_gpu import SHAPES, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", SHAPES)
def test_strange_values_behind_many_rows(shape, mx):
    c = make(shape, [300, 64, 129], [3, 2, 4], 16, seed=50, mx=mx).tree()
    c.mask[:, 0] = torch.tensor([0b001, 0b010, 0b101, 0b00, 0b11, 0b0001, 0b0010, 0b0100, 0b1111])
    at = lambda s, r: (c.table[s, r // 16].long(), r % 16)  # noqa: E731
    for b in c.bufs:
        if mx and b.shape[3] == c.bufs[0].shape[3] // 32:
            b[at(0, 301)] = 255   # the scales of a draft that token 1 alone sees
            b[at(1, 65)] = 255    # token 4 alone
        elif not mx:
            b[at(0, 301)] = math.nan
            b[at(1, 65)] = math.inf
            b[at(2, 131)][..., 7] = -math.inf  # tokens 7 and 8
    want = c.expected()
    assert torch.isfinite(want[0][0]).all() and not torch.isfinite(want[0][1]).any()
    check(*c.run(), want, c.q.shape[2])
    check(*c.run(max_len=40000), want, c.q.shape[2])


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("n", [1, 3])
def test_committed_values_that_are_not_finite(shape, n):
    """In whole tiles and in the one that the drafts share, up to the last committed row: all tokens see them."""
    c = make(shape, [300, 45, 32, 7], [n] * 4, 16, seed=51).tree()
    at = lambda s, r: (c.table[s, r // 16].long(), r % 16)  # noqa: E731
    v = c.bufs[-1]
    if len(c.bufs) == 1:
        c.q[..., :8] = 0
        c.q[..., 0] = 2.0 ** -20  # (an infinite key element times 0 would be NaN)
    v[at(0, 17)][..., 5] = math.nan
    v[at(0, 290)][..., 6] = math.nan
    v[at(1, 44)][..., 1] = math.nan
    v[at(2, 31)][..., 2] = math.nan
    if len(c.bufs) > 1:
        v[at(0, 298)][..., 3], v[at(0, 299)][..., 4] = math.inf, -math.inf
        v[at(3, 6)][..., 0], v[at(3, 2)][..., 0], v[at(3, 3)][..., 7] = math.inf, math.inf, -math.inf
    want = c.expected()
    assert not torch.isfinite(want[0]).all() and torch.isfinite(want[0]).any()
    check(*c.run(), want, c.q.shape[2])
