"""mla_tree_attention at the ends of fp32's range: scores that rise along the cache, and values so large that a sum
taken relative to an early, smaller score leaves the range although the result does not. The bound of an output
element is that of test_decode_attention_gpu; the largest values here are 2^127, so that a result that is off by
half a bf16 step is still finite."""
import math

import pytest
import torch

from tests.test_decode_attention_gpu import SHAPES, check, make

pytestmark = pytest.mark.gpu


def row(c, seq, r):
    return c.table[seq, r // c.page].long(), r % c.page


def lift(c, seq, r, t, h, powers):
    """Move key row r of the sequence along query (t, h), so that their score is `powers` powers of two."""
    pg, rr = row(c, seq, r)
    q = c.q[t, h].double()
    k = c.bufs[0][pg, rr, h // (c.q.shape[1] // c.bufs[0].shape[2])]
    k += (q * ((powers * math.log(2) / c.scale - k.double() @ q) / (q @ q))).to(k.dtype)


def quantize(c):
    """The case with an MXFP8 cache."""
    import mla_up_projection_amd as m
    out = []
    for b in c.bufs:
        codes = torch.empty(b.shape, dtype=torch.uint8, device="cuda")
        sc = torch.empty(*b.shape[:-1], b.shape[-1] // 32, dtype=torch.uint8, device="cuda")
        m.mxfp8_quantize(b.view(-1, b.shape[-1]).cuda(), codes.view(-1, b.shape[-1]), sc.view(-1, b.shape[-1] // 32))
        out += [codes.cpu(), sc.cpu()]
    c.bufs, c.mx = out, True
    return c


def scores(c, t, h, seq):
    """Of the committed rows, in powers of two."""
    from tests import decode_ref as ref
    key, _ = ref.cache_values(c.bufs, c.mx)
    at = [row(c, seq, r) for r in range(c.lens[seq])]
    k = torch.stack([key[pg, rr, h // (c.q.shape[1] // key.shape[2])] for pg, rr in at])
    return (k @ c.q[t, h].double()) * c.scale / math.log(2)


def values(c):
    """The value columns of a bf16 case, with the queries zero where a latent cache's large columns are: [.., 32]."""
    if len(c.bufs) == 1:
        c.q[..., :32] = 0
        return c.bufs[0][..., :32]
    return c.bufs[1][..., :32]


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("power", [70, 100])
@pytest.mark.parametrize("shape", SHAPES)
def test_large_values_behind_a_rising_score(shape, power, mx):
    """Scores rise by 60 powers of two after the first tile, less than makes a row start again by itself, with values
    of 2^70 and 2^100: relative to the first tile's scores the sums reach 2^130 and 2^160."""
    c = make(shape, [150, 9], [2, 1], 16, seed=40)
    v = values(c)
    v *= 2.0 ** power
    lift(c, 0, 100, 0, 0, 60)
    lift(c, 0, 140, 1, 1, 58)
    if mx:
        quantize(c)
    s = scores(c, 0, 0, 0)
    assert 50 < s.max() - s[:32].max() < 64
    want = c.expected()
    assert torch.isfinite(want[0]).all()
    check(*c.run(), want, c.q.shape[2])


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("rows", [40, 700])
def test_values_near_the_end_of_the_range(shape, rows, mx):
    """Values of 2^126 to 2^127 of one sign and scores that differ little: every partial sum and the sum over the parts
    leave the range, the mean does not."""
    c = make(shape, [rows], [2], 16, seed=41)
    v = values(c)
    v.copy_(v.abs().clamp(2.0 ** -6, 1) * 2.0 ** 126 + 2.0 ** 126)
    if mx:
        quantize(c)
    want = c.expected()
    assert torch.isfinite(want[0]).all() and want[0].max() > 2.0 ** 126
    check(*c.run(), want, c.q.shape[2])


@pytest.mark.parametrize("shape", ["latent", "per head"])
def test_large_values_beside_an_infinity_that_some_do_not_see(shape):
    c = make(shape, [40], [3], 16, seed=42).tree()
    v = values(c)
    v.copy_(v.abs().clamp(2.0 ** -6, 1) * 2.0 ** 126 + 2.0 ** 126)
    c.mask[0, 0], c.mask[1, 0], c.mask[2, 0] = 0b001, 0b011, 0b111
    (c.bufs[1] if len(c.bufs) > 1 else c.bufs[0])[row(c, 0, 42)][:, 5] = -math.inf
    want = c.expected()
    assert torch.isfinite(want[0][:2]).all()
    # (a latent cache's infinity is a key too, whose product with a query of 0 is NaN)
    assert (torch.isneginf if shape == "per head" else torch.isnan)(want[0][2, :, 5]).all()
    check(*c.run(), want, c.q.shape[2])


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("bound", [None, 30000])
def test_scores_that_rise_too_far_for_some_rows(shape, bound, mx):
    """By 100 and 150 powers of two after the first tile, within a part and from part to part, for one head of one
    token each; the other rows of the same workgroup stay as they were."""
    c = make(shape, [300, 70], [3, 2], 16, seed=43).tree()
    lift(c, 0, 100, 0, 0, 100)
    lift(c, 0, 290, 2, 1, 150)
    lift(c, 1, 60, 4, 2, 120)
    if mx:
        quantize(c)
    for t, h, seq in ((0, 0, 0), (2, 1, 0), (4, 2, 1)):
        s = scores(c, t, h, seq)
        assert s.max() - s[:32].max() > 64
    assert scores(c, 1, 0, 0).max() < 64
    check(*c.run(**({} if bound is None else dict(max_len=bound))), c.expected(), c.q.shape[2])
