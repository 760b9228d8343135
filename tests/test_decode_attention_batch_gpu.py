"""mla_tree_attention on the paths that batches of size take: steps numbered through over the workgroups with items cut
anywhere, parts of items joined in blocks of many vectors, and workgroups of two and four waves of every width. The
bound is that of test_decode_attention_gpu. Where the path depends on the division of the work, the test works the
division out and says so."""
import math

import pytest
import torch

from tests import decode_ref as ref
from tests import decode_ref_batch as batch
from tests.test_decode_attention_gpu import SHAPES, Case, check, make

pytestmark = pytest.mark.gpu


def expected(c):
    key, value = ref.cache_values(c.bufs, c.mx)
    return batch.attend(c.q, key, value, c.d_v, c.page, c.table, c.lens, c.order, c.cu, c.scale, c.mask)


def division(c):
    """Of a 576/512 call: items, steps of the longest, steps per part (0: numbered through), workgroups."""
    heads, cus = c.q.shape[1], torch.cuda.get_device_properties(0).multi_processor_count
    tiles = [-(-(c.lens[s] + d) // 32) for s, d in zip(c.order, c.drafts)]
    rts = [-(-d * heads // 128) for d in c.drafts]
    W, items = sum(a * b for a, b in zip(tiles, rts)), sum(rts)
    bound = len(c.order) * -(-c.max_q * heads // 128)
    steps = bound * ((c.max_len - 1) // 32 + 1)
    groups = min(cus, steps, math.floor(math.sqrt(17 * steps + 84 * bound)) + 1)
    G = min(groups, W, int(math.sqrt((2 * W + 10 * items) / (0.12 + 0.2 / items))))
    quantum = -(-W // (G - items)) if 4 * items <= G else 0
    return items, max(tiles), quantum, G


def lengths(n, low, high, seed):
    g = torch.Generator().manual_seed(seed)
    return [int(x) for x in torch.exp(torch.rand(n, generator=g) * math.log(high / low)) * low]


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("n,heads,drafts,high", [(70, 17, [1], 1500), (40, 128, [1, 2, 2], 1100), (130, 16, [3, 0, 8, 1], 900),
                                                 (300, 9, [1, 5], 700)])
def test_items_cut_anywhere(n, heads, drafts, high, mx):
    """More items than a quarter of the workgroups: their steps are numbered through, and items of more than 16 steps are
    cut where a workgroup's share ends. Twice the same bits."""
    c = make("latent", lengths(n, 20, high, 70), [drafts[k % len(drafts)] for k in range(n)], 16, seed=70, mx=mx, heads=heads).tree()
    items, longest, quantum, G = division(c)
    assert quantum == 0 and longest > 16 and items > G / 4
    out, lse = c.run()
    check(out, lse, expected(c), 576)
    again, _ = c.run()
    assert torch.equal(again, out)


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
def test_equal_parts_of_many_rows(mx):
    """Few items, each cut into equal parts, with enough rows that the join takes 16 vectors at a time."""
    c = make("latent", lengths(18, 300, 2500, 71), [1] * 18, 64, seed=71, mx=mx, heads=128)
    items, longest, quantum, _ = division(c)
    assert 0 < quantum < longest and 4 * items >= 64
    check(*c.run(), expected(c), 576)


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("shape,kv_heads", [("per head", 128), ("grouped", 32), ("narrow", 64)])
def test_parts_of_many_heads(shape, kv_heads, mx):
    """128 heads on many key heads, so many groups of rows, and lengths of several chunks."""
    d_k, d_v = SHAPES[shape][:2]
    c = Case([1400, 700, 129], [2, 1, 3], 16, 128, kv_heads, d_k, d_v, False, mx, 72).tree()
    check(*c.run(), expected(c), d_k)


WAVES = {"latent small": (15, 40), "per head": (50, 80), "grouped": (15, 40), "narrow": (25, 40)}  # drafts for two and four


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("waves", [2, 4])
@pytest.mark.parametrize("shape", WAVES)
def test_workgroups_of_several_waves(shape, waves, mx):
    """Row tiles of 64 and 128 rows, the last one with rows missing; one chunk and several."""
    n = WAVES[shape][waves // 4]
    _, _, _, h, hk = SHAPES[shape]
    rows = n * (h // hk)
    assert (32 < rows <= 64) if waves == 2 else 64 < rows
    for lens in ([70, 0, 33], [900, 65, 1]):
        c = make(shape, lens, [n, n - 7, 3], 16, seed=73, mx=mx).tree()
        check(*c.run(), expected(c), c.q.shape[2])


@pytest.mark.parametrize("shape", ["latent", "per head"])
def test_large_values_in_a_large_batch(shape):
    """Sums over the parts leave fp32's range although the parts and the result do not."""
    d_k, d_v = SHAPES[shape][:2]
    if shape == "latent":
        c = make(shape, lengths(17, 300, 900, 74), [1] * 17, 16, seed=74, heads=128)
        c.q[..., :24] = 0  # the large columns are keys too
    else:
        c = Case([1000, 600], [1, 2], 16, 128, 128, d_k, d_v, False, False, 74)
    v = c.bufs[-1][..., :24]
    v.copy_(v.abs().clamp(2.0 ** -6, 1) * 2.0 ** 126 + 2.0 ** 126)
    want = expected(c)
    assert torch.isfinite(want[0]).all()
    check(*c.run(), want, d_k)
