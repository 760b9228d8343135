"""mla_tree_attention with lengths that mean nothing: committed rows behind the held pages, up to the largest numbers,
are NaN for the sequence's tokens at once (they would be minutes of work) and change nothing for the others."""
import pytest
import torch

import mla_up_projection_amd as m
from tests.test_decode_attention_gpu import SHAPES, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", SHAPES)
def test_lengths_behind_the_held_pages(shape, mx):
    c = make(shape, [40, 30, 20], [2, 3, 1], 16, seed=60, mx=mx).tree()
    bound = 2 ** 31 - 1 if shape == "latent" else 10 ** 6  # (the other widths' workspaces grow with it)
    good, lse = c.run(max_len=bound)
    check(good, lse, c.expected(), c.q.shape[2])
    others = [0, 1, 5]
    for length in (c.held[1] * 16 + 1, 10 ** 6 - 3, 2 * 10 ** 9, 2 ** 31 - 33, 2 ** 31 - 4):
        if length > bound:
            continue
        c.lens[1] = length
        out, l2 = c.run(max_len=bound)
        assert torch.isnan(out[2:5].float()).all() and torch.isnan(l2[2:5]).all()
        assert torch.equal(out[others], good[others]) and torch.equal(l2[others], lse[others])
    c.held[1] = -3
    out, _ = c.run(max_len=bound)
    assert torch.isnan(out[2:5].float()).all() and torch.equal(out[others], good[others])
    c.lens[1], c.held[1] = -1, 3
    out, _ = c.run(max_len=bound)
    assert torch.isnan(out[2:5].float()).all() and torch.equal(out[others], good[others])


@pytest.mark.parametrize("shape", ["latent", "per head"])
def test_drafts_behind_the_held_pages(shape):
    """NaN for the tokens that see such a draft, nothing for those that do not."""
    c = make(shape, [30], [4], 16, seed=61).tree()
    c.mask[:, 0] = torch.tensor([0b0001, 0b0011, 0b0101, 0b1001])
    good, lse = c.run()
    c.held[0] = 2  # rows 0 to 31: drafts 2 and 3 have no page
    out, l2 = c.run()
    assert torch.isnan(out[2:].float()).all() and torch.isnan(l2[2:]).all()
    check(out[:2], l2[:2], [x[:2] for x in c.expected()], c.q.shape[2])


@pytest.mark.parametrize("shape", ["latent small", "latent"])
def test_a_sequence_of_more_rows_than_are_taken(shape):
    """One page named by the whole table, so that the rows are there; beside it a short sequence of the same page."""
    d_k, d_v = SHAPES[shape][:2]
    page, pages = 31, (2 ** 31 - 1) // 31
    buf = torch.randn(2, page, 1, d_k, device="cuda").to(torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = m.PagePool([buf], i32([pages, 0]), torch.zeros(2, pages, dtype=torch.int32, device="cuda"),
                      i32([2 ** 31 - 100, 31]), i32([pages, 2]))
    q = torch.randn(2, 3, d_k, device="cuda").to(torch.bfloat16)
    out = torch.empty(2, 3, d_v, dtype=torch.bfloat16, device="cuda")
    kw = dict(max_q=1, max_len=2 ** 31 - 1, scale=0.1)
    n = m.mla_tree_attention_workspace_size(q, pool, out, i32([0, 1]), i32([0, 1, 2]), **kw)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    m.mla_tree_attention(q, pool, out, i32([0, 1]), i32([0, 1, 2]), workspace=ws, **kw)
    alone = torch.empty(1, 3, d_v, dtype=torch.bfloat16, device="cuda")
    kw["max_len"] = 32
    n = m.mla_tree_attention_workspace_size(q[1:], pool, alone, i32([1]), i32([0, 1]), **kw)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    m.mla_tree_attention(q[1:], pool, alone, i32([1]), i32([0, 1]), workspace=ws, **kw)
    assert torch.isnan(out[0].float()).all() and torch.equal(out[1:], alone) and torch.isfinite(alone.float()).all()
