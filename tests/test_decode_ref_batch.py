"""The batch form of the attention's reference against the one that takes one query row at a time."""
import math

import pytest
import torch

from tests import decode_ref as ref
from tests import decode_ref_batch as batch


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_batch_form(latent, masked):
    g = torch.Generator().manual_seed(1)
    d_k, d_v, Hk, G, page = 24, 16, 1 if latent else 2, 3, 5
    lens, drafts, seqs = [13, 0, 40, 7], [3, 2, 1, 0], [2, 1, 0, 3]
    cu = [0, 3, 5, 6, 6]
    table = torch.randperm(60, generator=g).view(4, 15).int()
    key = torch.randn(60, page, Hk, d_k, generator=g, dtype=torch.float64)
    value = None if latent else torch.randn(60, page, Hk, d_v, generator=g, dtype=torch.float64)
    q = torch.randn(6, Hk * G, d_k, generator=g)
    mask = torch.tensor([[1], [0], [5], [0], [2], [1]]) if masked else None
    a = ref.attend(q, key, value, d_v, page, table, lens, seqs, cu, 0.3, mask)
    b = batch.attend(q, key, value, d_v, page, table, lens, seqs, cu, 0.3, mask)
    for x, y in zip(a, b):
        assert torch.equal(torch.isinf(x), torch.isinf(y))
        f = torch.isfinite(x)
        assert (x[f] - y[f]).abs().max() <= 1e-12 * max(1, x[f].abs().max())
    assert not masked or (math.isinf(b[1][3, 0]) and (b[0][3] == 0).all())
