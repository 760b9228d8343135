"""The 64-bit implementations that the layer operators are tested against, pinned by automatic differentiation and
by differences."""
import pytest
import torch

import layer_ref as ref

F64 = torch.float64


def inputs(seed=0, B=2, H=4, hk=2, Sq=5, Sk=7, dk=6, dv=4):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, dtype=F64)  # noqa: E731
    sees = torch.rand(B, Sq, Sk, generator=g) < 0.6
    sees[0, 1] = False  # a row that sees nothing
    return r(B, H, Sq, dk), r(B, hk, Sk, dk), r(B, hk, Sk, dv), r(B, H, Sq, dv), sees


@pytest.mark.parametrize("cap, slope", [(0.0, False), (1.5, False), (0.0, True), (2.0, True)])
def test_attention_gradients(cap, slope):
    q, k, v, do, sees = inputs()
    slopes = torch.tensor([0.5, 0.25, 0.1, 0.0], dtype=F64) if slope else None
    f = lambda q, k, v: ref.attention(q, k, v, sees, 0.4, cap, slopes)  # noqa: E731
    out, lse, p, c = f(q, k, v)
    grads = [g for g, _ in ref.attention_grad(q, k, v, do, p, c, out, 0.4)]
    assert (out[0, :, 1] == 0).all() and (lse[0, :, 1] == -float("inf")).all() and (grads[0][0, :, 1] == 0).all()
    e = 1e-5
    for which, (x, got) in enumerate(zip((q, k, v), grads)):
        for at in (0, 7, x.numel() // 2, x.numel() - 1):
            d = torch.zeros_like(x).view(-1)
            d[at] = e
            d = d.view(x.shape)
            args = [[q, k, v], [q, k, v]]
            args[0][which], args[1][which] = x + d, x - d
            diff = ((f(*args[0])[0] - f(*args[1])[0]) * do).sum() / (2 * e)
            assert abs(diff - got.view(-1)[at]) < 1e-8 + 1e-6 * abs(diff)


def test_norm_gradients():
    g = torch.Generator().manual_seed(1)
    h, gamma, dy = (torch.randn(*s, generator=g, dtype=F64) for s in ((3, 8), (8,), (3, 8)))
    f = lambda h, gamma: (ref.norm(h, gamma, 1e-3)[2] * dy).sum()  # noqa: E731
    d, dg = ref.norm_grad(dy, h, ref.norm(h, gamma, 1e-3)[1], gamma)
    e = 1e-6
    for i in range(8):
        x = torch.zeros_like(h)
        x[1, i] = e
        assert abs((f(h + x, gamma) - f(h - x, gamma)) / (2 * e) - d[1, i]) < 1e-7
        x = torch.zeros_like(gamma)
        x[i] = e
        assert abs((f(h, gamma + x) - f(h, gamma - x)) / (2 * e) - dg[i]) < 1e-7


def test_weights_sum_to_one_and_the_cap_bounds_scores():
    q, k, v, _, sees = inputs(3)
    _, lse, p, _ = ref.attention(q * 50, k, v, sees, 1.0, cap=2.0)
    s = p.sum(-1)
    assert ((s - 1).abs() < 1e-12)[s > 0].all()
    t, _ = ref.scores(q * 50, k, 1.0, cap=2.0)
    assert t.abs().max() <= 2.0
    assert (lse[lse > -float("inf")] <= 2.0 + torch.log(torch.tensor(7.0))).all()


def test_masked_values_that_are_not_finite_take_no_part():
    q, k, v, _, sees = inputs(4)
    want = ref.attention(q, k, v, sees, 0.4)[0]
    v2 = v.clone()
    sees[:, :, 3] = False
    want = ref.attention(q, k, v, sees, 0.4)[0]
    v2[:, :, 3] = float("nan")
    assert torch.allclose(ref.attention(q, k, v2, sees, 0.4)[0], want, atol=1e-14)
