"""The up-projection in 8-bit integers against 64 bits. Sums of products are exact; the product with the two scales
(and the bias and the rotation) takes a few roundings of 2^-24, and the output one of bf16 (2^-8) or E4M3 (2^-4)."""
import pytest
import torch

import layer_ref as ref
import mla_up_projection_amd as m

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64, BF = torch.float64, torch.bfloat16


def case(T, K, H, dn, dr, seed, bias=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    N = H * (dn + dr)
    x = torch.randint(-128, 128, (T, K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-128, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
    xs = torch.rand(T, generator=g, device=DEV) * 0.02 + 1e-3
    ws = torch.rand(N, generator=g, device=DEV) * 1e-3 + 1e-4
    b = torch.randn(N, generator=g, device=DEV).to(BF) if bias else None
    cos = torch.empty(512, max(dr // 2, 1), device=DEV)
    sin = torch.empty_like(cos)
    if dr:
        m.rope_cache_build(cos, sin, dr)
    return x, w, xs, ws, b, cos, sin


def want(x, w, xs, ws, b, cos, sin, H, dn, dr, pos):
    """[T, H, D] and the magnitude that rounding is relative to."""
    T = x.shape[0]
    q = (x.to(F64) @ w.to(F64).t()) * xs.to(F64)[:, None] * ws.to(F64)
    if b is not None:
        size = q.abs() + b.to(F64).abs()
        q = q + b.to(F64)
    else:
        size = q.abs()
    q, size = q.view(T, H, dn + dr), size.view(T, H, dn + dr).clone()
    if dr:
        c, s = cos.to(F64)[pos][:, None], sin.to(F64)[pos][:, None]
        a, d = q[..., dn::2].clone(), q[..., dn + 1::2].clone()
        sz = size[..., dn::2] + size[..., dn + 1::2]
        q = q.clone()
        q[..., dn::2], q[..., dn + 1::2] = a * c - d * s, a * s + d * c
        size[..., dn::2], size[..., dn + 1::2] = sz, sz
    return q, size


SHAPES = [(1, 64, 1, 128, 64), (1, 1536, 16, 128, 64), (16, 192, 3, 64, 64), (17, 320, 5, 0, 64), (33, 1536, 8, 128, 64),
          (17, 64, 43, 128, 64), (33, 576, 64, 64, 64), (64, 1088, 257, 0, 32), (32, 512, 129, 64, 0), (50, 1536, 128, 128, 64),
          (64, 128, 2, 32, 0), (65, 64, 1, 128, 64), (130, 192, 3, 16, 16), (300, 1536, 5, 128, 64), (129, 128, 7, 0, 64)]


@pytest.mark.parametrize("T, K, H, dn, dr", SHAPES)
@pytest.mark.parametrize("bias", [False, True])
def test_bf16_output(T, K, H, dn, dr, bias):
    a = case(T, K, H, dn, dr, T + K, bias)
    pos = torch.randint(0, 512, (T,), device=DEV, dtype=torch.int32)
    D = dn + dr
    out = torch.full((1, H, T, D), 7.0, dtype=BF, device=DEV)
    x, w, xs, ws, b, cos, sin = a
    kw = dict(H=H, d_nope=dn, d_rope=dr) | (dict(cos=cos, sin=sin) if dr else {})
    m.mla_qup_fwd_i8(x, xs, w, ws, out, positions=pos, bias=b, **kw)
    q, size = want(*a, H, dn, dr, pos.long())
    ref.within(out[0].transpose(0, 1), q, q.abs() * ref.BF16 + size * 2.0 ** -21 + 1e-30, "out")


@pytest.mark.parametrize("T, K, H, dn, dr", [(1, 64, 1, 128, 64), (17, 320, 5, 0, 64), (33, 576, 64, 64, 64), (64, 1088, 257, 0, 32),
                                            (130, 192, 3, 16, 16), (300, 1536, 5, 128, 64)])
def test_mxfp8_output(T, K, H, dn, dr):
    a = case(T, K, H, dn, dr, T)
    pos = torch.arange(T, device=DEV, dtype=torch.int32)
    D = dn + dr
    out = torch.empty(1, H, T, D, dtype=torch.uint8, device=DEV)
    sc = torch.empty(1, H, T, D // 32, dtype=torch.uint8, device=DEV)
    x, w, xs, ws, b, cos, sin = a
    m.mla_qup_fwd_i8(x, xs, w, ws, out, out_scales=sc, H=H, d_nope=dn, d_rope=dr, cos=cos, sin=sin)  # positions 0 .. T - 1
    q, size = want(*a, H, dn, dr, pos.long())
    s = 2.0 ** (sc[0].to(F64) - 127)[..., None]
    v = (out[0].view(torch.float8_e4m3fn).to(F64).unflatten(-1, (-1, 32)) * s).transpose(0, 1)
    s, q, size = s.transpose(0, 1), q.unflatten(-1, (-1, 32)), size.unflatten(-1, (-1, 32))
    amax = q.abs().amax(-1, keepdim=True)
    assert ((s * 256 <= amax * (1 + 2.0 ** -18)) & (s * 512 > amax * (1 - 2.0 ** -18))).all()
    bound = torch.maximum(q.abs() * 2.0 ** -4, s * 2.0 ** -10) + size * 2.0 ** -20
    ref.within(v, q, torch.where(q.abs() > 448 * s, q.abs() - 448 * s + size * 2.0 ** -20, bound), "out")


@pytest.mark.parametrize("fmt, T", [("bshd", 60), ("sbhd", 60), ("thd", 60), ("bshd", 210), ("sbhd", 210), ("thd", 210)])
@pytest.mark.parametrize("H", [3, 45])
def test_token_formats(fmt, T, H):
    dn, dr, K = 128, 64, 256
    a = case(T, K, H, dn, dr, 11)
    x, w, xs, ws, b, cos, sin = a
    kw = dict(H=H, d_nope=dn, d_rope=dr, cos=cos, sin=sin)
    B, S = 3, T // 3
    t = torch.arange(T, device=DEV)
    if fmt == "thd":
        cu = torch.tensor([0, 7, 7, T - 20, T], dtype=torch.int32, device=DEV)
        kw |= dict(fmt=m.FMT_THD, cu_seqlens=cu, max_seqlen=512)
        j = (t[:, None] >= cu[None, 1:]).sum(1)
        pos, out = t - cu[j], torch.empty(1, H, T, dn + dr, dtype=BF, device=DEV)
        got = lambda: out[0].transpose(0, 1)  # noqa: E731
    else:
        kw |= dict(fmt=m.FMT_BSHD if fmt == "bshd" else m.FMT_SBHD, B=B, S=S)
        pos, out = (t % S if fmt == "bshd" else t // B), torch.empty(B, H, S, dn + dr, dtype=BF, device=DEV)
        got = lambda: (out.permute(0, 2, 1, 3) if fmt == "bshd" else out.permute(2, 0, 1, 3)).reshape(T, H, -1)  # noqa: E731
    m.mla_qup_fwd_i8(x, xs, w, ws, out, **kw)
    q, size = want(*a, H, dn, dr, pos.long())
    ref.within(got(), q, q.abs() * ref.BF16 + size * 2.0 ** -21 + 1e-30, fmt)


@pytest.mark.parametrize("T", [3, 100])
def test_positions_outside_the_table_are_nan_in_the_rope_slice(T):
    a = case(T, 64, 2, 64, 64, 3)
    x, w, xs, ws, b, cos, sin = a
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    pos[1], pos[2] = -1, 512
    out = torch.empty(1, 2, T, 128, dtype=BF, device=DEV)
    m.mla_qup_fwd_i8(x, xs, w, ws, out, H=2, d_nope=64, d_rope=64, cos=cos, sin=sin, positions=pos)
    nan = torch.isnan(out[0])
    assert nan[:, 1:3, 64:].all() and not nan[:, 1:3, :64].any() and not nan[:, 0].any()


@pytest.mark.parametrize("T", [5, 70])
def test_extreme_sums_are_exact_and_scales_that_are_not_finite_spread(T):
    K = 65536
    x = torch.full((T, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((64, K), -128, dtype=torch.int8, device=DEV)
    xs, ws = torch.ones(T, device=DEV), torch.full((64,), 2.0 ** -30, device=DEV)
    xs[1] = float("nan")
    out = torch.empty(1, 1, T, 64, dtype=BF, device=DEV)
    m.mla_qup_fwd_i8(x, xs, w, ws, out, H=1, d_nope=64, d_rope=0)
    assert (out[0, 0, [0, 2, T - 1]] == 1).all() and torch.isnan(out[0, 0, 1]).all()


def test_against_the_norm_that_feeds_it():
    """Norm, integer projection and the bf16 path agree up to what 8 bits lose."""
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    T, K, H = 100, 1536, 4
    x, gamma = torch.randn(T, K, generator=g, device=DEV).to(BF), torch.ones(K, dtype=BF, device=DEV)
    w = (torch.randn(H * 192, K, generator=g, device=DEV) * 0.02).to(BF)
    wq, ws = torch.empty(H * 192, K, dtype=torch.int8, device=DEV), torch.empty(H * 192, device=DEV)
    m.int8_quantize(w, wq, ws)
    c, s = torch.empty(T, K, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    m.mla_rmsnorm_fwd(x, gamma, codes=c, scales=s)
    out = torch.empty(1, H, T, 192, dtype=BF, device=DEV)
    m.mla_qup_fwd_i8(c, s, wq, ws, out, H=H, d_nope=192, d_rope=0)
    y = ref.norm(x, gamma, 1e-6)[2]
    q = (y @ w.to(F64).t()).view(T, H, 192).transpose(0, 1)
    # half a code of each factor: |sum| <= sum (|y| ws / 2 + |w| s / 2 + s ws / 4)
    e = (y.abs() @ torch.ones_like(w).to(F64).t() * ws.to(F64) / 2 + s.to(F64)[:, None] / 2 * w.to(F64).abs().sum(1)
         + K * s.to(F64)[:, None] * ws.to(F64) / 4)
    ref.within(out[0], q, q.abs() * ref.BF16 + e.view(T, H, 192).transpose(0, 1) * 1.01, "projection")
