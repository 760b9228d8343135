"""mxfp4_quantize and mla_qup_fwd_w4 against the 64-bit forms.

Bound of a projected element before its last rounding, with e = 2^-24: products
of bf16 and E2M1 x 2^k are exact in fp32, K additions (and the bias) give
(K + 1) e A with A = sum |x w| + |bias|; a rotation of two such values with table
entries of at most 1 in magnitude: the table's roundings e and three fp32
operations, (K + 6) e (A_a + A_b). A bf16 output adds 2^-8 of its value."""
import pytest
import torch

import mla_up_projection_amd as m
from tests import decode_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
E = 2.0 ** -24


def quantize(w):
    codes = torch.empty(w.shape[0], w.shape[1] // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(w.shape[0], w.shape[1] // 32, dtype=torch.uint8, device=DEV)
    m.mxfp4_quantize(w.to(DEV), codes, scales)
    return codes, scales


def test_mxfp4_every_bf16_pattern():
    """All 65536 bf16 patterns at the head of a block whose other elements set different scales."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    for other in (0.0, 1.0, 5.0, 3e-38, 3e38):
        x = torch.full((65536 // 8, 32), other).to(torch.bfloat16)
        x[:, :8] = bits.view(torch.bfloat16).view(-1, 8)
        codes, scales = quantize(x)
        wc, ws = ref.mx4_quantize(x.double())
        assert torch.equal(scales.cpu(), ws)
        assert torch.equal(codes.cpu(), wc)


def test_mxfp4_fp32_strides_and_ties():
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(37, 160, generator=g)
    wide[3, 32:64] = 0
    wide[4, 0] = float("inf")
    wide[5, 95] = float("nan")
    wide[6, :32] = 2.0 ** -140
    wide[7, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4) * 2.0 ** 20
    wide[8, :32] = torch.nextafter(wide[7, :32], torch.zeros(32))
    wide[9, :32] = -torch.nextafter(wide[7, :32], torch.full((32,), 1e30))
    for x in (wide, wide.to(torch.bfloat16)):
        x = x.to(DEV)[:, :96]
        codes = torch.empty(37, 48, dtype=torch.uint8, device=DEV)
        scales = torch.empty(37, 3, dtype=torch.uint8, device=DEV)
        m.mxfp4_quantize(x, codes, scales)
        wc, ws = ref.mx4_quantize(x.cpu().double())
        assert torch.equal(scales.cpu(), ws)
        assert torch.equal(codes.cpu(), wc)


def rope(rows, d_rope):
    cos = torch.empty(rows, d_rope // 2, dtype=torch.float32, device=DEV)
    sin = torch.empty_like(cos)
    m.rope_cache_build(cos, sin, d_rope)
    return cos, sin


def projected(x, codes, scales, bias, H, dn, dr, cos, sin, pos):
    """[T, H, D] in 64 bits and the bound of the fp32 value."""
    T, K = x.shape
    w = ref.mx4_values(codes.cpu(), scales.cpu())
    q = x.cpu().double() @ w.t()
    A = x.cpu().double().abs() @ w.abs().t()
    if bias is not None:
        q, A = q + bias.cpu().double(), A + bias.cpu().double().abs()
    q, A = q.view(T, H, -1).clone(), A.view(T, H, -1)
    bound = (K + 1) * E * A
    if dr:
        c, s = (t.cpu().double()[pos.clamp(0, t.shape[0] - 1)][:, None] for t in (cos, sin))
        bad = (pos < 0) | (pos >= cos.shape[0])
        a, b = q[..., dn::2].clone(), q[..., dn + 1::2].clone()
        q[..., dn::2], q[..., dn + 1::2] = a * c - b * s, a * s + b * c
        q[bad, :, dn:] = torch.nan
        both = (K + 6) * E * (A[..., dn::2] + A[..., dn + 1::2])
        bound = torch.cat([bound[..., :dn], both.repeat_interleave(2, -1)], -1)
    return q, bound


def check(q, bound, out, out_scales):
    """q, bound [T, H, D]; out [1, H, T, D]."""
    got = out[0].transpose(0, 1).cpu()
    if out_scales is None:
        g = got.double()
        assert torch.equal(torch.isnan(g), torch.isnan(q))
        fin = torch.isfinite(q)
        assert torch.equal(g[~fin & ~torch.isnan(q)], q[~fin & ~torch.isnan(q)])
        assert ((g - q).abs() <= bound + 2.0 ** -8 * (q.abs() + bound))[fin].all()
        return
    # MXFP8: the scale is that of a block maximum within the bound, each element within half a step of its value
    sc = out_scales[0].transpose(0, 1).cpu()
    blocks, bb = q.unflatten(-1, (-1, 32)), bound.unflatten(-1, (-1, 32))
    nan = ~torch.isfinite(blocks).all(-1)
    assert torch.equal(sc == 255, nan)
    assert (got.unflatten(-1, (-1, 32))[nan] == 0x7F).all()
    top, tb = blocks.abs().amax(-1), bb.amax(-1)
    e = sc.double() - 127
    lo, hi = (torch.floor(torch.log2((top + d).clamp(min=2.0 ** -140))).clamp(min=-119) - 8 for d in (-tb, tb))
    assert ((e >= lo) & (e <= hi))[~nan].all()
    v = ref.mx8_values(got.contiguous(), sc.contiguous()).unflatten(-1, (-1, 32))
    lim = 448 * torch.exp2(e)[..., None]
    want = blocks.clamp(-lim, lim)
    # half an E4M3 step at the value: 2^-4 of it, 2^(e - 10) among the subnormals
    step = torch.maximum(2.0 ** -4 * (want.abs() + bb), torch.exp2(e - 10)[..., None])
    assert ((v - want).abs() <= step + bb)[~nan].all()


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("T", [1, 3, 16, 17, 33, 64, 65, 130])
def test_tokens(T, mx):
    run_case(T, 256, 3, 64, 32, mx)


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 512, 544, 1536, 1568])
def test_depths(K):
    for T in (2, 20, 50):
        run_case(T, K, 2, 16, 16, K % 64 == 0)


@pytest.mark.parametrize("dn,dr", [(128, 64), (0, 64), (96, 0), (30, 2), (2, 30)])
def test_head_widths(dn, dr):
    for mx in (False, True):
        run_case(5, 128, 5, dn, dr, mx, bias=True)


def run_case(T, K, H, dn, dr, mx, bias=False, x=None, codes=None, scales=None, pos=None):
    D = dn + dr
    g = torch.Generator().manual_seed(T * 1000 + K + dn)
    if x is None:
        x = torch.randn(T, K, generator=g).to(torch.bfloat16).to(DEV)
    if codes is None:
        codes, scales = quantize((torch.randn(H * D, K, generator=g) * 0.05).to(torch.bfloat16))
    b = torch.randn(H * D, generator=g).to(torch.bfloat16).to(DEV) if bias else None
    cos, sin = rope(5000, dr) if dr else (None, None)
    if pos is None:
        pos = torch.randint(0, 5000, (T,), generator=g)
    out = torch.full((1, H, T, D), 7, dtype=torch.uint8 if mx else torch.bfloat16, device=DEV)
    sc = torch.empty(1, H, T, D // 32, dtype=torch.uint8, device=DEV) if mx else None
    m.mla_qup_fwd_w4(x, codes, scales, out, H=H, d_nope=dn, d_rope=dr, cos=cos, sin=sin,
                     positions=pos.int().to(DEV), bias=b, out_scales=sc)
    q, bound = projected(x, codes, scales, b, H, dn, dr, cos, sin, pos)
    check(q, bound, out, sc)
    return out, sc


def test_full_shape():
    run_case(7, 1536, 128, 128, 64, False)
    run_case(40, 1536, 128, 128, 64, True)


@pytest.mark.parametrize("T", [1, 20, 40])
def test_heads_of_one_block(T):
    """Weight rows that end inside a workgroup's, few and many."""
    for H in (1, 511, 513):
        run_case(T, 96, H, 16, 16, H == 513)
    run_case(T, 1056, 3, 30, 2, False)


def test_positions_outside_the_table():
    run_case(6, 64, 2, 32, 32, False, pos=torch.tensor([0, -1, 4999, 5000, 2 ** 31 - 1, -2 ** 31]))
    run_case(6, 64, 2, 32, 32, True, pos=torch.tensor([0, -1, 4999, 5000, 2 ** 31 - 1, -2 ** 31]))


def test_special_weights_and_inputs():
    """NaN blocks, the smallest and largest scales, infinite and NaN activations: each stays in its row."""
    g = torch.Generator().manual_seed(3)
    codes = torch.randint(0, 256, (96, 64), generator=g, dtype=torch.uint8)
    scales = torch.randint(118, 130, (96, 4), generator=g, dtype=torch.uint8)
    scales[3, 2] = 255
    scales[40] = torch.tensor([0, 1, 2, 5], dtype=torch.uint8)
    scales[41] = 0
    scales[42] = torch.tensor([200, 190, 10, 210], dtype=torch.uint8)
    x = torch.randn(18, 128, generator=g).to(torch.bfloat16)
    x[2, 5] = float("inf")
    x[3, 7], x[3, 8] = float("inf"), float("-inf")
    x[4, 100] = float("nan")
    x[17, 0] = 1e30
    run_case(18, 128, 3, 32, 0, False, x=x.to(DEV), codes=codes.to(DEV), scales=scales.to(DEV))


def test_token_formats():
    """Without positions the token format places and rotates tokens, as in the forward."""
    T, K, H, dn, dr = 12, 64, 2, 32, 32
    g = torch.Generator().manual_seed(5)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).to(DEV)
    codes, scales = quantize((torch.randn(H * 64, K, generator=g) * 0.1).to(torch.bfloat16))
    w = ref.mx4_values(codes.cpu(), scales.cpu()).to(torch.bfloat16).to(DEV)  # exact in bf16
    cos, sin = rope(16, dr)
    cu = torch.tensor([0, 5, 5, 12], dtype=torch.int32, device=DEV)
    for kw in (dict(B=3, S=4), dict(fmt=m.FMT_SBHD, B=3, S=4), dict(fmt=m.FMT_THD, cu_seqlens=cu, max_seqlen=7)):
        shape = (kw.get("B", 1), H, kw.get("S", T), 64)
        a, b = (torch.empty(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        kw |= dict(H=H, d_nope=dn, d_rope=dr, cos=cos, sin=sin)
        m.mla_qup_fwd_w4(x, codes, scales, a, **kw)
        m.mla_qup_fwd(x, w, b, **kw)
        # both are within half a bf16 step and the fp32 bound of one 64-bit value
        lim = 2.0 ** -7 * b.double().abs() + 4 * (K + 6) * E * (x.double().abs() @ w.double().abs().t()).max()
        assert ((a.double() - b.double()).abs() <= lim).all()


def test_other_stream_and_graph():
    T, K, H = 4, 512, 8
    g = torch.Generator().manual_seed(6)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).to(DEV)
    codes, scales = quantize((torch.randn(H * 64, K, generator=g) * 0.1).to(torch.bfloat16))
    cos, sin = rope(64, 32)
    pos = torch.tensor([3, 4, 5, 60], dtype=torch.int32, device=DEV)
    kw = dict(H=H, d_nope=32, d_rope=32, cos=cos, sin=sin, positions=pos)
    a, b = (torch.empty(1, H, T, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    m.mla_qup_fwd_w4(x, codes, scales, a, **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    m.mla_qup_fwd_w4(x, codes, scales, b, stream=s, **kw)
    s.synchronize()
    assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.mla_qup_fwd_w4(x, codes, scales, b, **kw)
    for k in range(3):
        x.mul_(0.5)
        pos.add_(1).clamp_(max=63)
        graph.replay()
        m.mla_qup_fwd_w4(x, codes, scales, a, **kw)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
