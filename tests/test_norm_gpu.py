"""RMS norm with the residual's addition and outputs in 8 bits, and its backward, against 64 bits. Bounds count
roundings: half a bf16 step is 2^-8 of the value; fp32 sums over a row, each lane taking at most 32 elements in turn
before a tree of 10 levels, are off by less than 2^-18 of the sum of magnitudes."""
import pytest
import torch

import layer_ref as ref
import mla_up_projection_amd as m

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64, BF, F32 = torch.float64, torch.bfloat16, torch.float32
SUM = 2.0 ** -18


def rand(g, *s, sigma=1.0, dtype=BF):
    return (torch.randn(*s, generator=g, device=DEV) * sigma).to(dtype)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


SIZES = [(1, 8), (3, 40), (1, 1536), (7, 512), (5, 520), (65, 2048), (4, 2080), (130, 7168), (2, 8192), (3, 8224), (2, 32768)]


@pytest.mark.parametrize("T, K", SIZES)
@pytest.mark.parametrize("res", [None, BF, F32])
def test_forward(T, K, res):
    g = gen(T * 7 + K)
    x, gamma = rand(g, T, K), rand(g, K)
    r = None if res is None else rand(g, T, K, sigma=3.0, dtype=res)
    h = None if res is None else torch.full((T, K), 9.0, dtype=res, device=DEV)
    y, rstd = torch.full_like(x, 9.0), torch.empty(T, dtype=F32, device=DEV)
    codes, scales = torch.empty(T, K, dtype=torch.int8, device=DEV), torch.empty(T, dtype=F32, device=DEV)
    m.mla_rmsnorm_fwd(x, gamma, eps=1e-5, res=r, h=h, y=y, rstd=rstd, codes=codes, scales=scales)
    wh, wr, wy = ref.norm(x, gamma, 1e-5, r)
    if h is not None:
        assert torch.equal(h.to(F64), wh)
    ref.within(rstd, wr, wr * SUM, "rstd")
    ref.within(y, wy, wy.abs() * (ref.BF16 + SUM) + 1e-30, "y")
    ref.within(scales, wy.abs().amax(1) / 127, wy.abs().amax(1) * SUM, "scales")
    # a code is the nearest integer, up to what fp32 knows of the value
    ref.within(codes, wy / (wy.abs().amax(1, keepdim=True) / 127), torch.tensor(0.5 + 127 * 2 * SUM, device=DEV, dtype=F64), "codes")


@pytest.mark.parametrize("T, K", [(1, 32), (9, 96), (65, 1536), (33, 7168), (2, 8224)])
@pytest.mark.parametrize("gamma_dtype", [None, BF, F32])
def test_mxfp8_codes(T, K, gamma_dtype):
    g = gen(T + K)
    x = rand(g, T, K)
    x[0, :32] = 0
    gamma = None if gamma_dtype is None else rand(g, K, dtype=gamma_dtype)
    codes = torch.empty(T, K, dtype=torch.uint8, device=DEV)
    scales = torch.empty(T, K // 32, dtype=torch.uint8, device=DEV)
    m.mla_rmsnorm_fwd(x, gamma, eps=1e-6, codes=codes, scales=scales)
    _, _, y = ref.norm(x, gamma, 1e-6)
    b = y.unflatten(1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.floor(torch.log2(amax)) - 8, -127)
    near = (torch.log2(amax) - torch.round(torch.log2(amax))).abs() < 4 * SUM  # fp32 may take the next power there
    got = scales.to(F64) - 127
    assert torch.equal(got[~near], e[~near])
    s = 2.0 ** got[..., None]
    v = codes.view(torch.float8_e4m3fn).to(F64).unflatten(1, (-1, 32)) * s
    # half a step of E4M3 (2^-4), or of its smallest values (2^-10), or saturation at 448 of up to 512
    bound = torch.maximum(b.abs() * (2.0 ** -4 + SUM), s * 2.0 ** -10 * (1 + SUM))
    bound = torch.where(b.abs() > 448 * s, b.abs() - 448 * s * (1 - SUM), bound)
    ref.within(v, b, bound + 1e-30, "codes")


def test_rows_apart_in_memory_and_the_norm_alone():
    # the query latents lie in front of the key latents in the down-projection's output
    g = gen(5)
    wide = rand(g, 37, 1536 + 576)
    x, gamma = wide[:, :1536], rand(g, 1536)
    y = torch.empty(37, 1536, dtype=BF, device=DEV)
    m.mla_rmsnorm_fwd(x, gamma, eps=1e-6, y=y)
    want = torch.empty_like(y)
    m.mla_rmsnorm_fwd(x.contiguous(), gamma, eps=1e-6, y=want)
    assert torch.equal(y, want)


def test_rows_of_zeros_and_rows_that_are_not_finite():
    x = torch.zeros(4, 64, dtype=BF, device=DEV)
    x[1] = 1
    x[2, 5] = float("nan")
    x[3, 5] = float("inf")
    codes = torch.full((4, 64), 99, dtype=torch.int8, device=DEV)
    scales, rstd = torch.empty(4, device=DEV), torch.empty(4, device=DEV)
    m.mla_rmsnorm_fwd(x, None, eps=0.0, codes=codes, scales=scales, rstd=rstd)
    assert rstd[0].isinf() and rstd[1] == 1
    assert scales[1] > 0 and (codes[1] == 127).all()
    # 0 * inf: without eps a row of zeros has no norm
    assert scales[0].isnan() and scales[2].isnan() and scales[3].isnan() and (codes[[0, 2, 3]] == 0).all()
    m.mla_rmsnorm_fwd(x[:1], None, eps=1e-6, codes=codes[:1], scales=scales[:1])
    assert scales[0] == 0 and (codes[0] == 0).all()


@pytest.mark.parametrize("T, K", [(1, 8), (3, 40), (700, 512), (333, 1536), (65, 2048), (1500, 2080), (129, 7168), (2, 8192), (300, 8224), (3, 32768)])
@pytest.mark.parametrize("kind", ["plain", "bf16", "fp32"])
def test_backward(T, K, kind):
    g = gen(T + 3 * K)
    hd = F32 if kind == "fp32" else BF
    h, gamma, dy = rand(g, T, K, sigma=2.0, dtype=hd), rand(g, K, dtype=F32 if kind == "fp32" else BF), rand(g, T, K)
    dh = None if kind == "plain" else rand(g, T, K, dtype=hd)
    h64, r64, _ = ref.norm(h, gamma, 1e-6)
    rstd = r64.to(F32)
    dx, dg = torch.empty(T, K, dtype=BF, device=DEV), torch.empty(K, dtype=F32, device=DEV)
    dres = torch.empty(T, K, dtype=F32, device=DEV) if kind == "fp32" else None
    ws = torch.empty(m.mla_rmsnorm_bwd_workspace_size(T, K), dtype=torch.uint8, device=DEV)
    m.mla_rmsnorm_bwd(dy, h, rstd, gamma, dh=dh, dx=dx, dres=dres, dgamma=dg, workspace=ws)
    want, wg = ref.norm_grad(dy, h64, r64, gamma, dh)
    gd, xh = dy.to(F64) * gamma.to(F64), h64 * r64[:, None]
    size = r64[:, None] * (gd.abs() + xh.abs() * (gd * xh).abs().mean(1, keepdim=True)) + (0 if dh is None else dh.to(F64).abs())
    ref.within(dx, want, want.abs() * ref.BF16 + size * SUM + 1e-30, "dx")
    if dres is not None:
        ref.within(dres, want, size * SUM + 1e-30, "dres")
    # a sum over T rows: at most T / groups + 16 + groups / 16 roundings in a row
    steps = 64 + T / 256 + 128
    ref.within(dg, wg, (dy.to(F64) * xh).abs().sum(0) * steps * 2.0 ** -24 + 1e-30, "dgamma")
    again = torch.empty_like(dg)
    m.mla_rmsnorm_bwd(dy, h, rstd, gamma, dgamma=again, workspace=ws)
    assert torch.equal(again, dg)


@pytest.mark.parametrize("hd", [BF, F32])
@pytest.mark.parametrize("T, K", [(5, 96), (700, 1536), (3, 8224)])
def test_backward_gives_each_output_alone(T, K, hd):
    g = gen(T)
    h, gamma, dy, dh = rand(g, T, K, dtype=hd), rand(g, K), rand(g, T, K), rand(g, T, K, dtype=hd)
    rstd = ref.norm(h, gamma, 1e-6)[1].to(F32)
    ws = torch.empty(m.mla_rmsnorm_bwd_workspace_size(T, K), dtype=torch.uint8, device=DEV)
    new = dict(dx=lambda: torch.full((T, K), 9.0, dtype=BF, device=DEV), dres=lambda: torch.full((T, K), 9.0, device=DEV),
               dgamma=lambda: torch.full((K,), 9.0, device=DEV))
    all_of = {n: f() for n, f in new.items()}
    m.mla_rmsnorm_bwd(dy, h, rstd, gamma, dh=dh, workspace=ws, **all_of)
    assert torch.equal(all_of["dres"].to(BF), all_of["dx"])
    for n, f in new.items():
        one = f()
        m.mla_rmsnorm_bwd(dy, h, rstd, gamma, dh=dh, workspace=ws if n == "dgamma" else None, **{n: one})
        assert torch.equal(one, all_of[n]), n


def test_no_rows():
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    m.mla_rmsnorm_fwd(e, None, y=torch.empty_like(e))
    dg = torch.full((64,), 5.0, device=DEV)
    ws = torch.empty(m.mla_rmsnorm_bwd_workspace_size(0, 64), dtype=torch.uint8, device=DEV)
    m.mla_rmsnorm_bwd(e, e, torch.empty(0, device=DEV), None, dgamma=dg, workspace=ws)
    assert (dg == 0).all()


@pytest.mark.parametrize("rows, cols, dtype", [(1, 8, BF), (5, 1000, F32), (130, 1536, BF), (3, 40000, F32), (24576, 64, BF)])
def test_int8_quantize(rows, cols, dtype):
    g = gen(rows)
    x = rand(g, rows, cols + 8, dtype=dtype)[:, :cols]
    codes, scales = torch.empty(rows, cols, dtype=torch.int8, device=DEV), torch.empty(rows, device=DEV)
    m.int8_quantize(x, codes, scales)
    s = x.to(F64).abs().amax(1) / 127
    ref.within(scales, s, s * 2.0 ** -23, "scales")
    ref.within(codes, x.to(F64) / s[:, None], torch.tensor(0.5 + 1e-4, device=DEV, dtype=F64), "codes")


def test_rows_past_32_bits_of_offset():
    T, K = 530000, 8192  # 2^32 elements and more
    x, y = (torch.empty(T, K, dtype=BF, device=DEV) for _ in range(2))
    g = gen(3)
    at = [0, 1, T - 2, T - 1]
    x[at] = rand(g, len(at), K)
    m.mla_rmsnorm_fwd(x, None, eps=1e-6, y=y)
    want = ref.norm(x[at], None, 1e-6)[2]
    ref.within(y[at], want, want.abs() * (ref.BF16 + SUM) + 1e-30, "y")


@pytest.mark.parametrize("T", [512, 513, 2048, 2049])
@pytest.mark.parametrize("K", [544, 2048, 2080, 7168])
def test_both_divisions_of_rows_agree(T, K):
    """Few rows are divided over more waves than many: codes and scales as they are for each row alone."""
    g = gen(T + K)
    x, gamma = rand(g, T, K), rand(g, K)
    codes, scales = torch.empty(T, K, dtype=torch.uint8, device=DEV), torch.empty(T, K // 32, dtype=torch.uint8, device=DEV)
    y, one = torch.empty_like(x), torch.empty(1, K, dtype=BF, device=DEV)
    m.mla_rmsnorm_fwd(x, gamma, y=y, codes=codes, scales=scales)
    m.mla_rmsnorm_fwd(x[T - 1:], gamma, y=one)
    want = ref.norm(x[T - 1:], gamma, 1e-6)[2]
    for got in (y[T - 1:], one):
        ref.within(got, want, want.abs() * (ref.BF16 + SUM) + 1e-30, "y")
