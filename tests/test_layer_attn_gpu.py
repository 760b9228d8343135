"""Attention over documents and its backward against 64 bits, element by element within what the roundings to bf16
of weights, dS and results allow (layer_ref)."""
import math

import pytest
import torch

import layer_ref as ref
import mla_up_projection_amd as m

pytestmark = pytest.mark.gpu
DEV = "cuda"
F64, BF, F32, I32 = torch.float64, torch.bfloat16, torch.float32, torch.int32


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rand(g, *s, sigma=1.0):
    return (torch.randn(*s, generator=g, device=DEV) * sigma).to(BF)


def forward(q, k, v, **kw):
    B, H, Sq, _ = q.shape
    out = torch.full((B, H, Sq, v.shape[3]), 7.0, dtype=BF, device=DEV)
    lse = torch.full((B, H, Sq), 7.0, device=DEV)
    ws = torch.empty(m.mla_attn_fwd_workspace_size(q, k, v, out, **kw) or 1, dtype=torch.uint8, device=DEV)
    m.mla_attn_fwd(q, k, v, out, lse=lse, workspace=ws, **kw)
    return out, lse


def backward(dout, q, k, v, out, lse, **kw):
    dq, dk, dv = torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    args = (dout, q, k, v, out, lse, dq, dk, dv)
    ws = torch.empty(m.mla_attn_bwd_workspace_size(*args, **kw) or 1, dtype=torch.uint8, device=DEV)
    m.mla_attn_bwd(*args, workspace=ws, **kw)
    return dq, dk, dv


def check(q, k, v, sees, *, scale, cap=0.0, slopes=None, spans=None, at=None, dout=None):
    kw = dict(scale=scale, cap=cap, slopes=slopes, spans=spans, at=at)
    out, lse = forward(q, k, v, **kw)
    o, l, p, c = ref.attention(q, k, v, sees, scale, cap, slopes, at)
    ref.within(out, o, ref.attention_bound(q, v, o, p), "out")
    ref.within(lse, l, 2e-5 * (1 + l.abs()), "lse")
    if dout is not None:
        got = backward(dout, q, k, v, out, lse, **kw)
        for name, x, (y, bound) in zip(("dq", "dk", "dv"), got, ref.attention_grad(q, k, v, dout, p, c, o, scale)):
            ref.within(x, y, bound, name)
    return out, lse


def make(seed, B, H, hk, Sq, Sk, dk, dv):
    g = gen(seed)
    return rand(g, B, H, Sq, dk), rand(g, B, hk, Sk, dk), rand(g, B, hk, Sk, dv), rand(g, B, H, Sq, dv)


def spans_of(B, Sq, Sk, with_at=False, **kw):
    s = torch.empty(B, Sq, 2, dtype=I32, device=DEV)
    at = torch.empty(B, Sq, dtype=I32, device=DEV) if with_at else None
    tensors = {n: (None if x is None else torch.tensor(x, dtype=I32, device=DEV)) if n not in ("causal", "window") else x
               for n, x in kw.items()}
    m.mla_attn_spans(s, at, Sk=Sk, **tensors)
    return s, at


# ------------------------------------------------------------------ masks
@pytest.mark.parametrize("kw", [
    dict(B=1, Sq=40, Sk=40, cu_q=[0, 7, 7, 30, 36]),
    dict(B=1, Sq=40, Sk=40, cu_q=[0, 7, 7, 30, 40], prefix=[3, 5, 100, 0]),
    dict(B=1, Sq=20, Sk=50, cu_q=[0, 5, 11, 20], cu_k=[0, 20, 26, 50], prefix=[0, 2, 9], window=4),
    dict(B=3, Sq=9, Sk=17, len_q=[9, 0, 4], len_k=[17, 5, 4]),
    dict(B=3, Sq=9, Sk=17, len_q=[9, 2, 4], len_k=[17, 5, 0], causal=False, window=6),
    dict(B=2, Sq=1, Sk=8, window=3),
    dict(B=2, Sq=6, Sk=3),
    dict(B=1, Sq=5, Sk=0),
])
def test_spans(kw):
    B, Sq, Sk = kw["B"], kw["Sq"], kw["Sk"]
    rest = {n: x for n, x in kw.items() if n not in ("B", "Sq", "Sk")}
    s, at = spans_of(B, Sq, Sk, True, **rest)
    sees, places = ref.spans(B, Sq, Sk, **rest)
    assert torch.equal(ref.span_mask(s, Sk).cpu(), sees)
    assert torch.equal(at.cpu().long()[sees.any(2)], places[sees.any(2)])
    assert ((s[..., 1] >= s[..., 0]) & (s >= 0).all(2)).all()


def test_sequence_bounds_outside_the_rows_are_cut():
    s, _ = spans_of(1, 10, 10, cu_q=[0, 4, 1000], prefix=[-5, 1 << 30])
    assert (s[0, 4:] == torch.tensor([4, 10], device=DEV)).all()
    s, _ = spans_of(2, 10, 10, len_q=[-3, 99], len_k=[99, 99])
    assert (s[0] == 0).all() and (s[1, :, 1] == torch.arange(1, 11, device=DEV)).all()


# ------------------------------------------------------------------ values
WIDTHS = [(192, 128), (128, 128), (64, 64), (96, 64), (8, 8), (40, 24), (72, 128), (136, 120), (24, 96), (192, 8)]


@pytest.mark.parametrize("dk, dv", WIDTHS)
@pytest.mark.parametrize("Sq, Sk", [(1, 1), (33, 33), (130, 130)])
def test_causal(dk, dv, Sq, Sk):
    q, k, v, do = make(dk + Sq, 2, 3, 3, Sq, Sk, dk, dv)
    s, _ = spans_of(2, Sq, Sk)
    check(q, k, v, ref.span_mask(s, Sk), scale=1 / math.sqrt(dk), spans=s, dout=do)


@pytest.mark.parametrize("Sq, Sk", [(1, 64), (1, 517), (1, 5000), (1, 6500), (300, 2300), (2, 1777), (32, 700), (64, 300), (65, 900), (127, 128), (128, 64),
                                    (129, 65), (200, 63), (257, 511)])
@pytest.mark.parametrize("dk, dv", [(192, 128), (64, 64)])
def test_all_keys(Sq, Sk, dk, dv):
    q, k, v, do = make(Sq + Sk, 1, 2, 1, Sq, Sk, dk, dv)
    check(q, k, v, torch.ones(1, Sq, Sk, dtype=torch.bool, device=DEV), scale=0.11, dout=do)


@pytest.mark.parametrize("cap, slope, scale", [(20.0, False, 0.09), (0.0, True, 0.09), (5.0, True, 0.2), (0.0, False, -0.09),
                                               (0.0, False, 0.0), (3.0, False, -0.3)])
@pytest.mark.parametrize("dk, dv", [(192, 128), (128, 128), (64, 64)])
def test_caps_and_distances(cap, slope, scale, dk, dv):
    B, H, hk, Sq, Sk = 2, 4, 2, 150, 150
    q, k, v, do = make(int(cap) + dk, B, H, hk, Sq, Sk, dk, dv)
    slopes = torch.tensor([0.5, 0.1, 0.01, 0.0], device=DEV) if slope else None
    s, at = spans_of(B, Sq, Sk, slope, len_q=[150, 77], len_k=[150, 77], prefix=[0, 30])
    check(q, k, v, ref.span_mask(s, Sk), scale=scale, cap=cap, slopes=slopes, spans=s, at=at, dout=do)


@pytest.mark.parametrize("cap, slope", [(0.0, False), (0.0, True), (20.0, True)])
@pytest.mark.parametrize("dk, dv", [(192, 128), (128, 128), (64, 64)])
@pytest.mark.parametrize("B, H, hk, S", [(3, 88, 88, 130), (1, 64, 2, 600), (1, 40, 40, 600)])
def test_more_rows_than_compute_units(B, H, hk, S, dk, dv, cap, slope):
    """More tiles of 128 queries than the chip has compute units, with as many key tiles and with few; as many as it has
    of each together. The backward's kernels run in turn or at once, with one part or several."""
    q, k, v, do = make(S + dk, B, H, hk, S, S, dk, dv)
    slopes = torch.rand(H, device=DEV, generator=gen(5)) if slope else None
    s, at = spans_of(B, S, S, slope, len_q=[S, 77, 1][:B], len_k=[S, 77, 1][:B])
    check(q, k, v, ref.span_mask(s, S), scale=0.09, cap=cap, slopes=slopes, spans=s, at=at, dout=do)


@pytest.mark.parametrize("Sq, Sk", [(1, 700), (40, 90), (200, 200)])
def test_distances_without_places(Sq, Sk):
    """Without `at` the queries are the last of the keys; without spans they see all of them; lse need not be asked for."""
    q, k, v, do = make(Sq, 2, 4, 4, Sq, Sk, 64, 64)
    slopes = torch.tensor([0.5, 0.1, 0.01, 0.0], device=DEV)
    out, _ = check(q, k, v, torch.ones(2, Sq, Sk, dtype=torch.bool, device=DEV), scale=0.2, slopes=slopes, dout=do)
    alone = torch.empty_like(out)
    ws = torch.empty(m.mla_attn_fwd_workspace_size(q, k, v, scale=0.2) or 1, dtype=torch.uint8, device=DEV)
    m.mla_attn_fwd(q, k, v, alone, scale=0.2, slopes=slopes, workspace=ws)
    assert torch.equal(alone, out)


@pytest.mark.parametrize("H, hk", [(8, 8), (8, 2), (6, 1)])
def test_packed_documents(H, hk):
    cu = [0, 1, 64, 64, 200, 333, 460]  # rows 460 .. 499 are padding
    S = 500
    q, k, v, do = make(H, 1, H, hk, S, S, 192, 128)
    s, at = spans_of(1, S, S, True, cu_q=cu, prefix=[0, 10, 0, 100, 5, 200])
    sees = ref.spans(1, S, S, cu_q=cu, prefix=[0, 10, 0, 100, 5, 200])[0].to(DEV)
    out, lse = check(q, k, v, sees, scale=0.07, spans=s, at=at, dout=do)
    assert (out[0, :, 460:] == 0).all() and (lse[0, :, 460:] == -math.inf).all()


def test_chunks_of_prompts_and_windows():
    cu_q, cu_k = [0, 40, 41, 190], [0, 300, 377, 640]
    q, k, v, do = make(3, 1, 4, 2, 190, 640, 128, 128)
    s, at = spans_of(1, 190, 640, True, cu_q=cu_q, cu_k=cu_k, window=100)
    sees = ref.spans(1, 190, 640, cu_q=cu_q, cu_k=cu_k, window=100)[0].to(DEV)
    slopes = torch.tensor([0.3, 0.03, 0.003, 0.0], device=DEV)
    check(q, k, v, sees, scale=0.1, slopes=slopes, spans=s, at=at, dout=do)


def test_spans_of_any_kind():
    """Spans that follow no order, reach outside the keys or are empty."""
    B, H, Sq, Sk = 2, 2, 300, 400
    q, k, v, do = make(9, B, H, 1, Sq, Sk, 64, 64)
    g = gen(10)
    s = torch.randint(-50, Sk + 50, (B, Sq, 2), generator=g, device=DEV, dtype=I32)
    cut = s.clamp(0, Sk)
    check(q, k, v, ref.span_mask(cut, Sk), scale=0.2, spans=s, dout=do)
    none = torch.zeros_like(s)
    out, lse = forward(q, k, v, scale=0.2, spans=none)
    assert (out == 0).all() and (lse == -math.inf).all()
    for t in backward(do, q, k, v, out, lse, scale=0.2, spans=none):
        assert (t == 0).all()


@pytest.mark.parametrize("Sq, Sk", [(0, 5), (5, 0), (0, 0)])
def test_no_rows(Sq, Sk):
    q, k, v, do = make(1, 2, 4, 2, Sq, Sk, 64, 64)
    out, lse = forward(q, k, v, scale=0.2)
    assert (out == 0).all() and (lse == -math.inf).all()
    for t in backward(do, q, k, v, out, lse, scale=0.2):
        assert (t == 0).all()


def test_large_scores_and_a_maximum_that_rises_late():
    q, k, v, do = make(4, 1, 2, 2, 130, 700, 64, 64)
    k = (k.float() * torch.linspace(0.1, 30, 700, device=DEV)[None, None, :, None]).to(BF)
    check(q, k, v, torch.ones(1, 130, 700, dtype=torch.bool, device=DEV), scale=1.0, dout=do)


@pytest.mark.parametrize("H, hk, S", [(2, 1, 4500), (4, 1, 4200), (1, 1, 8300), (16, 1, 130), (24, 1, 60)])
def test_many_tiles(H, hk, S):
    """More than 64 tiles of 64 queries, so that the list of those that see a key has several words, for every head; or
    few rows and many heads to a key head, whose tiles go to many workgroups."""
    cu = [0, 5, 1000, 4100, S - 30]
    q, k, v, do = make(S, 1, H, hk, S, S, 64, 64)
    s, _ = spans_of(1, S, S, cu_q=cu)
    check(q, k, v, ref.span_mask(s, S), scale=0.15, spans=s, dout=do)


@pytest.mark.parametrize("Sq", [3, 150])
def test_keys_that_batch_entries_share(Sq):
    """Keys and values of one entry seen by all of the batch (stride 0)."""
    q, k, v, _ = make(Sq, 3, 4, 2, Sq, 333, 128, 128)
    k, v = k[:1].expand(3, -1, -1, -1), v[:1].expand(3, -1, -1, -1)
    assert k.stride(0) == 0
    check(q, k, v, torch.ones(3, Sq, 333, dtype=torch.bool, device=DEV), scale=0.1)


def test_rows_past_32_bits_of_offset():
    """Batch entries 2^31 elements apart, in bytes past 2^32."""
    B, H, S, d = 2, 1, 70, 64
    far = (1 << 31) + 64
    g = gen(21)
    t = {n: torch.as_strided(torch.empty(far + H * S * d, dtype=BF, device=DEV), (B, H, S, d), (far, S * d, d, 1))
         for n in ("q", "k", "v", "do")}
    for x in t.values():
        x.copy_(rand(g, B, H, S, d))
    s, _ = spans_of(B, S, S)
    check(t["q"], t["k"], t["v"], ref.span_mask(s, S), scale=0.1, spans=s, dout=t["do"])


@pytest.mark.parametrize("Sq, Sk", [(5, 900), (150, 300)])
def test_values_at_the_end_of_the_range(Sq, Sk):
    """A mean of values up to 2^127 is finite, also where their sum is not."""
    q, k, v, _ = make(31, 1, 2, 2, Sq, Sk, 64, 64)
    v = torch.where(v.float() > 0, 2.0 ** 127, 2.0 ** 126).to(BF)
    k = (k.float() * torch.linspace(0.2, 8, Sk, device=DEV)[None, None, :, None]).to(BF)
    s = torch.ones(1, Sq, Sk, dtype=torch.bool, device=DEV)
    out, _ = forward(q, k, v, scale=1.0)
    o, _, p, _ = ref.attention(q, k, v, s, 1.0)
    ref.within(out, o, ref.attention_bound(q, v, o, p), "out")


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e-6])
def test_scales_near_nothing(scale):
    q, k, v, do = make(32, 1, 2, 2, 100, 100, 64, 64)
    s, _ = spans_of(1, 100, 100)
    check(q, k, v, ref.span_mask(s, 100), scale=scale, spans=s, dout=do)


# ------------------------------------------------------------------ what is not seen
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
@pytest.mark.parametrize("Sq", [20, 200])
def test_rows_that_are_not_seen_have_no_influence(bad, Sq):
    """Padding keys, values and query rows (and their gradients) hold what was left there."""
    B, H, hk, Sk = 2, 4, 2, 300
    q, k, v, do = make(7, B, H, hk, Sq, Sk, 128, 64)
    lq, lk = [Sq, Sq // 2], [300, 201]
    s, _ = spans_of(B, Sq, Sk, len_q=lq, len_k=lk)
    clean, clean_lse = forward(q, k, v, scale=0.1, spans=s)
    grads = backward(do, q, k, v, clean, clean_lse, scale=0.1, spans=s)
    q2, k2, v2, do2 = (t.clone() for t in (q, k, v, do))
    q2[1, :, lq[1]:], do2[1, :, lq[1]:], k2[1, :, lk[1]:], v2[1, :, lk[1]:] = bad, bad, bad, bad
    out, lse = forward(q2, k2, v2, scale=0.1, spans=s)
    assert torch.equal(lse, clean_lse)
    # rows done again differ by roundings only
    ref.within(out, clean.to(F64), clean.to(F64).abs() * 2 * ref.BF16 + 0.02, "out")
    assert (out[1, :, lq[1]:] == 0).all()
    for name, a, b in zip(("dq", "dk", "dv"), backward(do2, q2, k2, v2, out, lse, scale=0.1, spans=s), grads):
        assert torch.isfinite(a).all(), name
        ref.within(a, b.to(F64), b.to(F64).abs() * 4 * ref.BF16 + 0.02 * b.float().abs().max(), name)


@pytest.mark.parametrize("cap", [0.0, 20.0, 50.0, 1e4])
def test_one_key_far_below_the_cap(cap):
    """Its lse is the score. Eight exact products are added (8 2^-23 of their magnitudes); scale, series and cap are at
    most 16 roundings relative to the score."""
    q, k, v, _ = make(int(cap), 2, 3, 3, 70, 1, 8, 8)
    _, lse = forward(q, k, v, scale=0.1, cap=cap)
    prod = q.to(F64) * k.to(F64)
    s = prod.sum(-1) * 0.1
    s = cap * torch.tanh(s / cap) if cap else s
    ref.within(lse, s, 8 * 2.0 ** -23 * 0.1 * prod.abs().sum(-1) + 2.0 ** -20 * s.abs(), "lse")


@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_holes_between_rows(cap):
    """Rows that see nothing in front of, between and behind others, all with NaN: gradients of the others are finite
    and what they are without them."""
    Sq, Sk = 260, 300
    q, k, v, do = make(17, 1, 4, 2, Sq, Sk, 64, 64)
    s, _ = spans_of(1, Sq, Sk, causal=False)
    s[:, :, 0], s[:, :, 1] = 30, 250
    for a, b in ((0, 5), (64, 70), (100, 101), (120, 192), (255, 260)):
        s[:, a:b] = 7
    sees = ref.span_mask(s, Sk)
    kw = dict(scale=0.1, cap=cap, spans=s)
    check(q, k, v, sees, dout=do, **kw)
    out, lse = forward(q, k, v, **kw)
    want = backward(do, q, k, v, out, lse, **kw)
    dead = ~sees[0].any(1)
    q[:, :, dead], do[:, :, dead] = float("nan"), float("inf")
    k[:, :, :30], k[:, :, 250:], v[:, :, :30], v[:, :, 250:] = float("nan"), float("nan"), float("inf"), float("nan")
    again, lse2 = forward(q, k, v, **kw)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    for name, a, b in zip(("dq", "dk", "dv"), backward(do, q, k, v, again, lse2, **kw), want):
        assert torch.isfinite(a).all(), name
        ref.within(a, b.to(F64), b.to(F64).abs() * 4 * ref.BF16 + 0.02 * b.float().abs().max(), name)
    assert (want[1][:, :, :30] == 0).all() and (want[1][:, :, 250:] == 0).all()


def test_a_value_that_some_see():
    """Rows that see a NaN value have it in their result, those that do not have none."""
    q, k, v, do = make(8, 1, 2, 2, 150, 150, 64, 64)
    v[0, 0, 70, 5] = float("nan")
    v[0, 1, 71, 6] = float("inf")
    s, _ = spans_of(1, 150, 150)
    out, lse = forward(q, k, v, scale=0.2, spans=s)
    o, l, p, _ = ref.attention(q, k, v, ref.span_mask(s, 150), 0.2)
    finite = torch.isfinite(o)
    assert torch.isnan(out[0, 0, 70:, 5]).all() and torch.isfinite(out[0, 0, :70]).all()
    assert torch.isinf(out[0, 1, 71:, 6]).all()
    vv = torch.where(torch.isfinite(v), v, 0.0)
    ref.within(out[finite], o[finite], ref.attention_bound(q, vv, o, p)[finite], "out")
    ref.within(lse, l, 2e-5 * (1 + l.abs()), "lse")


# ------------------------------------------------------------------ layouts, streams, graphs
def test_strided_rows():
    """Token-major queries inside wider rows, keys and values interleaved as one tensor."""
    g = gen(2)
    B, H, hk, S, dk, dv = 2, 4, 2, 140, 128, 64
    wide = rand(g, B, S, H, dk + 64)
    q = wide[..., :dk].transpose(1, 2)
    kv = rand(g, B, S, hk, dk + dv)
    k, v = kv[..., :dk].transpose(1, 2), kv[..., dk:].transpose(1, 2)
    do = rand(g, B, S, H, dv).transpose(1, 2)
    s, _ = spans_of(B, S, S)
    kw = dict(scale=0.1, spans=s)
    want, wl = forward(*(t.contiguous() for t in (q, k, v)), **kw)
    out = torch.empty(B, S, H, dv, dtype=BF, device=DEV).transpose(1, 2)
    lse = torch.empty(B, H, S, device=DEV)
    ws = torch.empty(m.mla_attn_fwd_workspace_size(q, k, v, out, **kw) or 1, dtype=torch.uint8, device=DEV)
    m.mla_attn_fwd(q, k, v, out, lse=lse, workspace=ws, **kw)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    grads = backward(*(t.contiguous() for t in (do, q, k, v, want)), wl, **kw)
    dkv = torch.full((B, S, hk, dk + dv + 8), 3.0, dtype=BF, device=DEV)
    dq = torch.empty(B, S, H, dk, dtype=BF, device=DEV).transpose(1, 2)
    args = (do, q, k, v, out, lse, dq, dkv[..., :dk].transpose(1, 2), dkv[..., dk:dk + dv].transpose(1, 2))
    ws = torch.empty(m.mla_attn_bwd_workspace_size(*args, **kw), dtype=torch.uint8, device=DEV)
    m.mla_attn_bwd(*args, workspace=ws, **kw)
    for a, b in zip(args[6:], grads):
        assert torch.equal(a, b)
    assert (dkv[..., dk + dv:] == 3).all()


def test_results_do_not_depend_on_timing():
    q, k, v, do = make(5, 1, 4, 1, 300, 900, 192, 128)
    a = forward(q, k, v, scale=0.1)
    ga = backward(do, q, k, v, *a, scale=0.1)
    for _ in range(3):
        b = forward(q, k, v, scale=0.1)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert all(torch.equal(x, y) for x, y in zip(ga, backward(do, q, k, v, *b, scale=0.1)))


def test_a_captured_layer_replays_with_other_lengths():
    """Norm, integer projection, masks, attention and the way back in one graph, replayed on other data."""
    B, S, K, H, dn, dr, dv = 2, 70, 256, 2, 64, 64, 64
    D = dn + dr
    g = gen(6)
    x, gamma = rand(g, B * S, K), rand(g, K)
    w, ws_ = torch.empty(H * D, K, dtype=torch.int8, device=DEV), torch.empty(H * D, device=DEV)
    m.int8_quantize(rand(g, H * D, K, sigma=0.05), w, ws_)
    cos, sin = torch.empty(S, dr // 2, device=DEV), torch.empty(S, dr // 2, device=DEV)
    m.rope_cache_build(cos, sin, dr)
    k, v, do = rand(g, B, H, S, D), rand(g, B, H, S, dv), rand(g, B, H, S, dv)
    lens = torch.tensor([S, 33], dtype=I32, device=DEV)
    codes, sc = torch.empty(B * S, K, dtype=torch.int8, device=DEV), torch.empty(B * S, device=DEV)
    q, out = torch.empty(B, H, S, D, dtype=BF, device=DEV), torch.empty(B, H, S, dv, dtype=BF, device=DEV)
    lse, spans = torch.empty(B, H, S, device=DEV), torch.empty(B, S, 2, dtype=I32, device=DEV)
    dq, dk, dvv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    kw = dict(scale=0.1, spans=spans)
    wf = torch.empty(m.mla_attn_fwd_workspace_size(q, k, v, out, **kw) or 1, dtype=torch.uint8, device=DEV)
    wb = torch.empty(m.mla_attn_bwd_workspace_size(do, q, k, v, out, lse, dq, dk, dvv, **kw), dtype=torch.uint8, device=DEV)

    def step():
        m.mla_rmsnorm_fwd(x, gamma, codes=codes, scales=sc)
        m.mla_qup_fwd_i8(codes, sc, w, ws_, q, H=H, d_nope=dn, d_rope=dr, cos=cos, sin=sin, B=B, S=S)
        m.mla_attn_spans(spans, Sk=S, len_q=lens, len_k=lens)
        m.mla_attn_fwd(q, k, v, out, lse=lse, workspace=wf, **kw)
        m.mla_attn_bwd(do, q, k, v, out, lse, dq, dk, dvv, workspace=wb, **kw)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in (33, 1, 0, 70):
        lens[1] = n
        x.copy_(rand(g, B * S, K))
        graph.replay()
        got = [t.clone() for t in (q, out, lse, dq, dk, dvv)]
        step()
        for a, b in zip(got, (q, out, lse, dq, dk, dvv)):
            assert torch.equal(a, b)
        assert (out[1, :, n:] == 0).all() and (dk[1, :, n:] == 0).all()


def test_two_streams_at_once():
    q, k, v, do = make(11, 1, 4, 4, 300, 300, 192, 128)
    s, _ = spans_of(1, 300, 300)
    want = forward(q, k, v, scale=0.1, spans=s)
    grads = backward(do, q, k, v, *want, scale=0.1, spans=s)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for st in (a, b, a, b):
        with torch.cuda.stream(st):
            o = forward(q, k, v, scale=0.1, spans=s)
            got.append(o + backward(do, q, k, v, *o, scale=0.1, spans=s))
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(x, y) for x, y in zip(r, want + grads))


def test_training_chain():
    """Norm -> projection -> attention and all the way back to the norm's input, against 64 bits with the library's
    own stored tensors, each product's error bounded by its operands' roundings."""
    g = gen(12)
    T, K, H, dn, dr, dv = 96, 256, 2, 64, 64, 64
    D, N = dn + dr, H * (dn + dr)
    x, gamma, w = rand(g, T, K), rand(g, K), rand(g, N, K, sigma=0.06)
    cos, sin = torch.empty(T, dr // 2, device=DEV), torch.empty(T, dr // 2, device=DEV)
    m.rope_cache_build(cos, sin, dr)
    k, v, do = rand(g, 1, H, T, D), rand(g, 1, H, T, dv), rand(g, 1, H, T, dv)
    y, rstd = torch.empty(T, K, dtype=BF, device=DEV), torch.empty(T, device=DEV)
    m.mla_rmsnorm_fwd(x, gamma, y=y, rstd=rstd)
    q = torch.empty(1, H, T, D, dtype=BF, device=DEV)
    kw = dict(H=H, d_nope=dn, d_rope=dr, cos=cos, sin=sin, B=1, S=T)
    m.mla_qup_fwd(y, w, q, **kw)
    s, _ = spans_of(1, T, T)
    out, lse = forward(q, k, v, scale=0.09, spans=s)
    dq = torch.empty(T, H, D, dtype=BF, device=DEV)
    dk, dvv = torch.empty_like(k), torch.empty_like(v)
    args = (do, q, k, v, out, lse, dq[None].transpose(1, 2), dk, dvv)
    ws = torch.empty(m.mla_attn_bwd_workspace_size(*args, scale=0.09, spans=s), dtype=torch.uint8, device=DEV)
    m.mla_attn_bwd(*args, scale=0.09, spans=s, workspace=ws)
    dq_pre, dy, dw = (torch.empty(n, dtype=BF, device=DEV) for n in ((T, N), (T, K), (N, K)))
    nb = m.mla_qup_bwd_workspace_size(dq, y, w, dq_pre, dx=dy, dw=dw, **kw)
    m.mla_qup_bwd(dq, y, w, dq_pre, dx=dy, dw=dw, workspace=torch.empty(nb, dtype=torch.uint8, device=DEV) if nb else None, **kw)
    dx, dg = torch.empty_like(x), torch.empty(K, device=DEV)
    ws = torch.empty(m.mla_rmsnorm_bwd_workspace_size(T, K), dtype=torch.uint8, device=DEV)
    m.mla_rmsnorm_bwd(dy, x, rstd, gamma, dx=dx, dgamma=dg, workspace=ws)
    # in 64 bits from the start, by automatic differentiation
    x64, g64, w64 = (t.to(F64).requires_grad_() for t in (x, gamma, w))
    y64 = x64 / torch.sqrt(x64.square().mean(1, keepdim=True) + 1e-6) * g64
    p64 = (y64 @ w64.t()).view(T, H, D)
    c, sn = cos.to(F64)[:, None], sin.to(F64)[:, None]
    a, b = p64[..., dn::2], p64[..., dn + 1::2]
    q64 = torch.cat([p64[..., :dn], torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2)], -1).transpose(0, 1)[None]
    o64 = ref.attention(q64, k, v, ref.span_mask(s, T), 0.09)[0]
    (o64 * do.to(F64)).sum().backward()
    # roundings to bf16 on the way: y, q, P, out, dS, dq, dq_pre, dy and the result itself; independent of each
    # other, so in the 2-norm their sum stays below nine times one
    for name, got, want in (("out", out, o64.detach()), ("dx", dx, x64.grad), ("dgamma", dg, g64.grad), ("dw", dw, w64.grad)):
        err = (got.to(F64) - want).norm() / want.norm()
        assert err <= 9 * ref.BF16, (name, err.item())
