"""Plain 64-bit implementations of the operators around the projection in a layer, with bounds of what the kernels'
roundings may do to each value. A rounding to bf16 is off by at most 2^-8 of the value, to fp32 by 2^-24."""
import torch

F64 = torch.float64
BF16 = 2.0 ** -8
SLACK = 2.0 ** -11  # fp32 sums, products and exponentials: far below the bf16 roundings next to them


# ------------------------------------------------------------------ norm
def norm(x, gamma, eps, res=None):
    """h (as it is stored), rstd and y."""
    h = x.to(F64)
    if res is not None:
        h = (h + res.to(F64)).to(torch.float32).to(res.dtype).to(F64)  # one fp32 sum, rounded to its type
    rstd = 1 / torch.sqrt(h.square().mean(1) + eps)
    y = h * rstd[:, None] * (1 if gamma is None else gamma.to(F64))
    return h, rstd, y


def norm_grad(dy, h, rstd, gamma, dh=None):
    xh = h * rstd[:, None]
    g = dy.to(F64) * (1 if gamma is None else gamma.to(F64))
    d = (g - xh * (g * xh).mean(1, keepdim=True)) * rstd[:, None]
    return d if dh is None else d + dh.to(F64), (dy.to(F64) * xh).sum(0)


# ------------------------------------------------------------------ masks
def spans(B, Sq, Sk, cu_q=None, cu_k=None, len_q=None, len_k=None, prefix=None, causal=True, window=0):
    """[B, Sq, Sk] truth values, from the words of the mask's definition, and the rows' places."""
    sees = torch.zeros(B, Sq, Sk, dtype=torch.bool)
    at = torch.zeros(B, Sq, dtype=torch.int64)
    for b in range(B):
        for i in range(Sq):
            if cu_q is not None:
                ck = cu_q if cu_k is None else cu_k
                docs = [j for j in range(len(cu_q) - 1) if cu_q[j] <= i < cu_q[j + 1]]
                if not docs:
                    continue
                j = docs[-1]
                q0, q1, k0, k1 = cu_q[j], cu_q[j + 1], ck[j], ck[j + 1]
            else:
                j, q0, k0 = b, 0, 0
                q1 = Sq if len_q is None else len_q[b]
                k1 = Sk if len_k is None else len_k[b]
                if i >= q1:
                    continue
            place = k1 - (q1 - i)
            at[b, i] = place
            for k in range(k0, k1):
                ok = True
                if causal:
                    ok = k <= place or (prefix is not None and k - k0 < prefix[j])
                if window:
                    ok = ok and place - k < window
                sees[b, i, k] = ok
    return sees, at


def span_mask(span, Sk):
    """[B, Sq, Sk] of spans [B, Sq, 2]."""
    k = torch.arange(Sk, device=span.device)
    return (k >= span[..., :1]) & (k < span[..., 1:])


# ------------------------------------------------------------------ attention
def scores(q, k, scale, cap=0.0, slopes=None, at=None):
    """Scores [B, H, Sq, Sk] and the cap's derivative."""
    B, H, Sq, _ = q.shape
    Sk = k.shape[2]
    k = k.repeat_interleave(H // k.shape[1], 1)
    t = scale * (q @ k.transpose(2, 3))
    c = torch.ones_like(t)
    if cap:
        th = torch.tanh(t / cap)
        t, c = cap * th, 1 - th * th
    if slopes is not None:
        if at is None:
            at = (torch.arange(Sq, device=q.device) + Sk - Sq).expand(B, Sq)
        far = (at[:, :, None] - torch.arange(Sk, device=q.device)).abs().to(F64)
        t = t - slopes.to(F64)[None, :, None, None] * far[:, None]
    return t, c


def attention(q, k, v, sees, scale, cap=0.0, slopes=None, at=None):
    """out, lse, P and the cap's derivative, in 64 bits. What a row does not see takes no part: rows of k and v that
    are not finite are left out of the products of rows that do not see them."""
    q, k, v = (t.to(F64) for t in (q, k, v))
    t, c = scores(q, k, scale, cap, slopes, at)
    t = torch.where(sees[:, None], t, -float("inf"))
    m = t.amax(-1, keepdim=True) if t.shape[-1] else torch.full_like(t[..., :1].sum(-1, keepdim=True), -float("inf"))
    m = torch.where(m == -float("inf"), 0.0, m)
    e = torch.exp(t - m)
    l = e.sum(-1, keepdim=True)
    p = e / torch.where(l == 0, 1.0, l)
    return times(p, v.repeat_interleave(q.shape[1] // v.shape[1], 1)), (m + torch.log(l))[..., 0], p, c


def times(p, v):
    """p @ v, with 0 * anything = 0."""
    if torch.isfinite(v).all():
        return p @ v
    out = p @ torch.where(torch.isfinite(v), v, 0.0)
    bad = ~torch.isfinite(v)
    for b, h, j, d in torch.nonzero(bad).tolist():
        w = p[b, h, :, j]
        out[b, h, :, d] += torch.where(w == 0, 0.0, w * v[b, h, j, d])
    return out


def attention_bound(q, v, out, p):
    """How far an element of out may be off: the weights' rounding times what they weigh, and its own."""
    v = v.to(F64).repeat_interleave(q.shape[1] // v.shape[1], 1).abs()
    return BF16 * out.abs() * (1 + SLACK) + (BF16 + SLACK) * times(p, v) + 1e-30


def attention_grad(q, k, v, dout, p, c, out, scale):
    """dq, dk, dv and bounds of each: P and dS are rounded to bf16, delta comes from out, which is rounded."""
    q, k, v, dout = (t.to(F64) for t in (q, k, v, dout))
    H, hk = q.shape[1], k.shape[1]
    kk, vv = k.repeat_interleave(H // hk, 1), v.repeat_interleave(H // hk, 1)
    share = lambda t: t.unflatten(1, (hk, H // hk)).sum(2)  # noqa: E731
    dp = dout @ vv.transpose(2, 3)
    delta = (dout * out).sum(-1, keepdim=True)
    ds = p * (dp - delta) * c
    d_delta = (dout.abs() * attention_bound(q, v, out, p)).sum(-1, keepdim=True)
    size = dout.abs() @ vv.abs().transpose(2, 3) + (dout * out).abs().sum(-1, keepdim=True)
    off = (BF16 + SLACK) * ds.abs() + p * (d_delta + SLACK * 2.0 ** -4 * size)
    dq, dk, dv = scale * (ds @ kk), scale * share(ds.transpose(2, 3) @ q), share(p.transpose(2, 3) @ dout)
    s = abs(scale)
    return ((dq, BF16 * dq.abs() + s * (off @ kk.abs()) + 1e-30),
            (dk, BF16 * dk.abs() + s * share(off.transpose(2, 3) @ q.abs()) + 1e-30),
            (dv, BF16 * dv.abs() + (BF16 + SLACK) * share(p.transpose(2, 3) @ dout.abs()) + 1e-30))


def within(got, want, bound, what=""):
    got, want = got.to(F64), want.to(F64)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), f"{what}: infinities"
    off = (got - want).abs()[fine]
    b = bound.expand_as(want)[fine]
    if off.numel():
        worst = (off / b).max().item()
        assert worst <= 1, f"{what}: {worst:.3g} times the bound"
