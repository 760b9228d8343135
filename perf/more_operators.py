"""Cases and plain forms of the operators on both sides of the query
up-projection: the RMS norm in front of it with its 8-bit output, the projection
itself in 8-bit integers, and attention over documents behind it, with the
gradients of norm and attention.

`run` computes an operator in elementary torch operations in 32 bits, or, with
`own` set, through the library's entry points. Shapes are DeepSeek-V3's MLA
(q_lora_rank 1536, 128 heads of 128 + 64, values of 128), its head-parallel
shards, and generic ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BF16, F8, E8 = torch.bfloat16, torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------ the cases
def listed():
    mla = dict(d_k=192, d_v=128)
    plain = dict(packed=False, causal=True, window=0, prefix=0, cap=0.0, slopes=False, ragged=False, doc_lo=0,
                 doc_hi=0, backward=False)
    return [
        # one decoded token entering a layer: nothing but latency
        dict(name="norm one token", op="norm", T=1, K=7168, residual="bf16", quant="mxfp8", keep=False, backward=False),
        # the query latents of two prompts on their way into the MXFP8 projection, kept in bf16 for its backward
        dict(name="norm latents mxfp8", op="norm", T=8192, K=1536, residual="none", quant="mxfp8", keep=True,
             backward=False),
        # a layer's entry in training, both directions
        dict(name="norm train", op="norm", T=4096, K=7168, residual="bf16", quant="none", keep=True, backward=True),
        # one token's latent through norm and integer projection
        dict(name="project one token", op="project", T=1, K=1536, heads=128, d_nope=128, d_rope=64, out="bf16"),
        # the drafts of a small batch, queries in 8 bits
        dict(name="project drafts", op="project", T=52, K=1536, heads=128, d_nope=128, d_rope=64, out="mxfp8"),
        # a prompt: the matrix units bound it
        dict(name="project prompt", op="project", T=4096, K=1536, heads=128, d_nope=128, d_rope=64, out="bf16"),
        # one token of one conversation on a contiguous cache
        dict(plain, name="attend one token", op="attend", B=1, Sq=1, Sk=1777, heads=128, kv_heads=128, **mla),
        # the next chunk of four padded prompts on a head shard
        dict(plain, name="attend chunk", op="attend", B=4, Sq=200, Sk=2100, heads=16, kv_heads=16, ragged=True, **mla),
        # packed documents with prefixes that all their tokens see, one rank's heads
        dict(plain, name="attend documents", op="attend", B=1, Sq=16384, Sk=16384, heads=16, kv_heads=16, packed=True,
             prefix=300, doc_lo=512, doc_hi=4096, **mla),
        # short ragged sequences in training, capped scores, heads that share keys
        dict(plain, name="train short", op="attend", B=3, Sq=333, Sk=333, heads=8, kv_heads=2, ragged=True, cap=30.0,
             backward=True, d_k=128, d_v=128),
        # one sequence on all heads, both directions: the matrix units bound it
        dict(plain, name="train causal", op="attend", B=1, Sq=4096, Sk=4096, heads=128, kv_heads=128, backward=True,
             **mla),
        # packed documents in training with a distance bias
        dict(plain, name="train documents", op="attend", B=1, Sq=8192, Sk=8192, heads=16, kv_heads=16, packed=True,
             slopes=True, doc_lo=256, doc_hi=3000, backward=True, **mla),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "project", "project", "attend", "attend", "attend", "attend"])
    if op == "norm":
        K = 32 * _log(rng, 2, 256)
        backward = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, min(16000, 30e6 / K)), K=K, residual=rng.choice(["none", "bf16", "fp32"]),
                    quant="none" if backward else rng.choice(["none", "mxfp8", "int8"]), keep=True, backward=backward)
    if op == "project":
        H, K = rng.choice([1, 5, 8, 16, 32, 128]), 64 * _log(rng, 1, 32)
        return dict(op=op, T=_log(rng, 1, min(5000, 800e6 / (H * K))), K=K, heads=H, d_nope=rng.choice([128, 128, 64, 0]),
                    d_rope=64, out=rng.choice(["bf16", "mxfp8"]))
    heads, kv, d_k, d_v = rng.choice([(16, 16, 192, 128), (128, 128, 192, 128), (12, 12, 192, 128), (32, 8, 128, 128),
                                      (8, 2, 128, 128), (14, 7, 64, 64), (6, 6, 96, 64), (10, 1, 128, 128)])
    backward = rng.random() < 0.5
    packed = rng.random() < 0.4
    B = 1 if packed else _log(rng, 1, 8)
    Sk = _log(rng, 1, min(16384, math.sqrt((1e9 if backward else 3e9) / (B * heads))))
    Sq = Sk if packed or backward else rng.choice([Sk, _log(rng, 1, Sk)])
    hi = _log(rng, 1, Sk)
    return dict(op=op, B=B, Sq=Sq, Sk=Sk, heads=heads, kv_heads=kv, d_k=d_k, d_v=d_v, packed=packed,
                causal=rng.random() < 0.8, window=rng.choice([0, 0, 0, _log(rng, 1, Sk)]),
                prefix=rng.choice([0, 0, rng.randint(0, hi)]), cap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                slopes=rng.random() < 0.3, ragged=not packed and rng.random() < 0.5, doc_lo=rng.randint(0, hi),
                doc_hi=hi, backward=backward)


# ------------------------------------------------------------------ inputs
def _normal(g, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * sigma).to(BF16)


def _lens(case):
    """Query and key lengths of the sequences (packed: of the documents) and their prefixes. They follow the
    case alone, so that outputs of different seeds have one shape."""
    r = random.Random(case["Sq"] * 7919 + case["Sk"] * 31 + case["doc_lo"] * 3 + case["B"])
    if case["packed"]:
        q, left = [], case["Sk"]
        while left > 0 and len(q) < 4000:
            n = min(left, r.randint(case["doc_lo"], case["doc_hi"]))
            q.append(n)
            left -= n
        k = list(q)  # rows that no document takes are padding
    else:
        k = [r.randint(0 if i else case["Sk"], case["Sk"]) if case["ragged"] else case["Sk"] for i in range(case["B"])]
        q = [min(r.randint(0 if i else case["Sq"], case["Sq"]), n) if case["ragged"] else case["Sq"]
             for i, n in enumerate(k)]
        if case["Sq"] == case["Sk"]:
            q = list(k)
    p = [min(n, r.randint(0, case["prefix"])) if case["prefix"] else 0 for n in k]
    return q, k, p


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(v):
    return _ints([sum(v[:i]) for i in range(len(v) + 1)])


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        T, K = case["T"], case["K"]
        s |= dict(x=_normal(g, T, K), gamma=1 + _normal(g, K, sigma=0.2), dy=None, dh=None, res=None)
        if case["residual"] != "none":
            s["res"] = _normal(g, T, K, sigma=3.0)
            s["res"] = s["res"].float() * 1.003 if case["residual"] == "fp32" else s["res"]
        if case["backward"]:
            s["dy"] = _normal(g, T, K, sigma=1e-2)
            s["dh"] = None if s["res"] is None else torch.randn(T, K, generator=g, device=DEV).mul_(1e-2).to(s["res"].dtype)
        return s
    if case["op"] == "project":
        T, K, H, D = case["T"], case["K"], case["heads"], case["d_nope"] + case["d_rope"]
        w = _normal(g, H * D, K, sigma=0.02).float()
        s["w_scales"] = w.abs().amax(1) / 127
        s["w"] = torch.round(w / s["w_scales"][:, None]).clamp(-127, 127).to(torch.int8)
        a = torch.arange(8192, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (
            -2.0 * torch.arange(case["d_rope"] // 2, device=DEV, dtype=torch.float64) / case["d_rope"])
        s |= dict(cos=a.cos().float(), sin=a.sin().float(), x=_normal(g, T, K), gamma=1 + _normal(g, K, sigma=0.2),
                  positions=torch.randint(0, 8192, (T,), generator=g, device=DEV, dtype=torch.int32))
        return s
    B, Sq, Sk, H, hk, d_k, d_v = (case[n] for n in ("B", "Sq", "Sk", "heads", "kv_heads", "d_k", "d_v"))
    s |= dict(q=_normal(g, B, H, Sq, d_k), k=_normal(g, B, hk, Sk, d_k), v=_normal(g, B, hk, Sk, d_v), dout=None,
              slopes=None, scale=1 / math.sqrt(d_k))
    if case["backward"]:
        s["dout"] = _normal(g, B, Sq, H, d_v, sigma=1e-2)  # token-major, as an output projection's gradient comes
    if case["slopes"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device=DEV) / H)
    q, k, p = _lens(case)
    s |= dict(cu=_starts(q), len_q=_ints(q), len_k=_ints(k), prefix=_ints(p) if case["prefix"] else None)
    return s


# ------------------------------------------------------------------ plain forms
def _mx8(x):
    """MXFP8 codes and scale bytes of x along its last axis (OCP MX, blocks of 32)."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 9).clamp(-127, 127)
    e = torch.where(amax == 0, -127, e)
    codes = torch.ldexp(b, -e[..., None]).clamp(-448, 448).float().to(F8)
    return codes.flatten(-2), (e + 127).to(torch.uint8).view(E8)


def _int8(y):
    """Codes of each row of y, as numbers, and its scale."""
    scale = y.abs().amax(-1) / 127
    return torch.round(y / torch.where(scale == 0, 1.0, scale)[..., None]).clamp(-127, 127), scale


def _int8_values(codes, scale):
    return codes * scale.to(BF16)[:, None]


def _norm_plain(s):
    c = s["case"]
    h = s["x"].float()
    if s["res"] is not None:
        h = (h + s["res"].float()).to(s["res"].dtype).float()
    rstd = torch.rsqrt(h.square().mean(-1) + 1e-6)
    xhat, gamma = h * rstd[:, None], s["gamma"].float()
    y = xhat * gamma
    out = {"rstd": rstd}
    if s["res"] is not None:
        out["h"] = h.to(s["res"].dtype)
    if c["keep"]:
        out["y"] = y.to(BF16)
    if c["quant"] == "mxfp8":
        out["codes"], out["scales"] = _mx8(y)
    if c["quant"] == "int8":
        codes, scale = _int8(y)
        out |= {"codes": _int8_values(codes.to(BF16), scale), "scales": scale}
    if c["backward"]:
        dy = s["dy"].float()
        g = dy * gamma
        dx = (g - xhat * (g * xhat).mean(-1, keepdim=True)) * rstd[:, None]
        dx = dx if s["dh"] is None else dx + s["dh"].float()
        out |= {"dx": dx.to(BF16), "dgamma": (dy * xhat).sum(0)}
        if c["residual"] == "fp32":
            out["dres"] = dx
    return out


def _rotate(x, cos, sin):
    """Pairs (2i, 2i + 1) of the last axis turned by the angles of cos, sin."""
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _project_plain(s):
    c = s["case"]
    x = s["x"].float()
    codes, scale = _int8(x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s["gamma"].float())
    # whole sums of products of 8-bit codes pass 2^24, where 32-bit floats begin to lose them
    q = torch.matmul(codes.double(), s["w"].double().t()).float()
    q = (q * scale[:, None] * s["w_scales"]).view(c["T"], c["heads"], -1)
    pos, dn = s["positions"].long(), c["d_nope"]
    q = torch.cat([q[..., :dn], _rotate(q[..., dn:], s["cos"][pos][:, None], s["sin"][pos][:, None])], -1)
    q = q.transpose(0, 1).contiguous()[None]  # [1, H, T, D]
    if c["out"] == "bf16":
        return {"out": q.to(BF16)}
    codes, scales = _mx8(q)
    return {"codes": codes, "scales": scales}


def _sees(s):
    """[B, Sq, Sk]: which keys a query sees, and how far behind the query's own place they lie."""
    c = s["case"]
    i, j = torch.arange(c["Sq"], device=DEV), torch.arange(c["Sk"], device=DEV)
    if c["packed"]:
        cu = s["cu"].long()
        doc = (i[:, None] >= cu[None, 1:]).sum(1)
        inside = doc < cu.numel() - 1
        doc = doc.clamp(max=cu.numel() - 2)
        at, start = i[None], cu[doc][None]
        prefix = s["prefix"].long()[doc][None, :, None] if s["prefix"] is not None else 0
        local = j[None, None, :] - start[..., None]
        sees = (doc[:, None] == doc[None, :]) & inside[:, None] & inside[None, :]
        sees = sees[None]
    else:
        at = i[None] + (s["len_k"] - s["len_q"]).long()[:, None]
        local = j[None, None, :]
        prefix = s["prefix"].long()[:, None, None] if s["prefix"] is not None else 0
        sees = (i[None, :, None] < s["len_q"][:, None, None]) & (local < s["len_k"][:, None, None])
    far = at[..., None] - j[None, None, :]
    if c["causal"]:
        sees = sees & ((far >= 0) | (local < prefix))
    if c["window"]:  # how far back a row sees; a prefix in front of that is out of sight too
        sees = sees & (far < c["window"])
    return sees, far


def _attend_plain(s):
    c = s["case"]
    sees, far = _sees(s)
    shared = torch.arange(c["heads"], device=DEV) * c["kv_heads"] // c["heads"]
    q, k, v = s["q"].float(), s["k"][:, shared].float(), s["v"][:, shared].float()
    t = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(s["scale"])
    if c["cap"]:
        t = torch.tanh_(t.div_(c["cap"]))
    sc = t * c["cap"] if c["cap"] else t
    if s["slopes"] is not None:
        sc = sc - s["slopes"][None, :, None, None] * far.abs().float()[:, None]
    sc = torch.where(sees[:, None], sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(sc.sub_(m))
    l = p.sum(-1, keepdim=True)
    p.div_(torch.where(l == 0, 1.0, l))
    out = torch.matmul(p, v)
    res = {"out": out.transpose(1, 2), "lse": (m + torch.log(l))[..., 0]}
    if c["backward"]:
        do = s["dout"].transpose(1, 2).float().contiguous()
        dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
        ds = torch.matmul(do, v.transpose(2, 3).contiguous())
        ds.sub_((do * out).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
        if c["cap"]:
            ds.mul_(1 - t.square_())
        dq = torch.matmul(ds, k)
        dk = torch.matmul(ds.transpose(2, 3).contiguous(), q)
        # heads that share a key head add their gradients
        dk, dv = (x.unflatten(1, (c["kv_heads"], -1)).sum(2) for x in (dk, dv))
        res |= {"dq": dq.transpose(1, 2), "dk": dk, "dv": dv}
    return {n: x if n == "lse" else x.to(BF16) for n, x in res.items()}


# ------------------------------------------------------------------ the library's calls
def _ws(s, size):
    """The workspace that the caller keeps, grown where a call asks for more."""
    if "ws" not in s or s["ws"].numel() < size:
        s["ws"] = torch.empty(max(1, size), dtype=torch.uint8, device=DEV)
    return s["ws"]


def _norm_own(s):
    import mla_up_projection_amd as m
    c = s["case"]
    x, res, T, K = s["x"], s["res"], c["T"], c["K"]
    rstd = torch.empty(T, dtype=torch.float32, device=DEV)
    h = None if res is None else torch.empty_like(res)
    y = torch.empty(T, K, dtype=BF16, device=DEV) if c["keep"] else None
    codes = scales = None
    if c["quant"] == "mxfp8":
        codes = torch.empty(T, K, dtype=torch.uint8, device=DEV)
        scales = torch.empty(T, K // 32, dtype=torch.uint8, device=DEV)
    if c["quant"] == "int8":
        codes = torch.empty(T, K, dtype=torch.int8, device=DEV)
        scales = torch.empty(T, dtype=torch.float32, device=DEV)
    m.mla_rmsnorm_fwd(x, s["gamma"], eps=1e-6, res=res, h=h, y=y, codes=codes, scales=scales, rstd=rstd)
    out = {"rstd": rstd} | ({} if h is None else {"h": h}) | ({} if y is None else {"y": y})
    if c["quant"] == "mxfp8":
        out |= {"codes": codes.view(F8), "scales": scales.view(E8)}
    if c["quant"] == "int8":
        out |= {"codes": _int8_values(codes, scales), "scales": scales}
    if c["backward"]:
        dx = torch.empty(T, K, dtype=BF16, device=DEV)
        dres = torch.empty(T, K, dtype=torch.float32, device=DEV) if c["residual"] == "fp32" else None
        dgamma = torch.empty(K, dtype=torch.float32, device=DEV)
        ws = _ws(s, m.mla_rmsnorm_bwd_workspace_size(T, K))
        m.mla_rmsnorm_bwd(s["dy"], x if h is None else h, rstd, s["gamma"], dh=s["dh"], dx=dx, dres=dres,
                          dgamma=dgamma, workspace=ws)
        out |= {"dx": dx, "dgamma": dgamma} | ({} if dres is None else {"dres": dres})
    return out


def _project_own(s):
    import mla_up_projection_amd as m
    c = s["case"]
    T, K, H, D = c["T"], c["K"], c["heads"], c["d_nope"] + c["d_rope"]
    codes = torch.empty(T, K, dtype=torch.int8, device=DEV)
    scales = torch.empty(T, dtype=torch.float32, device=DEV)
    m.mla_rmsnorm_fwd(s["x"], s["gamma"], eps=1e-6, codes=codes, scales=scales)
    kw = dict(H=H, d_nope=c["d_nope"], d_rope=c["d_rope"], cos=s["cos"], sin=s["sin"], positions=s["positions"])
    if c["out"] == "bf16":
        out = torch.empty(1, H, T, D, dtype=BF16, device=DEV)
        m.mla_qup_fwd_i8(codes, scales, s["w"], s["w_scales"], out, **kw)
        return {"out": out}
    out = torch.empty(1, H, T, D, dtype=torch.uint8, device=DEV)
    sc = torch.empty(1, H, T, D // 32, dtype=torch.uint8, device=DEV)
    m.mla_qup_fwd_i8(codes, scales, s["w"], s["w_scales"], out, out_scales=sc, **kw)
    return {"codes": out.view(F8), "scales": sc.view(E8)}


def _attend_own(s):
    import mla_up_projection_amd as m
    c = s["case"]
    B, Sq, Sk, H = c["B"], c["Sq"], c["Sk"], c["heads"]
    kw = dict(scale=s["scale"], cap=c["cap"], slopes=s["slopes"])
    if c["packed"] or c["causal"] and Sq > 1 or c["ragged"] or c["window"] or c["prefix"]:
        spans = torch.empty(B, Sq, 2, dtype=torch.int32, device=DEV)
        at = torch.empty(B, Sq, dtype=torch.int32, device=DEV) if c["slopes"] else None
        which = dict(cu_q=s["cu"], cu_k=s["cu"]) if c["packed"] else dict(len_q=s["len_q"], len_k=s["len_k"])
        m.mla_attn_spans(spans, at, Sk=Sk, prefix=s["prefix"], causal=c["causal"], window=c["window"], **which)
        kw |= dict(spans=spans, at=at)
    out = torch.empty(B, Sq, H, c["d_v"], dtype=BF16, device=DEV)
    lse = torch.empty(B, H, Sq, dtype=torch.float32, device=DEV)
    args = (s["q"], s["k"], s["v"], out.transpose(1, 2))
    m.mla_attn_fwd(*args, lse=lse, workspace=_ws(s, m.mla_attn_fwd_workspace_size(*args, **kw)), **kw)
    r = {"out": out, "lse": lse}
    if c["backward"]:
        dq = torch.empty(B, Sq, H, c["d_k"], dtype=BF16, device=DEV)
        dk, dv = torch.empty_like(s["k"]), torch.empty_like(s["v"])
        args = (s["dout"].transpose(1, 2), *args, lse, dq.transpose(1, 2), dk, dv)
        m.mla_attn_bwd(*args, workspace=_ws(s, m.mla_attn_bwd_workspace_size(*args, **kw)), **kw)
        r |= {"dq": dq, "dk": dk, "dv": dv}
    return r


def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm": _norm_own, "project": _project_own, "attend": _attend_own}[op](s)
    return {"norm": _norm_plain, "project": _project_plain, "attend": _attend_plain}[op](s)


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(case):
    """Visible (query, key) pairs of a head."""
    total = 0
    for n, k, p in zip(*_lens(case)):
        for i in range(n):
            at = i + k - n
            lo = max(0, at - case["window"] + 1) if case["window"] else 0
            hi = max(at + 1, p) if case["causal"] else k
            total += max(0, min(hi, k) - lo)
    return total


def work(case):
    if case["op"] == "norm":
        n = case["T"] * case["K"]
        r = {"none": 0, "bf16": 2, "fp32": 4}[case["residual"]]
        b = 2 + 2 * r + 2 * case["keep"] + {"none": 0, "mxfp8": 33 / 32, "int8": 1}[case["quant"]]
        if case["backward"]:
            b += 2 + (r or 2) + r + 2 + (4 if r == 4 else 0)
        return {"bytes": n * b + 4 * case["T"] + 2 * case["K"], "flops": 4 * n}
    if case["op"] == "project":
        T, K, N = case["T"], case["K"], case["heads"] * (case["d_nope"] + case["d_rope"])
        return {"bytes": N * K + 2 * T * K + T * N * (2 if case["out"] == "bf16" else 33 / 32), "flops": 2 * T * N * K}
    B, Sq, Sk, H, hk, d_k, d_v = (case[n] for n in ("B", "Sq", "Sk", "heads", "kv_heads", "d_k", "d_v"))
    b = 2 * B * (H * Sq * (d_k + d_v) + hk * Sk * (d_k + d_v)) + 4 * B * H * Sq
    f = 2 * (d_k + d_v)
    if case["backward"]:
        b, f = b * 2 + 2 * B * H * Sq * d_v, f + 2 * (3 * d_k + 2 * d_v)
    return {"bytes": b, "flops": f * H * max(1, _pairs(case))}


# ------------------------------------------------------------------ the definition in 64 bits
def _mx8_exact(y):
    """What MXFP8 makes of y, in 64 bits: elements as E4M3 values next to their block's scale."""
    b = y.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    scale = 2.0 ** (torch.floor(torch.log2(amax.clamp(min=2.0 ** -119))) - 8)
    m = b / scale
    step = 2.0 ** (torch.floor(torch.log2(m.abs().clamp(min=2.0 ** -6))) - 3)
    return {"codes": (torch.round(m / step) * step).clamp(-448, 448).flatten(-2), "scales": scale[..., 0]}


def exact(case, seed):
    s, c = prepare(case, seed), case
    d = torch.float64
    if c["op"] == "norm":
        h = s["x"].to(d)
        if s["res"] is not None:
            h = h + s["res"].to(d)
            h = h.to(s["res"].dtype).to(d)  # the sum is held in the residual's type
        gamma, K = s["gamma"].to(d), c["K"]
        r = 1 / torch.sqrt((h * h).sum(1) / K + 1e-6)
        y = torch.einsum("tk,t,k->tk", h, r, gamma)
        out = {"rstd": r, "h": None if s["res"] is None else h, "y": y if c["keep"] else None}
        if c["quant"] == "mxfp8":
            out |= _mx8_exact(y)
        if c["quant"] == "int8":
            a = y.abs().max(1)[0] / 127
            out |= {"codes": torch.round(y / a[:, None]) * a[:, None], "scales": a}
        if c["backward"]:
            dy = s["dy"].to(d)
            inner = torch.einsum("tk,tk,k->t", dy, h, gamma) * r ** 3 / K
            dx = dy * gamma * r[:, None] - h * inner[:, None]
            dx = dx if s["dh"] is None else dx + s["dh"].to(d)
            out |= {"dx": dx, "dgamma": torch.einsum("tk,tk,t->k", dy, h, r),
                    "dres": dx if c["residual"] == "fp32" else None}
        return {k: v for k, v in out.items() if v is not None}
    if c["op"] == "project":
        x = s["x"].to(d)
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / c["K"] + 1e-6) * s["gamma"].to(d)
        a = y.abs().max(1, keepdim=True)[0] / 127
        w = s["w"].to(d) * s["w_scales"].to(d)[:, None]
        q = ((torch.round(y / a) * a) @ w.t()).view(c["T"], c["heads"], -1)
        pos = s["positions"].long()
        turn = torch.complex(s["cos"].to(d)[pos], s["sin"].to(d)[pos])[:, None]
        tail = torch.view_as_complex(q[..., c["d_nope"]:].unflatten(-1, (-1, 2)).contiguous()) * turn
        q = torch.cat([q[..., : c["d_nope"]], torch.view_as_real(tail).flatten(-2)], -1).permute(1, 0, 2)[None]
        return {"out": q} if c["out"] == "bf16" else _mx8_exact(q)
    B, Sq, Sk, H, hk = (c[n] for n in ("B", "Sq", "Sk", "heads", "kv_heads"))
    if B * H * Sq * Sk * (5 if c["backward"] else 2) > 12e9:
        return None
    out = {"out": torch.zeros(B, Sq, H, c["d_v"], dtype=d, device=DEV),
           "lse": torch.full((B, H, Sq), -math.inf, dtype=d, device=DEV)}
    if c["backward"]:
        out |= {"dq": torch.zeros(B, Sq, H, c["d_k"], dtype=d, device=DEV),
                "dk": torch.zeros(s["k"].shape, dtype=d, device=DEV), "dv": torch.zeros(s["v"].shape, dtype=d, device=DEV)}
    q0 = k0 = 0
    for n, (lq, lk, pre) in enumerate(zip(*_lens(c))):  # one sequence or document at a time
        b = 0 if c["packed"] else n
        rows, cols = slice(q0, q0 + lq), slice(k0, k0 + lk)
        i, j = torch.arange(lq, device=DEV)[:, None] + lk - lq, torch.arange(lk, device=DEV)[None]
        ok = (j <= i) | (j < pre) if c["causal"] else torch.ones(lq, lk, dtype=torch.bool, device=DEV)
        if c["window"]:
            ok = ok & (j > i - c["window"])
        some = ok.any(1)
        for h in range(H if lq and lk else 0):
            q, k, v = (s[t][b, g, r].to(d) for t, g, r in (("q", h, rows), ("k", h * hk // H, cols), ("v", h * hk // H, cols)))
            z = q @ k.t() * s["scale"]
            th = torch.tanh(z / c["cap"]) if c["cap"] else None
            z = th * c["cap"] if c["cap"] else z
            if s["slopes"] is not None:
                z = z - s["slopes"][h].to(d) * (i - j).abs()
            z = z.masked_fill(~ok, -math.inf)
            lse = torch.logsumexp(z, 1)
            p = torch.exp(z - torch.where(some, lse, 0.0)[:, None])
            out["out"][b, rows, h] = p @ v
            out["lse"][b, h, rows] = lse
            if c["backward"]:
                do = s["dout"][b, rows, h].to(d)
                dp = do @ v.t()
                ds = p * (dp - (p * dp).sum(1, keepdim=True)) * s["scale"]
                ds = ds * (1 - th * th) if c["cap"] else ds
                out["dq"][b, rows, h] = ds @ k
                out["dk"][b, h * hk // H, cols] += ds.t() @ q
                out["dv"][b, h * hk // H, cols] += p.t() @ do
        if c["packed"]:
            q0, k0 = q0 + lq, k0 + lk
    return out
