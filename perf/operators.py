"""Cases and plain forms of the decode-side operators: the up-projection with
4-bit weights, key rows into a paged cache, attention of drafted tokens over
that cache, and the bookkeeping of its pages.

`run` computes an operator in elementary torch operations in 32 bits, or, with
`own` set, through the library's entry points. Shapes are DeepSeek-V3's MLA
(q_lora_rank 1536, 128 heads of 128 + 64, latent rows of 512 + 64) and its
head-parallel shards.
"""
import math

import torch

own = False

DEV = "cuda"
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token of one short conversation: nothing but latency
        dict(name="attend one token", op="attend", cache="bf16", nseq=1, max_q=1, heads=128, kv_heads=1,
             d_k=576, d_v=512, page=64, len_lo=517, len_hi=517, tree=False),
        # a 4-way head shard verifying small trees, short pages, one fresh sequence
        dict(name="attend trees shard", op="attend", cache="bf16", nseq=8, max_q=13, heads=32, kv_heads=1,
             d_k=576, d_v=512, page=16, len_lo=0, len_hi=2111, tree=True),
        # a full batch of trees on all heads: the matrix units bound it
        dict(name="attend trees batch", op="attend", cache="bf16", nseq=32, max_q=8, heads=128, kv_heads=1,
             d_k=576, d_v=512, page=64, len_lo=2900, len_hi=6000, tree=True),
        # long documents in an 8-bit cache, two tokens at a time
        dict(name="attend long mxfp8", op="attend", cache="mxfp8", nseq=16, max_q=2, heads=128, kv_heads=1,
             d_k=576, d_v=512, page=64, len_lo=20000, len_hi=32000, tree=False),
        # keys and values kept per head, as mla_kv_rope makes them; pages of 48 end inside a tile
        dict(name="attend per head", op="attend", cache="bf16", nseq=4, max_q=7, heads=128, kv_heads=128,
             d_k=192, d_v=128, page=48, len_lo=300, len_hi=1500, tree=True),
        # drafted tokens of a few sequences into latent pages
        dict(name="append drafts", op="append", cache="bf16", nseq=4, max_q=6, heads=1, d_nope=512, d_rope=64,
             d_v=0, page=64, len_lo=100, len_hi=4000),
        # a prompt's chunk into per-head 8-bit pages
        dict(name="append prompt mxfp8", op="append", cache="mxfp8", nseq=3, max_q=700, heads=128, d_nope=128,
             d_rope=64, d_v=128, page=64, len_lo=0, len_hi=500),
        # one conversation continued four ways: fork, room for six drafts, accept, drop
        dict(name="branch one", op="branch", parents=1, children=4, len_lo=1000, len_hi=1000, new=6, page=64,
             pages=512),
        # the same over a serving batch
        dict(name="branch batch", op="branch", parents=64, children=4, len_lo=500, len_hi=6000, new=9, page=64,
             pages=8192),
        # sequences leave between others; the pages that stay are packed to the front
        dict(name="pack pages", op="pack", base=16, others=48, new=1500, page=64, pages=8192),
        # one token through the up-projection
        dict(name="project one token", op="project", T=1, K=1536, heads=128, d_nope=128, d_rope=64, out="bf16"),
        # the drafts of a small batch, quantized for an 8-bit attention
        dict(name="project drafts mxfp8", op="project", T=52, K=1536, heads=128, d_nope=128, d_rope=64,
             out="mxfp8"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "branch", "pack", "project", "project"])
    page = rng.choice([16, 32, 48, 64, 100, 128])
    if op == "attend":
        d_k, d_v, heads, kv_heads = rng.choice(
            [(576, 512, h, 1) for h in (128, 64, 32, 8, 20)] +
            [(192, 128, 128, 128), (192, 128, 12, 12), (128, 128, 32, 8), (128, 128, 40, 2), (64, 64, 14, 7),
             (96, 64, 24, 1)])
        nseq, max_q = _log(rng, 1, 40), _log(rng, 1, 64)
        most = min(150e6 / (nseq * max_q * heads), 400e6 / (nseq * kv_heads * (d_k + d_v)), 32000)
        hi = _log(rng, 1, max(2, int(most)))
        return dict(op=op, cache=rng.choice(["bf16", "mxfp8"]), nseq=nseq, max_q=max_q, heads=heads,
                    kv_heads=kv_heads, d_k=d_k, d_v=d_v, page=page, len_lo=rng.randint(0, hi), len_hi=hi,
                    tree=rng.random() < 0.6)
    if op == "append":
        heads, dn, dr, dv = rng.choice([(1, 512, 64, 0), (1, 512, 64, 0), (128, 128, 64, 128), (12, 128, 64, 128),
                                        (8, 64, 64, 64)])
        nseq = _log(rng, 1, 40)
        return dict(op=op, cache=rng.choice(["bf16", "mxfp8"]), nseq=nseq,
                    max_q=_log(rng, 1, 2000 if heads == 1 else max(2, 2000 // nseq)), heads=heads, d_nope=dn,
                    d_rope=dr, d_v=dv, page=page, len_lo=0, len_hi=_log(rng, 1, 300))
    if op == "branch":
        parents, children, hi = _log(rng, 1, 64), rng.randint(1, 4), _log(rng, 1, 6000)
        return dict(op=op, parents=parents, children=children, len_lo=rng.randint(0, hi), len_hi=hi,
                    new=rng.randint(1, 40), page=page,
                    pages=parents * (-(-hi // page) + children * (2 + 40 // page)) + rng.randint(0, 500))
    if op == "pack":
        base, others, new = rng.randint(0, 16), _log(rng, 1, 48), _log(rng, 1, 1500)
        return dict(op=op, base=base, others=others, new=new, page=page,
                    pages=(base + 2 * others) * -(-new // page) + rng.randint(0, 500))
    return dict(op=op, T=_log(rng, 1, 64), K=32 * _log(rng, 2, 64), heads=rng.choice([1, 5, 8, 32, 128]),
                d_nope=rng.choice([128, 128, 64, 0]), d_rope=64, out=rng.choice(["bf16", "mxfp8"]))


# ------------------------------------------------------------------ inputs
def _rows(g, n, lo, hi):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _normal(g, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * sigma).to(torch.bfloat16)


def _mx8(x):
    """MXFP8 codes and scale bytes of x along its last axis (OCP MX, blocks of 32)."""
    b = x.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax)[1] - 9).clamp(-127, 127)
    e = torch.where(amax == 0, -127, e)
    codes = torch.ldexp(b, -e[..., None]).clamp(-448, 448).to(F8)
    return codes.flatten(-2).view(torch.uint8), (e + 127).to(torch.uint8)


def _mx8_values(codes, scales):
    v = codes.view(F8).float().unflatten(-1, (-1, 32))
    return torch.ldexp(v, scales.to(torch.int32)[..., None] - 127).flatten(-2)


def _mx4(w):
    """MXFP4 (E2M1) codes, two to a byte with the even column low, and scale bytes."""
    b = w.float().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = torch.where(amax == 0, -127, (torch.frexp(amax)[1] - 3).clamp(-127, 127))
    m = torch.ldexp(b, -e[..., None]).clamp(-6, 6)
    a = m.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.round(a / step) * step  # half to even: the even multiple is the even code
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=w.device)
    code = torch.bucketize(q, grid) | (torch.signbit(m).to(torch.int64) << 3)
    code = code.flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _table(rows, d_rope, base=10000.0):
    """cos, sin [rows, d_rope / 2], from angles in 64 bits."""
    a = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * base ** (
        -2.0 * torch.arange(d_rope // 2, device=DEV, dtype=torch.float64) / d_rope)
    return a.cos().float(), a.sin().float()


def _pool(g, shapes, page, num_pages, held, extra_seqs=0, fill=True):
    """Buffers of num_pages pages and a table whose rows hold `held` pages each, in random order."""
    n = held.numel()
    order = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    start = torch.cumsum(held, 0) - held
    most = max(1, -(-num_pages // max(1, n)), int(held.max()) + 8) if n else 8
    k = torch.arange(most, device=DEV)
    at = (start[:, None] + k).clamp(max=num_pages - 1)
    table = torch.where(k < held[:, None], order[at], -1)
    refs = torch.zeros(num_pages, dtype=torch.int32, device=DEV)
    refs[order[: int(held.sum())].long()] = 1
    pad = torch.full((extra_seqs, most), -1, dtype=torch.int32, device=DEV)
    bufs = [_normal(g, num_pages, page, *s) if fill else torch.zeros(num_pages, page, *s, dtype=torch.bfloat16,
                                                                    device=DEV) for s in shapes]
    zeros = torch.zeros(extra_seqs, dtype=torch.int32, device=DEV)
    return dict(bufs=bufs, refs=refs, table=torch.cat([table, pad]).to(torch.int32).contiguous(),
                held=torch.cat([held.to(torch.int32), zeros]), page=page)


def _mx8_bufs(bufs):
    return [t for b in bufs for t in _mx8(b)]


def _lengths(case):
    """Lengths and drafted tokens of the sequences: they follow the case alone, so that outputs of
    different seeds have one shape."""
    g = torch.Generator(device=DEV)
    g.manual_seed(case["nseq"] * 1000003 + case["max_q"] * 101 + case["len_hi"])
    nseq, max_q = case["nseq"], case["max_q"]
    lens = _rows(g, nseq, case["len_lo"], case["len_hi"])
    n = _rows(g, nseq, 1, max_q)
    n[torch.randint(nseq, (1,), generator=g, device=DEV)] = max_q
    cu = torch.zeros(nseq + 1, dtype=torch.int32, device=DEV)
    cu[1:] = torch.cumsum(n, 0)
    return lens, n, cu


def _tree_mask(g, n, max_q):
    """Bit masks [T, words]: each drafted token sees itself and its ancestors in a random tree."""
    nseq, i = n.numel(), torch.arange(max_q, device=DEV)
    parent = (torch.rand(nseq, max_q, generator=g, device=DEV) * (i + 1)).long() - 1  # -1: a root
    see = torch.zeros(nseq, max_q, max_q + 1, dtype=torch.bool, device=DEV)
    for d in range(max_q):
        p = parent[:, d]
        up = torch.gather(see, 1, p.clamp(min=0)[:, None, None].expand(-1, 1, max_q + 1))[:, 0]
        see[:, d] = up & (p >= 0)[:, None]
        see[:, d, d] = True
    see = see[:, :, :max_q]
    words = -(-max_q // 32)
    bits = torch.nn.functional.pad(see, (0, 32 * words - max_q)).unflatten(-1, (words, 32)).long()
    mask = (bits << torch.arange(32, device=DEV)).sum(-1)
    mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32)
    return mask[i < n[:, None]].contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "attend":
        nseq, hk, dk, dv = case["nseq"], case["kv_heads"], case["d_k"], case["d_v"]
        lens, n, cu = _lengths(case)
        held = -(-(lens + n) // case["page"])
        shared = hk == 1
        s |= _pool(g, [(hk, dk)] if shared else [(hk, dk), (hk, dv)], case["page"], int(held.sum()) + 3, held)
        if case["cache"] == "mxfp8":
            s["bufs"] = _mx8_bufs(s["bufs"])
        s["lens"] = lens
        s["seqs"] = torch.randperm(nseq, generator=g, device=DEV).to(torch.int32)
        n = n[s["seqs"].long()]  # rows of q follow the order of seqs
        cu = torch.cat([cu[:1], torch.cumsum(n, 0)]).to(torch.int32)
        T = int(cu[-1])
        s |= dict(cu_q=cu, T=T, q=_normal(g, T, case["heads"], dk), mask=None, scale=1 / math.sqrt(192.0),
                  max_len=int((lens[s["seqs"].long()] + n).max()))
        if case["tree"]:
            s["mask"] = _tree_mask(g, n, case["max_q"])
            s["mask"][T - 1] = 0  # a padding token: it sees no draft
        return s
    if case["op"] == "append":
        nseq, H, dn, dr, dv = (case[k] for k in ("nseq", "heads", "d_nope", "d_rope", "d_v"))
        lens, n, cu = _lengths(case)
        held = -(-(lens + n) // case["page"])
        shapes = [(H, dn + dr)] + ([(H, dv)] if dv else [])
        s |= _pool(g, shapes, case["page"], int(held.sum()) + 3, held, fill=False)
        if case["cache"] == "mxfp8":
            s["bufs"] = _mx8_bufs(s["bufs"])
        s["cos"], s["sin"] = _table(case["len_hi"] + case["max_q"], dr)
        T = int(cu[-1])
        s |= dict(lens=lens, seqs=torch.arange(nseq, dtype=torch.int32, device=DEV), cu_q=cu, T=T,
                  kv=_normal(g, T, H, dn + dv), pe=_normal(g, T, dr))
        return s
    if case["op"] == "branch":
        np_, nc, page = case["parents"], case["children"], case["page"]
        lens = _rows(g, np_, case["len_lo"], case["len_hi"])
        held = -(-lens // page)
        s |= _pool(g, [(1, 576)], page, case["pages"], held, np_ * nc)
        room = torch.full((np_ * (nc + 1), 2 + (case["new"] + page - 1) // page), -1, dtype=torch.int32, device=DEV)
        s["table"] = torch.cat([s["table"], room], 1).contiguous()
        s["lens"] = torch.cat([lens, torch.zeros(np_ * nc, dtype=torch.int32, device=DEV)])
        s["src"] = torch.arange(np_, dtype=torch.int32, device=DEV).repeat_interleave(nc)
        s["dst"] = torch.arange(np_, np_ * (nc + 1), dtype=torch.int32, device=DEV)
        s["new"] = torch.full_like(s["dst"], case["new"])
        s["n_acc"] = _rows(g, np_ * nc, 0, case["new"])
        pick = torch.rand(np_ * nc, case["new"], generator=g, device=DEV).argsort(1)
        pick = torch.where(torch.arange(case["new"], device=DEV) < s["n_acc"][:, None], pick, case["new"])
        s["path"] = pick.sort(1)[0].to(torch.int32).contiguous()  # increasing; n_acc of them count
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        return s
    if case["op"] == "pack":
        base, others, page = case["base"], case["others"], case["page"]
        lens = _rows(g, base, 1, case["new"])
        held = -(-lens // page)
        s |= _pool(g, [(1, 576)], page, case["pages"], held, 2 * others)
        need = max(s["table"].shape[1], -(-case["new"] // page) + 1)
        s["table"] = torch.nn.functional.pad(s["table"], (0, need - s["table"].shape[1]), value=-1).contiguous()
        zero = torch.zeros(2 * others, dtype=torch.int32, device=DEV)
        s["lens"] = torch.cat([lens, zero])
        s["both"] = torch.arange(base, base + 2 * others, dtype=torch.int32, device=DEV)
        s["go"], s["stay"] = s["both"][0::2].contiguous(), s["both"][1::2].contiguous()
        s["new"] = _rows(g, 2 * others, 1, case["new"])
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["used"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        return s
    T, K, H, D = case["T"], case["K"], case["heads"], case["d_nope"] + case["d_rope"]
    s["codes"], s["scales"] = _mx4(_normal(g, H * D, K, sigma=0.02))
    s["cos"], s["sin"] = _table(8192, case["d_rope"])
    s |= dict(x=_normal(g, T, K), positions=_rows(g, T, 0, 8191))
    return s


# ------------------------------------------------------------------ plain forms
def _seq_of(cu, T):
    t = torch.arange(T, device=DEV)
    j = (t[:, None] >= cu[None, 1:]).sum(1)
    return j, t - cu[j]


def _cache_rows(s, rows):
    """Key and value rows in 32 bits: [..., kv heads, d]."""
    c = s["case"]
    flat = [b.flatten(0, 1) for b in s["bufs"]]
    if c["cache"] == "mxfp8":
        vals = [_mx8_values(flat[k][rows], flat[k + 1][rows]) for k in range(0, len(flat), 2)]
    else:
        vals = [b[rows].float() for b in flat]
    return (vals[0], vals[1]) if len(vals) == 2 else (vals[0], vals[0][..., : c["d_v"]])


def _attend_plain(s):
    c, cu, T = s["case"], s["cu_q"].long(), s["T"]
    Q, L, H, hk = c["max_q"], s["max_len"], c["heads"], c["kv_heads"]
    seqs, lens, table = s["seqs"].long(), s["lens"].long(), s["table"].long()
    n, own_len = cu[1:] - cu[:-1], lens[seqs]
    pos = torch.arange(L, device=DEV)
    inside = pos < (own_len + n)[:, None]
    pages = table[seqs][:, pos // c["page"]]
    k, v = _cache_rows(s, torch.where(inside, pages * c["page"] + pos % c["page"], 0))
    i = torch.arange(Q, device=DEV)
    t = (cu[:-1, None] + i).clamp(max=T - 1)
    nseq = seqs.numel()
    q = s["q"].float()[t].view(nseq, Q, hk, H // hk, -1).permute(0, 2, 1, 3, 4).reshape(nseq, hk, Q * (H // hk), -1)
    sc = torch.matmul(q, k.permute(0, 2, 3, 1).contiguous()) * s["scale"]
    draft = pos - own_len[:, None]  # [nseq, L]
    if s["mask"] is None:
        sees = draft[:, None, :] <= i[:, None]
    else:
        d = draft.clamp(0, Q - 1)[:, None, :].expand(-1, Q, -1)
        word = torch.gather(s["mask"].long()[t], 2, d >> 5)
        sees = (draft < 0)[:, None, :] | (((word >> (d & 31)) & 1) > 0)
    sees = (sees & inside[:, None, :]).repeat_interleave(H // hk, 1)[:, None]
    sc = torch.where(sees, sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(sc - m0)
    l = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v.transpose(1, 2).contiguous()) / torch.where(l == 0, 1.0, l)
    lse = (m0 + torch.log(l))[..., 0]
    j, ii = _seq_of(cu, T)
    out = out.view(nseq, hk, Q, H // hk, -1).transpose(1, 2)[j, ii].reshape(T, H, -1)
    lse = lse.view(nseq, hk, Q, H // hk).transpose(1, 2)[j, ii].reshape(T, H)
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _rotate(x, cos, sin):
    """Pairs (2i, 2i + 1) of the last axis turned by the angles of cos, sin."""
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _append_plain(s):
    c, cu, T = s["case"], s["cu_q"].long(), s["T"]
    j, i = _seq_of(cu, T)
    seq = s["seqs"].long()[j]
    pos = s["lens"].long()[seq] + i
    rows = s["table"].long()[seq, pos // c["page"]] * c["page"] + pos % c["page"]
    kv = s["kv"].float()
    pe = _rotate(s["pe"].float(), s["cos"][pos], s["sin"][pos])
    key = torch.cat([kv[..., : c["d_nope"]], pe[:, None].expand(-1, c["heads"], -1)], -1)
    parts = [key] + ([kv[..., c["d_nope"]:]] if c["d_v"] else [])
    if c["cache"] == "mxfp8":
        parts = [t for p in parts for t in _mx8(p)]
    for b, p in zip(s["bufs"], parts):
        b.flatten(0, 1)[rows] = p.to(b.dtype)
    return _append_out(s)


def _append_out(s):
    if s["case"]["cache"] == "bf16":
        return {"bufs": s["bufs"]}
    return {"codes": [b.view(F8) for b in s["bufs"][0::2]], "scales": [b.view(E8) for b in s["bufs"][1::2]]}


def _free_plain(s, seqs):
    """The pages of seqs lose a reference; their rows of the table are cleared."""
    seqs = seqs.long()
    k = torch.arange(s["table"].shape[1], device=DEV)
    pages = s["table"][seqs][k < s["held"][seqs][:, None]].long()
    s["refs"].index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))
    s["table"][seqs] = -1
    s["held"][seqs] = 0
    s["lens"][seqs] = 0


def _fork_plain(s, src, dst):
    src, dst, page = src.long(), dst.long(), s["page"]
    k = torch.arange(s["table"].shape[1], device=DEV)
    n = (s["lens"][src] + page - 1) // page
    row = torch.where(k < n[:, None], s["table"][src], -1)
    shared = row[row >= 0].long()
    s["refs"].index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    s["table"][dst] = row
    s["held"][dst] = n
    s["lens"][dst] = s["lens"][src]


def _reserve_plain(s, seqs, new):
    seqs, page, n = seqs.long(), s["page"], seqs.numel()
    lens, held = s["lens"][seqs].long(), s["held"][seqs].long()
    last = s["table"][seqs, lens // page].long()  # the page that the next token falls into
    shared = (lens % page > 0) & (new > 0)
    last = torch.where(shared, last, -1 - torch.arange(n, device=DEV))
    before = torch.tril(last[:, None] == last[None, :], -1).sum(1)
    copy = shared & (s["refs"][last.clamp(min=0)] - before > 1)
    add = ((lens + new + page - 1) // page - held).clamp(min=0)
    need = add + copy
    start = torch.cumsum(need, 0) - need
    free = torch.nonzero(s["refs"] == 0)[:, 0]
    total = int(need.sum())
    s["status"].fill_(max(0, total - free.numel()))
    if total > free.numel():
        return
    owner = torch.repeat_interleave(torch.arange(n, device=DEV), need)
    at = torch.arange(total, device=DEV) - start[owner]  # the copied page first, then the added ones
    slot = torch.where(at < copy[owner], lens[owner] // page, held[owner] + at - copy[owner].long())
    free = free[:total]
    s["refs"].index_add_(0, last[copy], torch.full((int(copy.sum()),), -1, dtype=torch.int32, device=DEV))
    s["refs"][free] = 1
    s["table"][seqs[owner], slot] = free.to(torch.int32)
    s["held"][seqs] = (held + add).to(torch.int32)
    row = torch.arange(page, device=DEV)
    live = row < (lens[copy] % page)[:, None]
    source = (last[copy][:, None] * page + row)[live]
    target = (free[start[copy]][:, None] * page + row)[live]
    flat = s["bufs"][0].flatten(0, 1)
    flat[target] = flat[source]


def _accept_plain(s, seqs, path, n_acc):
    seqs, page = seqs.long(), s["page"]
    lens, table = s["lens"][seqs].long()[:, None], s["table"][seqs].long()
    a = torch.arange(path.shape[1], device=DEV)[None]
    live = a < n_acc[:, None]
    source, target = lens + torch.where(live, path.long(), 0), lens + torch.where(live, a, 0)
    row = lambda p: (torch.gather(table, 1, p // page) * page + p % page)[live]  # noqa: E731
    flat = s["bufs"][0].flatten(0, 1)
    flat[row(target)] = flat[row(source)]
    s["lens"][seqs] += n_acc


def _pack_plain(s):
    refs, n = s["refs"], s["refs"].numel()
    used = refs > 0
    count = int(used.sum())
    ids = torch.arange(n, device=DEV)
    source = ids[used & (ids >= count)]
    target = ids[~used & (ids < count)]
    to = ids.clone()
    to[source] = target
    s["bufs"][0][target] = s["bufs"][0][source]
    refs[target] = refs[source]
    refs[source] = 0
    s["table"].copy_(torch.where(s["table"] >= 0, to[s["table"].clamp(min=0).long()].to(torch.int32), -1))
    s["used"].fill_(count)


def _pages_out(s):
    return {k: s[k] for k in ("refs", "table", "held", "lens", "status")} | {
        "pages": s["bufs"][0].view(torch.int16)} | ({"used": s["used"]} if "used" in s else {})


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _project_plain(s):
    c = s["case"]
    H, dn = c["heads"], c["d_nope"]
    grid = torch.tensor(_E2M1, device=DEV)
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).flatten(-2)
    w = torch.ldexp(grid[codes.long()].unflatten(-1, (-1, 32)), s["scales"].to(torch.int32)[..., None] - 127)
    q = torch.matmul(s["x"].float(), w.flatten(-2).t()).view(c["T"], H, -1)
    pos = s["positions"].long()
    q = torch.cat([q[..., :dn], _rotate(q[..., dn:], s["cos"][pos][:, None], s["sin"][pos][:, None])], -1)
    q = q.transpose(0, 1).contiguous()[None]  # [1, H, T, D]
    if c["out"] == "bf16":
        return {"out": q.to(torch.bfloat16)}
    codes, scales = _mx8(q)
    return {"codes": codes.view(F8), "scales": scales.view(E8)}


# ------------------------------------------------------------------ the library's calls
def _pool_of(s):
    import mla_up_projection_amd as m
    if "pool" not in s:
        s["pool"] = m.PagePool(s["bufs"], s["refs"], s["table"], s["lens"], s["held"])
        s["ws"] = torch.empty(max(1, m.mla_pages_workspace_size(s["pool"])), dtype=torch.uint8, device=DEV)
    return m, s["pool"]


def _run_own(s):
    c = s["case"]
    op = c["op"]
    if op == "attend":
        m, pool = _pool_of(s)
        out = torch.empty(s["T"], c["heads"], c["d_v"], dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(s["T"], c["heads"], dtype=torch.float32, device=DEV)
        kw = dict(max_q=c["max_q"], max_len=s["max_len"], scale=s["scale"], lse=lse, mask=s["mask"])
        if "attend_ws" not in s:
            size = m.mla_tree_attention_workspace_size(s["q"], pool, out, s["seqs"], s["cu_q"], **kw)
            s["attend_ws"] = torch.empty(max(1, size), dtype=torch.uint8, device=DEV)
        m.mla_tree_attention(s["q"], pool, out, s["seqs"], s["cu_q"], workspace=s["attend_ws"], **kw)
        return {"out": out, "lse": lse}
    if op == "append":
        m, pool = _pool_of(s)
        m.mla_kv_rope_paged(s["kv"], s["pe"], pool, s["seqs"], s["cu_q"], H=c["heads"], d_nope=c["d_nope"],
                            d_rope=c["d_rope"], d_v=c["d_v"], cos=s["cos"], sin=s["sin"], max_q=c["max_q"])
        return _append_out(s)
    if op == "branch":
        m, pool = _pool_of(s)
        m.mla_pages_free(pool, s["dst"])
        m.mla_pages_fork(pool, s["src"], s["dst"])
        m.mla_pages_reserve(pool, s["dst"], s["new"], s["status"], workspace=s["ws"])
        m.mla_draft_accept(pool, s["dst"], s["path"], s["n_acc"])
        return _pages_out(s)
    if op == "pack":
        m, pool = _pool_of(s)
        m.mla_pages_free(pool, s["both"])
        m.mla_pages_reserve(pool, s["both"], s["new"], s["status"], workspace=s["ws"])
        m.mla_pages_free(pool, s["go"])
        m.mla_pages_compact(pool, s["used"], workspace=s["ws"])
        return _pages_out(s)
    import mla_up_projection_amd as m
    T, H, D = c["T"], c["heads"], c["d_nope"] + c["d_rope"]
    kw = dict(H=H, d_nope=c["d_nope"], d_rope=c["d_rope"], cos=s["cos"], sin=s["sin"], positions=s["positions"])
    if c["out"] == "bf16":
        out = torch.empty(1, H, T, D, dtype=torch.bfloat16, device=DEV)
        m.mla_qup_fwd_w4(s["x"], s["codes"], s["scales"], out, **kw)
        return {"out": out}
    out = torch.empty(1, H, T, D, dtype=torch.uint8, device=DEV)
    sc = torch.empty(1, H, T, D // 32, dtype=torch.uint8, device=DEV)
    m.mla_qup_fwd_w4(s["x"], s["codes"], s["scales"], out, out_scales=sc, **kw)
    return {"codes": out.view(F8), "scales": sc.view(E8)}


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "attend":
        return _attend_plain(s)
    if op == "append":
        return _append_plain(s)
    if op == "branch":
        _free_plain(s, s["dst"])
        _fork_plain(s, s["src"], s["dst"])
        _reserve_plain(s, s["dst"], s["new"])
        _accept_plain(s, s["dst"], s["path"], s["n_acc"])
        return _pages_out(s)
    if op == "pack":
        _free_plain(s, s["both"])
        _reserve_plain(s, s["both"], s["new"])
        _free_plain(s, s["go"])
        _pack_plain(s)
        return _pages_out(s)
    return _project_plain(s)


# ------------------------------------------------------------------ sizes of a pass
def work(case):
    op = case["op"]
    if op == "attend":
        mean_len, mean_q = (case["len_lo"] + case["len_hi"]) / 2, (1 + case["max_q"]) / 2
        rows = case["nseq"] * (mean_len + mean_q)
        width = case["d_k"] + (0 if case["kv_heads"] == 1 else case["d_v"])
        per = 33 / 32 if case["cache"] == "mxfp8" else 2
        q = case["nseq"] * mean_q * case["heads"]
        return {"bytes": rows * case["kv_heads"] * width * per + q * (2 * (case["d_k"] + case["d_v"]) + 4),
                "flops": 2 * q * (mean_len + mean_q / 2) * (case["d_k"] + case["d_v"])}
    if op == "append":
        T = case["nseq"] * (1 + case["max_q"]) / 2
        H, dn, dr, dv = (case[k] for k in ("heads", "d_nope", "d_rope", "d_v"))
        per = 33 / 32 if case["cache"] == "mxfp8" else 2
        return {"bytes": T * (2 * H * (dn + dv) + 2 * dr + 4 * dr + H * (dn + dr + dv) * per),
                "flops": T * 3 * dr}
    if op == "branch":
        n, page = case["parents"] * case["children"], case["page"]
        mean = (case["len_lo"] + case["len_hi"]) / 2
        moved = n * (page / 2 + case["new"] / 2) * 1152 * 2  # rows copied on write and rows accepted
        return {"bytes": moved + 16 * n * -(-mean // page) + 4 * case["pages"], "flops": 0}
    if op == "pack":
        mean = case["new"] / 2 / case["page"] + 0.5
        moved = case["others"] * mean / 2 * case["page"] * 1152 * 2  # about half of those that stay
        return {"bytes": moved + 8 * case["pages"] + 24 * case["others"] * mean, "flops": 0}
    T, K, D = case["T"], case["K"], case["d_nope"] + case["d_rope"]
    N = case["heads"] * D
    return {"bytes": N * K * 17 / 32 + 2 * T * K + T * N * (2 if case["out"] == "bf16" else 33 / 32),
            "flops": 2 * T * N * K}


# ------------------------------------------------------------------ in 64 bits
def _values64(codes, scales):
    v = codes.view(F8).double()
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _quantize64(x):
    """The E4M3 values and the scales 2^e of x [.., d] in 64 bits."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1)
    e = (torch.floor(torch.log2(top.clamp(min=2.0 ** -140))) - 8).clamp(-127, 127)
    m = (b * torch.exp2(-e)[..., None]).clamp(-448, 448)
    ulp = torch.exp2((torch.floor(torch.log2(m.abs().clamp(min=2.0 ** -40)))).clamp(min=-6) - 3)
    return (torch.round(m / ulp) * ulp).flatten(-2), torch.exp2(e)


def _exact_attend(s):
    c = s["case"]
    outs, lses = [], []
    cu, seqs, lens = s["cu_q"].tolist(), s["seqs"].tolist(), s["lens"].tolist()
    group = c["heads"] // c["kv_heads"]
    for j, seq in enumerate(seqs):
        n, past = cu[j + 1] - cu[j], lens[seq]
        ids = s["table"][seq, : -(-(past + n) // c["page"])].long()
        got = [b[ids].flatten(0, 1)[: past + n] for b in s["bufs"]]
        if c["cache"] == "mxfp8":
            got = [_values64(got[k], got[k + 1]) for k in range(0, len(got), 2)]
        k = got[0].double().transpose(0, 1)
        v = got[1].double().transpose(0, 1) if len(got) > 1 else k[..., : c["d_v"]]
        keep = torch.ones(n, past + n, dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            keep[:, past:] = torch.tril(keep[:, past:])
        else:
            words = s["mask"][cu[j]: cu[j + 1]]
            bit = torch.arange(n, device=DEV)
            keep[:, past:] = ((words[:, bit // 32] >> (bit % 32)) & 1).bool()
        q = s["q"][cu[j]: cu[j + 1]].double().unflatten(1, (c["kv_heads"], group)).permute(1, 2, 0, 3)
        sc = torch.matmul(q.flatten(1, 2), k.transpose(1, 2).contiguous()).unflatten(1, (group, n)) * s["scale"]
        sc = sc.masked_fill(~keep, -math.inf)
        lse = torch.logsumexp(sc, -1)
        p = torch.exp(sc - lse[..., None].nan_to_num(neginf=0.0))
        o = torch.matmul(p.flatten(1, 2), v.contiguous()).unflatten(1, (group, n))
        outs.append(o.permute(2, 0, 1, 3).flatten(1, 2))
        lses.append(lse.permute(2, 0, 1).flatten(1, 2))
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _turn64(x, pos):
    d = x.shape[-1]
    w = 10000.0 ** (-torch.arange(0, d, 2, device=DEV).double() / d)
    z = torch.view_as_complex(x.double().unflatten(-1, (-1, 2)).contiguous())
    return torch.view_as_real(z * torch.polar(torch.ones_like(w), pos.double()[..., None] * w)).flatten(-2)


def _exact_append(s):
    c, cu, lens = s["case"], s["cu_q"].tolist(), s["lens"].tolist()
    H, dn = c["heads"], c["d_nope"]
    pos = torch.cat([torch.arange(p, p + b - a, device=DEV) for a, b, p in zip(cu, cu[1:], lens)])
    seq = torch.repeat_interleave(torch.arange(len(lens), device=DEV), s["cu_q"][1:] - s["cu_q"][:-1])
    page, row = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    key = torch.cat([s["kv"][..., :dn].double(), _turn64(s["pe"], pos)[:, None].expand(-1, H, -1)], -1)
    parts = [key] + ([s["kv"][..., dn:].double()] if c["d_v"] else [])

    def placed(p, empty=0.0):
        b = torch.full((s["bufs"][0].shape[0], c["page"], *p.shape[1:]), empty, dtype=torch.float64, device=DEV)
        b[page, row] = p
        return b

    if c["cache"] == "bf16":
        return {"bufs": [placed(p) for p in parts]}
    both = [_quantize64(p) for p in parts]
    return {"codes": [placed(a) for a, _ in both], "scales": [placed(b, 2.0 ** -127) for _, b in both]}


def _exact_project(s):
    c = s["case"]
    lo, hi = (s["codes"] & 15).int(), (s["codes"] >> 4).int()
    code = torch.stack([lo, hi], -1).flatten(-2)
    e, frac = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, frac * 0.5, (1 + frac * 0.5) * torch.exp2(e.double() - 1))
    w = torch.where(code >= 8, -mag, mag) * torch.exp2(s["scales"].double() - 127).repeat_interleave(32, -1)
    q = torch.matmul(w, s["x"].double().t().contiguous()).unflatten(0, (c["heads"], -1)).transpose(1, 2)
    q = torch.cat([q[..., : c["d_nope"]], _turn64(q[..., c["d_nope"]:], s["positions"])], -1)[None]
    if c["out"] == "bf16":
        return {"out": q}
    codes, scales = _quantize64(q)
    return {"codes": codes, "scales": scales}


def exact(case, seed):
    if case["op"] in ("branch", "pack"):
        return None  # whole numbers and copies
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "project": _exact_project}[case["op"]](s)
