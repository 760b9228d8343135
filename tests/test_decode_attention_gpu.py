"""mla_tree_attention against the 64-bit form, element by element.

Bound of an output element, from the formula, with u = 2^-8 (half a bf16 step
relative to the value) and e = 2^-24 (fp32): the result is rounded once (u |out|)
and each weight once (u A, A = sum of weight times |value|); a score is off by
at most (d_k + 4) e D for D = scale sum |q k| (products exact, d_k additions in
fp32, the scale's rounding and the subtraction of the maximum), plus the
exponential's two units, which moves weights by that relative amount and their
sum as much again: 2 ((d_k + 4) e D + 4 e + 4 e (|s| + |m|)) A with |s|, |m| <= D; sums over L rows in fp32: 2 L e A.
lse: the score's error, 2 L e for the sum and 4 e |lse| + 4 e."""
import math

import pytest
import torch

import mla_up_projection_amd as m
from tests import decode_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
U, E = 2.0 ** -8, 2.0 ** -24


def normal(seed, *shape, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * sigma).to(torch.bfloat16)


class Case:
    """A pool with sequences of lens[i] committed rows and drafts[i] new ones, pages in random order."""

    def __init__(self, lens, drafts, page, heads, kv_heads, d_k, d_v, latent, mx=False, seed=0, spare=3, order=None):
        self.lens, self.drafts, self.page, self.d_v, self.mx = lens, drafts, page, d_v, mx
        g = torch.Generator().manual_seed(seed + 77)
        n = len(lens)
        order = list(range(n)) if order is None else order
        held = [-(-a // page) for a in lens]
        for j, s in enumerate(order):
            held[s] = max(held[s], -(-(lens[s] + drafts[j]) // page))  # a sequence may be listed twice
        num = sum(held) + spare
        num += num % 2 if mx else 0  # an even number of rows
        ids = torch.randperm(num, generator=g).tolist()
        self.table = torch.full((n, max(1, max(held)) + 1), -1, dtype=torch.int32)
        for i in range(n):
            for k in range(held[i]):
                self.table[i, k] = ids.pop()
        widths = [d_k] if latent else [d_k, d_v]
        bufs = [normal(seed + 5 + k, num, page, kv_heads, w) for k, w in enumerate(widths)]
        if mx:
            out = []
            for b in bufs:
                codes = torch.empty(b.shape, dtype=torch.uint8, device=DEV)
                sc = torch.empty(*b.shape[:-1], b.shape[-1] // 32, dtype=torch.uint8, device=DEV)
                m.mxfp8_quantize(b.view(-1, b.shape[-1]).to(DEV), codes.view(-1, b.shape[-1]),
                                 sc.view(-1, b.shape[-1] // 32))
                out += [codes.cpu(), sc.cpu()]
            bufs = out
        self.bufs, self.held, self.order = bufs, held, order
        self.cu = [0]
        for d in drafts:
            self.cu.append(self.cu[-1] + d)
        self.T = self.cu[-1]
        self.q = normal(seed + 9, self.T, heads, d_k)
        self.scale = 1 / math.sqrt(d_k)
        self.mask = None
        self.max_q, self.max_len = max(drafts + [1]), max([lens[s] + d for s, d in zip(order, drafts)] + [1])

    def tree(self, seed=1, words=None):
        g = torch.Generator().manual_seed(seed)
        words = -(-self.max_q // 32) if words is None else words
        self.mask = torch.zeros(self.T, words, dtype=torch.int64)
        for j, n in enumerate(self.drafts):
            see = []
            for i in range(n):
                parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
                see.append((see[parent] if parent >= 0 else set()) | {i})
                for k in see[i]:
                    self.mask[self.cu[j] + i, k // 32] |= 1 << (k % 32)
        return self

    def device(self):
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
        num = self.bufs[0].shape[0]
        pool = m.PagePool([b.to(DEV) for b in self.bufs], torch.ones(num, dtype=torch.int32, device=DEV),
                          self.table.to(DEV), i32(self.lens), i32(self.held))
        mask = None
        if self.mask is not None:
            mask = torch.where(self.mask >= 1 << 31, self.mask - (1 << 32), self.mask).to(torch.int32).to(DEV)
        return pool, i32(self.order), i32(self.cu), mask

    def run(self, q=None, out=None, lse=None, **kw):
        pool, seqs, cu, mask = self.device()
        q = self.q.to(DEV) if q is None else q
        out = torch.full((q.shape[0], q.shape[1], self.d_v), 7.0, dtype=torch.bfloat16, device=DEV) if out is None else out
        lse = torch.full(q.shape[:2], 7.0, device=DEV) if lse is None else lse
        a = dict(max_q=self.max_q, max_len=self.max_len, scale=self.scale, lse=lse, mask=mask) | kw
        size = m.mla_tree_attention_workspace_size(q, pool, out, seqs, cu, **a)
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV) if size else None  # NaN patterns
        m.mla_tree_attention(q, pool, out, seqs, cu, workspace=ws, **a)
        torch.cuda.synchronize()
        return out.cpu(), lse.cpu()

    def expected(self):
        key, value = ref.cache_values(self.bufs, self.mx)
        return ref.attend(self.q, key, value, self.d_v, self.page, self.table, self.lens, self.order, self.cu,
                          self.scale, self.mask)


def check(out, lse, want, d_k):
    o, l, A, D, L = want
    ds = (d_k + 4) * E * D + 4 * E + 8 * E * D
    bound = U * o.abs() + (U + 2 * ds[..., None] + 2 * L[:, None, None] * E) * A
    got = out.double()
    assert torch.isnan(got).equal(torch.isnan(o)), "NaN in other places"
    inf = torch.isinf(o)
    assert got[inf].equal(o[inf])
    ok = torch.isfinite(o)
    bad = ok & ~((got - o).abs() <= bound)
    assert not bad.any(), (bad.nonzero()[:4], got[bad][:4], o[bad][:4], bound[bad][:4])
    fin = torch.isfinite(l)
    assert torch.equal(torch.isnan(lse.double()), torch.isnan(l))
    assert torch.equal(lse.double()[torch.isinf(l)], l[torch.isinf(l)])
    err = (lse.double() - l).abs()[fin]
    assert (err <= (ds + 2 * L[:, None] * E + 4 * E * l.abs() + 4 * E)[fin]).all(), err.max()


SHAPES = {  # d_k, d_v, latent, heads, kv heads
    "latent": (576, 512, True, 5, 1),
    "latent small": (96, 64, True, 3, 1),
    "per head": (192, 128, False, 3, 3),
    "grouped": (128, 128, False, 6, 2),
    "narrow": (64, 64, False, 14, 7),
}


def make(shape, lens, drafts, page, seed=0, mx=False, heads=None, **kw):
    d_k, d_v, latent, h, hk = SHAPES[shape]
    return Case(lens, drafts, page, heads or h, hk, d_k, d_v, latent, mx, seed, **kw)


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", SHAPES)
def test_one_tile(shape, mx):
    c = make(shape, [13], [2], 16, mx=mx)
    check(*c.run(), c.expected(), c.q.shape[2])


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("page", [1, 16, 48])
def test_ragged_trees(shape, mx, page):
    c = make(shape, [37, 0, 200, 31, 1], [3, 5, 1, 0, 7], page, seed=3, mx=mx).tree()
    check(*c.run(), c.expected(), c.q.shape[2])


@pytest.mark.parametrize("heads", [1, 17, 40, 70, 128])
def test_row_tiles(heads):
    """Workgroups of one, two and four waves, the last rows of a tile missing."""
    c = make("latent", [65, 7], [3, 1], 7, seed=4, heads=heads).tree()
    check(*c.run(), c.expected(), 576)


@pytest.mark.parametrize("n", [33, 64, 70])
def test_more_drafts_than_a_mask_word(n):
    for words in (None, 4):
        c = make("narrow", [5, 40], [n, 3], 16, seed=n).tree(words=words)
        check(*c.run(), c.expected(), 64)
    c = make("latent small", [5], [n], 16, seed=n)  # a chain
    check(*c.run(), c.expected(), 96)


@pytest.mark.parametrize("shape", ["latent", "per head"])
def test_long_ragged_chunks(shape):
    """Lengths around chunk and tile borders; the plan's bound far above the actual lengths as well."""
    c = make(shape, [2047, 128, 511, 1024, 3], [1, 2, 1, 4, 1], 64, seed=8, heads=None if shape == "per head" else 2).tree()
    out, lse = c.run()
    check(out, lse, c.expected(), c.q.shape[2])
    out2, lse2 = c.run(max_len=20000, max_q=9)
    check(out2, lse2, c.expected(), c.q.shape[2])


def test_rows_that_see_nothing_and_strange_values_they_do_not_see():
    """Empty masks; NaN and infinities in drafts that a row masks, behind the sequence's end and in free pages."""
    for shape in ("latent", "per head", "latent small"):
        c = make(shape, [0, 40, 10], [3, 4, 2], 16, seed=11).tree()
        c.mask[:, :] = 0
        c.mask[3, 0], c.mask[4, 0], c.mask[5, 0] = 0b1, 0b0010, 0b1001
        used = torch.zeros(c.bufs[0].shape[:2], dtype=torch.bool)
        for s, (a, d) in enumerate(zip(c.lens, c.drafts)):
            for r in range(a + d):
                used[c.table[s, r // 16].long(), r % 16] = True
        for b in c.bufs:
            b[~used] = math.nan
            p = lambda r: (c.table[1, r // 16].long(), r % 16)  # noqa: B023, E731
            b[p(42)] = math.inf     # draft 2 of the second sequence: seen by nobody
            b[p(43)] = -math.inf    # draft 3: nobody either
            b[p(41)][..., 3] = math.nan  # draft 1: seen by token 4 alone
        want = c.expected()
        out, lse = c.run()
        check(out, lse, want, c.q.shape[2])
        assert (out[:3] == 0).all() and torch.isneginf(lse[:3]).all()  # nothing committed, no draft seen
        assert torch.isnan(lse[4]).all() and torch.isfinite(out[3].float()).all()


def test_infinite_values_in_rows_that_are_seen():
    c = make("per head", [40], [3], 16, seed=12).tree()
    c.mask[0, 0], c.mask[1, 0], c.mask[2, 0] = 0b001, 0b011, 0b111
    p = lambda r: (c.table[0, r // 16].long(), r % 16)  # noqa: E731
    c.bufs[1][p(41)][:, 5] = math.inf
    c.bufs[1][p(42)][:, 5] = -math.inf
    c.bufs[1][p(42)][:, 6] = -math.inf
    c.bufs[1][p(7)][:, 9] = math.inf
    out, lse = c.run()
    check(out, lse, c.expected(), 192)
    assert (out[:, :, 9] == math.inf).all() and (out[1, :, 5] == math.inf).all() and torch.isnan(out[2, :, 5]).all()


def test_large_scores_and_a_rising_maximum():
    """Scores that grow along the cache by far more than the maximum may lag; and all scores equal."""
    c = make("latent", [300], [2], 16, seed=13, heads=3)
    ramp = torch.linspace(0, 6, 320)
    for r in range(302):
        c.bufs[0][c.table[0, r // 16].long(), r % 16] *= ramp[r]
    check(*c.run(), c.expected(), 576)
    c.q.zero_()
    check(*c.run(), c.expected(), 576)


def test_mxfp8_special_scales():
    """A scale of 0xFF makes its block NaN for those who see it; the smallest scales are values, not zero."""
    c = make("latent", [20], [2], 16, seed=14, mx=True, heads=2).tree()
    c.mask[0, 0], c.mask[1, 0] = 0b01, 0b11
    p = lambda r: (c.table[0, r // 16].long(), r % 16)  # noqa: E731
    c.bufs[1][p(21)] = 255
    c.bufs[1][p(3)][..., :2] = 2
    out, lse = c.run()
    check(out, lse, c.expected(), 576)
    assert torch.isnan(out[1].float()).all() and torch.isfinite(out[0].float()).all()


def test_strides_and_order_of_sequences():
    """Queries in BHSD as mla_qup_fwd writes them, outputs into a wider buffer, sequences in another order and one
    listed twice."""
    c = make("per head", [30, 9, 50], [2, 3, 1], 16, seed=15, order=[2, 0, 1]).tree()
    want = c.expected()
    qh = c.q.transpose(0, 1).contiguous().to(DEV)  # [H, T, D]
    wide = torch.full((c.T, 3, 200), 7.0, dtype=torch.bfloat16, device=DEV)
    out, lse = c.run(q=qh.transpose(0, 1), out=wide[..., :128])
    check(out, lse, want, 192)
    assert (wide[..., 128:] == 7).all()
    hm = torch.empty(3, c.T, 128, dtype=torch.bfloat16, device=DEV)
    out2, _ = c.run(out=hm.transpose(0, 1))
    assert torch.equal(out2, out)
    d = make("per head", [30, 9, 50], [2, 3, 1], 16, seed=15, order=[2, 0, 0])
    check(*d.run(), d.expected(), 192)


def test_rows_behind_the_last_sequence_stay():
    c = make("latent small", [30, 9], [2, 3], 16, seed=16)
    q = torch.cat([c.q, c.q[:3]]).to(DEV)
    out, lse = c.run(q=q)
    assert (out[5:] == 7).all() and (lse[5:] == 7).all()
    check(out[:5], lse[:5], c.expected(), 96)


def test_bad_pages_and_outgrown_bounds_give_nan():
    """Page ids outside the pool, rows without a held page, more drafts or rows than announced, an invalid entry."""
    for shape in ("latent", "per head"):
        c = make(shape, [40, 20], [2, 2], 16, seed=17)
        good, _ = c.run()
        c.table[0, 1] = 10 ** 6
        out, lse = c.run()
        assert torch.isnan(out[:2].float()).all() and torch.isnan(lse[:2]).all() and torch.equal(out[2:], good[2:])
        c.table[0, 1] = -5
        assert torch.isnan(c.run()[0][:2].float()).all()
        c = make(shape, [40, 20], [2, 2], 16, seed=17)
        c.held[1] = 1
        out, _ = c.run()
        assert torch.equal(out[:2], good[:2]) and torch.isnan(out[2:].float()).all()
        c = make(shape, [40, 20], [2, 2], 16, seed=17)
        out, lse = c.run(max_len=30)
        assert torch.isnan(out[:2].float()).all() and torch.equal(out[2:], good[2:]) and torch.isnan(lse[:2]).all()
        out, lse = c.run(max_q=1)
        assert torch.isnan(out.float()).all() and torch.isnan(lse).all()
        c.order = [0, 2]
        out, _ = c.run()
        assert torch.equal(out[:2], good[:2]) and torch.isnan(out[2:].float()).all()


def test_offsets_beyond_32_bits():
    """Pages whose bytes lie behind 4 GiB of the buffer."""
    page, num = 64, 60000  # 4.4 GB of latent pages
    buf = torch.empty(num, page, 1, 576, dtype=torch.bfloat16, device=DEV)
    rows = normal(18, 3 * page, 576)
    ids = [59999, 2, 59000]
    for k, p in enumerate(ids):
        buf[p, :, 0] = rows[k * page: (k + 1) * page].to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pool = m.PagePool([buf], torch.ones(num, dtype=torch.int32, device=DEV), i32([ids]), i32([150]), i32([3]))
    q = normal(19, 2, 4, 576)
    out = torch.empty(2, 4, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(2, 4, device=DEV)
    kw = dict(max_q=2, max_len=152, scale=1 / 24, lse=lse)
    n = m.mla_tree_attention_workspace_size(q.to(DEV), pool, out, i32([0]), i32([0, 2]), **kw)
    m.mla_tree_attention(q.to(DEV), pool, out, i32([0]), i32([0, 2]),
                         workspace=torch.empty(n, dtype=torch.uint8, device=DEV) if n else None, **kw)
    want = ref.attend(q, rows.double().view(3, page, 1, 576), None, 512, page, torch.tensor([[0, 1, 2]]), [150], [0],
                      [0, 2], 1 / 24, None)
    check(out.cpu(), lse.cpu(), want, 576)


def test_same_bits_every_time_on_any_stream_and_in_a_graph():
    c = make("latent", [700, 90, 5], [3, 2, 4], 48, seed=20, heads=32).tree()
    pool, seqs, cu, mask = c.device()
    q = c.q.to(DEV)
    new = lambda: (torch.empty(c.T, 32, 512, dtype=torch.bfloat16, device=DEV), torch.empty(c.T, 32, device=DEV))  # noqa: E731
    out, lse = new()
    kw = dict(max_q=c.max_q, max_len=c.max_len, scale=c.scale, mask=mask)
    size = m.mla_tree_attention_workspace_size(q, pool, out, seqs, cu, lse=lse, **kw)
    assert size > 0
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    m.mla_tree_attention(q, pool, out, seqs, cu, lse=lse, workspace=ws, **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    o2, l2 = new()
    with torch.cuda.stream(st):
        m.mla_tree_attention(q, pool, o2, seqs, cu, lse=l2, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.mla_tree_attention(q, pool, o2, seqs, cu, lse=l2, workspace=ws, **kw)
    for k in range(3):
        o2.fill_(k)
        pool.lens[1] = 90 - k  # what the graph reads may change between replays
        g.replay()
        o3, l3 = new()
        m.mla_tree_attention(q, pool, o3, seqs, cu, lse=l3, workspace=ws, **kw)
        torch.cuda.synchronize()
        assert torch.equal(o2, o3) and torch.equal(l2, l3)
        if k == 0:
            assert torch.equal(o2, out)


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("n", [65, 300, 600])
def test_many_sequences(n, mx):
    """More sequences than lanes and than threads, some without drafts, some listed twice, some outgrown."""
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 90, (n,), generator=g).tolist()
    drafts = torch.randint(0, 3, (n,), generator=g).tolist()
    order = torch.randperm(n, generator=g).tolist()
    order[7] = order[-1]
    for shape in ("latent", "latent small"):
        c = make(shape, lens, drafts, 16, seed=21, mx=mx, heads=2, order=order).tree()
        want = c.expected()
        check(*c.run(), want, c.q.shape[2])
        for j, s in enumerate(order):
            if lens[s] + drafts[j] > 80:
                for x in want[:2]:
                    x[c.cu[j]: c.cu[j + 1]] = math.nan
        check(*c.run(max_len=80), want, c.q.shape[2])


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
def test_more_row_tiles_than_workgroups(mx):
    """Several items, and parts of items, to a workgroup."""
    g = torch.Generator().manual_seed(22)
    lens = torch.randint(0, 150, (80,), generator=g).tolist()
    c = make("latent", lens, [1] * 80, 16, seed=22, mx=mx, heads=128)
    check(*c.run(), c.expected(), 576)
    c = make("latent", lens[:30], [4, 1, 3] * 10, 16, seed=23, mx=mx, heads=70).tree()
    check(*c.run(), c.expected(), 576)


@pytest.mark.parametrize("shape", ["latent", "per head"])
def test_drafts_that_see_only_themselves(shape):
    """Rows whose first tiles are masked as a whole."""
    c = make(shape, [0, 3, 64], [70, 40, 33], 16, seed=24)
    c.mask = torch.zeros(c.T, 3, dtype=torch.int64)
    for j, n in enumerate(c.drafts):
        for i in range(n):
            c.mask[c.cu[j] + i, i // 32] = 1 << (i % 32)
    out, lse = c.run()
    check(out, lse, c.expected(), c.q.shape[2])


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
def test_parts_longer_than_the_list_of_pages(mx):
    """Pages of one row, and parts of more rows than the kernel lists pages at a time, with rows behind the first
    list that carry all the weight: scores 130 above the others, beyond what the running reference may lag. Eight
    such rows at distances of 25500 share it; without one of them the outputs change by an eighth."""
    n, d = 211000, 576
    g = torch.Generator().manual_seed(25)
    rows = torch.randn(n, d, generator=g).to(torch.bfloat16)
    q = normal(26, 1, 1, d)
    qd = q.double().view(-1)
    at = [1000 + 25500 * k for k in range(8)]
    for r in at:
        v = rows[r].double()
        rows[r] = (v + qd * ((130 * 24 - v @ qd) / (qd @ qd))).to(torch.bfloat16)
    c = Case.__new__(Case)
    c.lens, c.drafts, c.page, c.d_v, c.mx, c.order, c.cu, c.T = [n - 1], [1], 1, 512, mx, [0], [0, 1], 1
    c.held, c.table = [n], torch.randperm(n, generator=g).to(torch.int32).view(1, n)
    buf = torch.empty(n, d, dtype=torch.bfloat16)
    buf[c.table[0].long()] = rows
    c.bufs = [buf.view(n, 1, 1, d)]
    if mx:
        codes, sc = (torch.empty(n, w, dtype=torch.uint8, device=DEV) for w in (d, d // 32))
        m.mxfp8_quantize(buf.to(DEV), codes, sc)
        c.bufs = [codes.cpu().view(n, 1, 1, d), sc.cpu().view(n, 1, 1, d // 32)]
    c.q, c.scale, c.mask, c.max_q, c.max_len = q, 1 / 24, None, 1, n
    check(*c.run(), c.expected(), d)


def test_a_graph_follows_the_lengths_on_the_device():
    """Captured once, replayed with other lengths, orders of magnitude apart, in the same buffers."""
    c = make("latent", [700, 90, 5, 0], [3, 2, 4, 1], 48, seed=27, heads=32)
    pool, seqs, cu, _ = c.device()
    q = c.q.to(DEV)
    out, lse = torch.empty(c.T, 32, 512, dtype=torch.bfloat16, device=DEV), torch.empty(c.T, 32, device=DEV)
    kw = dict(max_q=c.max_q, max_len=c.max_len, scale=c.scale, lse=lse)
    size = m.mla_tree_attention_workspace_size(q, pool, out, seqs, cu, **kw)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.mla_tree_attention(q, pool, out, seqs, cu, workspace=ws, **kw)
    for lens in ([700, 90, 5, 0], [0, 0, 0, 0], [31, 28, 5, 0], [650, 1, 0, 0], [700, 90, 5, 0]):
        pool.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7)
        lse.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        c.lens = lens
        check(out.cpu(), lse.cpu(), c.expected(), 576)
        again = out.clone()
        ws.fill_(0xFF)
        m.mla_tree_attention(q, pool, out, seqs, cu, workspace=ws, **kw)
        torch.cuda.synchronize()
        assert torch.equal(again, out)


def test_no_tokens_and_no_sequences():
    c = make("latent", [40], [0], 16, seed=28, heads=2)
    out, lse = c.run()
    assert out.numel() == 0 and lse.numel() == 0
    c = make("latent", [40], [2], 16, seed=28, heads=2)
    c.cu, c.order = [0], []
    out, lse = c.run()
    assert (out == 7).all() and (lse == 7).all()


def test_bounds_far_above_the_call():
    g = torch.Generator().manual_seed(29)
    lens = torch.randint(0, 40, (1000,), generator=g).tolist()
    c = make("latent", lens, [1, 2] * 500, 16, seed=29, heads=8)
    check(*c.run(max_q=512, max_len=50000), c.expected(), 576)
    check(*c.run(max_len=2 ** 31 - 1), c.expected(), 576)


def test_calls_at_once():
    """Two streams over one pool, each with its own workspace, several times over."""
    c = make("latent", [3000, 90, 5, 1200], [3, 2, 4, 1], 48, seed=30, heads=32).tree()
    pool, seqs, cu, mask = c.device()
    q = c.q.to(DEV)
    kw = dict(max_q=c.max_q, max_len=c.max_len, scale=c.scale, mask=mask)
    outs = [torch.empty(c.T, 32, 512, dtype=torch.bfloat16, device=DEV) for _ in range(9)]
    size = m.mla_tree_attention_workspace_size(q, pool, outs[0], seqs, cu, **kw)
    ws = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    m.mla_tree_attention(q, pool, outs[8], seqs, cu, workspace=ws[0], **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(8):
        m.mla_tree_attention(q, pool, outs[k], seqs, cu, workspace=ws[k % 2], stream=streams[k % 2], **kw)
    torch.cuda.synchronize()
    for k in range(8):
        assert torch.equal(outs[k], outs[8])
