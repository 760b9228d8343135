"""Page bookkeeping, accepted paths and paged appends on the GPU. Bookkeeping and
copies are exact: every array and every byte must equal the list form's."""
import math

import numpy as np
import pytest
import torch

import mla_up_projection_amd as m
from tests import decode_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Both:
    """A pool on the GPU and its list form, driven side by side."""

    def __init__(self, num_pages, page, max_seqs, max_pages, row_shapes=((1, 96),), mx=False, seed=0):
        rng = np.random.default_rng(seed)
        dt = np.uint8 if mx else np.int16
        self.ref = ref.Pages(num_pages, page, max_seqs, max_pages,
                             [rng.integers(0, 127, (num_pages, page, *s)).astype(dt) for s in row_shapes])
        bufs = [torch.from_numpy(r).to(DEV) for r in self.ref.rows]
        self.bufs = bufs if mx else [b.view(torch.bfloat16) for b in bufs]
        self.ref.rows = [r.copy() for r in self.ref.rows]
        z = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
        self.pool = m.PagePool(self.bufs, z(num_pages), torch.full((max_seqs, max_pages), -1, dtype=torch.int32, device=DEV),
                               z(max_seqs), z(max_seqs))
        self.ws = torch.full((m.mla_pages_workspace_size(self.pool),), 0xAB, dtype=torch.uint8, device=DEV)
        self.status = i32([99])

    def set_lens(self, lens):
        self.ref.lens = list(lens)
        self.pool.lens.copy_(i32(lens))

    def reserve(self, seqs, new):
        m.mla_pages_reserve(self.pool, i32(seqs), i32(new), self.status, workspace=self.ws)
        want = self.ref.reserve(seqs, new)
        self.same()
        assert self.status.item() == want
        return want

    def fork(self, src, dst):
        m.mla_pages_fork(self.pool, i32(src), i32(dst))
        self.ref.fork(src, dst)
        self.same()

    def free(self, seqs, keep=None):
        m.mla_pages_free(self.pool, i32(seqs), None if keep is None else i32(keep))
        self.ref.free(seqs, keep)
        self.same()

    def compact(self):
        used = i32([-1])
        m.mla_pages_compact(self.pool, used, workspace=self.ws)
        assert used.item() == self.ref.compact()
        self.same()

    def accept(self, seqs, path, n_acc):
        m.mla_draft_accept(self.pool, i32(seqs), i32(path), i32(n_acc))
        self.ref.accept(seqs, path, n_acc)
        self.same()

    def same(self):
        r, p = self.ref, self.pool
        assert p.refs.tolist() == r.refs
        assert p.held.tolist() == [len(t) for t in r.table]
        assert p.lens.tolist() == r.lens
        table = p.table.tolist()
        for s, t in enumerate(r.table):
            assert table[s][: len(t)] == t
        for a, b in zip(self.bufs, r.rows):
            assert np.array_equal(a.view(torch.uint8 if a.dtype == torch.uint8 else torch.int16).cpu().numpy(), b)


POOLS = {
    "latent bf16": (((1, 96),), False),
    "latent mxfp8": (((1, 576), (1, 18)), True),  # scale rows of 18 bytes
    "heads bf16": (((3, 64), (3, 64)), False),
    "heads mxfp8": (((3, 32), (3, 1), (3, 96), (3, 3)), True),
}


@pytest.mark.parametrize("kind", POOLS)
@pytest.mark.parametrize("page", [1, 7, 16])
def test_a_random_life_of_a_pool(kind, page):
    shapes, mx = POOLS[kind]
    for seed in range(3):
        rng = np.random.default_rng(1000 * page + seed)
        b = Both(60, page, 9, 12, shapes, mx, seed)
        for step in range(40):
            what = rng.choice(["reserve", "reserve", "fork", "free", "cut", "accept", "compact"])
            n = int(rng.integers(1, 6))
            seqs = rng.integers(-1, 10, n).tolist()  # ids outside and twice among them
            if what == "reserve":
                b.reserve(seqs, rng.integers(0, 3 * page + 2, n).tolist())
            elif what == "fork":
                b.fork(seqs, rng.integers(0, 10, n).tolist())
            elif what == "free":
                b.free(seqs[:2])
            elif what == "cut":
                b.free(seqs, rng.integers(-2, 6 * page, n).tolist())
            elif what == "accept":
                # accepted rows are written in place: a server reserves first
                new = [4] * n
                if b.reserve(seqs, new) == 0:
                    path = [sorted(rng.choice(4, 3, replace=False).tolist()) for _ in range(n)]
                    b.accept(seqs, path, rng.integers(0, 4, n).tolist())
            else:
                b.compact()


def test_reserve_refuses_as_a_whole():
    b = Both(10, 4, 4, 6)
    assert b.reserve([0, 1], [16, 20]) == 0        # 4 + 5 pages
    assert b.reserve([2, 3], [4, 8]) == 2          # 3 wanted, 1 free
    assert b.reserve([2], [25]) == -1              # 7 pages of 6
    assert b.reserve([2, 3], [4, -1]) == -1
    assert b.reserve([2], [4]) == 0
    assert b.reserve([], []) == 0
    assert b.reserve([3], [1]) == 1
    assert b.reserve([3], [0]) == 0


def test_copy_on_write_by_many_children():
    """All who share a partly filled page in one call: the last listed keeps it; with the parent outside, none."""
    b = Both(400, 8, 300, 4, seed=5)
    b.reserve([0], [20])
    b.set_lens([20] + [0] * 299)
    kids = list(range(1, 251))
    b.fork([0] * 250, kids)
    assert max(b.ref.refs) == 251
    b.reserve(kids, [1] * 250)
    b.free(kids)
    b.fork([0] * 250, kids)
    b.reserve([0] + kids, [3] * 251)
    b.free([0])
    b.compact()


def test_longest_list_and_a_large_pool():
    b = Both(70000, 1, 1024, 80, seed=6, row_shapes=((1, 32),))
    rng = np.random.default_rng(2)
    seqs = rng.permutation(1024).tolist()
    b.reserve(seqs, rng.integers(0, 70, 1024).tolist())
    b.free(rng.permutation(1024)[:500].tolist())
    b.reserve(seqs, rng.integers(0, 60, 1024).tolist())
    b.compact()


def test_fork_rules():
    b = Both(30, 4, 6, 6)
    b.reserve([0, 1], [10, 3])
    b.set_lens([10, 3, 0, 0, 0, 0])
    b.fork([0, 1, 2], [2, 2, 3])   # 2 twice: the first counts; its source 2 is a destination of the call
    b.fork([0], [1])               # holds pages
    b.fork([4, 9, 0], [5, 4, -1])  # an empty source, ids outside
    b.fork([0, 0], [0, 3])         # itself (and 0 is then a destination: the second is skipped too)


def test_accept_rules():
    b = Both(40, 4, 5, 8, (((2, 64)),), seed=3)
    b.reserve([0, 1, 2, 3], [20, 20, 20, 20])
    b.set_lens([5, 0, 9, 2, 0])
    long = list(range(1, 14))
    pad = lambda p: p + [99] * (13 - len(p))  # noqa: E731
    b.accept([0, 1, 0, 2], [pad([1, 4, 5]), pad([0, 1, 2]), pad([2]), pad([10, 11])], [3, 2, 1, 2])  # last: behind the pages
    b.accept([3], [long], [13])                      # more rows than are loaded at once
    b.accept([2, 1, 0], [pad([3, 3]), pad([4, 2]), pad([-1])], [2, 2, 1])  # no strictly increasing path
    b.accept([2, 1, -7, 5], [pad([1])] * 4, [14, -1, 1, 1])


def test_lengths_that_cannot_be():
    """Lengths outside what the pages hold change nothing but their own sequence."""
    big = 2 ** 31 - 1
    for bad in (-1, -big - 1, big):
        b = Both(30, 4, 6, 6)
        b.reserve([0, 1], [10, 3])
        b.pool.lens.copy_(i32([bad, 3, 0, 0, 0, 0]))
        table, refs = b.pool.table.clone(), b.pool.refs.clone()
        m.mla_pages_reserve(b.pool, i32([0]), i32([1]), b.status, workspace=b.ws)
        assert b.status.item() == -1
        m.mla_draft_accept(b.pool, i32([0]), i32([[0, 1]]), i32([2]))
        assert b.pool.lens[0].item() == bad and torch.equal(b.pool.table, table) and torch.equal(b.pool.refs, refs)
        m.mla_pages_fork(b.pool, i32([0]), i32([2]))
        m.mla_pages_free(b.pool, i32([0]), i32([big]))
        assert b.pool.held[0].item() == (3 if bad > 0 else 0)
        assert b.pool.held[2].item() == (3 if bad > 0 else 0)
        assert torch.equal(b.pool.table[1], table[1]) and (b.pool.table[3:] == -1).all()


def test_copy_pages():
    shapes, mx = POOLS["heads mxfp8"]
    for page in (1, 16):
        a, b = Both(40, page, 2, 4, shapes, mx, 1), Both(50, page, 3, 4, shapes, mx, 2)
        src, dst = [3, 39, 7, 7, 40, -1, 5, 0], [49, 0, 11, 12, 1, 2, 0, 50]
        m.mla_pages_copy(a.pool, b.pool, i32(src), i32(dst))
        a.ref.copy(b.ref, src, dst)
        a.same()
        b.same()
        src, dst = [1, 2, 3, 4], [10, 3, 11, 10]  # 3 is a source too; 10 twice
        m.mla_pages_copy(a.pool, a.pool, i32(src), i32(dst))
        a.ref.copy(a.ref, src, dst)
        a.same()


def test_a_step_in_a_graph_replays():
    """free, fork, reserve, accept and compact recorded once; every replay equals the list form's next round."""
    b = Both(64, 4, 6, 10, seed=9)
    b.reserve([0], [14])
    b.set_lens([14, 0, 0, 0, 0, 0])
    kids, used = i32([1, 2, 3]), i32([0])
    src, new = i32([0, 0, 0]), i32([5, 6, 7])
    path, n_acc = i32([[1, 2], [0, 3], [4, 6]]), i32([2, 1, 2])

    def step():
        m.mla_pages_free(b.pool, kids)
        m.mla_pages_fork(b.pool, src, kids)
        m.mla_pages_reserve(b.pool, kids, new, b.status, workspace=b.ws)
        m.mla_draft_accept(b.pool, kids, path, n_acc)
        m.mla_pages_compact(b.pool, used, workspace=b.ws)

    def plain():
        b.ref.free([1, 2, 3])
        b.ref.fork([0, 0, 0], [1, 2, 3])
        assert b.ref.reserve([1, 2, 3], [5, 6, 7]) == 0
        b.ref.accept([1, 2, 3], path.tolist(), n_acc.tolist())
        return b.ref.compact()

    step()
    plain()
    torch.cuda.synchronize()
    b.same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert used.item() == plain()
        b.same()
        b.free([2])
        b.ws.fill_(0xCD)


# ------------------------------------------------------------------ append --
def table(rows, d_rope):
    cos = torch.empty(rows, d_rope // 2, dtype=torch.float32, device=DEV)
    sin = torch.empty_like(cos)
    m.rope_cache_build(cos, sin, d_rope)
    return cos, sin


APPENDS = {  # H, d_nope, d_rope, d_v
    "latent": (1, 512, 64, 0),
    "heads": (5, 128, 64, 128),
    "many heads": (130, 32, 32, 32),
    "odd widths": (3, 24, 8, 40),
    "no rope": (2, 64, 0, 32),
    "no nope": (2, 0, 64, 32),
}


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
@pytest.mark.parametrize("kind", APPENDS)
@pytest.mark.parametrize("page", [1, 16, 7])
def test_append(kind, mx, page):
    """Rows as mla_kv_rope makes them (which is pinned by its own tests), bit for bit; all else untouched."""
    H, dn, dr, dv = APPENDS[kind]
    if mx and ((dn + dr) % 32 or dv % 32):
        pytest.skip("MXFP8 rows are whole blocks of 32")
    lens, n, seqs = [5, 0, 33, 2, 70], [3, 0, 20, 1], [2, 1, 0, 4]
    T = sum(n)
    g = torch.Generator().manual_seed(page)
    kv = torch.randn(T + 2, H, dn + dv, generator=g).to(torch.bfloat16).to(DEV)  # two rows behind the last sequence
    pe = torch.randn(T + 2, dr, generator=g).to(torch.bfloat16).to(DEV)
    cos, sin = table(200, dr) if dr else (None, None)
    width = [(dn + dr), dv] if dv else [dn + dr]
    shapes = [s for w in width for s in (((H, w), (H, w // 32)) if mx else ((H, w),))]
    b = Both(220, page, 6, 100, shapes, mx)
    b.reserve([0, 2, 4, 3], [25, 36, 71, 2])
    b.set_lens(lens + [0])
    cu = [0, 3, 3, 23, 24]
    before = [x.clone() for x in b.bufs]
    pos = torch.cat([torch.arange(lens[s], lens[s] + k) for s, k in zip(seqs, [3, 0, 20, 1])]).int()
    for positions in (None, (pos * 7 + 1) % 150):
        use = pos if positions is None else positions
        # mla_kv_rope over a table whose row t is the row of token t's position
        rows = lambda t: t[use.long().to(DEV)].contiguous()  # noqa: B023, E731
        key = torch.empty(1, H, T, dn + dr, dtype=torch.uint8 if mx else torch.bfloat16, device=DEV)
        val = torch.empty(1, H, T, dv, dtype=key.dtype, device=DEV) if dv else None
        ks = torch.empty(1, H, T, (dn + dr) // 32, dtype=torch.uint8, device=DEV) if mx else None
        vs = torch.empty(1, H, T, dv // 32, dtype=torch.uint8, device=DEV) if mx and dv else None
        m.mla_kv_rope(kv[:T], pe[:T], key, val, H=H, d_nope=dn, d_rope=dr, d_v=dv, cos=rows(cos) if dr else None,
                      sin=rows(sin) if dr else None, key_scales=ks, value_scales=vs, B=1, S=T)
        made = [x for x in ((key, ks, val, vs) if mx else (key, val)) if x is not None]
        want = [x.clone() for x in before]
        for t in range(T):
            j = max(k for k in range(4) if cu[k] <= t and cu[k + 1] > cu[k])
            p, r = b.ref.at(seqs[j], lens[seqs[j]] + t - cu[j])
            for w, x in zip(want, made):
                w[p, r] = x[0, :, t]
        for x, y in zip(b.bufs, before):
            x.copy_(y)
        m.mla_kv_rope_paged(kv, pe, b.pool, i32(seqs), i32(cu), H=H, d_nope=dn, d_rope=dr, d_v=dv, cos=cos, sin=sin,
                            positions=None if positions is None else
                            torch.cat([positions, positions[:2]]).to(DEV))
        for x, y in zip(b.bufs, want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_append_what_is_not_written():
    """No held page, a page id outside the pool, an entry outside the table, a sequence listed twice; a position
    outside the table of angles gives NaN."""
    b = Both(20, 4, 4, 5)
    b.reserve([0, 1, 2], [8, 8, 8])
    b.set_lens([6, 0, 0, 0])
    kv, pe = torch.ones(12, 1, 64, dtype=torch.bfloat16, device=DEV), torch.ones(12, 32, dtype=torch.bfloat16, device=DEV)
    cos, sin = table(7, 32)
    b.pool.table[1, 1] = 500
    before = b.bufs[0].clone()
    m.mla_kv_rope_paged(kv, pe, b.pool, i32([0, 1, 7, 0, 2]), i32([0, 4, 9, 10, 11, 12]), H=1, d_nope=64, d_rope=32,
                        d_v=0, cos=cos, sin=sin)
    got = b.bufs[0]
    rows = {b.ref.at(0, 6): 6, b.ref.at(0, 7): 7, **{b.ref.at(1, r): r for r in range(4)}, b.ref.at(2, 0): 0}
    for p in range(20):
        for r in range(4):
            if (p, r) in rows:
                assert (got[p, r, 0, :64] == 1).all()
                assert torch.isnan(got[p, r, 0, 64:].float()).all() == (rows[p, r] >= 7)
            else:
                assert torch.equal(got[p, r].view(torch.int16), before[p, r].view(torch.int16))


def test_append_stops_at_max_q():
    b = Both(20, 4, 4, 5)
    b.reserve([0, 1], [8, 8])
    kv = torch.ones(9, 1, 96, dtype=torch.bfloat16, device=DEV)
    before = b.bufs[0].clone()
    m.mla_kv_rope_paged(kv, None, b.pool, i32([1, 0]), i32([0, 3, 9]), H=1, d_nope=96, d_rope=0, d_v=0, max_q=4)
    rows = {b.ref.at(1, r) for r in range(3)} | {b.ref.at(0, r) for r in range(4)}
    for p in range(20):
        for r in range(4):
            want = torch.ones_like(before[p, r]) if (p, r) in rows else before[p, r]
            assert torch.equal(b.bufs[0][p, r].view(torch.int16), want.view(torch.int16))


def test_many_tokens_one_sequence_many_sequences():
    """More chunks than one workgroup's, and the longest list of sequences."""
    for nseq, each in ((1, 5000), (1024, 2)):
        b = Both(nseq * each + 5, 1, nseq, 5000, (((1, 64)),))
        b.reserve(list(range(nseq)), [each] * nseq)
        kv = torch.randn(nseq * each, 1, 64, device=DEV).to(torch.bfloat16)
        m.mla_kv_rope_paged(kv, torch.empty(nseq * each, 0, dtype=torch.bfloat16, device=DEV), b.pool,
                            torch.arange(nseq, device=DEV, dtype=torch.int32),
                            torch.arange(0, nseq * each + 1, each, device=DEV, dtype=torch.int32), H=1, d_nope=64,
                            d_rope=0, d_v=0)
        flat = torch.tensor([p for t in b.ref.table for p in t], device=DEV)
        assert torch.equal(b.bufs[0][flat, 0].view(torch.int16), kv.view(torch.int16))
