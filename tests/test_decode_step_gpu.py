"""The decode-side operators together, as a server that drafts tokens calls them:
4-bit projection, room, append, tree attention, acceptance, release; sequences
fork, end and are packed in between. The cache must hold exactly the accepted
history of every sequence, and attention must be that over the history and the
drafts' ancestors (bounds as in test_decode_attention_gpu)."""
import pytest
import torch

import mla_up_projection_amd as m
from tests import decode_ref as ref
from tests.test_decode_attention_gpu import check

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, DN, DR, K, PAGE = 4, 64, 32, 128, 7


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("mx", [False, True], ids=["bf16", "mxfp8"])
def test_speculative_decoding(mx):
    g = torch.Generator().manual_seed(21)
    w = (torch.randn(H * (DN + DR), K, generator=g) * 0.1).to(torch.bfloat16).to(DEV)
    codes = torch.empty(w.shape[0], K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(w.shape[0], K // 32, dtype=torch.uint8, device=DEV)
    m.mxfp4_quantize(w, codes, scales)
    cos, sin = (torch.empty(400, DR // 2, device=DEV) for _ in range(2))
    m.rope_cache_build(cos, sin, DR)
    seqs_max, pages = 6, 90
    shape = (pages, PAGE, 1, DN + DR)
    bufs = [torch.zeros(shape, dtype=torch.uint8, device=DEV), torch.zeros(*shape[:3], 3, dtype=torch.uint8, device=DEV)] \
        if mx else [torch.zeros(shape, dtype=torch.bfloat16, device=DEV)]
    z = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    pool = m.PagePool(bufs, z(pages), torch.full((seqs_max, 30), -1, dtype=torch.int32, device=DEV), z(seqs_max), z(seqs_max))
    ws = torch.empty(m.mla_pages_workspace_size(pool), dtype=torch.uint8, device=DEV)
    status, used = i32([0]), i32([0])
    history = {s: [] for s in range(seqs_max)}  # rows (one tensor per buffer) of the committed tokens
    alive = [0, 1, 2]

    def row_of(latent, pe, pos):
        """A cache row as mla_kv_rope makes it."""
        key = torch.empty(1, 1, 1, DN + DR, dtype=torch.uint8 if mx else torch.bfloat16, device=DEV)
        ks = torch.empty(1, 1, 1, 3, dtype=torch.uint8, device=DEV) if mx else None
        m.mla_kv_rope(latent.view(1, DN), pe.view(1, DR), key, None, H=1, d_nope=DN, d_rope=DR, d_v=0,
                      cos=cos[pos: pos + 1].contiguous(), sin=sin[pos: pos + 1].contiguous(), key_scales=ks, B=1, S=1)
        return [x.flatten() for x in ([key, ks] if mx else [key])]

    for step in range(7):
        if step == 2:  # two branches of a running sequence, one sequence ends
            m.mla_pages_fork(pool, i32([1, 1]), i32([3, 4]))
            history[3], history[4] = list(history[1]), list(history[1])
            m.mla_pages_free(pool, i32([0]))
            history[0] = []
            alive = [4, 1, 2, 3]
        if step == 4:
            m.mla_pages_compact(pool, used, workspace=ws)
        n = torch.randint(1, 6, (len(alive),), generator=g).tolist()
        if step == 0:
            n = [20, 9, 1]  # prompts: chains, accepted whole
        cu = [0]
        for k in n:
            cu.append(cu[-1] + k)
        T = cu[-1]
        parent = [int(torch.randint(-1, i, (1,), generator=g)) if i and step else i - 1 for k in n for i in range(k)]
        see, depth = [], []
        for j, k in enumerate(n):
            for i in range(k):
                p = parent[cu[j] + i]
                see.append((see[cu[j] + p] if p >= 0 else 0) | 1 << i)
                depth.append(depth[cu[j] + p] + 1 if p >= 0 else 0)
        pos = [len(history[s]) + depth[cu[j] + i] for j, s in enumerate(alive) for i in range(n[j])]
        x = torch.randn(T, K, generator=g).to(torch.bfloat16).to(DEV)
        latent = torch.randn(T, 1, DN, generator=g).to(torch.bfloat16).to(DEV)
        pe = torch.randn(T, DR, generator=g).to(torch.bfloat16).to(DEV)
        q = torch.empty(1, H, T, DN + DR, dtype=torch.bfloat16, device=DEV)
        seqs, cuq, positions = i32(alive), i32(cu), i32(pos)

        m.mla_qup_fwd_w4(x, codes, scales, q, H=H, d_nope=DN, d_rope=DR, cos=cos, sin=sin, positions=positions)
        m.mla_pages_reserve(pool, seqs, i32(n), status, workspace=ws)
        m.mla_kv_rope_paged(latent, pe, pool, seqs, cuq, H=1, d_nope=DN, d_rope=DR, d_v=0, cos=cos, sin=sin,
                            positions=positions)
        out = torch.empty(T, H, DN, dtype=torch.bfloat16, device=DEV)
        lse = torch.empty(T, H, device=DEV)
        longest = max(len(history[s]) + k for s, k in zip(alive, n))
        kw = dict(max_q=max(n), max_len=longest, scale=0.1, lse=lse, mask=i32([[v] for v in see]))
        size = m.mla_tree_attention_workspace_size(q[0].transpose(0, 1), pool, out, seqs, cuq, **kw)
        aws = torch.empty(size, dtype=torch.uint8, device=DEV) if size else None
        m.mla_tree_attention(q[0].transpose(0, 1), pool, out, seqs, cuq, workspace=aws, **kw)
        # a random root-to-leaf path of each sequence is accepted, up to a random length
        path, n_acc, width = [], [], max(n)
        for j, k in enumerate(n):
            leaf = int(torch.randint(0, k, (1,), generator=g)) if step else k - 1
            p = [i for i in range(k) if see[cu[j] + leaf] >> i & 1]
            n_acc.append(len(p) if step in (0, 3) else int(torch.randint(0, len(p) + 1, (1,), generator=g)))
            path.append(p + [0] * (width - len(p)))
        drafts = [row_of(latent[t], pe[t], pos[t]) for t in range(T)]
        dense = [history[s] + drafts[cu[j]: cu[j + 1]] for j, s in enumerate(alive)]
        m.mla_draft_accept(pool, seqs, i32(path), i32(n_acc))
        m.mla_pages_free(pool, seqs, pool.lens[seqs.long()])  # what the drafts no longer need
        torch.cuda.synchronize()
        assert status.item() == 0

        # attention, over the rows the history says there are
        rows = max(len(d) for d in dense)
        flat = [torch.zeros(len(alive), rows, 1, b.shape[3], dtype=b.dtype) for b in bufs]
        for j, d in enumerate(dense):
            for r, parts in enumerate(d):
                for f, v in zip(flat, parts):
                    f[j, r, 0] = v.cpu()
        key, _ = ref.cache_values(flat, mx)
        want = ref.attend(q[0].transpose(0, 1).cpu(), key, None, DN, rows, torch.arange(len(alive))[:, None],
                          [len(history[s]) for s in alive], list(range(len(alive))), cu, 0.1, torch.tensor(see)[:, None])
        check(out.cpu(), lse.cpu(), want, DN + DR)
        for j, s in enumerate(alive):
            history[s] = history[s] + [drafts[cu[j] + i] for i in path[j][: n_acc[j]]]
        # the cache holds the history
        assert pool.lens.tolist() == [len(history[s]) for s in range(seqs_max)]
        assert pool.held.tolist() == [-(-len(history[s]) // PAGE) for s in range(seqs_max)]
        table = pool.table.tolist()
        refs = [0] * pages
        for s in range(seqs_max):
            for k in range(pool.held[s].item()):
                refs[table[s][k]] += 1
            for r, parts in enumerate(history[s]):
                for b, v in zip(bufs, parts):
                    assert torch.equal(b[table[s][r // PAGE], r % PAGE].flatten().view(torch.uint8), v.view(torch.uint8))
        assert pool.refs.tolist() == refs
    assert max(len(h) for h in history.values()) > PAGE  # the run went over page borders
