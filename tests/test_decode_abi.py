"""Refusals of the decode-side entry points, without a GPU: validation compares
and aligns the addresses it is given and never dereferences them, so made-up
ones serve. Every listed call must return its status before anything is
enqueued."""
import ctypes
import os
import subprocess

import pytest
import torch

import mla_up_projection_amd as m
from mla_up_projection_amd import binding as bd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7F0000000000


def addr(i, off=0):
    return BASE + i * (1 << 36) + off


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bd.LIB_PATH):
        from mla_up_projection_amd import build
        build.build()
    return bd.lib()


def test_struct_layouts_match_c(tmp_path):
    structs = [bd.mla_pool, bd.mla_qup_w4_args, bd.mla_kv_paged_args, bd.mla_tree_attn_args]
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "mla_qup.h"', "int main(void){"]
    for s in structs:
        lines.append(f'printf("{s.__name__} %zu\\n", sizeof({s.__name__}));')
        lines += [f'printf("{s.__name__}.{f} %zu\\n", offsetof({s.__name__}, {f}));' for f, _ in s._fields_]
    (tmp_path / "l.c").write_text("\n".join(lines + ["return 0;}"]))
    exe = tmp_path / "l"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o", str(exe)], check=True)
    out = dict(x.split() for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for s in structs:
        assert int(out[s.__name__]) == ctypes.sizeof(s)
        for f, _ in s._fields_:
            assert int(out[f"{s.__name__}.{f}"]) == getattr(s, f).offset, (s.__name__, f)


def put(obj, over):
    for k, v in over.items():
        *path, last = k.split("__")
        o = obj
        for p in path:
            o = o[int(p)] if p.isdigit() else getattr(o, p)
        if last.isdigit():
            o[int(last)] = v
        else:
            setattr(o, last, v)
    return obj


def pool(**over):
    p = bd.mla_pool()
    p.num_pages, p.page_size, p.max_seqs, p.max_pages = 100, 64, 8, 20
    p.refs, p.table, p.lens, p.held = addr(1), addr(2), addr(3), addr(4)
    p.nbuf, p.buf[0], p.page_bytes[0] = 1, addr(5), 64 * 1152
    return put(p, over)


BAD_POOLS = [dict(num_pages=0), dict(num_pages=(1 << 20) + 1), dict(page_size=0), dict(page_size=4097), dict(max_seqs=0),
             dict(max_pages=0), dict(max_pages=1 << 26), dict(refs=0), dict(table=addr(2, 2)), dict(lens=0), dict(held=0),
             dict(nbuf=0), dict(nbuf=5), dict(nbuf=2), dict(buf__0=addr(5, 8)), dict(page_bytes__0=0),
             dict(page_bytes__0=64 * 1152 + 1), dict(page_bytes__0=1 << 41)]
WS = 1 << 20


def calls(L):
    """name -> a call of it on a pool, with every other argument valid."""
    r = ctypes.byref
    return {
        "copy": lambda p: L.mla_pages_copy(r(p), r(p), addr(10), addr(11), 3, None),
        "reserve": lambda p: L.mla_pages_reserve(r(p), addr(10), addr(11), 3, addr(12), addr(13), WS, None),
        "fork": lambda p: L.mla_pages_fork(r(p), addr(10), addr(11), 3, None),
        "free": lambda p: L.mla_pages_free(r(p), addr(10), None, 3, None),
        "compact": lambda p: L.mla_pages_compact(r(p), addr(12), addr(13), WS, None),
        "accept": lambda p: L.mla_draft_accept(r(p), addr(10), addr(11), addr(12), 3, 5, None),
    }


@pytest.mark.parametrize("over", BAD_POOLS, ids=str)
def test_invalid_pools(L, over):
    p = pool(**over)
    for name, call in calls(L).items():
        assert call(p) == bd.MLA_EINVAL, name
    assert L.mla_pages_workspace_size(ctypes.byref(p)) == 0
    assert L.mla_tree_attention(ctypes.byref(attn(pool=p)), None) == bd.MLA_EINVAL
    assert L.mla_kv_rope_paged(ctypes.byref(paged(pool=p)), None) == bd.MLA_EINVAL
    assert L.mla_pages_fork(None, addr(10), addr(11), 3, None) == bd.MLA_EINVAL


@pytest.mark.parametrize("over", [dict(table=addr(1)), dict(lens=addr(2, 16)), dict(held=addr(3)), dict(refs=addr(2, 8))],
                         ids=str)
def test_arrays_of_a_pool_that_overlap(L, over):
    p = pool(**over)
    for name, call in calls(L).items():
        if name != "copy":  # copies buffers alone
            assert call(p) == bd.MLA_EALIAS, name


def test_lists_and_workspaces(L):
    r, p = ctypes.byref, pool()
    assert L.mla_pages_workspace_size(r(p)) == 4 * (3 * 1024 + 32 + 200)
    E = bd.MLA_EINVAL
    for n in (-1, 1025):
        assert L.mla_pages_reserve(r(p), addr(10), addr(11), n, addr(12), addr(13), WS, None) == E
        assert L.mla_pages_fork(r(p), addr(10), addr(11), n, None) == E
        assert L.mla_pages_free(r(p), addr(10), None, n, None) == E
        assert L.mla_draft_accept(r(p), addr(10), addr(11), addr(12), n, 5, None) == E
    assert L.mla_pages_copy(r(p), r(p), addr(10), addr(11), -1, None) == E
    assert L.mla_pages_copy(r(p), r(p), addr(10), addr(11), 65537, None) == E
    assert L.mla_pages_copy(r(p), r(p), 0, addr(11), 1, None) == E
    assert L.mla_pages_copy(r(p), r(p), addr(10), addr(11, 2), 1, None) == E
    assert L.mla_pages_copy(r(p), r(p), addr(5, 64), addr(11), 1, None) == bd.MLA_EALIAS
    assert L.mla_pages_copy(r(p), r(pool(buf__0=addr(6), page_size=32, page_bytes__0=64 * 1152)), addr(10), addr(11), 1, None) == E
    assert L.mla_pages_copy(r(p), r(pool(buf__0=addr(6), page_bytes__0=64 * 576)), addr(10), addr(11), 1, None) == E
    assert L.mla_pages_copy(r(p), r(pool(buf__0=addr(5, 4096))), addr(10), addr(11), 1, None) == bd.MLA_EALIAS
    assert L.mla_pages_copy(r(p), r(pool(num_pages=50)), addr(10), addr(11), 1, None) == bd.MLA_EALIAS
    assert L.mla_pages_reserve(r(p), 0, addr(11), 1, addr(12), addr(13), WS, None) == E
    assert L.mla_pages_reserve(r(p), addr(10), 0, 1, addr(12), addr(13), WS, None) == E
    assert L.mla_pages_reserve(r(p), addr(10), addr(11), 1, 0, addr(13), WS, None) == E
    assert L.mla_pages_reserve(r(p), addr(10), addr(11), 1, addr(12), 0, WS, None) == bd.MLA_EWORKSPACE
    assert L.mla_pages_reserve(r(p), addr(10), addr(11), 1, addr(12), addr(13), 13215, None) == bd.MLA_EWORKSPACE
    assert L.mla_pages_reserve(r(p), addr(10), addr(11), 1, addr(12), addr(13, 8), WS, None) == E
    assert L.mla_pages_reserve(r(p), addr(10), addr(3), 1, addr(12), addr(13), WS, None) == bd.MLA_EALIAS
    assert L.mla_pages_reserve(r(p), addr(10), addr(11), 1, addr(4, 4), addr(13), WS, None) == bd.MLA_EALIAS
    assert L.mla_pages_compact(r(p), 0, addr(13), WS, None) == E
    assert L.mla_pages_compact(r(p), addr(12), 0, 0, None) == bd.MLA_EWORKSPACE
    assert L.mla_pages_compact(r(p), addr(13, 64), addr(13), WS, None) == bd.MLA_EALIAS
    assert L.mla_pages_free(r(p), addr(10), addr(11, 1), 1, None) == E
    assert L.mla_pages_free(r(p), addr(10), addr(3), 1, None) == bd.MLA_EALIAS
    assert L.mla_pages_fork(r(p), addr(2), addr(11), 1, None) == bd.MLA_EALIAS
    assert L.mla_draft_accept(r(p), addr(10), addr(11), addr(12), 1, 0, None) == E
    assert L.mla_draft_accept(r(p), addr(10), 0, addr(12), 1, 1, None) == E
    assert L.mla_draft_accept(r(p), addr(10), addr(5, 128), addr(12), 1, 1, None) == bd.MLA_EALIAS


def w4(**over):
    a = bd.mla_qup_w4_args()
    a.x, a.w, a.w_scales, a.K = addr(1), addr(2), addr(3), 1536
    a.H, a.d_nope, a.d_rope = 8, 128, 64
    a.tokens.fmt, a.tokens.B, a.tokens.S, a.tokens.T = bd.FMT_BSHD, 1, 7, 7
    a.rope.cos, a.rope.sin, a.rope.rows, a.rope.pairs = addr(4), addr(5), 7, 32
    a.out_dtype, a.out, a.out_scales = bd.DTYPE_MXFP8, addr(6), addr(7)
    return put(a, over)


@pytest.mark.parametrize("over,code", [
    (dict(K=0), 1), (dict(K=48), 1), (dict(H=0), 1), (dict(d_nope=100), 1), (dict(d_rope=3), 1), (dict(x=0), 1),
    (dict(w=0), 1), (dict(w_scales=0), 1), (dict(out=0), 1), (dict(out_scales=0), 1), (dict(x=addr(1, 8)), 1),
    (dict(w=addr(2, 4)), 1), (dict(out=addr(6, 2)), 1), (dict(bias=addr(8, 1)), 1), (dict(positions=addr(8, 2)), 1),
    (dict(out_dtype=1), 1), (dict(tokens__S=6), 1), (dict(tokens__fmt=3), 1), (dict(rope__cos=0), 1),
    (dict(rope__pairs=31), 2), (dict(rope__rows=6), 2), (dict(rope__rows=0, positions=addr(8)), 2),
    (dict(out=addr(1, 64)), 3), (dict(out=addr(2)), 3), (dict(out_scales=addr(6)), 3), (dict(out=addr(4)), 3),
    (dict(positions=addr(6)), 3), (dict(tokens__T=0, tokens__S=0), 1),
], ids=str)
def test_w4_refusals(L, over, code):
    assert L.mla_qup_fwd_w4(ctypes.byref(w4(**over)), None) == code
    assert L.mla_qup_fwd_w4(None, None) == bd.MLA_EINVAL


@pytest.mark.parametrize("args,code", [
    ((addr(1), 2, 4, 64, 64, addr(2), addr(3)), 1), ((addr(1), 0, -1, 64, 64, addr(2), addr(3)), 1),
    ((addr(1), 0, 4, 48, 64, addr(2), addr(3)), 1), ((addr(1), 0, 4, 64, 63, addr(2), addr(3)), 1),
    ((0, 0, 4, 64, 64, addr(2), addr(3)), 1), ((addr(1, 8), 0, 4, 64, 64, addr(2), addr(3)), 1),
    ((addr(1), 0, 4, 64, 68, addr(2), addr(3)), 1), ((addr(1), 0, 4, 64, 64, addr(2, 2), addr(3)), 1),
    ((addr(1), 0, 1 << 32, 64, 64, addr(2), addr(3)), 1), ((addr(1), 0, 4, 64, 1 << 62, addr(2), addr(3)), 1),
    ((addr(1), 0, 4, 64, 64, addr(1, 16), addr(3)), 3), ((addr(1), 0, 4, 64, 64, addr(2), addr(2, 8)), 3),
    ((0, 0, 0, 64, 64, 0, 0), 0),
], ids=str)
def test_mxfp4_refusals(L, args, code):
    assert L.mxfp4_quantize(*args, None) == code


def paged(**over):
    a = bd.mla_kv_paged_args()
    p = over.pop("pool", None) or pool()
    a.kv, a.k_pe, a.H, a.d_nope, a.d_rope, a.d_v, a.T = addr(11), addr(12), 1, 512, 64, 0, 9
    a.seqs, a.cu_q, a.nseq, a.max_q = addr(13), addr(14), 2, 5
    a.rope.cos, a.rope.sin, a.rope.rows, a.rope.pairs = addr(15), addr(16), 100, 32
    a.cache_dtype, a.pool = bd.DTYPE_BF16, ctypes.pointer(p)
    return put(a, over)


@pytest.mark.parametrize("over,code", [
    (dict(H=0), 1), (dict(H=2), 1), (dict(d_nope=510), 1), (dict(d_nope=504), 1), (dict(d_rope=264), 1), (dict(d_v=64), 1),
    (dict(T=-1), 1), (dict(T=1 << 31), 1), (dict(nseq=-1), 1), (dict(nseq=1025), 1), (dict(seqs=0), 1), (dict(cu_q=0), 1),
    (dict(cu_q=addr(14, 2)), 1), (dict(max_q=0), 1), (dict(cache_dtype=1), 1), (dict(cache_dtype=2), 1), (dict(kv=0), 1),
    (dict(k_pe=addr(12, 8)), 1), (dict(positions=addr(17, 1)), 1), (dict(rope__cos=0), 1), (dict(rope__pairs=16), 2),
    (dict(rope__rows=0), 2), (dict(kv=addr(5, 64)), 3), (dict(k_pe=addr(5)), 3), (dict(rope__cos=addr(5)), 3),
    (dict(T=0), 0), (dict(nseq=0), 0),
], ids=str)
def test_paged_refusals(L, over, code):
    assert L.mla_kv_rope_paged(ctypes.byref(paged(**over)), None) == code
    assert L.mla_kv_rope_paged(None, None) == bd.MLA_EINVAL


def attn(**over):
    a = bd.mla_tree_attn_args()
    p = over.pop("pool", None) or pool()
    a.q, a.q_stride_t, a.q_stride_h = addr(11), 128 * 576, 576
    a.out, a.out_stride_t, a.out_stride_h = addr(12), 128 * 512, 512
    a.lse, a.T, a.H, a.H_kv, a.d_k, a.d_v, a.scale = addr(13), 9, 128, 1, 576, 512, 0.07
    a.seqs, a.cu_q, a.nseq, a.max_q, a.max_len = addr(14), addr(15), 2, 5, 5000
    a.mask, a.mask_words = addr(16), 1
    a.cache_dtype, a.pool = bd.DTYPE_BF16, ctypes.pointer(p)
    a.workspace, a.workspace_bytes = addr(17), 1 << 36
    return put(a, over)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(H_kv=0), 1), (dict(H_kv=3), 1), (dict(H_kv=2), 1), (dict(nseq=-1), 1),
    (dict(nseq=65536), 1), (dict(max_q=0), 1), (dict(max_len=0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(cache_dtype=1), 1), (dict(d_k=512), 4), (dict(d_v=256), 4), (dict(d_k=0), 1),
    (dict(q=0), 1), (dict(out=0), 1), (dict(seqs=0), 1), (dict(cu_q=0), 1), (dict(q=addr(11, 8)), 1),
    (dict(out=addr(12, 4)), 1), (dict(lse=addr(13, 2)), 1), (dict(mask=addr(16, 2)), 1), (dict(q_stride_t=4), 1),
    (dict(q_stride_h=-576), 1), (dict(out_stride_h=500), 1), (dict(out_stride_t=127 * 512), 1), (dict(mask_words=0), 1),
    (dict(max_q=33), 1), (dict(workspace=0), 6), (dict(workspace_bytes=100), 6), (dict(workspace=addr(17, 16)), 1),
    (dict(max_q=1 << 30), 1), (dict(nseq=65535, max_q=1 << 20, mask=0), 1),
    (dict(out=addr(11, 64)), 3), (dict(out=addr(5)), 3), (dict(lse=addr(12)), 3), (dict(lse=addr(2)), 3),
    (dict(workspace=addr(5, 256)), 3), (dict(mask=addr(12)), 3), (dict(T=0), 0), (dict(nseq=0), 0),
], ids=str)
def test_attention_refusals(L, over, code):
    assert L.mla_tree_attention(ctypes.byref(attn(**over)), None) == code
    assert L.mla_tree_attention(None, None) == bd.MLA_EINVAL


def test_attention_limits(L):
    size = lambda **kw: L.mla_tree_attention_workspace_size(ctypes.byref(attn(**kw)))  # noqa: E731
    assert size(nseq=1024, max_q=64, mask_words=2) > 0  # 2^16 row tiles of 128
    assert size(nseq=8192, max_q=63, mask_words=2) > 0
    assert size(nseq=8192, max_q=64, mask_words=2) == 0  # 2^21 groups of 32 rows
    assert size(nseq=4096, max_q=64, mask_words=2, max_len=(1 << 31) - 1) == 0  # 2^44 steps
    assert size(max_len=(1 << 31) - 1) > 0
    heads = pool(nbuf=2, buf__1=addr(6), page_bytes__0=64 * 2 * 384, page_bytes__1=64 * 2 * 256)
    assert size(pool=heads, H=2, H_kv=2, d_k=192, d_v=128, q_stride_h=192, q_stride_t=384, out_stride_h=128,
                out_stride_t=256, max_len=(1 << 31) - 1) > 0
    a = attn(nseq=8192, max_q=64, mask_words=2)
    assert L.mla_tree_attention(ctypes.byref(a), None) == bd.MLA_EINVAL


def test_cache_must_fit_the_widths(L):
    two = dict(nbuf=2, buf__1=addr(6), page_bytes__1=64 * 1024)
    assert L.mla_tree_attention(ctypes.byref(attn(pool=pool(**two))), None) == bd.MLA_EUNSUPPORTED  # (576, 512) with values
    heads = dict(nbuf=2, buf__1=addr(6), page_bytes__0=64 * 2 * 384, page_bytes__1=64 * 2 * 256)
    a = dict(H=2, H_kv=2, d_k=192, d_v=128, q_stride_h=192, q_stride_t=384, out_stride_h=128, out_stride_t=256)
    assert L.mla_tree_attention_workspace_size(ctypes.byref(attn(pool=pool(**heads), **a))) > 0
    assert L.mla_tree_attention(ctypes.byref(attn(pool=pool(**(heads | dict(page_bytes__1=64 * 2 * 128))), **a)), None) == 1
    mx = dict(nbuf=2, buf__1=addr(6), page_bytes__0=64 * 576, page_bytes__1=64 * 18)
    assert L.mla_tree_attention_workspace_size(ctypes.byref(attn(pool=pool(**mx), cache_dtype=2))) > 0
    assert L.mla_tree_attention(ctypes.byref(attn(pool=pool(**(mx | dict(page_bytes__1=64 * 36))), cache_dtype=2)), None) == 1
    odd = mx | dict(num_pages=99, page_size=7, page_bytes__0=7 * 576, page_bytes__1=7 * 18)  # an odd number of rows
    assert L.mla_tree_attention(ctypes.byref(attn(pool=pool(**odd), cache_dtype=2)), None) == 1


def test_bindings_refuse_host_tensors_and_wrong_sizes(monkeypatch):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    buf = torch.zeros(10, 16, 1, 576, dtype=torch.bfloat16)
    good = dict(refs=i(10), table=i(3, 4), lens=i(3), held=i(3))
    with pytest.raises(ValueError, match="not on the GPU"):
        m.PagePool([buf], **good)
    monkeypatch.setattr(bd, "DEVICE_TYPE", "cpu")
    pool_ = m.PagePool([buf], **good)
    assert pool_.latent and pool_.c.page_bytes[0] == 16 * 1152 and pool_.c.num_pages == 10
    for bad in (dict(refs=i(9)), dict(table=i(12)), dict(lens=i(4)), dict(held=torch.zeros(3)), dict(lens=i(6)[::2])):
        with pytest.raises(ValueError):
            m.PagePool([buf], **(good | bad))
    for bufs in ([], [buf] * 5, [buf[0]], [buf, buf[:5]], [buf, buf, buf], [buf.to(torch.uint8)], [buf[:, :, :, ::2]],
                 [buf.to(torch.uint8), torch.zeros(10, 16, 1, 17, dtype=torch.uint8)], [buf.float()]):
        with pytest.raises(ValueError):
            m.PagePool(bufs, **good)
    q, out = torch.zeros(4, 2, 576, dtype=torch.bfloat16), torch.zeros(4, 2, 512, dtype=torch.bfloat16)
    kw = dict(max_q=2, max_len=9, scale=1.0)
    assert m.mla_tree_attention_workspace_size(q, pool_, out, i(2), i(3), **kw) == 0
    for a, b in ((q.float(), out), (q[:3], out), (q[..., :512], out), (q.transpose(1, 2), out), (q[0], out[0])):
        with pytest.raises(ValueError):
            m.binding.make_tree_attn_args(a, pool_, b, i(2), i(3), **kw)
    for over in (dict(lse=torch.zeros(4, 3)), dict(mask=i(3, 1)), dict(mask=i(4)), dict(workspace=torch.zeros(4))):
        with pytest.raises(ValueError):
            m.binding.make_tree_attn_args(q, pool_, out, i(2), i(3), **(kw | over))
    with pytest.raises(ValueError):
        m.binding.make_tree_attn_args(q, pool_, out, i(2), i(2), **kw)
    with pytest.raises(ValueError, match="PagePool"):
        m.mla_pages_fork(None, i(1), i(1))
    with pytest.raises(ValueError):
        m.mla_pages_fork(pool_, i(1), i(2))
    with pytest.raises(ValueError):
        m.mla_draft_accept(pool_, i(2), i(3, 2), i(2))
