"""Refusals of the operators around the projection, without a GPU: validation compares and aligns the addresses it is
given and never dereferences them, so made-up ones serve."""
import ctypes
import os
import subprocess

import pytest
import torch

import mla_up_projection_amd as m
from mla_up_projection_amd import binding as bd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BASE = 0x7F0000000000
OK, EINVAL, EROPE, EALIAS, EUNSUP, EDEVICE, EWS = range(7)
NAN, INF = float("nan"), float("inf")


def addr(i, off=0):
    return BASE + i * (1 << 36) + off


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bd.LIB_PATH):
        from mla_up_projection_amd import build
        build.build()
    return bd.lib()


def test_struct_layouts_match_c(tmp_path):
    structs = [bd.mla_rmsnorm_args, bd.mla_rmsnorm_bwd_args, bd.mla_qup_i8_args, bd.mla_attn_spans_args, bd.mla_attn_rows,
               bd.mla_attn_args, bd.mla_attn_bwd_args]
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
            o = getattr(o, p)
        setattr(o, last, v)
    return obj


def norm(**over):
    a = bd.mla_rmsnorm_args(x=addr(1), ld_x=64, res=addr(2), res_dtype=0, gamma=addr(3), gamma_dtype=0, eps=1e-6, T=5, K=64,
                            h=addr(4), rstd=addr(5), y=addr(6), q_dtype=2, codes=addr(7), scales=addr(8))
    return put(a, over)


@pytest.mark.parametrize("over, status", [
    (dict(T=-1), EINVAL), (dict(T=1 << 31), EINVAL), (dict(K=0), EINVAL), (dict(K=60), EINVAL), (dict(K=32776, ld_x=32776), EINVAL),
    (dict(K=40, ld_x=40), EINVAL), (dict(ld_x=56), EINVAL), (dict(ld_x=68), EINVAL), (dict(eps=-1.0), EINVAL), (dict(eps=NAN), EINVAL),
    (dict(eps=INF), EINVAL), (dict(x=None), EINVAL), (dict(x=addr(1, 8)), EINVAL), (dict(res_dtype=2), EINVAL),
    (dict(gamma_dtype=3), EINVAL), (dict(res=None), EINVAL), (dict(q_dtype=0), EINVAL), (dict(scales=None), EINVAL),
    (dict(codes=None), EINVAL), (dict(h=None, rstd=None, y=None, codes=None, scales=None), EINVAL), (dict(codes=addr(7, 4)), EINVAL),
    (dict(q_dtype=3, scales=addr(8, 2)), EINVAL), (dict(y=addr(1)), EALIAS), (dict(h=addr(2)), EALIAS), (dict(y=addr(6), h=addr(6, 16)), EALIAS),
    (dict(rstd=addr(3)), EALIAS), (dict(T=0, x=None), OK), (dict(T=1 << 22), EUNSUP),
])
def test_norm(L, over, status):
    assert L.mla_rmsnorm_fwd(ctypes.byref(norm(**over)), None) == status


def norm_bwd(**over):
    a = bd.mla_rmsnorm_bwd_args(dy=addr(1), h=addr(2), h_dtype=1, ld_h=64, rstd=addr(3), gamma=addr(4), gamma_dtype=1, dh=addr(5),
                                T=5, K=64, dx=addr(6), dres=addr(7), dgamma=addr(8), workspace=addr(9), workspace_bytes=1 << 20)
    return put(a, over)


@pytest.mark.parametrize("over, status", [
    (dict(K=4), EINVAL), (dict(ld_h=63), EINVAL), (dict(h_dtype=2), EINVAL), (dict(gamma_dtype=2), EINVAL), (dict(dy=None), EINVAL),
    (dict(rstd=None), EINVAL), (dict(dx=None, dres=None, dgamma=None), EINVAL), (dict(workspace=None), EWS), (dict(workspace_bytes=5 * 256 - 1), EWS),
    (dict(workspace=addr(9, 16)), EINVAL), (dict(dx=addr(1)), EALIAS), (dict(dres=addr(2)), EALIAS), (dict(workspace=addr(8)), EALIAS),
    (dict(dx=addr(6, 2)), EINVAL), (dict(dgamma=None, T=0), OK),
])
def test_norm_backward(L, over, status):
    assert L.mla_rmsnorm_bwd(ctypes.byref(norm_bwd(**over)), None) == status


def test_norm_workspace(L):
    assert L.mla_rmsnorm_bwd_workspace_size(5, 64) == 5 * 64 * 4
    assert L.mla_rmsnorm_bwd_workspace_size(0, 64) == 64 * 4
    assert L.mla_rmsnorm_bwd_workspace_size(-1, 64) == 0 and L.mla_rmsnorm_bwd_workspace_size(5, 12) == 0


@pytest.mark.parametrize("args, status", [
    ((addr(1), 2, 5, 64, 64, addr(2), addr(3)), EINVAL), ((addr(1), 0, -1, 64, 64, addr(2), addr(3)), EINVAL),
    ((addr(1), 0, 5, 60, 64, addr(2), addr(3)), EINVAL), ((addr(1), 0, 5, 64, 56, addr(2), addr(3)), EINVAL),
    ((addr(1), 0, 1 << 24, 64, 64, addr(2), addr(3)), EINVAL), ((None, 0, 5, 64, 64, addr(2), addr(3)), EINVAL),
    ((addr(1), 0, 5, 64, 68, addr(2), addr(3)), EINVAL), ((addr(1), 0, 5, 64, 64, addr(2, 4), addr(3)), EINVAL),
    ((addr(1), 0, 5, 64, 64, addr(1), addr(3)), EALIAS), ((addr(1), 0, 5, 64, 64, addr(2), addr(2)), EALIAS),
    ((None, 0, 0, 64, 64, None, None), OK),
])
def test_int8_quantize(L, args, status):
    assert L.int8_quantize(*args, None) == status


def i8(**over):
    a = bd.mla_qup_i8_args(x=addr(1), x_scales=addr(2), w=addr(3), w_scales=addr(4), K=128, H=2, d_nope=32, d_rope=32, out_dtype=0,
                           out=addr(5))
    put(a, dict(tokens__fmt=0, tokens__B=1, tokens__S=7, tokens__T=7, rope__cos=addr(6), rope__sin=addr(7), rope__rows=7, rope__pairs=16))
    return put(a, over)


@pytest.mark.parametrize("over, status", [
    (dict(K=96), EINVAL), (dict(K=65600), EINVAL), (dict(K=0), EINVAL), (dict(H=0), EINVAL), (dict(d_nope=33), EINVAL), (dict(d_rope=16), EINVAL),
    (dict(tokens__T=8), EINVAL), (dict(rope__rows=6), EROPE), (dict(rope__pairs=15), EROPE), (dict(rope__cos=None), EINVAL),
    (dict(rope__rows=0, positions=addr(8)), EROPE), (dict(out_dtype=1), EINVAL), (dict(out_dtype=2), EINVAL), (dict(out_scales=addr(9)), EINVAL),
    (dict(x=None), EINVAL), (dict(x_scales=None), EINVAL), (dict(w=addr(3, 8)), EINVAL), (dict(w_scales=addr(4, 2)), EINVAL), (dict(bias=addr(8, 4)), EINVAL),
    (dict(out=addr(1)), EALIAS), (dict(out=addr(6)), EALIAS), (dict(positions=addr(5)), EALIAS),
    (dict(H=1 << 23), EUNSUP), (dict(K=65536, H=2048), EUNSUP), (dict(tokens__T=0, tokens__S=1, tokens__B=1), EINVAL),
])
def test_i8(L, over, status):
    assert L.mla_qup_fwd_i8(ctypes.byref(i8(**over)), None) == status


def spans(**over):
    return put(bd.mla_attn_spans_args(spans=addr(1), at=addr(2), B=1, Sq=10, Sk=10, cu_q=addr(3), cu_k=addr(4), nseq=2, prefix=addr(5),
                                      causal=1, window=0), over)


@pytest.mark.parametrize("over, status", [
    (dict(B=0), EINVAL), (dict(B=2), EINVAL), (dict(Sq=-1), EINVAL), (dict(Sk=(1 << 27) + 1), EINVAL), (dict(nseq=0), EINVAL), (dict(window=-1), EINVAL),
    (dict(causal=2), EINVAL), (dict(len_q=addr(6)), EINVAL), (dict(cu_q=None), EINVAL), (dict(cu_k=None, Sk=11), EINVAL), (dict(spans=None), EINVAL),
    (dict(spans=addr(1, 4)), EINVAL), (dict(at=addr(2, 2)), EINVAL), (dict(at=addr(1, 8)), EALIAS), (dict(spans=addr(3)), EALIAS), (dict(Sq=0), OK),
])
def test_spans(L, over, status):
    assert L.mla_attn_spans(ctypes.byref(spans(**over)), None) == status


def rows(i, B, H, S, d):
    return bd.mla_attn_rows(addr(i), H * S * d, S * d, d)


def attn(**over):
    B, H, hk, Sq, Sk, dk, dv = 2, 4, 2, 100, 50, 64, 32
    a = bd.mla_attn_args(q=rows(1, B, H, Sq, dk), k=rows(2, B, hk, Sk, dk), v=rows(3, B, hk, Sk, dv), out=rows(4, B, H, Sq, dv),
                         lse=addr(5), B=B, H=H, H_kv=hk, Sq=Sq, Sk=Sk, d_k=dk, d_v=dv, scale=0.1, cap=0.0, slopes=addr(6), spans=addr(7),
                         at=addr(8), workspace=addr(9), workspace_bytes=1 << 30)
    return put(a, over)


BAD_ATTN = [
    (dict(B=0), EINVAL), (dict(H=3), EINVAL), (dict(H_kv=0), EINVAL), (dict(Sq=-1), EINVAL), (dict(Sk=-1), EINVAL), (dict(Sq=(1 << 27) + 1), EINVAL),
    (dict(d_k=60), EINVAL), (dict(d_v=0), EINVAL), (dict(d_k=200), EUNSUP), (dict(d_v=136), EUNSUP), (dict(scale=NAN), EINVAL), (dict(scale=INF), EINVAL),
    (dict(scale=3e38), EINVAL), (dict(cap=-1.0), EINVAL), (dict(cap=NAN), EINVAL), (dict(cap=1e-38, scale=100.0), EINVAL), (dict(q__p=None), EINVAL),
    (dict(k__p=addr(2, 8)), EINVAL), (dict(q__stride_s=68), EINVAL), (dict(q__stride_h=-8), EINVAL), (dict(v__stride_s=1 << 22), EUNSUP),
    (dict(lse=addr(5, 2)), EINVAL), (dict(spans=addr(7, 4)), EINVAL), (dict(Sq=1 << 24, H=32, H_kv=2), EUNSUP),
]


@pytest.mark.parametrize("over, status", BAD_ATTN + [
    (dict(out__stride_s=24), EINVAL), (dict(out__stride_h=0), EINVAL), (dict(out__stride_b=100 * 32), EINVAL), (dict(out__p=addr(1)), EALIAS),
    (dict(q__p=addr(4)), EALIAS), (dict(lse=addr(7)), EALIAS),
    (dict(Sq=1, Sk=9000, workspace=None), EWS), (dict(Sq=1, Sk=9000, workspace=addr(9, 8)), EINVAL), (dict(Sq=1, Sk=9000, workspace=addr(4)), EALIAS),
    (dict(Sq=0, q__p=None, out__p=None), OK),
])
def test_attention(L, over, status):
    assert L.mla_attn_fwd(ctypes.byref(attn(**over)), None) == status


def attn_bwd(**over):
    B, H, hk, Sq, Sk, dk, dv = 2, 4, 2, 100, 50, 64, 32
    a = bd.mla_attn_bwd_args(fwd=attn(workspace=None, workspace_bytes=0), dout=rows(10, B, H, Sq, dv), dq=rows(11, B, H, Sq, dk),
                             dk=rows(12, B, hk, Sk, dk), dv=rows(13, B, hk, Sk, dv), workspace=addr(14), workspace_bytes=1 << 30)
    return put(a, over)


@pytest.mark.parametrize("over, status", [({"fwd__" + k: v for k, v in o.items()}, s) for o, s in BAD_ATTN] + [
    (dict(fwd__lse=None), EINVAL), (dict(dout__p=None), EINVAL), (dict(dq__stride_s=32), EINVAL), (dict(dk__stride_h=0), EINVAL),
    (dict(dv__stride_s=8), EINVAL), (dict(workspace=None), EWS), (dict(workspace_bytes=100), EWS), (dict(workspace=addr(14, 128)), EINVAL),
    (dict(dq__p=addr(1)), EALIAS), (dict(dk__p=addr(12), dv__p=addr(12, 64)), EALIAS), (dict(dq__p=addr(10)), EALIAS), (dict(workspace=addr(13)), EALIAS),
])
def test_attention_backward(L, over, status):
    assert L.mla_attn_bwd(ctypes.byref(attn_bwd(**over)), None) == status


@pytest.mark.parametrize("off, status", [(64, EDEVICE), (72, EALIAS), (56, EALIAS)])
def test_slices_of_the_same_rows_may_take_two_gradients(L, off, status):
    """Key and value gradients beside each other in rows of 64 + 32: no aliasing (made-up addresses then end at the
    launch, without a device)."""
    wide = lambda o: bd.mla_attn_rows(addr(12, 2 * o), 50 * 2 * 96, 96, 2 * 96)  # noqa: E731
    if torch.cuda.is_available() and status == EDEVICE:
        pytest.skip("the call would be accepted")
    assert L.mla_attn_bwd(ctypes.byref(attn_bwd(dk=wide(0), dv=wide(off))), None) == status


def test_workspaces(L):
    assert L.mla_attn_fwd_workspace_size(ctypes.byref(attn())) == 0
    assert L.mla_attn_fwd_workspace_size(ctypes.byref(attn(Sq=1, Sk=9000))) > 0
    assert L.mla_attn_fwd_workspace_size(ctypes.byref(attn(d_k=200))) == 0
    assert L.mla_attn_bwd_workspace_size(ctypes.byref(attn_bwd(fwd__d_k=200))) == 0
    assert L.mla_attn_bwd_workspace_size(ctypes.byref(attn_bwd())) > 0
    for f in (L.mla_rmsnorm_fwd, L.mla_rmsnorm_bwd, L.mla_qup_fwd_i8, L.mla_attn_spans, L.mla_attn_fwd, L.mla_attn_bwd):
        assert f(None, None) == EINVAL


def test_binding_refuses_before_the_library_is_called(monkeypatch):
    monkeypatch.setattr(bd, "DEVICE_TYPE", "cpu")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="contiguous rows"):
        m.mla_rmsnorm_fwd(bf(64, 8).t(), None, y=bf(8, 64))
    with pytest.raises(ValueError, match="elements"):
        m.mla_rmsnorm_fwd(bf(8, 64), bf(63), y=bf(8, 64))
    with pytest.raises(ValueError, match="dtype"):
        m.mla_rmsnorm_fwd(bf(8, 64), None, y=torch.zeros(8, 64))
    with pytest.raises(ValueError, match="dtype"):
        m.mla_rmsnorm_fwd(bf(8, 64), None, codes=torch.zeros(8, 64, dtype=torch.int8), scales=torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="dtype"):
        m.mla_qup_fwd_i8(bf(8, 64), torch.zeros(8), torch.zeros(64, 64, dtype=torch.int8), torch.zeros(64), bf(1, 1, 8, 64), H=1, d_nope=64, d_rope=0)
    q, k, v = bf(1, 4, 9, 64), bf(1, 2, 9, 64), bf(1, 2, 9, 32)
    with pytest.raises(ValueError, match="out must be"):
        m.mla_attn_fwd(q, k, v, bf(1, 4, 9, 64), scale=1.0)
    with pytest.raises(ValueError, match="k must be"):
        m.mla_attn_fwd(q, bf(1, 2, 8, 64), v, bf(1, 4, 9, 32), scale=1.0)
    with pytest.raises(ValueError, match="dense"):
        m.mla_attn_fwd(q, k, v, bf(1, 4, 32, 9).transpose(2, 3), scale=1.0)
    with pytest.raises(ValueError, match="spans"):
        m.mla_attn_fwd(q, k, v, bf(1, 4, 9, 32), scale=1.0, spans=torch.zeros(1, 8, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="spans must be"):
        m.mla_attn_spans(torch.zeros(9, 2, dtype=torch.int32), Sk=9)
    with pytest.raises(ValueError, match="cu_k without"):
        m.mla_attn_spans(torch.zeros(1, 9, 2, dtype=torch.int32), Sk=9, cu_k=torch.zeros(2, dtype=torch.int32))
