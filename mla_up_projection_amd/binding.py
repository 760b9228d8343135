"""Thin ctypes binding of libmlaqup.so (include/mla_qup.h).

Argument marshalling only: every function takes torch tensors that already
live on the GPU, passes their device pointers and the current HIP stream to
the C entry point of the same name, and raises on any status other than
MLA_OK. Nothing here computes any part of the operation, and there is no
fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, Structure, c_char_p, c_double, c_float, c_int32, c_int64, c_size_t, c_void_p

import torch  # imported before the library so both share torch's HIP runtime

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmlaqup.so")

MLA_FWD_FP8_MFMA = 1
(MLA_OK, MLA_EINVAL, MLA_EROPE_TABLE, MLA_EALIAS, MLA_EUNSUPPORTED, MLA_EDEVICE, MLA_EWORKSPACE,
 MLA_ESCRATCH) = range(8)
MLA_BWD_SCRATCH_BYTES = 64 << 20
DTYPE_BF16, DTYPE_FP32, DTYPE_MXFP8 = 0, 1, 2
FMT_BSHD, FMT_SBHD, FMT_THD = 0, 1, 2

FUNCTIONS = ("rope_cache_build", "mxfp8_quantize", "mxfp8_quantize_t", "mla_qup_fwd", "mla_qup_bwd",
             "mla_qup_bwd_workspace_size", "mla_qup_bwd_noalloc", "mla_qup_bwd_mxfp8",
             "mla_qup_bwd_mxfp8_workspace_size", "mla_kv_rope", "mla_status_str",
             "mxfp4_quantize", "mla_qup_fwd_w4", "mla_pages_workspace_size", "mla_pages_copy",
             "mla_pages_reserve", "mla_pages_fork", "mla_pages_free", "mla_pages_compact",
             "mla_draft_accept", "mla_kv_rope_paged", "mla_tree_attention",
             "mla_tree_attention_workspace_size")


class mla_tokens(Structure):
    _fields_ = [("fmt", c_int32), ("B", c_int32), ("S", c_int32), ("T", c_int64),
                ("cu_seqlens", c_void_p), ("nseq", c_int32), ("max_seqlen", c_int32)]


class mla_yarn(Structure):
    _fields_ = [("factor", c_double), ("orig_max_pos", c_int32), ("beta_fast", c_double),
                ("beta_slow", c_double), ("mscale", c_double)]


class mla_rope(Structure):
    _fields_ = [("cos", c_void_p), ("sin", c_void_p), ("rows", c_int32), ("pairs", c_int32)]


class mla_qup_fwd_args(Structure):
    _fields_ = [("x", c_void_p), ("x_scales", c_void_p), ("x_dtype", c_int32),
                ("w", c_void_p), ("w_scales", c_void_p), ("w_dtype", c_int32),
                ("bias", c_void_p), ("K", c_int32), ("H", c_int32), ("d_nope", c_int32),
                ("d_rope", c_int32), ("tokens", mla_tokens), ("rope", mla_rope),
                ("out_dtype", c_int32), ("out", c_void_p), ("out_scales", c_void_p),
                ("flags", c_int32)]


class mla_kv_args(Structure):
    _fields_ = [("kv", c_void_p), ("k_pe", c_void_p), ("H", c_int32), ("d_nope", c_int32),
                ("d_rope", c_int32), ("d_v", c_int32), ("tokens", mla_tokens), ("rope", mla_rope),
                ("out_dtype", c_int32), ("key", c_void_p), ("key_scales", c_void_p),
                ("value", c_void_p), ("value_scales", c_void_p)]


class mla_qup_bwd_args(Structure):
    _fields_ = [("dq", c_void_p), ("x", c_void_p), ("w", c_void_p), ("K", c_int32),
                ("H", c_int32), ("d_nope", c_int32), ("d_rope", c_int32),
                ("tokens", mla_tokens), ("rope", mla_rope), ("dq_pre", c_void_p),
                ("dx", c_void_p), ("dw", c_void_p), ("dw_dtype", c_int32),
                ("use_bias", c_int32), ("db", c_void_p), ("workspace", c_void_p),
                ("workspace_bytes", c_size_t)]


class mla_pool(Structure):
    _fields_ = [("num_pages", c_int32), ("page_size", c_int32), ("max_seqs", c_int32), ("max_pages", c_int32),
                ("refs", c_void_p), ("table", c_void_p), ("lens", c_void_p), ("held", c_void_p),
                ("nbuf", c_int32), ("buf", c_void_p * 4), ("page_bytes", c_int64 * 4)]


class mla_qup_w4_args(Structure):
    _fields_ = [("x", c_void_p), ("w", c_void_p), ("w_scales", c_void_p), ("bias", c_void_p), ("K", c_int32),
                ("H", c_int32), ("d_nope", c_int32), ("d_rope", c_int32), ("tokens", mla_tokens),
                ("positions", c_void_p), ("rope", mla_rope), ("out_dtype", c_int32), ("out", c_void_p),
                ("out_scales", c_void_p)]


class mla_kv_paged_args(Structure):
    _fields_ = [("kv", c_void_p), ("k_pe", c_void_p), ("H", c_int32), ("d_nope", c_int32), ("d_rope", c_int32),
                ("d_v", c_int32), ("T", c_int64), ("seqs", c_void_p), ("cu_q", c_void_p), ("nseq", c_int32),
                ("max_q", c_int32), ("positions", c_void_p), ("rope", mla_rope), ("cache_dtype", c_int32),
                ("pool", POINTER(mla_pool))]


class mla_tree_attn_args(Structure):
    _fields_ = [("q", c_void_p), ("q_stride_t", c_int64), ("q_stride_h", c_int64), ("out", c_void_p),
                ("out_stride_t", c_int64), ("out_stride_h", c_int64), ("lse", c_void_p), ("T", c_int64),
                ("H", c_int32), ("H_kv", c_int32), ("d_k", c_int32), ("d_v", c_int32), ("scale", c_float),
                ("seqs", c_void_p), ("cu_q", c_void_p), ("nseq", c_int32), ("max_q", c_int32),
                ("max_len", c_int32), ("mask", c_void_p), ("mask_words", c_int32), ("cache_dtype", c_int32),
                ("pool", POINTER(mla_pool)), ("workspace", c_void_p), ("workspace_bytes", c_size_t)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmlaqup.so once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mla_up_projection_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.rope_cache_build.argtypes = [c_void_p, c_void_p, c_int32, c_int32, c_double,
                                       POINTER(mla_yarn), c_void_p]
        L.mxfp8_quantize.argtypes = [c_void_p, c_int32, c_int64, c_int64, c_int64, c_void_p,
                                     c_void_p, c_void_p]
        L.mxfp8_quantize_t.argtypes = [c_void_p, c_int64, c_int64, c_int64, c_int64, c_void_p,
                                       c_void_p, c_void_p]
        L.mla_qup_fwd.argtypes = [POINTER(mla_qup_fwd_args), c_void_p]
        L.mla_qup_bwd.argtypes = [POINTER(mla_qup_bwd_args), c_void_p]
        L.mla_qup_bwd_workspace_size.argtypes = [POINTER(mla_qup_bwd_args)]
        L.mla_qup_bwd_workspace_size.restype = c_size_t
        L.mla_qup_bwd_noalloc.argtypes = [POINTER(mla_qup_bwd_args), c_void_p]
        L.mla_qup_bwd_mxfp8.argtypes = [POINTER(mla_qup_bwd_args), c_int32, c_void_p]
        L.mla_qup_bwd_mxfp8_workspace_size.argtypes = [POINTER(mla_qup_bwd_args)]
        L.mla_qup_bwd_mxfp8_workspace_size.restype = c_size_t
        L.mla_kv_rope.argtypes = [POINTER(mla_kv_args), c_void_p]
        L.mla_status_str.argtypes = [c_int32]
        L.mla_status_str.restype = c_char_p
        pool = POINTER(mla_pool)
        L.mxfp4_quantize.argtypes = L.mxfp8_quantize.argtypes
        L.mla_qup_fwd_w4.argtypes = [POINTER(mla_qup_w4_args), c_void_p]
        L.mla_pages_workspace_size.argtypes = [pool]
        L.mla_pages_workspace_size.restype = c_size_t
        L.mla_pages_copy.argtypes = [pool, pool, c_void_p, c_void_p, c_int32, c_void_p]
        L.mla_pages_reserve.argtypes = [pool, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_size_t, c_void_p]
        L.mla_pages_fork.argtypes = [pool, c_void_p, c_void_p, c_int32, c_void_p]
        L.mla_pages_free.argtypes = [pool, c_void_p, c_void_p, c_int32, c_void_p]
        L.mla_pages_compact.argtypes = [pool, c_void_p, c_void_p, c_size_t, c_void_p]
        L.mla_draft_accept.argtypes = [pool, c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_void_p]
        L.mla_kv_rope_paged.argtypes = [POINTER(mla_kv_paged_args), c_void_p]
        L.mla_tree_attention.argtypes = [POINTER(mla_tree_attn_args), c_void_p]
        L.mla_tree_attention_workspace_size.argtypes = [POINTER(mla_tree_attn_args)]
        L.mla_tree_attention_workspace_size.restype = c_size_t
        for f in ("mxfp4_quantize", "mla_qup_fwd_w4", "mla_pages_copy", "mla_pages_reserve", "mla_pages_fork",
                  "mla_pages_free", "mla_pages_compact", "mla_draft_accept", "mla_kv_rope_paged",
                  "mla_tree_attention"):
            getattr(L, f).restype = c_int32
        for f in ("rope_cache_build", "mxfp8_quantize", "mxfp8_quantize_t", "mla_qup_fwd", "mla_qup_bwd",
                  "mla_qup_bwd_noalloc", "mla_qup_bwd_mxfp8", "mla_kv_rope"):
            getattr(L, f).restype = c_int32
        _lib = L
    return _lib


class MlaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {mla_status_str(status)}")
        self.status = status


def mla_status_str(status: int) -> str:
    return lib().mla_status_str(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != MLA_OK:
        raise MlaError(status, where)


# Device type every tensor argument must live on (the library receives raw
# device pointers and cannot tell a host address from a device one).
DEVICE_TYPE = "cuda"

_BF16, _FP32, _U8, _I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


class _Dev:
    """Checks of one call's tensor arguments before any pointer crosses the C
    ABI: every tensor on one device of DEVICE_TYPE, contiguous, of an
    accepted dtype and with the element count the C call will assume."""

    def __init__(self, where: str):
        self.where = where
        self.device = None

    def __call__(self, t, name: str, dtypes, numel=None, min_numel=None) -> int | None:
        if t is None:
            return None
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{self.where}: {name} must be a torch tensor")
        if t.device.type != DEVICE_TYPE:
            raise ValueError(f"{self.where}: {name} is on {t.device}, not on the GPU")
        if self.device is None:
            self.device = t.device
        elif t.device != self.device:
            raise ValueError(f"{self.where}: {name} is on {t.device}, other arguments on {self.device}")
        if t.dtype not in dtypes:
            raise ValueError(f"{self.where}: {name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
        if not t.is_contiguous():
            raise ValueError(f"{self.where}: {name} must be contiguous")
        if numel is not None and t.numel() != numel:
            raise ValueError(f"{self.where}: {name} has {t.numel()} elements, expected {numel}")
        if min_numel is not None and t.numel() < min_numel:
            raise ValueError(f"{self.where}: {name} has {t.numel()} elements, at least {min_numel} needed")
        return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _tokens(chk: _Dev, T, fmt, B, S, cu_seqlens, max_seqlen) -> mla_tokens:
    tk = mla_tokens()
    tk.fmt = fmt
    tk.T = T
    if fmt == FMT_THD:
        tk.B, tk.S = 1, T
        tk.cu_seqlens = chk(cu_seqlens, "cu_seqlens", (_I32,), min_numel=2)
        tk.nseq = cu_seqlens.numel() - 1 if cu_seqlens is not None else 0
        tk.max_seqlen = int(max_seqlen) if max_seqlen is not None else 0
    else:
        tk.B = B
        tk.S = S if S is not None else (T // B if B else 0)
    return tk


def _rope(chk: _Dev, cos, sin, d_rope) -> mla_rope:
    r = mla_rope()
    if cos is not None or sin is not None:
        if cos is None or sin is None or cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError(f"{chk.where}: cos and sin must be two tables of one shape [rows, pairs]")
        r.cos, r.sin = chk(cos, "cos", (_FP32,)), chk(sin, "sin", (_FP32,))
        r.rows = cos.shape[0]
        r.pairs = cos.shape[1]
    return r


def _yarn(yarn) -> mla_yarn | None:
    if yarn is None:
        return None
    y = mla_yarn()
    y.factor, y.orig_max_pos, y.beta_fast, y.beta_slow, y.mscale = yarn
    return y


# ------------------------------------------------------------- entry points --
def rope_cache_build(cos, sin, d_rope: int, base: float = 10000.0, yarn=None, stream=None):
    """Fill fp32 device tables cos/sin [rows, d_rope/2]; yarn = (factor, L,
    beta_fast, beta_slow, mscale) or None."""
    y = _yarn(yarn)
    chk = _Dev("rope_cache_build")
    if cos.dim() != 2 or cos.shape != sin.shape or cos.shape[1] != d_rope // 2:
        raise ValueError("rope_cache_build: cos and sin must both be [rows, d_rope/2]")
    pc, ps = chk(cos, "cos", (_FP32,)), chk(sin, "sin", (_FP32,))
    st = lib().rope_cache_build(pc, ps, cos.shape[0], d_rope, float(base),
                                ctypes.byref(y) if y is not None else None, _stream(stream))
    _check(st, "rope_cache_build")


def mxfp8_quantize(x, codes, scales, stream=None):
    """x [rows, cols] bf16/fp32 (row stride may exceed cols) -> codes uint8
    [rows, cols], scales uint8 [rows, cols/32]."""
    chk = _Dev("mxfp8_quantize")
    if x.dim() != 2 or x.stride(-1) != 1:
        raise ValueError("mxfp8_quantize: x must be 2-D with contiguous rows")
    rows, cols = x.shape
    # x may be a row-strided view: check it as the rows it spans
    span = x.as_strided(((rows - 1) * x.stride(0) + cols,) if rows else (0,), (1,))
    px = chk(span, "x", (_BF16, _FP32))
    dt = DTYPE_FP32 if x.dtype == torch.float32 else DTYPE_BF16
    pc = chk(codes, "codes", (_U8,), numel=rows * cols)
    psc = chk(scales, "scales", (_U8,), numel=rows * cols // 32)
    st = lib().mxfp8_quantize(px if rows else x.data_ptr(), dt, rows, cols, x.stride(0), pc, psc,
                              _stream(stream))
    _check(st, "mxfp8_quantize")


def mxfp8_quantize_t(x, codes_t, scales_t, rows_pad=None, stream=None):
    """x bf16 [rows, cols] (row stride may exceed cols) -> codes_t uint8
    [cols, rows_pad], scales_t uint8 [cols, rows_pad/32]: quantized along the
    columns, stored transposed; rows_pad defaults to codes_t.shape[1]."""
    chk = _Dev("mxfp8_quantize_t")
    if x.dim() != 2 or x.stride(-1) != 1:
        raise ValueError("mxfp8_quantize_t: x must be 2-D with contiguous rows")
    rows, cols = x.shape
    span = x.as_strided(((rows - 1) * x.stride(0) + cols,) if rows else (0,), (1,))
    px = chk(span, "x", (_BF16,))
    rp = codes_t.shape[1] if rows_pad is None else rows_pad
    pc = chk(codes_t, "codes_t", (_U8,), numel=cols * rp)
    psc = chk(scales_t, "scales_t", (_U8,), numel=cols * rp // 32)
    st = lib().mxfp8_quantize_t(px if rows else x.data_ptr(), rows, cols, x.stride(0), rp, pc, psc,
                                _stream(stream))
    _check(st, "mxfp8_quantize_t")


def make_fwd_args(x, w, out, *, H, d_nope, d_rope, cos=None, sin=None, x_scales=None,
                  w_scales=None, bias=None, out_scales=None, fmt=FMT_BSHD, B=1, S=None,
                  cu_seqlens=None, max_seqlen=None, fp8_mfma=False) -> mla_qup_fwd_args:
    chk = _Dev("mla_qup_fwd")
    a = mla_qup_fwd_args()
    a.flags = MLA_FWD_FP8_MFMA if fp8_mfma else 0
    if x.dim() != 2:
        raise ValueError("mla_qup_fwd: x must be [T, K]")
    T, K = x.shape
    N = H * (d_nope + d_rope)
    mx_in = x.dtype == torch.uint8
    a.x = chk(x, "x", (_BF16, _U8))
    a.x_scales = chk(x_scales, "x_scales", (_U8,), numel=T * K // 32)
    a.x_dtype = DTYPE_MXFP8 if mx_in else DTYPE_BF16
    a.w = chk(w, "w", (_BF16, _U8), numel=N * K)
    a.w_scales = chk(w_scales, "w_scales", (_U8,), numel=N * K // 32)
    a.w_dtype = DTYPE_MXFP8 if w.dtype == torch.uint8 else DTYPE_BF16
    a.bias = chk(bias, "bias", (_BF16,), numel=N)
    a.K, a.H, a.d_nope, a.d_rope = K, H, d_nope, d_rope
    a.tokens = _tokens(chk, T, fmt, B, S, cu_seqlens, max_seqlen)
    a.rope = _rope(chk, cos, sin, d_rope)
    a.out_dtype = DTYPE_MXFP8 if out.dtype == torch.uint8 else DTYPE_BF16
    a.out = chk(out, "out", (_BF16, _U8), numel=T * N)
    a.out_scales = chk(out_scales, "out_scales", (_U8,), numel=T * N // 32)
    return a


def mla_qup_fwd(x, w, out, *, stream=None, **kw):
    """Fused forward. x: bf16 [T,K] or uint8 codes with x_scales; w likewise
    [N,K]; out: bf16 or uint8 BHSD [B,H,S,D] (THD: [1,H,T,D]); out_scales
    uint8 [.., D/32] for MXFP8 output. fp8_mfma=True puts MXFP8 operands on
    the scaled FP8 MFMA (faster, lower accumulation precision)."""
    a = make_fwd_args(x, w, out, **kw)
    _check(lib().mla_qup_fwd(ctypes.byref(a), _stream(stream)), "mla_qup_fwd")


def make_bwd_args(dq, x, w, dq_pre, *, H, d_nope, d_rope, cos=None, sin=None, dx=None, dw=None,
                  db=None, use_bias=False, workspace=None, fmt=FMT_BSHD, B=1, S=None,
                  cu_seqlens=None, max_seqlen=None) -> mla_qup_bwd_args:
    chk = _Dev("mla_qup_bwd")
    a = mla_qup_bwd_args()
    if x.dim() != 2:
        raise ValueError("mla_qup_bwd: x must be [T, K]")
    T, K = x.shape
    N = H * (d_nope + d_rope)
    a.dq = chk(dq, "dq", (_BF16,), numel=T * N)
    a.x = chk(x, "x", (_BF16,))
    a.w = chk(w, "w", (_BF16,), numel=N * K)
    a.K, a.H, a.d_nope, a.d_rope = K, H, d_nope, d_rope
    a.tokens = _tokens(chk, T, fmt, B, S, cu_seqlens, max_seqlen)
    a.rope = _rope(chk, cos, sin, d_rope)
    a.dq_pre = chk(dq_pre, "dq_pre", (_BF16,), numel=T * N)
    a.dx = chk(dx, "dx", (_BF16,), numel=T * K)
    a.dw = chk(dw, "dw", (_BF16, _FP32), numel=N * K)
    a.dw_dtype = DTYPE_FP32 if (dw is not None and dw.dtype == torch.float32) else DTYPE_BF16
    a.use_bias = 1 if use_bias else 0
    a.db = chk(db, "db", (_BF16,), numel=N)
    if workspace is not None:
        a.workspace = chk(workspace, "workspace", (_U8,))
        a.workspace_bytes = workspace.numel()
    return a


def mla_qup_bwd_workspace_size(dq, x, w, dq_pre, **kw) -> int:
    kw.pop("stream", None)
    a = make_bwd_args(dq, x, w, dq_pre, **kw)
    return int(lib().mla_qup_bwd_workspace_size(ctypes.byref(a)))


def mla_qup_bwd(dq, x, w, dq_pre, *, stream=None, **kw):
    """Backward. dq bf16 [T,H,D], x bf16 [T,K], w bf16 [N,K] -> dq_pre bf16
    [T,N], dx bf16 [T,K] (optional), dw bf16/fp32 [N,K] (optional), db bf16
    [N] (use_bias). workspace: uint8 device tensor of at least
    mla_qup_bwd_workspace_size() bytes (None if that is 0)."""
    a = make_bwd_args(dq, x, w, dq_pre, **kw)
    _check(lib().mla_qup_bwd(ctypes.byref(a), _stream(stream)), "mla_qup_bwd")


def mla_qup_bwd_noalloc(dq, x, w, dq_pre, *, stream=None, **kw):
    """Backward as mla_qup_bwd, with the partial sums in the library's static
    scratch instead of a workspace (nothing is allocated; calls that overlap on
    one GPU race on that scratch). No workspace argument."""
    if kw.get("workspace") is not None:
        raise ValueError("mla_qup_bwd_noalloc takes no workspace")
    a = make_bwd_args(dq, x, w, dq_pre, **kw)
    _check(lib().mla_qup_bwd_noalloc(ctypes.byref(a), _stream(stream)), "mla_qup_bwd_noalloc")


def mla_qup_bwd_mxfp8_workspace_size(dq, x, w, dq_pre, **kw) -> int:
    kw.pop("stream", None)
    kw.pop("fp8_mfma", None)
    a = make_bwd_args(dq, x, w, dq_pre, **kw)
    return int(lib().mla_qup_bwd_mxfp8_workspace_size(ctypes.byref(a)))


def mla_qup_bwd_mxfp8(dq, x, w, dq_pre, *, fp8_mfma=False, stream=None, **kw):
    """MXFP8 backward: arguments and outputs as mla_qup_bwd; the dx and dw
    products take MXFP8 operands quantized along their reduction axes.
    workspace: at least mla_qup_bwd_mxfp8_workspace_size() bytes."""
    a = make_bwd_args(dq, x, w, dq_pre, **kw)
    _check(lib().mla_qup_bwd_mxfp8(ctypes.byref(a), 1 if fp8_mfma else 0, _stream(stream)),
           "mla_qup_bwd_mxfp8")


def mla_kv_rope(kv, k_pe, key, value, *, H, d_nope, d_rope, d_v, cos=None, sin=None,
                key_scales=None, value_scales=None, fmt=FMT_BSHD, B=1, S=None, cu_seqlens=None,
                max_seqlen=None, stream=None):
    """KV side: kv bf16 [T,H,d_nope+d_v], k_pe bf16 [T,d_rope] -> key [B,H,S,d_nope+d_rope]
    and value [B,H,S,d_v] (BHSD; THD: B=1, S=T), bf16 or uint8 E4M3 codes with
    key_scales / value_scales uint8 [.., D/32]."""
    chk = _Dev("mla_kv_rope")
    a = mla_kv_args()
    T = kv.shape[0]
    Dk, Dv = d_nope + d_rope, d_v
    a.kv = chk(kv, "kv", (_BF16,), numel=T * H * (d_nope + d_v))
    a.k_pe = chk(k_pe, "k_pe", (_BF16,), numel=T * d_rope)
    a.H, a.d_nope, a.d_rope, a.d_v = H, d_nope, d_rope, d_v
    a.tokens = _tokens(chk, T, fmt, B, S, cu_seqlens, max_seqlen)
    a.rope = _rope(chk, cos, sin, d_rope)
    out_dt = key.dtype if key is not None else value.dtype
    a.out_dtype = DTYPE_MXFP8 if out_dt == torch.uint8 else DTYPE_BF16
    a.key = chk(key, "key", (out_dt,), numel=T * H * Dk)
    a.value = chk(value, "value", (out_dt,), numel=T * H * Dv)
    a.key_scales = chk(key_scales, "key_scales", (_U8,), numel=T * H * Dk // 32)
    a.value_scales = chk(value_scales, "value_scales", (_U8,), numel=T * H * Dv // 32)
    _check(lib().mla_kv_rope(ctypes.byref(a), _stream(stream)), "mla_kv_rope")


# ------------------------------------------------------------------ decoding --
def _call(where, device, stream, fn, *args):
    """fn(*args, stream) on `device`: the given stream, or the device's current one, with the device current while
    the call lasts (a launch on the default stream goes to the current device)."""
    index = device.index if device is not None and device.type == "cuda" else None
    if stream is not None:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    elif index is not None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        raw = torch.cuda.current_stream().cuda_stream
    if index is None or index == torch._C._cuda_getDevice():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            status = fn(*args, raw)
    if status:
        raise MlaError(status, where)


def _is(t, dtype, numel, device) -> bool:
    """Whether t is what _Dev would accept; the slow check then says what is wrong with one that is not."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == numel and t.device == device
            and t.is_contiguous())


def _i32(chk, t, name, numel):
    """Device address of an int32 tensor."""
    if _is(t, _I32, numel, chk.device):
        return t.data_ptr()
    if t is None:
        raise ValueError(f"{chk.where}: {name} must be a torch tensor")
    return chk(t, name, (_I32,), numel=numel)


def mxfp4_quantize(x, codes, scales, stream=None):
    """x [rows, cols] bf16/fp32 (row stride may exceed cols) -> codes uint8
    [rows, cols/2] (even column in the low four bits), scales uint8 [rows, cols/32]."""
    chk = _Dev("mxfp4_quantize")
    if x.dim() != 2 or x.stride(-1) != 1:
        raise ValueError("mxfp4_quantize: x must be 2-D with contiguous rows")
    rows, cols = x.shape
    if rows > 1 and x.stride(0) < cols:
        raise ValueError("mxfp4_quantize: the rows of x overlap")
    ld = max(x.stride(0), cols) if rows > 1 else cols
    span = x.as_strided(((rows - 1) * ld + cols,) if rows else (0,), (1,))
    px = chk(span, "x", (_BF16, _FP32))
    dt = DTYPE_FP32 if x.dtype == torch.float32 else DTYPE_BF16
    pc = chk(codes, "codes", (_U8,), numel=rows * cols // 2)
    psc = chk(scales, "scales", (_U8,), numel=rows * cols // 32)
    _call("mxfp4_quantize", chk.device, stream, lib().mxfp4_quantize, px, dt, rows, cols, ld, pc, psc)


def mla_qup_fwd_w4(x, w, w_scales, out, *, H, d_nope, d_rope, cos=None, sin=None, positions=None, bias=None,
                   out_scales=None, fmt=FMT_BSHD, B=1, S=None, cu_seqlens=None, max_seqlen=None, stream=None):
    """Forward of few tokens with MXFP4 weights: x bf16 [T,K], w uint8 [N,K/2] and w_scales uint8 [N,K/32] from
    mxfp4_quantize; out and out_scales as mla_qup_fwd's. positions int32 [T]: each token's position, in place of
    the format's."""
    chk = _Dev("mla_qup_fwd_w4")
    a = mla_qup_w4_args()
    if x.dim() != 2:
        raise ValueError("mla_qup_fwd_w4: x must be [T, K]")
    T, K = x.shape
    N = H * (d_nope + d_rope)
    a.x = chk(x, "x", (_BF16,))
    a.w = chk(w, "w", (_U8,), numel=N * K // 2)
    a.w_scales = chk(w_scales, "w_scales", (_U8,), numel=N * K // 32)
    a.bias = chk(bias, "bias", (_BF16,), numel=N)
    a.K, a.H, a.d_nope, a.d_rope = K, H, d_nope, d_rope
    a.tokens = _tokens(chk, T, fmt, B, S, cu_seqlens, max_seqlen)
    a.positions = chk(positions, "positions", (_I32,), numel=T)
    a.rope = _rope(chk, cos, sin, d_rope)
    a.out_dtype = DTYPE_MXFP8 if out.dtype == torch.uint8 else DTYPE_BF16
    a.out = chk(out, "out", (_BF16, _U8), numel=T * N)
    a.out_scales = chk(out_scales, "out_scales", (_U8,), numel=T * N // 32)
    _call("mla_qup_fwd_w4", chk.device, stream, lib().mla_qup_fwd_w4, ctypes.byref(a))


class PagePool:
    """A paged cache (mla_pool): buffers [num_pages, page_size, heads, width] (bf16: key, then value unless the
    cache is latent; MXFP8, uint8: key codes, key scales [.., width/32], then value codes and scales), and
    int32 refs [num_pages], table [max_seqs, max_pages], lens [max_seqs], held [max_seqs]. The tensors are
    checked once, here; the pool keeps them alive and they must stay as they are (their values are the state)."""

    def __init__(self, bufs, refs, table, lens, held):
        chk = _Dev("PagePool")
        bufs = list(bufs)
        if not 1 <= len(bufs) <= 4 or any(b.dim() != 4 for b in bufs):
            raise ValueError("PagePool: one to four buffers [num_pages, page_size, heads, width]")
        if any(b.shape[:2] != bufs[0].shape[:2] or b.shape[2] != bufs[0].shape[2] or b.dtype != bufs[0].dtype
               for b in bufs):
            raise ValueError("PagePool: buffers must agree in pages, page size, heads and dtype")
        if table.dim() != 2:
            raise ValueError("PagePool: table must be [max_seqs, max_pages]")
        self.mx = bufs[0].dtype == torch.uint8
        if self.mx:
            if len(bufs) % 2 or any(bufs[k].shape[3] != 32 * bufs[k + 1].shape[3] for k in range(0, len(bufs), 2)):
                raise ValueError("PagePool: an MXFP8 cache has codes and scales [.., width/32] in pairs")
        elif len(bufs) > 2:
            raise ValueError("PagePool: a bf16 cache has a key and at most a value buffer")
        n, page = bufs[0].shape[:2]
        c = mla_pool()
        c.num_pages, c.page_size, c.max_seqs, c.max_pages = n, page, table.shape[0], table.shape[1]
        c.refs = chk(refs, "refs", (_I32,), numel=n)
        c.table = chk(table, "table", (_I32,))
        c.lens = chk(lens, "lens", (_I32,), numel=table.shape[0])
        c.held = chk(held, "held", (_I32,), numel=table.shape[0])
        c.nbuf = len(bufs)
        for k, b in enumerate(bufs):
            c.buf[k] = chk(b, f"bufs[{k}]", (_BF16, _U8))
            c.page_bytes[k] = b.stride(0) * b.element_size() if n > 1 else b.numel() * b.element_size()
        self.c, self.device = c, chk.device
        self.ref, self.ptr = ctypes.byref(c), ctypes.pointer(c)
        self.bufs, self.refs, self.table, self.lens, self.held = bufs, refs, table, lens, held
        self.heads, self.d_k = bufs[0].shape[2:]
        self.latent = len(bufs) == (2 if self.mx else 1)
        self.d_v = None if self.latent else bufs[2 if self.mx else 1].shape[3]


def _pool_chk(where, pool) -> _Dev:
    if not isinstance(pool, PagePool):
        raise ValueError(f"{where}: pool must be a PagePool")
    chk = _Dev(where)
    chk.device = pool.device
    return chk


def _workspace(chk, workspace):
    if workspace is None:
        return None, 0
    n = workspace.numel() if isinstance(workspace, torch.Tensor) else 0
    return (workspace.data_ptr() if _is(workspace, _U8, n, chk.device) else chk(workspace, "workspace", (_U8,))), n


def _count(where, t, name) -> int:
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{where}: {name} must be a torch tensor")
    return t.numel()


def mla_pages_workspace_size(pool) -> int:
    _pool_chk("mla_pages_workspace_size", pool)
    return int(lib().mla_pages_workspace_size(pool.ref))


def mla_pages_copy(src, dst, src_ids, dst_ids, stream=None):
    """Page src_ids[i] of pool src to page dst_ids[i] of pool dst (int32 tensors), every buffer."""
    chk = _pool_chk("mla_pages_copy", src)
    if not isinstance(dst, PagePool) or dst.device != src.device:
        raise ValueError("mla_pages_copy: dst must be a PagePool on src's device")
    n = _count(chk.where, src_ids, "src_ids")
    a, b = _i32(chk, src_ids, "src_ids", n), _i32(chk, dst_ids, "dst_ids", n)
    _call(chk.where, chk.device, stream, lib().mla_pages_copy, src.ref, dst.ref, a, b, n)


def mla_pages_reserve(pool, seqs, new_tokens, status, *, workspace, stream=None):
    """Room for new_tokens[i] rows behind sequence seqs[i] (int32 [n] each), copying shared pages on write.
    status int32 [1]: 0 when done, else nothing changed. workspace: mla_pages_workspace_size() bytes."""
    chk = _pool_chk("mla_pages_reserve", pool)
    n = _count(chk.where, seqs, "seqs")
    a, b = _i32(chk, seqs, "seqs", n), _i32(chk, new_tokens, "new_tokens", n)
    st = _i32(chk, status, "status", 1)
    w, size = _workspace(chk, workspace)
    _call(chk.where, chk.device, stream, lib().mla_pages_reserve, pool.ref, a, b, n, st, w, size)


def mla_pages_fork(pool, src, dst, stream=None):
    """Sequence dst[i] (empty) takes the committed rows of src[i] by sharing its pages."""
    chk = _pool_chk("mla_pages_fork", pool)
    n = _count(chk.where, src, "src")
    a, b = _i32(chk, src, "src", n), _i32(chk, dst, "dst", n)
    _call(chk.where, chk.device, stream, lib().mla_pages_fork, pool.ref, a, b, n)


def mla_pages_free(pool, seqs, keep=None, stream=None):
    """Cut sequences to keep[i] committed rows (None: none) and drop the pages behind them."""
    chk = _pool_chk("mla_pages_free", pool)
    n = _count(chk.where, seqs, "seqs")
    a, b = _i32(chk, seqs, "seqs", n), (None if keep is None else _i32(chk, keep, "keep", n))
    _call(chk.where, chk.device, stream, lib().mla_pages_free, pool.ref, a, b, n)


def mla_pages_compact(pool, used, *, workspace, stream=None):
    """Move the pages in use to the front of the pool; used int32 [1] receives their number."""
    chk = _pool_chk("mla_pages_compact", pool)
    u = _i32(chk, used, "used", 1)
    w, size = _workspace(chk, workspace)
    _call(chk.where, chk.device, stream, lib().mla_pages_compact, pool.ref, u, w, size)


def mla_draft_accept(pool, seqs, path, n_acc, stream=None):
    """Drafted rows path[i, :n_acc[i]] (counted behind the committed ones) of sequence seqs[i] become its next rows."""
    chk = _pool_chk("mla_draft_accept", pool)
    n = _count(chk.where, seqs, "seqs")
    if not isinstance(path, torch.Tensor) or path.dim() != 2 or path.shape[0] != n:
        raise ValueError("mla_draft_accept: path must be [n, max_path]")
    width = path.shape[1]
    a, b = _i32(chk, seqs, "seqs", n), _i32(chk, path, "path", n * width)
    c = _i32(chk, n_acc, "n_acc", n)
    _call(chk.where, chk.device, stream, lib().mla_draft_accept, pool.ref, a, b, c, n, width)


def mla_kv_rope_paged(kv, k_pe, pool, seqs, cu_q, *, H, d_nope, d_rope, d_v, cos=None, sin=None, positions=None,
                      max_q=None, stream=None):
    """Key and value rows of new tokens into the cache: kv bf16 [T,H,d_nope+d_v], k_pe bf16 [T,d_rope]; token
    cu_q[j] + i becomes row lens[seqs[j]] + i, i < max_q (None: all). positions int32 [T] or None for the rows
    themselves."""
    chk = _pool_chk("mla_kv_rope_paged", pool)
    a = mla_kv_paged_args()
    T = kv.shape[0]
    a.kv = chk(kv, "kv", (_BF16,), numel=T * H * (d_nope + d_v))
    a.k_pe = chk(k_pe, "k_pe", (_BF16,), numel=T * d_rope)
    a.H, a.d_nope, a.d_rope, a.d_v, a.T = H, d_nope, d_rope, d_v, T
    n = _count(chk.where, seqs, "seqs")
    a.nseq = n
    a.seqs, a.cu_q = _i32(chk, seqs, "seqs", n), _i32(chk, cu_q, "cu_q", n + 1)
    a.max_q = max(1, T) if max_q is None else max_q
    a.positions = None if positions is None else _i32(chk, positions, "positions", T)
    a.rope = _rope(chk, cos, sin, d_rope)
    a.cache_dtype = DTYPE_MXFP8 if pool.mx else DTYPE_BF16
    a.pool = pool.ptr
    _call(chk.where, chk.device, stream, lib().mla_kv_rope_paged, ctypes.byref(a))


def make_tree_attn_args(q, pool, out, seqs, cu_q, *, max_q, max_len, scale, lse=None, mask=None,
                        workspace=None) -> mla_tree_attn_args:
    where = "mla_tree_attention"
    chk = _pool_chk(where, pool)
    if q.dim() != 3 or out.dim() != 3 or q.shape[:2] != out.shape[:2]:
        raise ValueError(f"{where}: q must be [T, H, d_k] and out [T, H, d_v]")
    for t, name in ((q, "q"), (out, "out")):  # token and head strides are free, elements are dense
        if not isinstance(t, torch.Tensor) or t.device != pool.device or t.dtype != _BF16:
            raise ValueError(f"{where}: {name} must be a bf16 tensor on {pool.device}")
        if t.stride(2) != 1 and t.numel():
            raise ValueError(f"{where}: the elements of a row of {name} must be dense")
    T, H, d_k = q.shape
    d_v = out.shape[2]
    if d_k != pool.d_k or (not pool.latent and d_v != pool.d_v):
        raise ValueError(f"{where}: widths of q and out do not fit the cache")
    n = _count(where, seqs, "seqs")
    words = 0
    if mask is not None:
        if not isinstance(mask, torch.Tensor) or mask.dim() != 2 or mask.shape[0] != T:
            raise ValueError(f"{where}: mask must be [T, words]")
        words = mask.shape[1]
        mask = mask.data_ptr() if _is(mask, _I32, T * words, pool.device) else chk(mask, "mask", (_I32, torch.uint32))
    if lse is not None:
        lse = lse.data_ptr() if _is(lse, _FP32, T * H, pool.device) else chk(lse, "lse", (_FP32,), numel=T * H)
    ws, ws_bytes = _workspace(chk, workspace)
    sq, so = q.stride(), out.stride()
    return mla_tree_attn_args(
        q.data_ptr(), sq[0], sq[1], out.data_ptr(), so[0], so[1], lse, T, H, pool.heads, d_k, d_v, scale,
        _i32(chk, seqs, "seqs", n), _i32(chk, cu_q, "cu_q", n + 1), n, max_q, max_len, mask, words,
        DTYPE_MXFP8 if pool.mx else DTYPE_BF16, pool.ptr, ws, ws_bytes)


def mla_tree_attention_workspace_size(q, pool, out, seqs, cu_q, **kw) -> int:
    kw.pop("stream", None)
    a = make_tree_attn_args(q, pool, out, seqs, cu_q, **kw)
    with torch.cuda.device(pool.device if pool.device.type == "cuda" else -1):  # the plan asks for its compute units
        return int(lib().mla_tree_attention_workspace_size(ctypes.byref(a)))


def mla_tree_attention(q, pool, out, seqs, cu_q, *, stream=None, **kw):
    """Attention of drafted tokens over the cache: q bf16 [T,H,d_k] and out bf16 [T,H,d_v] (rows dense, token and
    head strides free), tokens cu_q[j] .. cu_q[j+1] belonging to sequence seqs[j] (int32). mask int32 [T, words]:
    the drafts of its sequence that a token sees, one bit each (None: a chain). max_q and max_len bound the drafts
    and the rows, drafts included, of any sequence. lse fp32 [T,H] or None; workspace:
    mla_tree_attention_workspace_size() bytes (None if that is 0)."""
    a = make_tree_attn_args(q, pool, out, seqs, cu_q, **kw)
    _call("mla_tree_attention", pool.device, stream, lib().mla_tree_attention, ctypes.byref(a))
