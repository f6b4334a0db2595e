"""Torch binding of the decoder-layer operators in include/moe_layer.h: the
residual addition with RMS norm and int8 quant, products with 4-bit weights,
and the paged int8 key / value cache with its attention.

Like the block's binding it only marshals arguments: dtypes, shapes, strides
and devices are checked here, sizes and alignment by the C entry points, and
raw pointers are passed on.  There is no CPU path.  Work is enqueued on
`stream` (the device's current stream without one); outputs that the caller
does not pass are allocated for that stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

P = ctypes.c_void_p
I32 = ctypes.c_int32
I64 = ctypes.c_int64

LAYER_EXPORTS = ["moe_layer_add_rmsnorm_quant", "moe_layer_w4_linear", "moe_layer_kv_append",
                 "moe_layer_kv_attention_workspace_size", "moe_layer_kv_attention"]
DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.int8: 3}


class NormArgs(ctypes.Structure):
    _fields_ = [("x", P), ("residual", P), ("weight", P), ("smooth", P), ("residual_out", P), ("y_out", P), ("q", P),
                ("q_scale", P), ("x_stride", I64), ("residual_stride", I64), ("residual_out_stride", I64),
                ("rows", I32), ("hidden", I32), ("dtype", I32), ("weight_dtype", I32), ("eps", ctypes.c_float)]


class W4Args(ctypes.Structure):
    _fields_ = [("x", P), ("x_scale", P), ("w", P), ("w_scale", P), ("w_zero", P), ("y", P), ("x_stride", I64),
                ("m", I32), ("n", I32), ("k", I32), ("group", I32), ("x_dtype", I32), ("scale_dtype", I32),
                ("out_dtype", I32)]


class KvCacheArgs(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("k_scale", P), ("v_scale", P), ("page_stride", I64), ("head_stride", I64),
                ("scale_stride", I64), ("num_pages", I32), ("kv_heads", I32), ("page_size", I32), ("head_dim", I32)]


class KvAppendArgs(ctypes.Structure):
    _fields_ = [("cache", KvCacheArgs), ("k_new", P), ("v_new", P), ("page_table", P), ("start", P),
                ("cu_tokens", P), ("k_stride", I64), ("v_stride", I64), ("table_stride", I64), ("tokens", I32),
                ("batch", I32), ("max_pages", I32), ("dtype", I32)]


class KvAttentionArgs(ctypes.Structure):
    _fields_ = [("cache", KvCacheArgs), ("q", P), ("out", P), ("page_table", P), ("seq_lens", P), ("cu_q", P),
                ("q_stride", I64), ("table_stride", I64), ("tokens", I32), ("batch", I32), ("max_pages", I32),
                ("max_q", I32), ("group_size", I32), ("window", I32), ("dtype", I32), ("sm_scale", ctypes.c_float)]


def declare(L: ctypes.CDLL) -> None:
    """Argument types of the entry points of a loaded library."""
    for name, args in (("moe_layer_add_rmsnorm_quant", NormArgs), ("moe_layer_w4_linear", W4Args),
                       ("moe_layer_kv_append", KvAppendArgs)):
        getattr(L, name).argtypes = [ctypes.POINTER(args), P]
    L.moe_layer_kv_attention.argtypes = [ctypes.POINTER(KvAttentionArgs), P, ctypes.c_size_t, P]
    L.moe_layer_kv_attention_workspace_size.argtypes = [I32, ctypes.POINTER(ctypes.c_size_t)]
    for name in LAYER_EXPORTS:
        getattr(L, name).restype = ctypes.c_int


_lib = None


def _call(name, args, stream: int, *more) -> None:
    global _lib
    if _lib is None:
        from . import lib
        _lib = lib()
    rc = getattr(_lib, name)(ctypes.byref(args), *more, stream)
    if rc:
        from . import MoeError
        raise MoeError(rc, name)


class _On:
    """The stream that a call runs on, as a context in which its device is
    current and its outputs are allocated."""

    __slots__ = ("raw", "ctx")

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream]):
        if device.type != "cuda":
            raise ValueError("the decoder-layer operators run on a CUDA device only")
        now = torch.cuda.current_stream(device)
        self.ctx = None
        if stream is not None and stream != now:
            if stream.device != device:
                raise ValueError("stream: on %s, expected %s" % (stream.device, device))
            self.ctx, now = torch.cuda.stream(stream), stream
        elif device.index != torch.cuda.current_device():
            self.ctx = torch.cuda.device(device)
        self.raw = now.cuda_stream

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.raw

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _act(t: torch.Tensor, name: str) -> int:
    if t.dtype != torch.bfloat16 and t.dtype != torch.float16:
        raise TypeError("%s: dtype %s, expected bfloat16 or float16" % (name, t.dtype))
    return DTYPE_CODES[t.dtype]


def _dense(t: Optional[torch.Tensor], name: str, dtype, shape, device) -> int:
    """Pointer of a contiguous tensor; 0 for None."""
    if t is None:
        return 0
    if t.dtype != dtype:
        raise TypeError("%s: dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.device != device:
        raise ValueError("%s: on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, dtype, shape, device) -> Tuple[int, int]:
    """Pointer and row stride of a tensor whose inner dimensions are dense."""
    if t.dtype != dtype:
        raise TypeError("%s: dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.device != device:
        raise ValueError("%s: on %s, expected %s" % (name, t.device, device))
    inner = 1
    for d in range(t.dim() - 1, 0, -1):
        if t.stride(d) != inner and shape[d] != 1:
            raise ValueError("%s: every dimension but the first must be dense" % name)
        inner *= shape[d]
    # a single row has no stride that matters
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else -(-inner // 16) * 16


def add_rmsnorm_quant(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                      residual: Optional[torch.Tensor] = None, smooth: Optional[torch.Tensor] = None,
                      want_y: bool = False, q: Optional[torch.Tensor] = None, q_scale: Optional[torch.Tensor] = None,
                      residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                      stream: Optional[torch.cuda.Stream] = None):
    """(q, q_scale, residual_out, y) of moe_layer_add_rmsnorm_quant.

    x [rows, hidden] bf16 or fp16, its rows may be strided, as residual's;
    weight [hidden] of x's dtype or fp32; smooth [hidden] fp32.  q int8 and
    q_scale fp32 [rows] are the quantised norm; residual_out is x + residual
    in x's dtype (None without residual; pass residual itself to add in
    place); y is the norm in x's dtype (None unless `want_y` or a tensor for
    it is given)."""
    code, device, shape = _act(x, "x"), x.device, x.shape
    if len(shape) != 2:
        raise ValueError("x: %d dimensions, expected 2" % len(shape))
    rows, hidden = shape
    a = NormArgs()
    a.x, a.x_stride = _rows(x, "x", x.dtype, shape, device)
    if weight.dtype != x.dtype and weight.dtype != torch.float32:
        raise TypeError("weight: dtype %s, expected %s or float32" % (weight.dtype, x.dtype))
    a.weight = _dense(weight, "weight", weight.dtype, (hidden,), device)
    a.smooth = _dense(smooth, "smooth", torch.float32, (hidden,), device)
    a.rows, a.hidden, a.dtype, a.weight_dtype, a.eps = rows, hidden, code, DTYPE_CODES[weight.dtype], eps
    with _On(device, stream) as raw:
        if q is None:
            q = torch.empty(shape, dtype=torch.int8, device=device)
        if q_scale is None:
            q_scale = torch.empty(rows, dtype=torch.float32, device=device)
        if residual is not None:
            a.residual, a.residual_stride = _rows(residual, "residual", x.dtype, shape, device)
            if residual_out is None:
                residual_out = torch.empty(shape, dtype=x.dtype, device=device)
            a.residual_out, a.residual_out_stride = _rows(residual_out, "residual_out", x.dtype, shape, device)
        elif residual_out is not None:
            raise ValueError("residual_out without residual")
        if y is None and want_y:
            y = torch.empty(shape, dtype=x.dtype, device=device)
        a.y_out = _dense(y, "y", x.dtype, shape, device)
        a.q = _dense(q, "q", torch.int8, shape, device)
        a.q_scale = _dense(q_scale, "q_scale", torch.float32, (rows,), device)
        _call("moe_layer_add_rmsnorm_quant", a, raw)
    return q, q_scale, residual_out, y


def w4_linear(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, zero: Optional[torch.Tensor] = None,
              x_scale: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
              out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """y [m, n] of moe_layer_w4_linear: x times the transposed 4-bit weights.

    x [m, k] bf16 or fp16, or int8 codes with x_scale [m] fp32 (as
    add_rmsnorm_quant leaves them); its rows may be strided.  w [n, k / 2]
    uint8 (even k in the low four bits), w_scale [n, k / group] bf16, fp16 or
    fp32, zero [n, k / group] uint8 or None (8 everywhere).  The group is what
    w_scale's shape says.  out_dtype: bf16, fp16 or fp32; x's dtype without
    it (bf16 for int8 x)."""
    device = x.device
    if x.dim() != 2 or w.dim() != 2 or w_scale.dim() != 2:
        raise ValueError("x, w and w_scale have 2 dimensions")
    m, k = x.shape
    n, groups = w_scale.shape
    if x.dtype == torch.int8:
        if x_scale is None:
            raise ValueError("x_scale is required with int8 x")
    else:
        _act(x, "x")
        if x_scale is not None:
            raise ValueError("x_scale is for int8 x only")
    if groups < 1 or k % groups:
        raise ValueError("w_scale: %d groups do not divide k = %d" % (groups, k))
    if w_scale.dtype not in DTYPE_CODES or w_scale.dtype == torch.int8:
        raise TypeError("w_scale: dtype %s, expected bfloat16, float16 or float32" % w_scale.dtype)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else (torch.bfloat16 if x.dtype == torch.int8 else x.dtype)
    if out_dtype not in DTYPE_CODES or out_dtype == torch.int8:
        raise TypeError("out_dtype: %s, expected bfloat16, float16 or float32" % out_dtype)
    a = W4Args()
    a.x, a.x_stride = _rows(x, "x", x.dtype, x.shape, device)
    a.x_scale = _dense(x_scale, "x_scale", torch.float32, (m,), device)
    a.w = _dense(w, "w", torch.uint8, (n, k // 2), device)
    a.w_scale = _dense(w_scale, "w_scale", w_scale.dtype, (n, groups), device)
    a.w_zero = _dense(zero, "zero", torch.uint8, (n, groups), device)
    a.m, a.n, a.k, a.group = m, n, k, k // groups
    a.x_dtype, a.scale_dtype, a.out_dtype = DTYPE_CODES[x.dtype], DTYPE_CODES[w_scale.dtype], DTYPE_CODES[out_dtype]
    with _On(device, stream) as raw:
        if out is None:
            out = torch.empty(m, n, dtype=out_dtype, device=device)
        a.y = _dense(out, "out", out_dtype, (m, n), device)
        _call("moe_layer_w4_linear", a, raw)
    return out


class KvCache:
    """A paged int8 cache of keys and values with one scale a page and head.

    k, v: int8 [num_pages, kv_heads, page_size, head_dim]; k_scale, v_scale:
    fp32 [num_pages, kv_heads].  Pages and heads may be strided (the same way
    for k and v: views of one larger tensor work); a head's slots are dense.
    The tensors stay the caller's and can be read at any time.  The handle
    keeps the attention's workspace, so calls on one handle must be ordered on
    the GPU.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        if k.dim() != 4 or k.shape != v.shape:
            raise ValueError("k and v: shapes %s and %s, expected one [num_pages, kv_heads, page_size, head_dim]" %
                             (tuple(k.shape), tuple(v.shape)))
        pages, heads, page_size, dim = k.shape
        for t, name in ((k, "k"), (v, "v")):
            if t.dtype != torch.int8:
                raise TypeError("%s: dtype %s, expected int8" % (name, t.dtype))
            if t.device != k.device:
                raise ValueError("%s: on %s, expected %s" % (name, t.device, k.device))
            if t.stride(3) != 1 or t.stride(2) != dim:
                raise ValueError("%s: the slots of a head must be dense" % name)
        if k.stride() != v.stride():
            raise ValueError("k and v must have the same strides")
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.dtype != torch.float32:
                raise TypeError("%s: dtype %s, expected float32" % (name, t.dtype))
            if t.shape != (pages, heads):
                raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), (pages, heads)))
            if t.device != k.device:
                raise ValueError("%s: on %s, expected %s" % (name, t.device, k.device))
            if t.stride(1) != 1 and heads != 1:
                raise ValueError("%s: the heads of a page must be dense" % name)
        if k_scale.stride(0) != v_scale.stride(0):
            raise ValueError("k_scale and v_scale must have the same strides")
        if k.device.type != "cuda":
            raise ValueError("the decoder-layer operators run on a CUDA device only")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.kv_heads, self.page_size, self.head_dim = k.device, heads, page_size, dim
        c = KvCacheArgs()
        c.k, c.v, c.k_scale, c.v_scale = k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr()
        c.page_stride, c.head_stride, c.scale_stride = k.stride(0), k.stride(1), k_scale.stride(0)
        c.num_pages, c.kv_heads, c.page_size, c.head_dim = pages, heads, page_size, dim
        self._args = c
        self._ws = None

    @classmethod
    def empty(cls, num_pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda") -> "KvCache":
        """A cache with tensors of its own (nothing in it counts until it is appended)."""
        k, v = (torch.zeros(num_pages, kv_heads, page_size, head_dim, dtype=torch.int8, device=device) for _ in "kv")
        ks, vs = (torch.zeros(num_pages, kv_heads, dtype=torch.float32, device=device) for _ in "kv")
        return cls(k, v, ks, vs)

    def workspace(self) -> torch.Tensor:
        """The attention's workspace, allocated at its first use."""
        if self._ws is None:
            from . import MoeError, lib
            nb = ctypes.c_size_t(0)
            with torch.cuda.device(self.device):
                rc = lib().moe_layer_kv_attention_workspace_size(self.head_dim, ctypes.byref(nb))
            if rc:
                raise MoeError(rc, "moe_layer_kv_attention_workspace_size")
            buf = torch.empty(nb.value + 256, dtype=torch.uint8, device=self.device)
            self._ws = buf[(-buf.data_ptr()) % 256:]
        return self._ws

    def _table(self, page_table: torch.Tensor) -> Tuple[int, int, int, int]:
        if page_table.dtype != torch.int32:
            raise TypeError("page_table: dtype %s, expected int32" % page_table.dtype)
        if page_table.dim() != 2:
            raise ValueError("page_table: %d dimensions, expected 2" % page_table.dim())
        if page_table.device != self.device:
            raise ValueError("page_table: on %s, expected %s" % (page_table.device, self.device))
        batch, pages = page_table.shape
        if pages > 1 and page_table.stride(1) != 1:
            raise ValueError("page_table: the pages of a sequence must be dense")
        return page_table.data_ptr(), batch, pages, page_table.stride(0) if batch > 1 else pages

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor,
               cu_tokens: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Write new tokens (moe_layer_kv_append).  k_new, v_new [tokens,
        kv_heads, head_dim] bf16 or fp16 (tokens may be strided); page_table
        [batch, max_pages] and start [batch] int32; cu_tokens [batch + 1]
        int32 where sequences get more or fewer tokens than one."""
        code, dev = _act(k_new, "k_new"), self.device
        if k_new.dim() != 3:
            raise ValueError("k_new: %d dimensions, expected 3" % k_new.dim())
        a = KvAppendArgs()
        a.cache = self._args
        a.page_table, a.batch, a.max_pages, a.table_stride = self._table(page_table)
        tokens = k_new.shape[0]
        shape = (tokens, self.kv_heads, self.head_dim)
        a.k_new, a.k_stride = _rows(k_new, "k_new", k_new.dtype, shape, dev)
        a.v_new, a.v_stride = _rows(v_new, "v_new", k_new.dtype, shape, dev)
        a.start = _dense(start, "start", torch.int32, (a.batch,), dev)
        a.cu_tokens = _dense(cu_tokens, "cu_tokens", torch.int32, (a.batch + 1,), dev)
        if cu_tokens is None and tokens != a.batch:
            raise ValueError("k_new: %d tokens for %d sequences without cu_tokens" % (tokens, a.batch))
        a.tokens, a.dtype = tokens, code
        with _On(dev, stream) as raw:
            _call("moe_layer_kv_append", a, raw)

    def attention(self, q: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                  cu_q: Optional[torch.Tensor] = None, max_q: int = 1, scale: Optional[float] = None, window: int = 0,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Attention of the query tokens over their sequences' keys
        (moe_layer_kv_attention).  q [tokens, heads, head_dim] bf16 or fp16
        (tokens may be strided), heads a multiple of kv_heads; seq_lens
        [batch] int32, the query tokens' own keys counted; cu_q [batch + 1]
        int32 with max_q, the most query tokens of a sequence, where that is
        not one each; scale: head_dim ** -0.5 without it; window: keys that a
        token sees at most, itself among them (0: no limit).  Returns out
        [tokens, heads, head_dim]."""
        code, dev = _act(q, "q"), self.device
        if q.dim() != 3:
            raise ValueError("q: %d dimensions, expected 3" % q.dim())
        tokens, heads, dim = q.shape
        if dim != self.head_dim or heads % self.kv_heads:
            raise ValueError("q: %d heads of %d do not fit %d kv heads of %d" %
                             (heads, dim, self.kv_heads, self.head_dim))
        a = KvAttentionArgs()
        a.cache = self._args
        a.page_table, a.batch, a.max_pages, a.table_stride = self._table(page_table)
        a.q, a.q_stride = _rows(q, "q", q.dtype, q.shape, dev)
        a.seq_lens = _dense(seq_lens, "seq_lens", torch.int32, (a.batch,), dev)
        a.cu_q = _dense(cu_q, "cu_q", torch.int32, (a.batch + 1,), dev)
        if cu_q is None and (tokens != a.batch or max_q != 1):
            raise ValueError("q: %d tokens (max_q %d) for %d sequences without cu_q" % (tokens, max_q, a.batch))
        a.tokens, a.max_q, a.group_size, a.window, a.dtype = tokens, max_q, heads // self.kv_heads, window, code
        a.sm_scale = dim ** -0.5 if scale is None else scale
        with _On(dev, stream) as raw:
            ws = self.workspace() if workspace is None else workspace
            if out is None:
                out = torch.empty(q.shape, dtype=q.dtype, device=dev)
            a.out = _dense(out, "out", q.dtype, q.shape, dev)
            _call("moe_layer_kv_attention", a, raw, ws.data_ptr(), ws.numel())
        return out
