"""Torch binding of the decoder-layer operators in include/moe_layer.h: the
residual addition with RMS norm and int8 quant, the same behind the norm and
gate of the block before, products with 4-bit and 8-bit weights, the paged int8
key / value cache with its attention and the plan of its pages, and log
probabilities of tokens.

Like the block's binding it only marshals arguments: dtypes, shapes, strides
and devices are checked here, sizes and alignment by the C entry points, and
raw pointers are passed on.  There is no CPU path.  Work is enqueued on
`stream` (the device's current stream without one); outputs that the caller
does not pass are allocated for that stream.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional, Tuple

import torch

P = ctypes.c_void_p
I32 = ctypes.c_int32
I64 = ctypes.c_int64

LAYER_EXPORTS = ["moe_layer_add_rmsnorm_quant", "moe_layer_w4_linear", "moe_layer_kv_append",
                 "moe_layer_kv_attention_workspace_size", "moe_layer_kv_attention", "moe_layer_kv_attention_status",
                 "moe_layer_norm_add_rmsnorm_quant", "moe_layer_w8_linear_workspace_size", "moe_layer_w8_linear",
                 "moe_layer_w8_linear_status", "moe_layer_page_plan", "moe_layer_token_logprobs"]
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


class NormPairArgs(ctypes.Structure):
    _fields_ = [("x", P), ("residual", P), ("post_weight", P), ("gate", P), ("weight", P), ("smooth", P),
                ("residual_out", P), ("y_out", P), ("q", P), ("q_scale", P), ("x_stride", I64), ("residual_stride", I64),
                ("gate_stride", I64), ("residual_out_stride", I64), ("rows", I32), ("hidden", I32), ("dtype", I32),
                ("weight_dtype", I32), ("eps", ctypes.c_float), ("branch_scale", ctypes.c_float)]


class W8Args(ctypes.Structure):
    _fields_ = [("x", P), ("x_scale", P), ("w", P), ("w_scale", P), ("y", P), ("x_stride", I64), ("m", I32), ("n", I32),
                ("k", I32), ("scale_dtype", I32), ("out_dtype", I32)]


class PagePlanArgs(ctypes.Structure):
    _fields_ = [("page_table", P), ("held", P), ("new_tokens", P), ("free_pages", P), ("taken", P), ("taken_out", P),
                ("unplaced", P), ("cu_tokens", P), ("seq_lens", P), ("sequence", P), ("position", P), ("slot", P),
                ("table_stride", I64), ("batch", I32), ("max_pages", I32), ("page_size", I32), ("num_pages", I32),
                ("num_free", I32), ("tokens", I32)]


class LogprobsArgs(ctypes.Structure):
    _fields_ = [("logits", P), ("tokens", P), ("logprob", P), ("entropy", P), ("top_logprob", P), ("top_id", P),
                ("logits_stride", I64), ("rows", I32), ("vocab", I32), ("num_tokens", I32), ("top", I32), ("dtype", I32),
                ("tokens_64", I32)]


def declare(L: ctypes.CDLL) -> None:
    """Argument types of the entry points of a loaded library."""
    for name, args in (("moe_layer_add_rmsnorm_quant", NormArgs), ("moe_layer_w4_linear", W4Args),
                       ("moe_layer_kv_append", KvAppendArgs), ("moe_layer_norm_add_rmsnorm_quant", NormPairArgs),
                       ("moe_layer_page_plan", PagePlanArgs), ("moe_layer_token_logprobs", LogprobsArgs)):
        getattr(L, name).argtypes = [ctypes.POINTER(args), P]
    L.moe_layer_kv_attention.argtypes = [ctypes.POINTER(KvAttentionArgs), P, ctypes.c_size_t, P]
    L.moe_layer_kv_attention_status.argtypes = [P, P]
    L.moe_layer_w8_linear.argtypes = [ctypes.POINTER(W8Args), P, ctypes.c_size_t, P]
    L.moe_layer_w8_linear_status.argtypes = [P, P]
    L.moe_layer_w8_linear_workspace_size.argtypes = [I32, I32, I32, ctypes.POINTER(ctypes.c_size_t)]
    L.moe_layer_kv_attention_workspace_size.argtypes = [I32, ctypes.POINTER(ctypes.c_size_t)]
    for name in LAYER_EXPORTS:
        getattr(L, name).restype = ctypes.c_int


_lib = None
# the current device's index, and the raw handle of a device's current stream: plain
# integers, without the objects of torch.cuda (which cost as much as a launch).
# A torch without CUDA has neither, and imports this module all the same.
_device_index = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_CONTIGUOUS = torch.contiguous_format


def _entry(name: str):
    global _lib
    if _lib is None:
        from . import lib
        _lib = lib()
    return getattr(_lib, name)


_I32_MAX = 2 ** 31 - 1


def _too_large(name: str, size: int):
    raise ValueError("%s: %d does not fit 32 bits" % (name, size))


def _raise(rc: int, name: str):
    from . import MoeError
    raise MoeError(rc, name)


class _On:
    """Context in which a tensor's device is current, and `stream` its stream."""

    def __init__(self, device: torch.device, stream: Optional[torch.cuda.Stream]):
        if device.type != "cuda":
            raise ValueError("the decoder-layer operators run on a CUDA device only")
        if stream is not None and stream.device != device:
            raise ValueError("stream: on %s, expected %s" % (stream.device, device))
        self.ctx = torch.cuda.device(device) if stream is None else torch.cuda.stream(stream)

    def __enter__(self):
        self.ctx.__enter__()

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)


def _act(t: torch.Tensor, name: str) -> int:
    code = DTYPE_CODES.get(t.dtype, 9)
    if code > 1:
        raise TypeError("%s: dtype %s, expected bfloat16 or float16" % (name, t.dtype))
    return code


def _dense(t: Optional[torch.Tensor], name: str, dtype, shape, index: int) -> int:
    """Pointer of a contiguous tensor; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype:
        raise TypeError("%s: dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.get_device() != index:
        raise ValueError("%s: on %s, expected cuda:%d" % (name, t.device, index))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _workspace(ws: torch.Tensor, index: int) -> Tuple[int, int]:
    """Pointer and bytes of a workspace of the caller's own."""
    if ws.get_device() != index:
        raise ValueError("workspace: on %s, expected cuda:%d" % (ws.device, index))
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _rows(t: torch.Tensor, name: str, dtype, shape, index: int) -> Tuple[int, int]:
    """Pointer and row stride of a tensor whose inner dimensions are dense."""
    if t.dtype is not dtype:
        raise TypeError("%s: dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s: shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.get_device() != index:
        raise ValueError("%s: on %s, expected cuda:%d" % (name, t.device, index))
    strides = t.stride()
    inner = 1
    for d in range(len(shape) - 1, 0, -1):
        if strides[d] != inner and shape[d] != 1:
            raise ValueError("%s: every dimension but the first must be dense" % name)
        inner *= shape[d]
    # a single row has no stride that matters
    return t.data_ptr(), strides[0] if shape[0] > 1 else -(-inner // 16) * 16


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
    code, shape, index = _act(x, "x"), x.shape, x.get_device()
    if len(shape) != 2:
        raise ValueError("x: %d dimensions, expected 2" % len(shape))
    if stream is not None or index < 0 or index != _device_index():
        with _On(x.device, stream):
            return add_rmsnorm_quant(x, weight, eps, residual, smooth, want_y, q, q_scale, residual_out, y)
    rows, hidden = shape
    if rows > _I32_MAX or hidden > _I32_MAX:
        _too_large("x", max(shape))
    dtype, wdtype = x.dtype, weight.dtype
    if wdtype is not dtype and wdtype is not torch.float32:
        raise TypeError("weight: dtype %s, expected %s or float32" % (wdtype, dtype))
    a = NormArgs()
    a.x, a.x_stride = _rows(x, "x", dtype, shape, index)
    a.weight = _dense(weight, "weight", wdtype, (hidden,), index)
    a.smooth = _dense(smooth, "smooth", torch.float32, (hidden,), index)
    a.rows, a.hidden, a.dtype, a.weight_dtype, a.eps = rows, hidden, code, DTYPE_CODES[wdtype], eps
    if q is None:
        q = torch.empty_like(x, dtype=torch.int8, memory_format=_CONTIGUOUS)
    if q_scale is None:
        q_scale = torch.empty(rows, dtype=torch.float32, device=x.device)
    if residual is not None:
        a.residual, a.residual_stride = _rows(residual, "residual", dtype, shape, index)
        if residual_out is None:
            residual_out = torch.empty_like(x, memory_format=_CONTIGUOUS)
        a.residual_out, a.residual_out_stride = _rows(residual_out, "residual_out", dtype, shape, index)
    elif residual_out is not None:
        raise ValueError("residual_out without residual")
    if y is None and want_y:
        y = torch.empty_like(x, memory_format=_CONTIGUOUS)
    a.y_out = _dense(y, "y", dtype, shape, index)
    a.q = _dense(q, "q", torch.int8, shape, index)
    a.q_scale = _dense(q_scale, "q_scale", torch.float32, (rows,), index)
    rc = _entry("moe_layer_add_rmsnorm_quant")(ctypes.byref(a), _raw_stream(index))
    if rc:
        _raise(rc, "moe_layer_add_rmsnorm_quant")
    return q, q_scale, residual_out, y


def norm_add_rmsnorm_quant(x: torch.Tensor, residual: torch.Tensor, post_weight: torch.Tensor, weight: torch.Tensor,
                           eps: float = 1e-6, gate: Optional[torch.Tensor] = None, branch_scale: float = 1.0,
                           smooth: Optional[torch.Tensor] = None, want_q: bool = True, want_y: bool = False,
                           q: Optional[torch.Tensor] = None, q_scale: Optional[torch.Tensor] = None,
                           residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                           stream: Optional[torch.cuda.Stream] = None):
    """(q, q_scale, residual_out, y) of moe_layer_norm_add_rmsnorm_quant: the
    norm of a block's output x, its gate and scale, the residual addition, and
    the norm before the next block.

    x, residual [rows, hidden] bf16 or fp16, their rows may be strided;
    post_weight and weight [hidden], both of x's dtype or both fp32; gate
    [hidden], or [rows, hidden] (rows may be strided), of x's dtype;
    smooth [hidden] fp32.  residual_out is residual + branch_scale * gate *
    norm(x) in x's dtype (pass residual itself to add in place); q int8 and
    q_scale fp32 [rows] are the quantised norm of that (None where `want_q` is
    false and no tensors are given), y the norm in x's dtype (None unless
    `want_y` or a tensor for it is given)."""
    code, shape, index = _act(x, "x"), x.shape, x.get_device()
    if len(shape) != 2:
        raise ValueError("x: %d dimensions, expected 2" % len(shape))
    if stream is not None or index < 0 or index != _device_index():
        with _On(x.device, stream):
            return norm_add_rmsnorm_quant(x, residual, post_weight, weight, eps, gate, branch_scale, smooth, want_q,
                                          want_y, q, q_scale, residual_out, y)
    rows, hidden = shape
    if rows > _I32_MAX or hidden > _I32_MAX:
        _too_large("x", max(shape))
    dtype, wdtype = x.dtype, weight.dtype
    if wdtype is not dtype and wdtype is not torch.float32:
        raise TypeError("weight: dtype %s, expected %s or float32" % (wdtype, dtype))
    a = NormPairArgs()
    a.x, a.x_stride = _rows(x, "x", dtype, shape, index)
    a.residual, a.residual_stride = _rows(residual, "residual", dtype, shape, index)
    a.post_weight = _dense(post_weight, "post_weight", wdtype, (hidden,), index)
    a.weight = _dense(weight, "weight", wdtype, (hidden,), index)
    if gate is not None:
        if gate.dim() == 1:
            a.gate = _dense(gate, "gate", dtype, (hidden,), index)
        else:
            a.gate, a.gate_stride = _rows(gate, "gate", dtype, shape, index)
    a.smooth = _dense(smooth, "smooth", torch.float32, (hidden,), index)
    a.rows, a.hidden, a.dtype, a.weight_dtype = rows, hidden, code, DTYPE_CODES[wdtype]
    a.eps, a.branch_scale = eps, branch_scale
    if residual_out is None:
        residual_out = torch.empty_like(x, memory_format=_CONTIGUOUS)
    a.residual_out, a.residual_out_stride = _rows(residual_out, "residual_out", dtype, shape, index)
    if want_q or q is not None or q_scale is not None:
        if q is None:
            q = torch.empty_like(x, dtype=torch.int8, memory_format=_CONTIGUOUS)
        if q_scale is None:
            q_scale = torch.empty(rows, dtype=torch.float32, device=x.device)
        a.q = _dense(q, "q", torch.int8, shape, index)
        a.q_scale = _dense(q_scale, "q_scale", torch.float32, (rows,), index)
    if y is None and want_y:
        y = torch.empty_like(x, memory_format=_CONTIGUOUS)
    a.y_out = _dense(y, "y", dtype, shape, index)
    rc = _entry("moe_layer_norm_add_rmsnorm_quant")(ctypes.byref(a), _raw_stream(index))
    if rc:
        _raise(rc, "moe_layer_norm_add_rmsnorm_quant")
    return q, q_scale, residual_out, y


def w8_linear_workspace(m: int, n: int, k: int, device="cuda") -> Optional[torch.Tensor]:
    """A workspace for w8_linear of these sizes; None where it needs none."""
    device = torch.device(device)
    with _On(device, None):
        nb = _w8_workspace_bytes(m, n, k, torch.cuda.current_device())
        if not nb:
            return None
        buf = torch.empty(nb + 256, dtype=torch.uint8, device="cuda")
        return buf[(-buf.data_ptr()) % 256:][:nb]


@functools.lru_cache(maxsize=1024)
def _w8_workspace_bytes(m: int, n: int, k: int, index: int) -> int:
    if max(m, n, k) > _I32_MAX or min(m, n, k) < -_I32_MAX:
        _too_large("w8_linear_workspace", max(m, n, k, key=abs))
    nb = ctypes.c_size_t(0)
    rc = _entry("moe_layer_w8_linear_workspace_size")(m, n, k, ctypes.byref(nb))
    if rc:
        _raise(rc, "moe_layer_w8_linear_workspace_size")
    return nb.value


def w8_linear(x: torch.Tensor, w: torch.Tensor, w_scale: torch.Tensor, x_scale: torch.Tensor,
              out_dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
              workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """y [m, n] of moe_layer_w8_linear: int8 codes times the transposed int8
    weights, exact in int32, times both scales.

    x [m, k] int8 with x_scale [m] fp32, as add_rmsnorm_quant leaves them; its
    rows may be strided.  w [n, k] int8, w_scale [n] bf16, fp16 or fp32.
    out_dtype: bf16 (without it), fp16 or fp32.  workspace: one of
    w8_linear_workspace; without it memory of torch's allocator is used for
    the call."""
    index, shape = x.get_device(), x.shape
    if stream is not None or index < 0 or index != _device_index():
        with _On(x.device, stream):
            return w8_linear(x, w, w_scale, x_scale, out_dtype, out, workspace)
    wshape = w.shape
    if len(shape) != 2 or len(wshape) != 2:
        raise ValueError("x and w have 2 dimensions")
    m, k = shape
    n = wshape[0]
    if m > _I32_MAX or k > _I32_MAX or n > _I32_MAX:
        _too_large("x or w", max(m, k, n))
    sdtype = w_scale.dtype
    scode = DTYPE_CODES.get(sdtype, 3)
    if scode == 3:
        raise TypeError("w_scale: dtype %s, expected bfloat16, float16 or float32" % sdtype)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else torch.bfloat16
    ocode = DTYPE_CODES.get(out_dtype, 3)
    if ocode == 3:
        raise TypeError("out_dtype: %s, expected bfloat16, float16 or float32" % out_dtype)
    a = W8Args()
    a.x, a.x_stride = _rows(x, "x", torch.int8, shape, index)
    a.x_scale = _dense(x_scale, "x_scale", torch.float32, (m,), index)
    a.w = _dense(w, "w", torch.int8, (n, k), index)
    a.w_scale = _dense(w_scale, "w_scale", sdtype, (n,), index)
    a.m, a.n, a.k, a.scale_dtype, a.out_dtype = m, n, k, scode, ocode
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=x.device)
        a.y = out.data_ptr()
    else:
        a.y = _dense(out, "out", out_dtype, (m, n), index)
    ws_at = ws_bytes = 0
    if workspace is not None:
        ws_at, ws_bytes = _workspace(workspace, index)
    elif m:
        need = _w8_workspace_bytes(m, n, k, index)
        if need:
            workspace = torch.empty(need + 256, dtype=torch.uint8, device=x.device)
            ws_at, ws_bytes = -(-workspace.data_ptr() // 256) * 256, need
    rc = _entry("moe_layer_w8_linear")(ctypes.byref(a), ws_at, ws_bytes, _raw_stream(index))
    if rc:
        _raise(rc, "moe_layer_w8_linear")
    return out


def w8_linear_status(workspace: torch.Tensor) -> int:
    """Synchronises the current stream; the code of the last w8_linear that
    used this workspace (there has to have been one): 0, or
    MOE_ERR_DEVICE_TIMEOUT where a wait inside it gave up."""
    with _On(workspace.device, None):
        index = workspace.get_device()
        return _entry("moe_layer_w8_linear_status")(_workspace(workspace, index)[0], _raw_stream(index))


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None, top: int = 0,
                   stream: Optional[torch.cuda.Stream] = None):
    """(logprob, entropy, top_logprob, top_id) of moe_layer_token_logprobs.

    logits [rows, vocab] bf16, fp16 or fp32, its rows may be strided; tokens
    [rows] or [rows, n] int32 or int64.  logprob fp32 has the shape of tokens
    (None without tokens), entropy fp32 [rows]; top_logprob fp32 and top_id
    int32 [rows, top] are the `top` (at most 32) likeliest tokens, the lower
    id first among equals (None with top 0)."""
    index, shape, code = logits.get_device(), logits.shape, DTYPE_CODES.get(logits.dtype, 3)
    if code == 3:
        raise TypeError("logits: dtype %s, expected bfloat16, float16 or float32" % logits.dtype)
    if stream is not None or index < 0 or index != _device_index():
        with _On(logits.device, stream):
            return token_logprobs(logits, tokens, top)
    if len(shape) != 2:
        raise ValueError("logits: %d dimensions, expected 2" % len(shape))
    rows, vocab = shape
    if rows > _I32_MAX or vocab > _I32_MAX:
        _too_large("logits", max(shape))
    if not 0 <= top <= min(32, vocab):
        raise ValueError("top: %d, expected 0 to %d" % (top, min(32, vocab)))
    a = LogprobsArgs()
    a.logits, a.logits_stride = _rows(logits, "logits", logits.dtype, shape, index)
    if rows == 1:
        a.logits_stride = vocab
    device = logits.device
    logprob = top_logprob = top_id = None
    if tokens is not None:
        tdtype, tshape = tokens.dtype, tokens.shape
        if tdtype is not torch.int32 and tdtype is not torch.int64:
            raise TypeError("tokens: dtype %s, expected int32 or int64" % tdtype)
        if not 1 <= len(tshape) <= 2 or tshape[0] != rows:
            raise ValueError("tokens: shape %s, expected [%d] or [%d, n]" % (tuple(tshape), rows, rows))
        if tokens.numel() > rows * _I32_MAX:
            _too_large("tokens", tshape[1])
        a.num_tokens = tshape[1] if len(tshape) == 2 else 1
        if a.num_tokens:
            a.tokens = _dense(tokens, "tokens", tdtype, tshape, index)
        a.tokens_64 = tdtype is torch.int64
        logprob = torch.empty(tshape, dtype=torch.float32, device=device)
        a.logprob = logprob.data_ptr()
    entropy = torch.empty(rows, dtype=torch.float32, device=device)
    a.entropy = entropy.data_ptr()
    if top:
        top_logprob = torch.empty((rows, top), dtype=torch.float32, device=device)
        top_id = torch.empty((rows, top), dtype=torch.int32, device=device)
        a.top_logprob, a.top_id = top_logprob.data_ptr(), top_id.data_ptr()
    a.rows, a.vocab, a.top, a.dtype = rows, vocab, top, code
    rc = _entry("moe_layer_token_logprobs")(ctypes.byref(a), _raw_stream(index))
    if rc:
        _raise(rc, "moe_layer_token_logprobs")
    return logprob, entropy, top_logprob, top_id


class PagePlan(NamedTuple):
    """What a step over a paged cache needs (moe_layer_page_plan): cu_tokens
    [batch + 1] and seq_lens [batch] as KvCache's append and attention take
    them; sequence, position (int32) and slot (int64) [tokens] of every token of
    the step, -1 past the last; taken [1], the entries of the list of free pages
    that are in use now; unplaced [1], how many tokens have no slot."""
    cu_tokens: torch.Tensor
    seq_lens: torch.Tensor
    sequence: torch.Tensor
    position: torch.Tensor
    slot: torch.Tensor
    taken: torch.Tensor
    unplaced: torch.Tensor


def page_plan(page_table: torch.Tensor, held: torch.Tensor, new_tokens: torch.Tensor, free_pages: torch.Tensor,
              page_size: int, num_pages: int, tokens: int, taken: Optional[torch.Tensor] = None,
              taken_out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> PagePlan:
    """Plan a step whose sequences hold `held` [batch] tokens and get
    `new_tokens` [batch] more (int32): writes the new pages, taken from
    free_pages (int32, from entry `taken` [1] on, 0 without it), into page_table
    [batch, max_pages] int32 and returns a PagePlan.

    num_pages: pages of the cache; tokens: rows of the step's buffers, at least
    as many as there are new tokens (those past it are left out).  taken_out:
    where to write the plan's `taken` (pass `taken` itself to move it on in
    place, as a captured step does)."""
    index = page_table.get_device()
    if stream is not None or index < 0 or index != _device_index():
        with _On(page_table.device, stream):
            return page_plan(page_table, held, new_tokens, free_pages, page_size, num_pages, tokens, taken, taken_out)
    table_at, batch, pages, stride = _page_table(page_table, index)
    num_free = free_pages.numel()
    if max(page_size, num_pages, tokens, num_free) > _I32_MAX or min(page_size, num_pages) < -_I32_MAX:
        _too_large("page_plan", max(page_size, num_pages, tokens, num_free, key=abs))
    if tokens < 0:
        raise ValueError("tokens: %d" % tokens)
    i32 = torch.int32
    # one allocation for the numbers of 32 bits (whole numbers: nothing differentiates through parts that torch does not
    # keep as views, which cost half as much)
    device = page_table.device
    buf = torch.empty(2 * tokens + 2 * batch + 3, dtype=i32, device=device)
    sequence, position, seq_lens, cu_tokens, unplaced, own_taken = torch.unsafe_split_with_sizes(
        buf, [tokens, tokens, batch, batch + 1, 1, 1])
    slot = torch.empty(tokens, dtype=torch.int64, device=device)
    sequence_at = buf.data_ptr()
    position_at = sequence_at + 4 * tokens
    lens_at = position_at + 4 * tokens
    cu_at = lens_at + 4 * batch
    counts_at = cu_at + 4 * batch + 4
    if taken_out is None:
        taken_out, taken_out_at = own_taken, counts_at + 4
    else:
        taken_out_at = _dense(taken_out, "taken_out", i32, (1,), index)
    a = PagePlanArgs(table_at, _dense(held, "held", i32, (batch,), index),
                     _dense(new_tokens, "new_tokens", i32, (batch,), index),
                     _dense(free_pages, "free_pages", i32, (num_free,), index),
                     0 if taken is None else _dense(taken, "taken", i32, (1,), index), taken_out_at, counts_at, cu_at,
                     lens_at, sequence_at, position_at, slot.data_ptr(), stride, batch, pages, page_size, num_pages, num_free, tokens)
    rc = _entry("moe_layer_page_plan")(ctypes.byref(a), _raw_stream(index))
    if rc:
        _raise(rc, "moe_layer_page_plan")
    return PagePlan(cu_tokens, seq_lens, sequence, position, slot, taken_out, unplaced)


def _page_table(page_table: torch.Tensor, index: int) -> Tuple[int, int, int, int]:
    """Pointer, batch, pages and row stride of a page table."""
    if page_table.dtype is not torch.int32:
        raise TypeError("page_table: dtype %s, expected int32" % page_table.dtype)
    shape, strides = page_table.shape, page_table.stride()
    if len(shape) != 2:
        raise ValueError("page_table: %d dimensions, expected 2" % len(shape))
    if page_table.get_device() != index:
        raise ValueError("page_table: on %s, expected cuda:%d" % (page_table.device, index))
    batch, pages = shape
    if batch > _I32_MAX or pages > _I32_MAX:
        _too_large("page_table", max(shape))
    if pages > 1 and strides[1] != 1:
        raise ValueError("page_table: the pages of a sequence must be dense")
    return page_table.data_ptr(), batch, pages, strides[0] if batch > 1 else pages


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
    index, shape, xdtype = x.get_device(), x.shape, x.dtype
    if stream is not None or index < 0 or index != _device_index():
        with _On(x.device, stream):
            return w4_linear(x, w, w_scale, zero, x_scale, out_dtype, out)
    gshape = w_scale.shape
    if len(shape) != 2 or len(gshape) != 2:
        raise ValueError("x and w_scale have 2 dimensions")
    m, k = shape
    n, groups = gshape
    if m > _I32_MAX or k > _I32_MAX or n > _I32_MAX:
        _too_large("x or w_scale", max(m, k, n))
    xcode = DTYPE_CODES.get(xdtype, 2)
    if xcode == 2:
        raise TypeError("x: dtype %s, expected bfloat16, float16 or int8" % xdtype)
    if (xcode == 3) != (x_scale is not None):
        raise ValueError("x_scale is required with int8 x, and for int8 x only")
    if groups < 1 or k % groups:
        raise ValueError("w_scale: %d groups do not divide k = %d" % (groups, k))
    sdtype = w_scale.dtype
    scode = DTYPE_CODES.get(sdtype, 3)
    if scode == 3:
        raise TypeError("w_scale: dtype %s, expected bfloat16, float16 or float32" % sdtype)
    if out_dtype is None:
        out_dtype = out.dtype if out is not None else (torch.bfloat16 if xcode == 3 else xdtype)
    ocode = DTYPE_CODES.get(out_dtype, 3)
    if ocode == 3:
        raise TypeError("out_dtype: %s, expected bfloat16, float16 or float32" % out_dtype)
    a = W4Args()
    a.x, a.x_stride = _rows(x, "x", xdtype, shape, index)
    if x_scale is not None:
        a.x_scale = _dense(x_scale, "x_scale", torch.float32, (m,), index)
    a.w = _dense(w, "w", torch.uint8, (n, k // 2), index)
    a.w_scale = _dense(w_scale, "w_scale", sdtype, gshape, index)
    if zero is not None:
        a.w_zero = _dense(zero, "zero", torch.uint8, gshape, index)
    a.m, a.n, a.k, a.group = m, n, k, k // groups
    a.x_dtype, a.scale_dtype, a.out_dtype = xcode, scode, ocode
    if out is None:
        out = torch.empty((m, n), dtype=out_dtype, device=x.device)
        a.y = out.data_ptr()
    else:
        a.y = _dense(out, "out", out_dtype, (m, n), index)
    rc = _entry("moe_layer_w4_linear")(ctypes.byref(a), _raw_stream(index))
    if rc:
        _raise(rc, "moe_layer_w4_linear")
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
        if max(k.shape) > _I32_MAX:
            _too_large("k and v", max(k.shape))
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
        self._index = k.get_device()
        self._ws, self._ws_at, self._ws_streams = None, (0, 0), set()

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
            self._ws_at, self._ws_streams = (self._ws.data_ptr(), self._ws.numel()), {_raw_stream(self._index)}
            self._ws[:256].zero_()  # the status words: status() may come before the first attention
        return self._ws

    def _table(self, a, page_table: torch.Tensor) -> int:
        """Sets the page table's fields of `a`; returns the batch."""
        a.cache = self._args
        a.page_table, a.batch, a.max_pages, a.table_stride = _page_table(page_table, self._index)
        return a.batch

    def plan(self, page_table: torch.Tensor, held: torch.Tensor, new_tokens: torch.Tensor, free_pages: torch.Tensor,
             tokens: int, taken: Optional[torch.Tensor] = None, taken_out: Optional[torch.Tensor] = None,
             stream: Optional[torch.cuda.Stream] = None) -> PagePlan:
        """page_plan for this cache's pages: held is then `start` of append,
        the plan's cu_tokens and seq_lens go to append and attention."""
        if page_table.get_device() != self._index:
            raise ValueError("page_table: on %s, expected %s" % (page_table.device, self.device))
        return page_plan(page_table, held, new_tokens, free_pages, self.page_size, self._args.num_pages, tokens, taken,
                         taken_out, stream)

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, page_table: torch.Tensor, start: torch.Tensor,
               cu_tokens: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Write new tokens (moe_layer_kv_append).  k_new, v_new [tokens,
        kv_heads, head_dim] bf16 or fp16 (tokens may be strided); page_table
        [batch, max_pages] and start [batch] int32; cu_tokens [batch + 1]
        int32 where sequences get more or fewer tokens than one."""
        code, index, shape, dtype = _act(k_new, "k_new"), self._index, k_new.shape, k_new.dtype
        if stream is not None or index < 0 or index != _device_index():
            with _On(self.device, stream):
                return self.append(k_new, v_new, page_table, start, cu_tokens)
        if len(shape) != 3 or shape[1] != self.kv_heads or shape[2] != self.head_dim:
            raise ValueError("k_new: shape %s, expected [tokens, %d, %d]" % (tuple(shape), self.kv_heads, self.head_dim))
        if shape[0] > _I32_MAX:
            _too_large("k_new", shape[0])
        a = KvAppendArgs()
        batch = self._table(a, page_table)
        a.k_new, a.k_stride = _rows(k_new, "k_new", dtype, shape, index)
        a.v_new, a.v_stride = _rows(v_new, "v_new", dtype, shape, index)
        a.start = _dense(start, "start", torch.int32, (batch,), index)
        if cu_tokens is not None:
            a.cu_tokens = _dense(cu_tokens, "cu_tokens", torch.int32, (batch + 1,), index)
        elif shape[0] != batch:
            raise ValueError("k_new: %d tokens for %d sequences without cu_tokens" % (shape[0], batch))
        a.tokens, a.dtype = shape[0], code
        rc = _entry("moe_layer_kv_append")(ctypes.byref(a), _raw_stream(index))
        if rc:
            _raise(rc, "moe_layer_kv_append")

    def attention(self, q: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                  cu_q: Optional[torch.Tensor] = None, max_q: Optional[int] = None, scale: Optional[float] = None, window: int = 0,
                  out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
        """Attention of the query tokens over their sequences' keys
        (moe_layer_kv_attention).  q [tokens, heads, head_dim] bf16 or fp16
        (tokens may be strided), heads a multiple of kv_heads; seq_lens
        [batch] int32, the query tokens' own keys counted; cu_q [batch + 1]
        int32 with max_q, the most query tokens of a sequence (tokens past
        it stay unwritten, so it has to be given), where that is not one
        each; scale: head_dim ** -0.5 without it; window: keys that a
        token sees at most, itself among them (0: no limit).  Returns out
        [tokens, heads, head_dim]."""
        code, index, shape, dtype = _act(q, "q"), self._index, q.shape, q.dtype
        if stream is not None or index < 0 or index != _device_index():
            with _On(self.device, stream):
                return self.attention(q, page_table, seq_lens, cu_q, max_q, scale, window, out, workspace)
        if len(shape) != 3:
            raise ValueError("q: %d dimensions, expected 3" % len(shape))
        tokens, heads, dim = shape
        if dim != self.head_dim or heads % self.kv_heads:
            raise ValueError("q: %d heads of %d do not fit %d kv heads of %d" %
                             (heads, dim, self.kv_heads, self.head_dim))
        if tokens > _I32_MAX or heads > _I32_MAX:
            _too_large("q", max(tokens, heads))
        a = KvAttentionArgs()
        batch = self._table(a, page_table)
        a.q, a.q_stride = _rows(q, "q", dtype, shape, index)
        a.seq_lens = _dense(seq_lens, "seq_lens", torch.int32, (batch,), index)
        if cu_q is not None:
            a.cu_q = _dense(cu_q, "cu_q", torch.int32, (batch + 1,), index)
            if max_q is None:
                raise ValueError("max_q is required with cu_q")
        else:
            max_q = 1 if max_q is None else max_q
            if tokens != batch or max_q != 1:
                raise ValueError("q: %d tokens (max_q %d) for %d sequences without cu_q" % (tokens, max_q, batch))
        if max_q > _I32_MAX:
            _too_large("max_q", max_q)
        # positions end below 2^31: a wider window sees what that sees
        a.window = -1 if window < 0 else window if window <= _I32_MAX else _I32_MAX
        a.tokens, a.max_q, a.group_size, a.dtype = tokens, max_q if max_q > 0 else 0, heads // self.kv_heads, code
        a.sm_scale = dim ** -0.5 if scale is None else scale
        s = _raw_stream(index)
        if workspace is not None:
            ws_at, ws_bytes = _workspace(workspace, self._index)
        else:
            if self._ws is None:
                self.workspace()
            ws_at, ws_bytes = self._ws_at
            if s not in self._ws_streams:  # its memory stays until this stream is done, whatever becomes of the handle
                self._ws.record_stream(torch.cuda.current_stream(index))
                self._ws_streams.add(s)
        if out is None:
            out = torch.empty_like(q, memory_format=_CONTIGUOUS)
            a.out = out.data_ptr()
        else:
            a.out = _dense(out, "out", dtype, shape, index)
        rc = _entry("moe_layer_kv_attention")(ctypes.byref(a), ws_at, ws_bytes, s)
        if rc:
            _raise(rc, "moe_layer_kv_attention")
        return out

    def status(self, workspace: Optional[torch.Tensor] = None) -> int:
        """Synchronises the current stream; the code of the last attention on
        this workspace that had query tokens: 0, or MOE_ERR_DEVICE_TIMEOUT
        where a wait inside it gave up.  A workspace of the caller's own has
        to have been used by one."""
        at = self.workspace().data_ptr() if workspace is None else _workspace(workspace, self._index)[0]
        return _entry("moe_layer_kv_attention_status")(at, torch.cuda.current_stream(self.device).cuda_stream)
