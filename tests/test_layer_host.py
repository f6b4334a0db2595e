"""The decoder-layer header and its binding agree, and the entry points refuse
what they cannot run, without a GPU: refusals come before any CUDA call."""
import ctypes
import os
import re
import subprocess

import pytest

import moe_expert_ffn_dispatch_gb300 as m
from moe_expert_ffn_dispatch_gb300 import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_layer.h")
STRUCTS = [("moe_layer_norm_args_t", layer.NormArgs), ("moe_layer_w4_args_t", layer.W4Args),
           ("moe_layer_kv_cache_t", layer.KvCacheArgs), ("moe_layer_kv_append_args_t", layer.KvAppendArgs),
           ("moe_layer_kv_attention_args_t", layer.KvAttentionArgs)]


@pytest.fixture(scope="module")
def built():
    from moe_expert_ffn_dispatch_gb300 import _build
    _build.build()
    return m.lib()


def test_exports_match_header(built):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(moe_layer_\w+)\s*\(", src)))
    assert declared == sorted(layer.LAYER_EXPORTS)
    for name in declared:
        getattr(built, name)


def test_struct_layouts_match_header(tmp_path):
    lines, want = [], []
    for c_name, py in STRUCTS:
        lines.append('printf("%%zu\\n", sizeof(%s));' % c_name)
        want.append(ctypes.sizeof(py))
        for field, _ in py._fields_:
            lines.append('printf("%%zu\\n", offsetof(%s, %s));' % (c_name, field))
            want.append(getattr(py, field).offset)
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_layer.h"\nint main(void) {\n' +
                    "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)])
    assert [int(v) for v in subprocess.check_output([str(exe)]).split()] == want


A = 1 << 20  # an aligned address that nothing reads


def norm_args(**kw):
    a = layer.NormArgs(x=A, weight=A, q=A, q_scale=A, x_stride=64, rows=2, hidden=64, dtype=0, weight_dtype=0, eps=1e-6)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def w4_args(**kw):
    a = layer.W4Args(x=A, w=A, w_scale=A, y=A, x_stride=256, m=1, n=16, k=256, group=128, x_dtype=0, scale_dtype=0,
                     out_dtype=0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def cache_args(**kw):
    c = layer.KvCacheArgs(k=A, v=A, k_scale=A, v_scale=A, page_stride=8 * 64 * 128, head_stride=64 * 128,
                          scale_stride=8, num_pages=4, kv_heads=8, page_size=64, head_dim=128)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def append_args(cache=None, **kw):
    a = layer.KvAppendArgs(cache=cache or cache_args(), k_new=A, v_new=A, page_table=A, start=A, k_stride=1024,
                           v_stride=1024, table_stride=4, tokens=2, batch=2, max_pages=4, dtype=0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def attention_args(cache=None, **kw):
    a = layer.KvAttentionArgs(cache=cache or cache_args(), q=A, out=A, page_table=A, seq_lens=A, q_stride=4096,
                              table_stride=4, tokens=2, batch=2, max_pages=4, max_q=1, group_size=4, window=0, dtype=0,
                              sm_scale=1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


INVALID, SHAPE, ALIGN = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED_SHAPE, m.MOE_ERR_ALIGNMENT


@pytest.mark.parametrize("kw, code", [
    (dict(x=0), INVALID), (dict(weight=0), INVALID), (dict(q=0), INVALID), (dict(q_scale=0), INVALID),
    (dict(dtype=2), INVALID), (dict(dtype=3), INVALID), (dict(weight_dtype=1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(residual=A), INVALID), (dict(residual_out=A), INVALID),
    (dict(x_stride=63), INVALID), (dict(residual=A, residual_out=A, residual_stride=64, residual_out_stride=8), INVALID),
    (dict(rows=-1), SHAPE), (dict(hidden=0), SHAPE), (dict(hidden=16385, x_stride=16385), SHAPE),
    (dict(x=A + 1), ALIGN), (dict(q_scale=A + 2), ALIGN), (dict(smooth=A + 2), ALIGN), (dict(y_out=A + 1), ALIGN),
    (dict(rows=0, x=0, q=0), m.MOE_OK)])
def test_norm_refusals(built, kw, code):
    assert built.moe_layer_add_rmsnorm_quant(ctypes.byref(norm_args(**kw)), 0) == code


@pytest.mark.parametrize("kw, code", [
    (dict(x=0), INVALID), (dict(w=0), INVALID), (dict(w_scale=0), INVALID), (dict(y=0), INVALID),
    (dict(x_dtype=2), INVALID), (dict(x_dtype=3), INVALID), (dict(x_scale=A), INVALID), (dict(out_dtype=3), INVALID),
    (dict(scale_dtype=3), INVALID), (dict(x_stride=255), INVALID), (dict(m=-1), SHAPE), (dict(n=0), SHAPE),
    (dict(k=0), SHAPE), (dict(k=255), SHAPE), (dict(group=16), SHAPE), (dict(group=96), SHAPE), (dict(group=0), SHAPE),
    (dict(k=320, x_stride=320), SHAPE), (dict(k=65536 + 128, x_stride=1 << 20), SHAPE), (dict(x=A + 8), ALIGN),
    (dict(x_stride=257), ALIGN), (dict(w=A + 8), ALIGN), (dict(w_scale=A + 1), ALIGN),
    (dict(scale_dtype=2, w_scale=A + 2), ALIGN), (dict(y=A + 1), ALIGN), (dict(m=0, x=0, y=0), m.MOE_OK)])
def test_w4_refusals(built, kw, code):
    assert built.moe_layer_w4_linear(ctypes.byref(w4_args(**kw)), 0) == code


CACHE_REFUSALS = [
    (dict(k=0), INVALID), (dict(v_scale=0), INVALID), (dict(num_pages=0), SHAPE), (dict(kv_heads=0), SHAPE),
    (dict(kv_heads=1025), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=256), SHAPE), (dict(head_dim=96), SHAPE),
    (dict(k=A + 8), ALIGN), (dict(page_stride=8 * 64 * 128 + 8), ALIGN), (dict(head_stride=100), ALIGN),
    (dict(page_stride=-16), INVALID)]


@pytest.mark.parametrize("kw, code", [
    (dict(k_new=0), INVALID), (dict(page_table=0), INVALID), (dict(start=0), INVALID), (dict(dtype=2), INVALID),
    (dict(tokens=3), INVALID), (dict(k_stride=1023), INVALID), (dict(table_stride=3), INVALID), (dict(tokens=-1), SHAPE),
    (dict(batch=4097, tokens=4097), SHAPE), (dict(max_pages=-1), SHAPE), (dict(k_new=A + 8), ALIGN),
    (dict(v_stride=1028), ALIGN), (dict(start=A + 1), ALIGN), (dict(cu_tokens=A + 2), ALIGN),
    (dict(tokens=0, k_new=0), m.MOE_OK), (dict(batch=0, tokens=0, start=0), m.MOE_OK)])
def test_append_refusals(built, kw, code):
    assert built.moe_layer_kv_append(ctypes.byref(append_args(**kw)), 0) == code


@pytest.mark.parametrize("kw, code", [
    (dict(q=0), INVALID), (dict(out=0), INVALID), (dict(seq_lens=0), INVALID), (dict(page_table=0), INVALID),
    (dict(dtype=2), INVALID), (dict(window=-1), INVALID), (dict(sm_scale=float("nan")), INVALID),
    (dict(tokens=3), INVALID), (dict(max_q=2), INVALID), (dict(q_stride=4095), INVALID), (dict(table_stride=3), INVALID),
    (dict(max_q=0), SHAPE), (dict(group_size=0), SHAPE), (dict(group_size=129), SHAPE), (dict(batch=4097), SHAPE),
    (dict(tokens=-1), SHAPE), (dict(q=A + 8), ALIGN), (dict(q_stride=4100), ALIGN), (dict(out=A + 8), ALIGN),
    (dict(seq_lens=A + 2), ALIGN), (dict(tokens=0, batch=0, q=0), m.MOE_OK)])
def test_attention_refusals(built, kw, code):
    a = attention_args(**kw)
    assert built.moe_layer_kv_attention(ctypes.byref(a), A, 1 << 30, 0) == code


@pytest.mark.parametrize("kw, code", CACHE_REFUSALS)
def test_cache_refusals(built, kw, code):
    c = cache_args(**kw)
    assert built.moe_layer_kv_append(ctypes.byref(append_args(cache=c)), 0) == code
    assert built.moe_layer_kv_attention(ctypes.byref(attention_args(cache=c)), A, 1 << 30, 0) == code


def test_null_arguments_and_workspace(built):
    for name in ("moe_layer_add_rmsnorm_quant", "moe_layer_w4_linear", "moe_layer_kv_append"):
        assert getattr(built, name)(None, 0) == INVALID
    assert built.moe_layer_kv_attention(None, A, 1 << 30, 0) == INVALID
    assert built.moe_layer_kv_attention(ctypes.byref(attention_args()), 0, 1 << 30, 0) == INVALID
    assert built.moe_layer_kv_attention(ctypes.byref(attention_args()), A + 16, 1 << 30, 0) == ALIGN
    nb = ctypes.c_size_t(0)
    assert built.moe_layer_kv_attention_workspace_size(128, None) == INVALID
    assert built.moe_layer_kv_attention_workspace_size(80, ctypes.byref(nb)) == SHAPE


def test_binding_has_no_cpu_path():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        m.add_rmsnorm_quant(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        m.w4_linear(x, torch.zeros(16, 32, dtype=torch.uint8), torch.ones(16, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        m.KvCache.empty(2, 1, 16, 64, device="cpu")
