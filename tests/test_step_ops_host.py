"""The serving step's operators refuse what they cannot run, without a GPU:
refusals come before any CUDA call."""
import ctypes
import os
import subprocess

import pytest

import moe_expert_ffn_dispatch_gb300 as m
from moe_expert_ffn_dispatch_gb300 import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = [("moe_layer_norm_pair_args_t", layer.NormPairArgs), ("moe_layer_w8_args_t", layer.W8Args),
           ("moe_layer_page_plan_args_t", layer.PagePlanArgs), ("moe_layer_logprobs_args_t", layer.LogprobsArgs)]
A = 1 << 20  # an aligned address that nothing reads
INVALID, SHAPE, ALIGN, OK = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED_SHAPE, m.MOE_ERR_ALIGNMENT, m.MOE_OK


@pytest.fixture(scope="module")
def built():
    from moe_expert_ffn_dispatch_gb300 import _build
    _build.build()
    return m.lib()


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


def pair_args(**kw):
    a = layer.NormPairArgs(x=A, residual=A, post_weight=A, weight=A, residual_out=A, q=A, q_scale=A, x_stride=64,
                           residual_stride=64, residual_out_stride=64, rows=2, hidden=64, eps=1e-6, branch_scale=1.0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw, code", [
    (dict(x=0), INVALID), (dict(residual=0), INVALID), (dict(post_weight=0), INVALID), (dict(weight=0), INVALID),
    (dict(residual_out=0), INVALID), (dict(q=0), INVALID), (dict(q_scale=0), INVALID), (dict(q=0, q_scale=0), INVALID),
    (dict(dtype=2), INVALID), (dict(weight_dtype=1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(branch_scale=float("nan")), INVALID), (dict(x_stride=63), INVALID), (dict(residual_stride=0), INVALID),
    (dict(residual_out_stride=63), INVALID), (dict(gate=A, gate_stride=63), INVALID), (dict(gate=A, gate_stride=-64), INVALID),
    (dict(rows=-1), SHAPE), (dict(hidden=0), SHAPE), (dict(hidden=16385), SHAPE), (dict(x=A + 1), ALIGN),
    (dict(gate=A + 1), ALIGN), (dict(weight=A + 1), ALIGN), (dict(weight_dtype=2, post_weight=A + 2), ALIGN),
    (dict(smooth=A + 2), ALIGN), (dict(q_scale=A + 1), ALIGN), (dict(y_out=A + 1), ALIGN), (dict(rows=0, x=0, q=0), OK)])
def test_pair_refusals(built, kw, code):
    assert built.moe_layer_norm_add_rmsnorm_quant(ctypes.byref(pair_args(**kw)), 0) == code


def w8_args(**kw):
    a = layer.W8Args(x=A, x_scale=A, w=A, w_scale=A, y=A, x_stride=256, m=2, n=16, k=256, scale_dtype=2, out_dtype=0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw, code", [
    (dict(x=0), INVALID), (dict(x_scale=0), INVALID), (dict(w=0), INVALID), (dict(w_scale=0), INVALID), (dict(y=0), INVALID),
    (dict(scale_dtype=3), INVALID), (dict(out_dtype=3), INVALID), (dict(x_stride=240), INVALID), (dict(m=-1), SHAPE),
    (dict(m=1000001), SHAPE), (dict(n=0), SHAPE), (dict(n=2 ** 31 - 2 ** 20), SHAPE), (dict(k=0), SHAPE), (dict(k=8), SHAPE),
    (dict(k=248), SHAPE), (dict(k=65552, x_stride=1 << 20), SHAPE), (dict(x=A + 8), ALIGN), (dict(x_stride=264), ALIGN),
    (dict(w=A + 8), ALIGN), (dict(x_scale=A + 2), ALIGN), (dict(w_scale=A + 2), ALIGN), (dict(scale_dtype=0, w_scale=A + 1), ALIGN),
    (dict(y=A + 1), ALIGN), (dict(out_dtype=2, y=A + 2), ALIGN), (dict(m=0, x=0, y=0), OK)])
def test_w8_refusals(built, kw, code):
    assert built.moe_layer_w8_linear(ctypes.byref(w8_args(**kw)), A, 1 << 40, 0) == code


def test_w8_workspace_refusals(built):
    nb = ctypes.c_size_t(0)
    size = built.moe_layer_w8_linear_workspace_size
    assert size(4, 4, 64, None) == INVALID
    for sizes in ((-1, 4, 64), (1000001, 4, 64), (4, 0, 64), (4, 4, 0), (4, 4, 40), (4, 4, 65552)):
        assert size(*sizes, ctypes.byref(nb)) == SHAPE
    assert built.moe_layer_w8_linear(ctypes.byref(w8_args()), A + 16, 1 << 40, 0) == ALIGN
    assert built.moe_layer_w8_linear_status(0, 0) == INVALID
    assert built.moe_layer_w8_linear_status(A + 16, 0) == ALIGN


def plan_args(**kw):
    a = layer.PagePlanArgs(page_table=A, held=A, new_tokens=A, free_pages=A, taken_out=A, unplaced=A, cu_tokens=A, seq_lens=A,
                           sequence=A, position=A, slot=A, table_stride=8, batch=2, max_pages=8, page_size=16, num_pages=4,
                           num_free=3, tokens=5)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw, code", [
    (dict(page_table=0), INVALID), (dict(held=0), INVALID), (dict(new_tokens=0), INVALID), (dict(free_pages=0), INVALID),
    (dict(taken_out=0), INVALID), (dict(unplaced=0), INVALID), (dict(cu_tokens=0), INVALID), (dict(seq_lens=0), INVALID),
    (dict(table_stride=7), INVALID), (dict(batch=-1), SHAPE), (dict(batch=4097), SHAPE), (dict(max_pages=-1), SHAPE),
    (dict(batch=4096, max_pages=1 << 19, table_stride=1 << 19), SHAPE), (dict(page_size=48), SHAPE), (dict(num_pages=-1), SHAPE),
    (dict(num_free=-1), SHAPE), (dict(tokens=-1), SHAPE), (dict(held=A + 2), ALIGN), (dict(taken=A + 1), ALIGN),
    (dict(slot=A + 4), ALIGN), (dict(position=A + 2), ALIGN), (dict(cu_tokens=A + 3), ALIGN)])
def test_plan_refusals(built, kw, code):
    assert built.moe_layer_page_plan(ctypes.byref(plan_args(**kw)), 0) == code


def logprobs_args(**kw):
    a = layer.LogprobsArgs(logits=A, tokens=A, logprob=A, entropy=A, top_logprob=A, top_id=A, logits_stride=100, rows=2,
                           vocab=100, num_tokens=1, top=5, dtype=0, tokens_64=0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw, code", [
    (dict(logits=0), INVALID), (dict(tokens=0), INVALID), (dict(logprob=0), INVALID), (dict(top_logprob=0), INVALID),
    (dict(top_id=0), INVALID), (dict(dtype=3), INVALID), (dict(tokens_64=2), INVALID), (dict(logits_stride=99), INVALID),
    (dict(rows=-1), SHAPE), (dict(vocab=0), SHAPE), (dict(num_tokens=-1), SHAPE), (dict(top=-1), SHAPE), (dict(top=33), SHAPE),
    (dict(vocab=4, top=5), SHAPE), (dict(logits=A + 1), ALIGN), (dict(dtype=2, logits=A + 2), ALIGN), (dict(tokens=A + 2), ALIGN),
    (dict(tokens_64=1, tokens=A + 4), ALIGN), (dict(entropy=A + 1), ALIGN), (dict(top_id=A + 2), ALIGN),
    (dict(rows=0, logits=0, tokens=0), OK)])
def test_logprobs_refusals(built, kw, code):
    assert built.moe_layer_token_logprobs(ctypes.byref(logprobs_args(**kw)), 0) == code


def test_null_arguments(built):
    for name in ("moe_layer_norm_add_rmsnorm_quant", "moe_layer_page_plan", "moe_layer_token_logprobs"):
        assert getattr(built, name)(None, 0) == INVALID
    assert built.moe_layer_w8_linear(None, A, 1 << 40, 0) == INVALID


def test_binding_has_no_cpu_path_and_checks_types():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    x8, one, i = torch.zeros(2, 64, dtype=torch.int8), torch.ones(2), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: m.norm_add_rmsnorm_quant(x, x, w, w), lambda: m.w8_linear(x8, x8, one, one),
                 lambda: m.token_logprobs(x), lambda: m.page_plan(i.view(2, 1), i, i, i, 16, 4, 2),
                 lambda: m.w8_linear_workspace(2, 2, 64, "cpu"), lambda: m.w8_linear_status(x8)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        m.norm_add_rmsnorm_quant(x8, x, w, w)
    with pytest.raises(TypeError):
        m.token_logprobs(x8)


def test_waits_of_the_w8_kernel_have_one_answer_for_a_warp():
    """As in the attention's tensor-memory kernel: lanes that decided alone could part for ever.  Every wait goes through
    the voted one, but for those after the roles, whose answers nobody takes."""
    import re
    src = open(os.path.join(ROOT, "moe_expert_ffn_dispatch_gb300", "csrc", "w8_linear_tc.cu")).read()
    src = re.sub(r"//[^\n]*", "", src)
    calls = [src[src.rfind("\n", 0, c.start()):src.index(";", c.start())].strip()
             for c in re.finditer(r"\bmbar_(wait_bounded|try_wait|test_wait)\s*\(", src)]
    voted = [c for c in calls if "__all_sync(0xffffffffu," in c]
    after = [c for c in calls if re.search(r"&full\[i\]|&bar\.drain", c)]
    assert len(voted) == 1 and len(voted) + len(after) == len(calls), calls
    # and each answer is taken: no call of the voted wait stands by itself
    assert not re.search(r"[;{}]\s*wait\(", src)


def test_waits_of_a_pair_of_ctas_in_the_w8_kernel():
    """What both CTAs of a pair complete is waited for over the cluster, by the voted wait of that kind, whose answer is
    taken; and nothing of the pair ends before the cluster's last barrier."""
    import re
    src = open(os.path.join(ROOT, "moe_expert_ffn_dispatch_gb300", "csrc", "w8_linear_tc.cu")).read()
    src = re.sub(r"//[^\n]*", "", src)
    over = [src[src.rfind("\n", 0, c.start()):src.index(";", c.start())] for c in re.finditer(r"mbar_wait_bounded<", src)]
    assert len(over) == 1 and "__all_sync(0xffffffffu," in over[0]
    assert not re.search(r"[;{}]\s*wait_both\(", src)
    takers = re.findall(r"ok = ok && wait_both\(&bar\.(\w+)", src)
    assert sorted(takers) == ["acc_empty", "full"] == sorted(re.findall(r"wait_both\(&bar\.(\w+)", src))
    assert src.index("pair_dealloc(tmem") > src.rindex("if constexpr (FORM == kTwo) cluster_sync();") > src.rindex("wait(&bar")
