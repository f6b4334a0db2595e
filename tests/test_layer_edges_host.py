"""What of the decoder-layer operators' edges shows without a GPU."""
import os
import re
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_expert_ffn_dispatch_gb300", "csrc")


def test_bounded_waits_of_the_chunk_kernel_have_one_answer_for_a_warp():
    """A wait that gives up ends its warp's role.  If lanes decided alone, one could pass the barrier in the poll in
    which its neighbour gives up, go on, and stand at the next warp-wide operation for ever, the neighbour being at the
    kernel's last barrier.  So every wait asks all lanes, at once or before any lane can leave or meet the others; the
    one after the last role, whose answer nobody takes, is the exception."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "kv_attention_chunk.cu")).read())
    calls = [m.start() for m in re.finditer(r"\bmbar_(wait_bounded|try_wait)\s*\(", src)]
    assert calls
    alone = []
    for at in calls:
        end = src.index(";", at)
        statement = src[max(src.rfind(c, 0, at) for c in ";{}") + 1:end]
        if "__all_sync(" in statement or re.search(r"&bar\.drain,[^;]*nullptr", statement):
            continue
        vote = src.find("if (!__all_sync(0xffffffffu, ok)) break;", end)
        if not re.search(r"\bok = (moe::)?mbar_wait_bounded", statement) or vote < 0 or \
                re.search(r"\b(break|return|continue|goto|wait|\w+_segment|pages_of_next|__\w+_sync|__sync\w+)\b", src[end:vote]):
            alone.append(statement.strip())
    assert alone == []
    # and each answer is taken: no call of the voted wait stands by itself
    assert not re.search(r"[;{}]\s*wait\(", src)


def test_the_package_imports_where_torch_has_no_cuda_build():
    prog = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import moe_expert_ffn_dispatch_gb300 as m
x, w = torch.ones(2, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
code, scale = torch.zeros(16, 32, dtype=torch.uint8), torch.ones(16, 2, dtype=torch.bfloat16)
for call in (lambda: m.add_rmsnorm_quant(x, w), lambda: m.w4_linear(x, code, scale),
             lambda: m.KvCache.empty(2, 1, 16, 64, device="cpu")):
    try:
        call()
    except ValueError as e:
        assert "CUDA" in str(e), e
    else:
        raise AssertionError("ran without a GPU")
print("imported")
"""
    out = subprocess.run([sys.executable, "-c", prog], cwd=ROOT, capture_output=True, text=True)
    assert out.returncode == 0 and "imported" in out.stdout, out.stderr


def test_w4_refuses_row_numbers_that_could_pass_32_bits():
    """The tiles of a launch go past n by up to 16 rows for each of 16 warps of every SM; a row number that wrapped
    would pass for one below n."""
    import ctypes
    import moe_expert_ffn_dispatch_gb300 as m
    from moe_expert_ffn_dispatch_gb300 import _build, layer
    _build.build()
    at = 1 << 20  # an aligned address that nothing reads
    for n, code in ((2 ** 31 - 1, m.MOE_ERR_UNSUPPORTED_SHAPE), (2 ** 31 - 2 ** 20, m.MOE_ERR_UNSUPPORTED_SHAPE),
                    (2 ** 31 - 2 ** 20 - 1, m.MOE_OK)):
        a = layer.W4Args(x=at, w=at, w_scale=at, y=at, x_stride=256, m=0, n=n, k=256, group=128, x_dtype=0, scale_dtype=0,
                         out_dtype=0)
        assert m.lib().moe_layer_w4_linear(ctypes.byref(a), 0) == code
    most = 2 ** 31 - 2 ** 20 - 1
    past = 16 * 16 * 1024  # a thousand SMs
    assert -(-most // 16) * 16 + past < 2 ** 31
