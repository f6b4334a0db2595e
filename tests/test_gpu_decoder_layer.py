"""The example's decoder layer against the same layer in plain fp32 torch:
dequantised weights, no quantisation of activations or cache.

The int8 steps (norm output, cache, both quants of the experts) each leave
about 0.5 to 1 % of a row's rms; four of them in a row stay within 6 %."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def norm(x, w, eps=1e-6):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.float()


def plain_layer(ex, layer, x, keys, values, pos0):
    """One sequence: x [tokens, hidden] fp32 at positions pos0 ..; keys, values: lists of what came before."""
    H, G, D, T = layer.kv_heads, layer.heads // layer.kv_heads, layer.head_dim, x.shape[0]
    pos = torch.arange(pos0, pos0 + T, device=x.device)
    qkv = (norm(x, layer.norm_attn) @ ex.unpack_w4(*layer.qkv).t()).view(T, (G + 2) * H, D)
    q, k = ex.rotate(qkv[:, :G * H], pos), ex.rotate(qkv[:, G * H:(G + 1) * H], pos)
    keys.append(k)
    values.append(qkv[:, (G + 1) * H:])
    k, v = torch.cat(keys), torch.cat(values)
    a = torch.einsum("tngd,snd->ntgs", q.view(T, H, G, D), k) * D ** -0.5
    a = a.masked_fill(torch.arange(k.shape[0], device=x.device) > pos[:, None, None], float("-inf")).softmax(-1)
    o = torch.einsum("ntgs,snd->tngd", a, v).reshape(T, -1)
    x = x + o @ ex.unpack_w4(*layer.out).t()
    y = norm(x, layer.norm_ffn)
    p = (y @ ex.unpack_w4(*layer.gate).t()).softmax(-1)
    w, ids = p.topk(layer.topk)
    w = w / w.sum(-1, keepdim=True)
    e = layer.experts

    def ffn(y, w1, s1, w2, s2):
        h = y @ (w1.float() * s1[:, None]).t()
        n = h.shape[-1] // 2
        return (torch.nn.functional.silu(h[:, :n]) * h[:, n:]) @ (w2.float() * s2[:, None]).t()

    out = ffn(y, e["share_w1"], e["share_w1_scale"], e["share_w2"], e["share_w2_scale"])
    for t in range(T):
        for j in range(layer.topk):
            i = int(ids[t, j])
            out[t] += w[t, j] * ffn(y[t:t + 1], e["w1"][i], e["w1_scale"][i], e["w2"][i], e["w2_scale"][i])[0]
    return x, out, p


def test_layer_matches_plain_torch():
    import decoder_layer as ex
    layer = ex.DecoderLayer(hidden=512, heads=8, kv_heads=2, head_dim=64, experts=8, topk=2, inter=256, pages=40,
                            page_size=16, max_tokens=128)
    lens = [37, 3, 20]
    table = torch.randperm(40, device="cuda")[:24].view(3, 8).int()
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(sum(lens), 512, device="cuda", generator=g).bfloat16()
    cu = torch.tensor([0, 37, 40, 60], dtype=torch.int32, device="cuda")
    start = torch.zeros(3, dtype=torch.int32, device="cuda")
    held = [([], []) for _ in lens]
    for step in range(3):
        got_x, got_y = layer(x, table, start, cu if step == 0 else None, max_q=37 if step == 0 else 1)
        ends = cu.tolist() if step == 0 else [0, 1, 2, 3]
        for b in range(3):
            rows = slice(ends[b], ends[b + 1])
            wx, wy, p = plain_layer(ex, layer, x[rows].float(), *held[b], int(start[b]))
            err = (got_x[rows].float() - wx).norm(dim=-1) / wx.norm(dim=-1)
            assert float(err.max()) < 0.06, (step, b, float(err.max()))
            # tokens whose choice of experts is not a near tie
            top = p.topk(layer.topk + 1).values
            sure = top[:, -2] > 1.1 * top[:, -1]
            err = ((got_y[rows].float() - wy).norm(dim=-1) / wy.norm(dim=-1))[sure]
            assert not len(err) or float(err.max()) < 0.06, (step, b, float(err.max()))
        assert layer.cache.status() == 0 and layer.moe.status()["rc"] == 0
        last = (cu[1:] - 1).long() if step == 0 else torch.arange(3, device="cuda")
        start = start + (torch.tensor(lens, dtype=torch.int32, device="cuda") if step == 0 else 1)
        x = (got_x + got_y)[last]
