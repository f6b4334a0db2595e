"""One decoder layer around the fused MoE expert block, from this package's
operators alone: RMS norm with int8 output, 4-bit projections, the paged int8
key / value cache with its attention, and the block.

  python examples/decoder_layer.py      # a prompt of three requests, then decode steps

Weights are random.  Rotary positions and the router's top-k are plain torch.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_ffn_dispatch_gb300 as m  # noqa: E402


def pack_w4(w: torch.Tensor, group: int):
    """(codes [n, k / 2] uint8, scales [n, k / group] bf16) of a weight [n, k], symmetric: zero point 8."""
    n, k = w.shape
    g = w.float().view(n, k // group, group)
    scale = (g.abs().amax(-1) / 7).clamp(min=1e-8).bfloat16()
    code = ((g / scale.float()[..., None]).round().clamp(-8, 7) + 8).to(torch.uint8).view(n, k)
    return code[:, 0::2] | (code[:, 1::2] << 4), scale


def unpack_w4(codes: torch.Tensor, scale: torch.Tensor) -> torch.Tensor:
    n, k = codes.shape[0], codes.shape[1] * 2
    w = torch.stack((codes & 15, codes >> 4), dim=-1).view(n, scale.shape[1], k // scale.shape[1]).float() - 8
    return (w * scale.float()[..., None]).view(n, k)


def rotate(x: torch.Tensor, pos: torch.Tensor) -> torch.Tensor:
    """Rotary positions: the two halves of a head as real and imaginary parts."""
    half = x.shape[-1] // 2
    freq = 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
    a = pos.float()[:, None, None] * freq
    re, im = x.float()[..., :half], x.float()[..., half:]
    return torch.cat((re * a.cos() - im * a.sin(), re * a.sin() + im * a.cos()), dim=-1).to(x.dtype)


class DecoderLayer:
    """Weights, a cache of `pages` pages and the expert block of one layer."""

    def __init__(self, hidden=1024, heads=8, kv_heads=2, head_dim=128, experts=16, topk=4, inter=512, pages=64,
                 page_size=64, max_tokens=512, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, std):
            return torch.randn(shape, device=device, generator=g) * std

        self.hidden, self.heads, self.kv_heads, self.head_dim, self.topk = hidden, heads, kv_heads, head_dim, topk
        qkv = (heads + 2 * kv_heads) * head_dim
        self.norm_attn = (torch.rand(hidden, device=device, generator=g) + 0.5).bfloat16()
        self.norm_ffn = (torch.rand(hidden, device=device, generator=g) + 0.5).bfloat16()
        self.qkv = pack_w4(randn(qkv, hidden, std=hidden ** -0.5), 64)
        self.out = pack_w4(randn(hidden, heads * head_dim, std=(heads * head_dim) ** -0.5), 128)
        self.gate = pack_w4(randn(experts, hidden, std=hidden ** -0.5), 32)
        self.cache = m.KvCache.empty(pages, kv_heads, page_size, head_dim, device)
        self.moe = m.MoeFused(max_tokens, hidden, experts, topk, inter, True, device)
        lim = 127

        def int8(*shape):
            return torch.randint(-lim, lim + 1, shape, device=device, generator=g, dtype=torch.int8)

        def scales(*shape, k):
            return (torch.rand(shape, device=device, generator=g) + 0.5) / (lim * k ** 0.5)

        self.experts = dict(
            w1=int8(experts, 2 * inter, hidden), w1_scale=scales(experts, 2 * inter, k=hidden),
            w2=int8(experts, hidden, inter), w2_scale=scales(experts, hidden, k=inter),
            share_w1=int8(2 * inter, hidden), share_w1_scale=scales(2 * inter, k=hidden),
            share_w2=int8(hidden, inter), share_w2_scale=scales(hidden, k=inter))

    def __call__(self, x, page_table, start, cu=None, max_q=1):
        """(residual stream after the attention, output of the experts) for
        tokens x [tokens, hidden] of sequences that hold `start` [batch] tokens
        already; cu [batch + 1] and max_q where they get more than one each.
        The next layer's norm adds the two."""
        H, G, D, T = self.kv_heads, self.heads // self.kv_heads, self.head_dim, x.shape[0]
        batch = start.shape[0]
        token = torch.arange(T, device=x.device)
        if cu is None:
            pos, lens = start, start + 1
        else:
            seq = (token[:, None] >= cu[1:]).sum(1)
            pos, lens = start[seq] + token - cu[seq], start + cu[1:] - cu[:-1]
        codes, scale, _, _ = m.add_rmsnorm_quant(x, self.norm_attn)
        qkv = m.w4_linear(codes, *self.qkv, x_scale=scale).view(T, (G + 2) * H, D)
        q, k, v = rotate(qkv[:, :G * H], pos), rotate(qkv[:, G * H:(G + 1) * H], pos), qkv[:, (G + 1) * H:]
        self.cache.append(k, v, page_table, start.int(), cu_tokens=cu)
        o = self.cache.attention(q, page_table, lens.int(), cu_q=cu, max_q=max_q)
        a = m.w4_linear(o.view(T, -1), *self.out)
        _, _, x, y = m.add_rmsnorm_quant(a, self.norm_ffn, residual=x, want_y=True)
        p = torch.softmax(m.w4_linear(y, *self.gate, out_dtype=torch.float32), dim=-1)
        w, ids = torch.topk(p, self.topk, dim=-1)
        routed, shared, _ = self.moe.forward_inputs(
            dict(x=y, expert_ids=ids.int(), expert_scales=(w / w.sum(-1, keepdim=True)).contiguous()), self.experts)
        assert batch == page_table.shape[0]
        return x, routed + shared


def main():
    layer = DecoderLayer()
    lens = [70, 5, 200]
    table = torch.arange(3 * 8, dtype=torch.int32, device="cuda").view(3, 8)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(sum(lens), layer.hidden, device="cuda", generator=g).bfloat16()
    cu = torch.tensor([0, 70, 75, 275], dtype=torch.int32, device="cuda")
    start = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, y = layer(x, table, start, cu, max_q=max(lens))
    print("prompt: %d tokens, residual rms %.3f, experts rms %.3f" % (x.shape[0], x.float().square().mean() ** 0.5,
                                                                      y.float().square().mean() ** 0.5))
    start = torch.tensor(lens, dtype=torch.int32, device="cuda")
    last = (cu[1:] - 1).long()
    x = (x + y)[last]
    for step in range(4):
        x, y = layer(x, table, start + step)
        x = x + y
    assert layer.cache.status() == 0 and layer.moe.status()["rc"] == 0
    print("4 decode steps of 3 requests: output rms %.3f" % (x.float().square().mean() ** 0.5))


if __name__ == "__main__":
    main()
