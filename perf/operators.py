"""The decoder-layer operators around the fused MoE expert block, as workloads.

Four operators: the residual addition with RMS norm and an int8 output
("norm"), products with 4-bit weights and group scales ("w4"), the quantised
write into the paged int8 key / value cache ("append") and attention over
that cache ("attention").  `run` computes each in plain torch operations, or,
where `own` is true, by this package's entry points.

The ragged lengths of a case come from the case alone (its "mix"), so that
`work` knows them; values come from the seed.
"""
import math
import random

import torch

own = False

BF16, FP16, F32 = "bfloat16", "float16", "float32"


def listed():
    return [
        # 8 tokens (4 requests x 2 rows) of the decode step, hidden size of the block's configurations
        dict(name="norm_decode8", op="norm", T=8, h=4096, dtype=BF16, residual=True, smooth=False, y=True),
        # a prefill batch that is not a round number of tokens, with smooth scales before the quant
        dict(name="norm_prefill", op="norm", T=4093, h=4096, dtype=BF16, residual=True, smooth=True, y=True),
        # attention output projection for a single token
        dict(name="w4_out_one", op="w4", M=1, N=4096, K=4096, group=128, dtype=BF16, x8=False, zero=False, out=BF16),
        # query / key / value projection of one decode step: 32 + 2 x 8 heads of 128, int8 activations, zeros
        dict(name="w4_qkv_decode8", op="w4", M=8, N=6144, K=4096, group=64, dtype=BF16, x8=True, zero=True, out=BF16),
        # output head over a large vocabulary, ragged N
        dict(name="w4_head16", op="w4", M=16, N=130001, K=4096, group=128, dtype=FP16, x8=False, zero=False, out=FP16),
        # one new token each for 64 requests
        dict(name="append_decode64", op="append", B=64, n=1, start=120, Hkv=8, D=128, page=64, dtype=BF16, mix=1),
        # four prompts written in one call, ragged
        dict(name="append_prompt", op="append", B=4, n=2048, start=100, Hkv=8, D=128, page=64, dtype=BF16, mix=2),
        # a single request with a short context: latency
        dict(name="attn_one_request", op="attention", B=1, qmax=1, ctx=1009, Hkv=8, G=4, D=128, page=64, dtype=BF16,
             window=0, mix=3),
        # decode step of 64 requests, ragged contexts (one of them empty)
        dict(name="attn_decode64", op="attention", B=64, qmax=1, ctx=8191, Hkv=8, G=8, D=128, page=64, dtype=BF16,
             window=0, mix=4),
        # two requests with very long contexts
        dict(name="attn_long", op="attention", B=2, qmax=1, ctx=200003, Hkv=8, G=4, D=128, page=128, dtype=FP16,
             window=0, mix=5),
        # checking of drafted tokens: up to 4 rows a request, sliding window, small pages and heads
        dict(name="attn_verify", op="attention", B=16, qmax=4, ctx=4001, Hkv=4, G=8, D=64, page=16, dtype=FP16,
             window=1024, mix=6),
        # pieces of long prompts: ragged chunks of up to 512 tokens over what the cache already holds
        dict(name="attn_chunk", op="attention", B=4, qmax=512, ctx=4500, Hkv=8, G=4, D=128, page=64, dtype=BF16,
             window=0, mix=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "w4", "append", "attention", "attention"])
    dtype = rng.choice([BF16, FP16])
    if op == "norm":
        h = _log(rng, 64, 16384)
        if rng.random() < 0.5:
            h = -(-h // 64) * 64
        T = _log(rng, 1, max(1, min(8192, 4093 * 4096 // h)))
        return dict(op=op, T=T, h=h, dtype=dtype, residual=rng.random() < 0.75, smooth=rng.random() < 0.5,
                    y=rng.random() < 0.75)
    if op == "w4":
        group = rng.choice([32, 64, 128])
        K = group * _log(rng, 2, 16384 // group)
        M = _log(rng, 1, 64)
        N = _log(rng, 1, max(1, min(130001, 130001 * 4096 // K, 16 * 130001 * 4096 // (M * K))))
        return dict(op=op, M=M, N=N, K=K, group=group, dtype=dtype, x8=rng.random() < 0.3, zero=rng.random() < 0.5,
                    out=F32 if rng.random() < 0.15 else dtype)
    D, page, Hkv = rng.choice([64, 128]), rng.choice([16, 32, 64, 128]), rng.choice([1, 2, 4, 8])
    mix = rng.randrange(1 << 20)
    if op == "append":
        n = 1 if rng.random() < 0.5 else _log(rng, 2, 2048)
        return dict(op=op, B=_log(rng, 1, max(1, min(256, 8192 // n))), n=n, start=_log(rng, 1, 500), Hkv=Hkv, D=D,
                    page=page, dtype=dtype, mix=mix)
    G = rng.choice([1, 2, 3, 4, 5, 8, 16])
    qmax = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 16, 512)])
    B = _log(rng, 1, 64 if qmax <= 8 else 4)
    top = min(200003, 64 * 8191 * 8 * 128 // (B * Hkv * D), 4 * 32 * 512 * 4500 // (B * qmax * Hkv * G))
    return dict(op=op, B=B, qmax=qmax, ctx=_log(rng, 1, max(2, top - qmax)), Hkv=Hkv, G=G, D=D, page=page,
                dtype=dtype, window=rng.choice([0, 0, _log(rng, 1, 4096)]), mix=mix)


# ------------------------------------------------------------ lengths of a case
def _append_lens(c):
    """Tokens that each sequence already has, and that it gets."""
    r = random.Random(c["mix"])
    start = [r.randint(0, c["start"]) for _ in range(c["B"])]
    n = [c["n"]] + [r.randint(1, c["n"]) for _ in range(c["B"] - 1)]
    return start, n


def _attn_lens(c):
    """Query tokens of each sequence and keys that it has (those of the query tokens among them)."""
    r = random.Random(c["mix"])
    qlen = [c["qmax"]] + [r.randint(1, c["qmax"]) for _ in range(c["B"] - 1)]
    held = [c["ctx"]] + [_log(r, 1, c["ctx"]) for _ in range(c["B"] - 1)]
    kv = [a + b - 1 for a, b in zip(held, qlen)]
    if c["B"] >= 8:
        kv[c["B"] // 2] = 0  # a slot of the batch that holds no request
    return qlen, kv


def _cum(v):
    out = [0]
    for x in v:
        out.append(out[-1] + x)
    return out


# ------------------------------------------------------------ inputs
def _paged(kv, page, g):
    """A page table [B, most pages] over a shuffled pool, -1 where a sequence has no page; the pool's size."""
    need = [-(-x // page) for x in kv]
    pool = sum(need) + 3
    ids = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(kv), max(1, max(need))), -1, dtype=torch.int32)
    at, where = _cum(need), ids.cpu()
    for b, m in enumerate(need):
        table[b, :m] = where[at[b]:at[b] + m]
    return table.cuda(), pool


def _pool(pool, c, g):
    """A filled cache: codes of normal values, scales of pages whose largest value varies."""
    shape = (pool, c["Hkv"], c["page"], c["D"])
    codes = []
    for _ in range(2):
        t = torch.empty(shape, dtype=torch.int8, device="cuda")
        step = max(1, (1 << 27) // (shape[1] * shape[2] * shape[3]))
        for i in range(0, pool, step):
            p = t[i:i + step]
            p.copy_(torch.empty(p.shape, device="cuda").normal_(0.0, 32.0, generator=g).round_().clamp_(-127, 127))
        codes.append(t)
    ks, vs = (torch.empty(shape[:2], device="cuda").uniform_(-0.5, 0.5, generator=g).exp_() * (4.0 / 127) for _ in "kv")
    return codes[0], codes[1], ks, vs


def prepare(case, seed):
    c, dt = case, getattr(torch, case["dtype"])
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g)

    def uniform(*shape, lo, hi):
        return torch.empty(shape, device="cuda").uniform_(lo, hi, generator=g)

    s = {"case": dict(c)}
    if c["op"] == "norm":
        big = torch.where(uniform(c["h"], lo=0, hi=1) < 0.01, 10.0, 1.0)  # a few channels are large, as in real activations
        s["x"] = (normal(c["T"], c["h"]) * big).to(dt)
        s["residual"] = normal(c["T"], c["h"], std=3.0).to(dt) if c["residual"] else None
        s["weight"] = uniform(c["h"], lo=0.5, hi=1.5).to(dt)
        s["smooth"] = uniform(c["h"], lo=0.8, hi=1.2) if c["smooth"] else None
        s["values"] = torch.empty(c["T"], c["h"], dtype=dt, device="cuda")
    elif c["op"] == "w4":
        M, N, K, gs = c["M"], c["N"], c["K"], c["group"]
        code = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 27) // K)
        for i in range(0, N, step):
            n = min(step, N - i)
            w = (normal(n, K, std=2.7).round_() + 8).clamp_(0, 15).to(torch.uint8)
            code[i:i + n] = w[:, 0::2] | (w[:, 1::2] << 4)
        s["code"] = code
        s["scale"] = (uniform(N, K // gs, lo=0.5, hi=1.5) / (2.7 * math.sqrt(K))).to(dt)
        s["zero"] = uniform(N, K // gs, lo=5.5, hi=10.5).round_().to(torch.uint8) if c["zero"] else None
        if c["x8"]:
            s["x"] = normal(M, K, std=30.0).round_().clamp_(-127, 127).to(torch.int8)
            s["x_scale"] = uniform(M, lo=0.02, hi=0.06)
        else:
            s["x"], s["x_scale"] = normal(M, K).to(dt), None
    elif c["op"] == "append":
        start, n = _append_lens(c)
        H, D, T = c["Hkv"], c["D"], sum(n)
        s["table"], pool = _paged([a + b for a, b in zip(start, n)], c["page"], g)
        k, v, ks, vs = _pool(pool, c, g)
        held = torch.tensor(start, device="cuda")[:, None] - torch.arange(s["table"].shape[1], device="cuda") * c["page"]
        fill = torch.zeros(pool, dtype=held.dtype, device="cuda")  # tokens that each page holds; none past them
        fill[s["table"].clamp(min=0).long().flatten()] = 0
        fill.scatter_reduce_(0, s["table"].clamp(min=0).long().flatten(), torch.where(s["table"] >= 0, held, 0).flatten(),
                             "amax")
        empty = (torch.arange(c["page"], device="cuda") >= fill[:, None])[:, None, :, None]
        s["k"], s["v"] = k.masked_fill_(empty, 0), v.masked_fill_(empty, 0)
        s["k_scale"], s["v_scale"] = ks, vs
        qkv = normal(T, 6 * H * D).to(dt)  # new keys and values lie in the projection's output rows, behind the queries
        s["k_new"], s["v_new"] = qkv[:, 4 * H * D:5 * H * D].view(T, H, D), qkv[:, 5 * H * D:].view(T, H, D)
        s["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
        s["cu"] = torch.tensor(_cum(n), dtype=torch.int32, device="cuda") if c["n"] > 1 else None
        s["k_values"], s["v_values"] = (torch.empty(k.shape, dtype=dt, device="cuda") for _ in "kv")
    else:
        qlen, kv = _attn_lens(c)
        H, G, D, T = c["Hkv"], c["G"], c["D"], sum(qlen)
        s["table"], pool = _paged(kv, c["page"], g)
        s["k"], s["v"], s["k_scale"], s["v_scale"] = _pool(pool, c, g)
        qkv = normal(T, (G + 2) * H * D, std=2.0).to(dt)  # queries lie in the projection's output rows
        s["q"] = qkv[:, :G * H * D].view(T, G * H, D)
        s["lens"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        s["cu"] = torch.tensor(_cum(qlen), dtype=torch.int32, device="cuda") if c["qmax"] > 1 else None
    if own and c["op"] in ("append", "attention"):
        # the handle that a serving program keeps with its cache: the four tensors and the workspace
        import moe_expert_ffn_dispatch_gb300 as m
        s["cache"] = m.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


# ------------------------------------------------------------ the pass
def run(state):
    return {"norm": _norm, "w4": _w4, "append": _append, "attention": _attention}[state["case"]["op"]](state)


def _norm(s):
    c, dt = s["case"], s["x"].dtype
    if own:
        import moe_expert_ffn_dispatch_gb300 as m
        q, scale, res, y = m.add_rmsnorm_quant(s["x"], s["weight"], 1e-6, residual=s["residual"], smooth=s["smooth"],
                                               want_y=c["y"])
    else:
        t = s["x"].float()
        res = None
        if s["residual"] is not None:
            t = t + s["residual"].float()
            res = t.to(dt)
        yf = t * torch.rsqrt((t * t).mean(dim=1, keepdim=True) + 1e-6) * s["weight"].float()
        y = yf.to(dt) if c["y"] else None
        if s["smooth"] is not None:
            yf = yf * s["smooth"]
        mul = 127.0 / yf.abs().amax(dim=1, keepdim=True).clamp(min=1e-4)
        q = (yf * mul).round().clamp(-127, 127).to(torch.int8)
        scale = (1.0 / mul)[:, 0]
    return {"values": torch.mul(q, scale[:, None], out=s["values"]), "scale": scale, "residual": res, "y": y}


def _w4(s):
    c, out = s["case"], getattr(torch, s["case"]["out"])
    if own:
        import moe_expert_ffn_dispatch_gb300 as m
        return m.w4_linear(s["x"], s["code"], s["scale"], zero=s["zero"], x_scale=s["x_scale"], out_dtype=out)
    N, K, gs = c["N"], c["K"], c["group"]
    w = torch.stack((s["code"] & 15, s["code"] >> 4), dim=-1).view(N, K // gs, gs).float()
    w = (w - (8.0 if s["zero"] is None else s["zero"].float()[:, :, None])) * s["scale"].float()[:, :, None]
    y = s["x"].float() @ w.view(N, K).t()
    if s["x_scale"] is not None:
        y = y * s["x_scale"][:, None]
    return y.to(out)


def _append(s):
    if own:
        s["cache"].append(s["k_new"], s["v_new"], s["table"], s["start"], cu_tokens=s["cu"])
    else:
        T, P = s["k_new"].shape[0], s["case"]["page"]
        t = torch.arange(T, device="cuda")
        b = t if s["cu"] is None else (t[:, None] >= s["cu"][1:]).sum(dim=1)
        pos = s["start"].long()[b] + (0 if s["cu"] is None else t - s["cu"][b])
        page, slot = s["table"][b, pos // P].long(), pos % P
        # how many tokens each page held before: the slot of its first new token
        first = torch.full((s["k"].shape[0],), P, device="cuda").scatter_reduce(0, page, slot, "amin")
        touched = (first < P)[:, None]
        for new, code, scale in ((s["k_new"].float(), s["k"], s["k_scale"]), (s["v_new"].float(), s["v"], s["v_scale"])):
            top = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand(T, scale.shape[1]), new.abs().amax(dim=2),
                                                         "amax")
            fresh = top.clamp(min=1e-4) / 127.0
            to = torch.where(touched, torch.where((first == 0)[:, None], fresh, torch.maximum(scale, top / 127.0)), scale)
            again = (code.float() * (scale / to)[:, :, None, None]).round().clamp(-127, 127).to(torch.int8)
            code.copy_(torch.where((touched & (to > scale) & (first > 0)[:, None])[:, :, None, None], again, code))
            scale.copy_(to)
            code[page, :, slot] = (new * (1.0 / to)[page][:, :, None]).round().clamp(-127, 127).to(torch.int8)
    # the cache's codes as the values that they stand for
    return {"k": torch.mul(s["k"], s["k_scale"][:, :, None, None], out=s["k_values"]), "k_scale": s["k_scale"],
            "v": torch.mul(s["v"], s["v_scale"][:, :, None, None], out=s["v_values"]), "v_scale": s["v_scale"]}


def _attention(s):
    c, q = s["case"], s["q"]
    scale = c["D"] ** -0.5
    if own:
        return s["cache"].attention(q, s["table"], s["lens"], cu_q=s["cu"], max_q=c["qmax"], scale=scale,
                                    window=c["window"])
    B, H, G, D, P, qm, T = c["B"], c["Hkv"], c["G"], c["D"], c["page"], c["qmax"], q.shape[0]
    L = s["table"].shape[1] * P
    at = s["table"].clamp(min=0).long()
    k = (s["k"][at].float() * s["k_scale"][at][..., None, None]).transpose(1, 2).reshape(B, H, L, D)
    v = (s["v"][at].float() * s["v_scale"][at][..., None, None]).transpose(1, 2).reshape(B, H, L, D)
    cu = torch.arange(B + 1, device="cuda", dtype=torch.int32) if s["cu"] is None else s["cu"]
    qlen = cu[1:] - cu[:-1]
    j = torch.arange(qm, device="cuda")
    rows = (cu[:-1, None] + j).clamp(max=T - 1).long()  # padded query tokens
    qp = q[rows].float().view(B, qm, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * qm, D)
    pos = (s["lens"] - qlen)[:, None] + j
    i = torch.arange(L, device="cuda")
    seen = i <= pos[..., None]
    if c["window"]:
        seen = seen & (i > pos[..., None] - c["window"])
    a = (qp @ k.transpose(2, 3) * scale).view(B, H, G, qm, L).masked_fill(~seen[:, None, None], float("-inf"))
    top = a.amax(dim=-1, keepdim=True)
    e = torch.exp(a - torch.where(top == float("-inf"), 0.0, top))
    total = e.sum(dim=-1, keepdim=True)
    o = (e.view(B, H, G * qm, L) @ v).view(B, H, G, qm, D) / torch.where(total > 0, total, 1.0)
    t = torch.arange(T, device="cuda")
    b = (t[:, None] >= cu[1:]).sum(dim=1)
    return o.permute(0, 3, 1, 2, 4)[b, t - cu[b]].reshape(T, H * G, D).to(q.dtype)


# ------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["h"]
        return {"bytes": n * (2 + 1 + 4 * c["residual"] + 2 * c["y"]) + c["h"] * (2 + 4 * c["smooth"]) + 4 * c["T"],
                "flops": 8 * n}
    if c["op"] == "w4":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K // 2 + N * (K // c["group"]) * (2 + c["zero"]) + M * (K if c["x8"] else 2 * K) +
                4 * M * c["x8"] + M * N * (4 if c["out"] == F32 else 2), "flops": 2 * M * N * K}
    H, D = c["Hkv"], c["D"]
    if c["op"] == "append":
        start, n = _append_lens(c)
        pages = sum(-(-(a + b) // c["page"]) - a // c["page"] for a, b in zip(start, n))
        return {"bytes": 2 * sum(n) * H * D * 3 + pages * (4 + 2 * H * 8) + 8 * c["B"], "flops": 2 * sum(n) * H * D * 4}
    qlen, kv = _attn_lens(c)
    keys = pairs = pages = 0
    for m, n in zip(qlen, kv):
        w = c["window"] or n + 1
        lo = max(0, n - m - w + 1)  # first key that any of the rows sees
        keys += max(0, n - lo)
        pages += max(0, -(-n // c["page"]) - lo // c["page"])
        pairs += sum(max(0, min(p + 1, w)) for p in range(n - m, n))
    T, G = sum(qlen), c["G"]
    return {"bytes": keys * H * D * 2 + pages * (4 + 8 * H) + 2 * 2 * T * G * H * D + 8 * c["B"],
            "flops": 4 * D * pairs * G * H}


# ------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c, f8 = case, torch.float64
    if c["op"] == "norm":
        t = s["x"].to(f8)
        res = None
        if s["residual"] is not None:
            t = t + s["residual"].to(f8)
            res = t
        y = t / ((t ** 2).sum(1, keepdim=True) / c["h"] + 1e-6).sqrt() * s["weight"].to(f8)
        z = y if s["smooth"] is None else y * s["smooth"].to(f8)
        return {"values": z, "scale": z.abs().amax(1).clamp(min=1e-4) / 127, "residual": res, "y": y if c["y"] else None}
    if c["op"] == "w4":
        x, out = s["x"].to(f8), torch.empty(c["M"], c["N"], dtype=f8, device="cuda")
        if s["x_scale"] is not None:
            x = x * s["x_scale"].to(f8)[:, None]
        step = max(1, (1 << 26) // c["K"])
        for i in range(0, c["N"], step):
            code = s["code"][i:i + step]
            w = torch.empty(code.shape[0], c["K"], dtype=f8, device="cuda")
            w[:, 0::2], w[:, 1::2] = code % 16, code // 16
            zero = 8 if s["zero"] is None else s["zero"][i:i + step].to(f8).repeat_interleave(c["group"], dim=1)
            w = (w - zero) * s["scale"][i:i + step].to(f8).repeat_interleave(c["group"], dim=1)
            out[:, i:i + step] = torch.einsum("mk,nk->mn", x, w)
        return out
    P = c["page"]
    if c["op"] == "append":
        start, n = _append_lens(c)
        cu, table = _cum(n), s["table"].tolist()
        out = {}
        for name in ("k", "v"):
            code, scale, new = s[name], s[name + "_scale"].to(f8), s[name + "_new"].to(f8)
            val, sc = code.to(f8) * scale[:, :, None, None], scale.clone()
            for b in range(c["B"]):
                for p in range(start[b] // P, (start[b] + n[b] - 1) // P + 1):
                    lo, hi = max(start[b], p * P), min(start[b] + n[b], (p + 1) * P)
                    x, at = new[cu[b] + lo - start[b]:cu[b] + hi - start[b]], table[b][p]
                    top = x.abs().amax(dim=(0, 2)) / 127
                    sc[at] = top.clamp(min=1e-4 / 127) if lo == p * P else torch.maximum(sc[at], top)
                    val[at, :, lo - p * P:hi - p * P] = x.transpose(0, 1)
            out[name], out[name + "_scale"] = val, sc
        return out
    qlen, kv = _attn_lens(c)
    cu, out = _cum(qlen), torch.zeros(s["q"].shape, dtype=f8, device="cuda")
    for b in range(c["B"]):
        m, n = qlen[b], kv[b]
        if not n:
            continue
        at = s["table"][b, :-(-n // P)].long()
        for h in range(c["Hkv"]):
            k, v = ((s[x][at, h].to(f8) * s[x + "_scale"][at, h].to(f8)[:, None, None]).reshape(-1, c["D"])[:n] for x in "kv")
            i = torch.arange(n, device="cuda")
            p = torch.arange(n - m, n, device="cuda")[:, None]
            seen = (i <= p) & (i > p - (c["window"] or n + m + 1))
            heads = slice(h * c["G"], (h + 1) * c["G"])
            a = torch.einsum("jgd,id->jgi", s["q"][cu[b]:cu[b + 1], heads].to(f8), k) / math.sqrt(c["D"])
            a = a.masked_fill(~seen[:, None], float("-inf"))
            out[cu[b]:cu[b + 1], heads] = torch.einsum("jgi,id->jgd", torch.softmax(a, dim=-1).nan_to_num(0.0), v)
    return out
