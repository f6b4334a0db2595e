"""Operators of one serving step around the decoder layer, as workloads.

Four operators: the plan of a step's pages ("plan": page table, prefix sums
and slots from request lengths), the norm after a block with its gate and
residual scale fused with the norm before the next ("norms"), products of int8
codes with scales a token and a channel ("w8"), and log probabilities of given
tokens with entropy and the top alternatives ("logprobs").  `run` computes each
in plain torch operations, or, where `own` is true, by this package's entry
points.

The ragged lengths of a plan come from the case alone (its "mix"), so that
`work` knows them; values come from the seed.
"""
import math
import random

import torch

own = False

BF16, FP16, F32 = "bfloat16", "float16", "float32"
EPS = 1e-6


def listed():
    return [
        # query / key / value projection of one decode step of 8 tokens: 32 + 2 x 8 heads of 128
        dict(name="w8_qkv_decode8", op="w8", M=8, N=6144, K=4096, scale=F32, out=BF16),
        # attention output projection of 64 requests
        dict(name="w8_out_decode64", op="w8", M=64, N=4096, K=4096, scale=F32, out=FP16),
        # output head over a large vocabulary, ragged N, logits in fp32
        dict(name="w8_head16", op="w8", M=16, N=130001, K=4096, scale=BF16, out=F32),
        # the projection of a prefill batch that is not a round number of tokens
        dict(name="w8_prompt", op="w8", M=4093, N=6144, K=4096, scale=F32, out=BF16),
        # between two blocks of a decode step: codes for the next projection
        dict(name="norms_decode8", op="norms", T=8, h=4096, dtype=BF16, gate="channel", codes=True, y=False),
        # the same of a prefill batch in front of the expert block, which takes the norm itself
        dict(name="norms_prefill", op="norms", T=4093, h=4096, dtype=BF16, gate="token", codes=False, y=True),
        # one request's sampled token: latency
        dict(name="logprobs_one", op="logprobs", T=1, V=130001, dtype=F32, n=1, top=5, masked=0.0),
        # a decode step, the vocabulary partly forbidden to some requests
        dict(name="logprobs_decode64", op="logprobs", T=64, V=130001, dtype=BF16, n=1, top=20, masked=0.25),
        # scoring of a prompt's tokens, two candidates each
        dict(name="logprobs_prompt", op="logprobs", T=2039, V=130001, dtype=BF16, n=2, top=5, masked=0.0),
        # one new token each for 64 requests
        dict(name="plan_decode64", op="plan", B=64, n=1, held=8191, page=64, mix=1),
        # a few prompts, ragged
        dict(name="plan_prompts", op="plan", B=5, n=2048, held=100, page=64, mix=2),
        # many requests, chunks of prompts among them, small pages
        dict(name="plan_many", op="plan", B=1024, n=64, held=2000, page=16, mix=3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["w8", "w8", "norms", "logprobs", "plan"])
    dtype = rng.choice([BF16, FP16])
    if op == "w8":
        K = 16 * _log(rng, 2, 1024)
        M = _log(rng, 1, 4093)
        N = _log(rng, 1, max(1, min(130001, 130001 * 4096 // K, 4093 * 6144 * 4096 // (M * K), 130001 * 16 * 8 // M)))
        return dict(op=op, M=M, N=N, K=K, scale=rng.choice([F32, BF16, FP16]), out=rng.choice([BF16, BF16, FP16, F32]))
    if op == "norms":
        h = _log(rng, 64, 16384)
        if rng.random() < 0.5:
            h = -(-h // 64) * 64
        codes = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, max(1, min(8192, 4093 * 4096 // h))), h=h, dtype=dtype,
                    gate=rng.choice(["none", "channel", "token"]), codes=codes, y=not codes or rng.random() < 0.3)
    if op == "logprobs":
        V = _log(rng, 32, 262144)
        T = _log(rng, 1, max(1, min(2039, 2039 * 130001 // V)))
        if rng.random() < 0.3 and T * V <= 2039 * 65000:
            dtype = F32
        return dict(op=op, T=T, V=V, dtype=dtype, n=rng.choice([1, 1, 4]), top=rng.choice([0, 1, 5, 20, 32]),
                    masked=rng.choice([0.0, 0.5]))
    n = 1 if rng.random() < 0.4 else _log(rng, 2, 2048)
    return dict(op=op, B=_log(rng, 1, max(1, min(1024, 65536 // n))), n=n, held=_log(rng, 1, 8191),
                page=rng.choice([16, 32, 64, 128]), mix=rng.randrange(1 << 20))


# ------------------------------------------------------------ lengths of a plan
def _plan_lens(c):
    """Tokens that each sequence holds, and that it gets (none, for a slot of the batch without a request)."""
    r = random.Random(c["mix"])
    held = [c["held"]] + [r.randint(0, c["held"]) for _ in range(c["B"] - 1)]
    new = [c["n"]] + [r.randint(1, c["n"]) for _ in range(c["B"] - 1)]
    if c["B"] >= 8:
        held[c["B"] // 2] = new[c["B"] // 2] = 0
    return held, new


def _pages(c):
    """Pages that each sequence holds, and that it holds after the step."""
    return zip(*((-(-a // c["page"]), -(-(a + b) // c["page"])) for a, b in zip(*_plan_lens(c))))


# ------------------------------------------------------------ inputs
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.empty(shape, device="cuda").normal_(0.0, std, generator=g)

    def uniform(*shape, lo, hi):
        return torch.empty(shape, device="cuda").uniform_(lo, hi, generator=g)

    def codes(n, k):
        t = torch.empty(n, k, dtype=torch.int8, device="cuda")
        step = max(1, (1 << 27) // k)
        for i in range(0, n, step):
            t[i:i + step] = normal(min(step, n - i), k, std=32.0).round_().clamp_(-127, 127)
        return t

    s = {"case": dict(c)}
    if c["op"] == "w8":
        M, N, K = c["M"], c["N"], c["K"]
        s["x"], s["w"] = codes(M, K), codes(N, K)
        s["x_scale"] = uniform(M, lo=0.02, hi=0.06)
        s["w_scale"] = (uniform(N, lo=0.5, hi=1.5) / (32 * math.sqrt(K))).to(getattr(torch, c["scale"]))
    elif c["op"] == "norms":
        T, h, dt = c["T"], c["h"], getattr(torch, c["dtype"])
        big = torch.where(uniform(h, lo=0, hi=1) < 0.01, 10.0, 1.0)  # a few channels are large, as in real activations
        s["x"] = (normal(T, h) * big).to(dt)
        s["residual"] = normal(T, h, std=3.0).to(dt)
        s["post_weight"], s["weight"] = (uniform(h, lo=0.5, hi=1.5).to(dt) for _ in "pw")
        s["gate"] = None
        if c["gate"] != "none":
            s["gate"] = torch.sigmoid(normal(*((T, h) if c["gate"] == "token" else (h,)))).to(dt)
        s["values"] = torch.empty(T, h, dtype=dt, device="cuda")
    elif c["op"] == "logprobs":
        T, V, dt = c["T"], c["V"], getattr(torch, c["dtype"])
        logits = torch.empty(T, V, dtype=dt, device="cuda")
        step = max(1, (1 << 27) // V)
        for i in range(0, T, step):
            t = min(step, T - i)
            sharp = uniform(t, 1, lo=1.0, hi=4.0)  # some positions are sure of their token, others are not
            part = normal(t, V) * sharp
            if c["masked"]:
                rows = uniform(t, 1, lo=0, hi=1) < c["masked"]
                part.masked_fill_((uniform(t, V, lo=0, hi=1) < 0.9) & rows, float("-inf"))
            logits[i:i + step] = part
        s["logits"] = logits
        shape = (T,) if c["n"] == 1 else (T, c["n"])
        s["tokens"] = torch.randint(0, V, shape, device="cuda", generator=g)
    else:
        held, new = _plan_lens(c)
        had, has = _pages(c)
        used = sum(had)
        ids = torch.randperm(sum(has) + 7, generator=g, device="cuda").to(torch.int32)
        where, at = ids.cpu(), 0
        table = torch.full((c["B"], max(1, max(has)) + 2), -1, dtype=torch.int32)
        for b, n in enumerate(had):
            table[b, :n] = where[at:at + n]
            at += n
        s["table"], s["pool"] = table.cuda(), ids.numel()
        s["free"] = ids[used:].contiguous()
        s["held"], s["new"] = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in (held, new))
        s["taken"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["tokens"] = -(-sum(new) // 64) * 64  # rows of the step's buffers, those past the last token unused
    return s


# ------------------------------------------------------------ the pass
def run(state):
    return {"w8": _w8, "norms": _norms, "logprobs": _logprobs, "plan": _plan}[state["case"]["op"]](state)


def _w8(s):
    out = getattr(torch, s["case"]["out"])
    if own:
        import moe_expert_ffn_dispatch_gb300 as m
        return m.w8_linear(s["x"], s["w"], s["w_scale"], s["x_scale"], out_dtype=out)
    return ((s["x"].float() @ s["w"].float().t()) * s["w_scale"].float() * s["x_scale"][:, None]).to(out)


def _norms(s):
    c, dt = s["case"], s["x"].dtype
    if own:
        import moe_expert_ffn_dispatch_gb300 as m
        q, scale, res, y = m.norm_add_rmsnorm_quant(s["x"], s["residual"], s["post_weight"], s["weight"], EPS,
                                                    gate=s["gate"], branch_scale=0.5, want_q=c["codes"], want_y=c["y"])
    else:
        x = s["x"].float()
        p = x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS) * s["post_weight"].float()
        if s["gate"] is not None:
            p = p * s["gate"].float()
        t = s["residual"].float() + 0.5 * p
        res = t.to(dt)
        yf = t * torch.rsqrt((t * t).mean(dim=1, keepdim=True) + EPS) * s["weight"].float()
        y = yf.to(dt) if c["y"] else None
        q = scale = None
        if c["codes"]:
            mul = 127.0 / yf.abs().amax(dim=1, keepdim=True).clamp(min=1e-4)
            q = (yf * mul).round().clamp(-127, 127).to(torch.int8)
            scale = (1.0 / mul)[:, 0]
    # the codes as the values that they stand for
    values = torch.mul(q, scale[:, None], out=s["values"]) if c["codes"] else None
    return {"values": values, "scale": scale, "residual": res, "y": y}


def _logprobs(s):
    c = s["case"]
    if own:
        import moe_expert_ffn_dispatch_gb300 as m
        logprob, entropy, top_logprob, top_id = m.token_logprobs(s["logits"], s["tokens"], top=c["top"])
    else:
        l = s["logits"].float()
        top = l.amax(dim=1, keepdim=True)
        z = l - top
        e = torch.exp(z)
        total = e.sum(dim=1, keepdim=True)
        lse = torch.log(total)  # of z
        entropy = (lse - torch.where(e > 0, e * z, 0.0).sum(dim=1, keepdim=True) / total)[:, 0]
        logprob = (z.gather(1, s["tokens"].view(c["T"], -1)) - lse).view(s["tokens"].shape)
        # order by value, then by the lower index: both in one whole number
        bits = (l + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) + (c["V"] - 1 - torch.arange(c["V"], device="cuda"))
        k = min(c["top"], c["V"])
        at = c["V"] - 1 - (torch.topk(key, k, dim=1).values & 0xFFFFFFFF)
        top_logprob, top_id = z.gather(1, at) - lse, at.int()
    return {"logprob": logprob, "entropy": entropy, "top_logprob": top_logprob, "top_id": top_id}


def _plan(s):
    c, table, n = s["case"], s["table"], s["tokens"]
    if own:
        import moe_expert_ffn_dispatch_gb300 as m
        p = m.page_plan(table, s["held"], s["new"], s["free"], c["page"], s["pool"], n, taken=s["taken"])
        return {"table": table, "cu": p.cu_tokens, "lens": p.seq_lens, "sequence": p.sequence, "position": p.position,
                "slot": p.slot, "taken": p.taken, "unplaced": p.unplaced}
    P, free = c["page"], s["free"]
    held, new = s["held"].long(), s["new"].long()
    cu = torch.cat((torch.zeros_like(new[:1]), new.cumsum(0)))
    lens = held + new
    first, last = (held + P - 1) // P, ((lens + P - 1) // P).clamp(max=table.shape[1])
    need = (last - first).clamp(min=0)
    at = s["taken"].long() + need.cumsum(0) - need
    i = torch.arange(table.shape[1], device="cuda")
    take = at[:, None] + i - first[:, None]
    fresh = torch.where(take < free.shape[0], free[take.clamp(0, free.shape[0] - 1)], -1)
    table.copy_(torch.where((i >= first[:, None]) & (i < last[:, None]), fresh, table))
    t = torch.arange(n, device="cuda")
    live = t < cu[-1]
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=c["B"] - 1)
    pos = held[b] + t - cu[b]
    inside = live & (pos < table.shape[1] * P)
    page = table[b, (pos // P).clamp(0, table.shape[1] - 1)].long()
    placed = inside & (page >= 0) & (page < s["pool"])
    slot = torch.where(placed, page * P + pos % P, -1)
    return {"table": table, "cu": cu.int(), "lens": lens.int(), "sequence": torch.where(live, b, -1).int(),
            "position": torch.where(live, pos, -1).int(), "slot": slot,
            "taken": (s["taken"] + need.sum()).clamp(max=free.shape[0]).int(), "unplaced": (live & ~placed).sum().int().view(1)}


# ------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    size = {BF16: 2, FP16: 2, F32: 4}
    if c["op"] == "w8":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K + M * K + N * size[c["scale"]] + 4 * M + M * N * size[c["out"]], "flops": 2 * M * N * K}
    if c["op"] == "norms":
        n, gate = c["T"] * c["h"], {"none": 0, "channel": c["h"], "token": c["T"] * c["h"]}[c["gate"]]
        return {"bytes": n * (2 + 2 + 2 + c["codes"] + 2 * c["y"]) + 2 * gate + 4 * c["h"] + 4 * c["T"] * c["codes"],
                "flops": 16 * n}
    if c["op"] == "logprobs":
        return {"bytes": c["T"] * (c["V"] * size[c["dtype"]] + c["n"] * 12 + 4 + 8 * c["top"]), "flops": 6 * c["T"] * c["V"]}
    held, new = _plan_lens(c)
    had, has = _pages(c)
    partly = sum(1 for a, b in zip(held, new) if b and a % c["page"])  # pages that are read from the table
    return {"bytes": 16 * c["B"] + 16 * (-(-sum(new) // 64) * 64) + 8 * (sum(has) - sum(had)) + 4 * partly + 20,
            "flops": 8 * sum(new)}


# ------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    c, f8 = case, torch.float64
    if c["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    if c["op"] == "w8":
        out = torch.empty(c["M"], c["N"], dtype=f8, device="cuda")
        x = s["x"].to(f8)
        step = max(1, (1 << 27) // c["K"])
        for i in range(0, c["N"], step):
            w = s["w"][i:i + step].to(f8) * s["w_scale"][i:i + step].to(f8)[:, None]
            out[:, i:i + step] = torch.einsum("mk,nk->mn", x, w)
        return out * s["x_scale"].to(f8)[:, None]
    if c["op"] == "norms":
        x, h = s["x"].to(f8), c["h"]
        branch = x / ((x ** 2).sum(1, keepdim=True) / h + EPS).sqrt() * s["post_weight"].to(f8)
        if s["gate"] is not None:
            branch = branch * s["gate"].to(f8)
        t = s["residual"].to(f8) + branch / 2
        y = t / ((t ** 2).sum(1, keepdim=True) / h + EPS).sqrt() * s["weight"].to(f8)
        step = y.abs().amax(1).clamp(min=1e-4) / 127
        values = (y / step[:, None]).round().clamp(-127, 127) * step[:, None] if c["codes"] else None
        return {"values": values, "scale": step if c["codes"] else None, "residual": t, "y": y if c["y"] else None}
    T, V, k = c["T"], c["V"], min(c["top"], c["V"])
    got = {"logprob": [], "entropy": [], "top_logprob": []}
    for rows in torch.arange(T, device="cuda").split(max(1, (1 << 26) // V)):
        p = torch.log_softmax(s["logits"][rows].to(f8), dim=1)
        got["logprob"].append(p.gather(1, s["tokens"].view(T, -1)[rows]))
        got["entropy"].append(torch.special.entr(p.exp()).sum(1))
        got["top_logprob"].append(torch.sort(p, dim=1, descending=True).values[:, :k])
    return {"logprob": torch.cat(got["logprob"]).view(s["tokens"].shape), "entropy": torch.cat(got["entropy"]),
            "top_logprob": torch.cat(got["top_logprob"]), "top_id": None}
