"""A serving loop made of the package's operators: page plan, norms, 8-bit products,
append and attention, 8-bit head, log probabilities.  Every operator is held to its
definition on the inputs that it got in the run; decode steps are captured into a
graph and replayed against steps run one by one."""
import pytest

torch = pytest.importorskip("torch")

import moe_expert_ffn_dispatch_gb300 as m  # noqa: E402
import test_gpu_step_ops as ops  # noqa: E402

pytestmark = pytest.mark.gpu
DEV, BF16, F32 = "cuda", torch.bfloat16, torch.float32


def quantise(w):
    scale = w.abs().amax(1).clamp(min=1e-8) / 127
    return (w / scale[:, None]).round().clamp(-127, 127).to(torch.int8), scale


class Model:
    """Two layers: norm, projections, attention over the paged cache, the norm pair, a gated product; then a head."""
    HEADS, KV, DIM, HIDDEN, FFN, VOCAB, PAGE, EPS = 8, 2, 64, 512, 1024, 5003, 16, 1e-5

    def __init__(self, pages=64, seed=0):
        g = ops.gen(seed)

        def weight(n, k):
            return quantise(ops.randn(n, k, g=g, std=k ** -0.5))

        self.embed = ops.randn(self.VOCAB, self.HIDDEN, g=g).to(BF16)
        self.layers = [dict(qkv=weight((self.HEADS + 2 * self.KV) * self.DIM, self.HIDDEN),
                            out=weight(self.HIDDEN, self.HEADS * self.DIM), up=weight(2 * self.FFN, self.HIDDEN),
                            down=weight(self.HIDDEN, self.FFN),
                            norms=[ops.rand(self.HIDDEN, g=g, lo=0.5, hi=1.5).to(BF16) for _ in range(3)],
                            gate=ops.rand(self.HIDDEN, g=g, lo=0.2, hi=1.0).to(BF16)) for _ in range(2)]
        self.last_norm = ops.rand(self.HIDDEN, g=g, lo=0.5, hi=1.5).to(BF16)
        self.ones = torch.ones(self.HIDDEN, dtype=BF16, device=DEV)
        self.head = weight(self.VOCAB, self.HIDDEN)
        self.caches = [m.KvCache.empty(pages, self.KV, self.PAGE, self.DIM) for _ in self.layers]
        self.free = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
        self.pages = pages

    def step(self, ids, table, held, new, taken, tokens, max_q, check=False, counts=None):
        """Logits of every token, and the plan."""
        plan = self.caches[0].plan(table, held, new, self.free, tokens, taken=taken, taken_out=taken)
        x = self.embed[ids]
        q8, qs, _, y = m.add_rmsnorm_quant(x, self.layers[0]["norms"][0], self.EPS, want_y=True)
        for i, (layer, cache) in enumerate(zip(self.layers, self.caches)):
            qkv = self.linear(q8, qs, layer["qkv"], check)
            q, k, v = (t.view(tokens, -1, self.DIM) for t in
                       qkv.split([self.HEADS * self.DIM, self.KV * self.DIM, self.KV * self.DIM], dim=1))
            cache.append(k, v, table, held, cu_tokens=plan.cu_tokens)
            o = cache.attention(q, table, plan.seq_lens, cu_q=plan.cu_tokens, max_q=max_q)
            o8, os, _, _ = m.add_rmsnorm_quant(o.view(tokens, -1), self.ones, self.EPS)
            a = self.linear(o8, os, layer["out"], check)
            q8, qs, x = self.pair(a, x, layer["norms"][1], layer["norms"][2], layer["gate"], check)
            up = self.linear(q8, qs, layer["up"], check)
            h = torch.nn.functional.silu(up[:, :self.FFN].float()) * up[:, self.FFN:].float()
            h8, hs, _, _ = m.add_rmsnorm_quant(h.to(BF16), torch.ones(self.FFN, dtype=BF16, device=DEV), self.EPS)
            f = self.linear(h8, hs, layer["down"], check)
            after = self.layers[i + 1]["norms"][0] if i + 1 < len(self.layers) else self.last_norm
            q8, qs, x = self.pair(f, x, layer["norms"][1], after, None, check)
        return self.linear(q8, qs, self.head, check, F32), plan

    def linear(self, q8, qs, w, check, out=BF16):
        y = m.w8_linear(q8, *w, qs, out_dtype=out)
        if check:
            assert torch.equal(y, ops.w8_reference(q8, w[0], w[1], qs, out))
        return y

    def pair(self, a, x, post, norm, gate, check):
        out = m.norm_add_rmsnorm_quant(a, x, post, norm, self.EPS, gate=gate, branch_scale=0.5, want_y=True)
        if check:
            ops.check_pair(a, x, post, norm, gate, 0.5, None, self.EPS, out)
        return out[0], out[1], out[2]


def prompts(model, lens, rows):
    """The state of a batch before its prompts, and their tokens in a buffer of `rows`."""
    g = ops.gen(5)
    B = len(lens)
    table = torch.full((B, 12), -1, dtype=torch.int32, device=DEV)
    ids = torch.randint(0, model.VOCAB, (rows,), device=DEV, generator=g)
    return dict(table=table, held=torch.zeros(B, dtype=torch.int32, device=DEV), new=ops.i32(lens), taken=ops.i32([0])), ids


def test_prompts_and_decode_steps():
    model, lens = Model(), [37, 1, 70, 16]
    st, ids = prompts(model, lens, sum(lens))
    logits, plan = model.step(ids, st["table"], st["held"], st["new"], st["taken"], sum(lens), max(lens), check=True)
    assert plan.cu_tokens.tolist() == [0, 37, 38, 108, 124] and plan.seq_lens.tolist() == lens
    assert int(plan.unplaced) == 0 and int(st["taken"]) == 3 + 1 + 5 + 1
    # every token's slot holds what was appended for it: the cache's rows at the slots differ from empty ones
    assert len(set(plan.slot.tolist())) == sum(lens)
    k = model.caches[1].k.permute(0, 2, 1, 3).reshape(-1, model.KV * model.DIM)
    assert (k[plan.slot].abs().amax(1) > 0).all()
    rest = torch.ones(k.shape[0], dtype=torch.bool, device=DEV)
    rest[plan.slot] = False
    assert (k[rest] == 0).all()
    # the prompt's own tokens scored: token t + 1 under the logits of t
    out = m.token_logprobs(logits, ids.roll(-1), 5)
    ops.check_logprobs(logits, ids.roll(-1), 5, out)
    last = (plan.cu_tokens[1:] - 1).long()
    nxt = out[3][last, 0].contiguous()
    held, one = plan.seq_lens, torch.ones(4, dtype=torch.int32, device=DEV)
    for step in range(20):
        logits, plan = model.step(nxt.long(), st["table"], held, one, st["taken"], 4, 1, check=step in (0, 19))
        out = m.token_logprobs(logits, nxt, 3)
        ops.check_logprobs(logits, nxt, 3, out)
        assert torch.equal(out[3][:, 0].long(), logits.argmax(1))
        nxt, held = out[3][:, 0].contiguous(), plan.seq_lens
    assert held.tolist() == [n + 20 for n in lens] and int(plan.unplaced) == 0
    used = sum(-(-(n + 20) // model.PAGE) for n in lens)
    assert int(st["taken"]) == used
    pages = st["table"][st["table"] >= 0]
    assert pages.numel() == used == pages.unique().numel()
    assert all(c.status() == 0 for c in model.caches)


def test_a_prompt_in_chunks_sees_what_the_whole_prompt_sees():
    """One sequence's prompt at once, and in chunks beside others: the same log probabilities within what the cache's
    quantisation does to them (a page that fills over several calls is quantised anew when its scale grows)."""
    whole, lens = Model(), [64]
    st, ids = prompts(whole, lens, 64)
    a, _ = whole.step(ids, st["table"], st["held"], st["new"], st["taken"], 64, 64)
    parts = Model()
    B = 3
    table = torch.full((B, 12), -1, dtype=torch.int32, device=DEV)
    taken, held = ops.i32([0]), ops.i32([0, 0, 0])
    got = []
    for lo in range(0, 64, 16):  # whole pages: each is quantised once, as in the whole prompt
        new = ops.i32([3, 16, 0])
        toks = torch.cat((ids[:3], ids[lo:lo + 16]))
        logits, plan = parts.step(toks, table, held, new, taken, 19, 16)
        got.append(logits[3:])
        held = plan.seq_lens
    assert held.tolist() == [12, 64, 0] and plan.sequence.tolist() == [0] * 3 + [1] * 16
    assert plan.position.tolist()[3:] == list(range(48, 64))
    b = torch.cat(got)
    # the attention's sums are ordered otherwise, which can move an int8 code of a later layer by one: a step of 1 / 127 of
    # a row's largest, through two layers
    assert (torch.log_softmax(a.double(), 1) - torch.log_softmax(b.double(), 1)).abs().max() < 0.5
    assert (a - b).abs().mean() < 0.02 * a.abs().mean()


@pytest.mark.parametrize("batch", [3, 40])
def test_captured_decode_steps(batch):
    """A decode step as a graph: plan (pages taken on in place), layers, head, log probabilities, the next tokens."""
    def start():
        model = Model(pages=400)
        lens = [(7 * i) % 30 + 1 for i in range(batch)]
        st, ids = prompts(model, lens, sum(lens))
        logits, plan = model.step(ids, st["table"], st["held"], st["new"], st["taken"], sum(lens), max(lens))
        nxt = m.token_logprobs(logits[(plan.cu_tokens[1:] - 1).long()], None, 1)[3][:, 0].long()
        return model, st, nxt, plan.seq_lens.clone(), torch.ones(batch, dtype=torch.int32, device=DEV)

    def one(model, st, nxt, held, new):
        logits, plan = model.step(nxt, st["table"], held, new, st["taken"], batch, 1)
        lp, ent, _, ids = m.token_logprobs(logits, None, 2)
        lp = m.token_logprobs(logits, ids)[0]
        nxt.copy_(ids[:, 0])
        held.copy_(plan.seq_lens)
        return lp, ent, ids, plan.slot, plan.unplaced

    state = start()
    want = [[t.clone() for t in one(*state)] for _ in range(12)]
    state = start()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        first = [t.clone() for t in one(*state)]  # workspaces exist before the capture
        with torch.cuda.graph(graph, stream=side):
            out = one(*state)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, want[0]))
    for step in range(1, 12):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want[step]):
            assert torch.equal(a, b), step
    assert int(out[4]) == 0
