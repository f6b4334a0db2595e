"""Calls of the serving-step operators that their documentation allows and that lie off the ordinary paths: sums that
need every bit that fp32 has, workspaces of the caller's own, rows of logits in the forms that many rows get."""

import pytest

torch = pytest.importorskip("torch")

import moe_expert_ffn_dispatch_gb300 as m  # noqa: E402
from test_gpu_step_ops import (BF16, DEV, F32, FP16, check_logprobs, gen, i32, pair_inputs, rand, randn,  # noqa: E402
                               w8_inputs, w8_reference)

pytestmark = pytest.mark.gpu

# tokens, weight rows: few tokens in integer products, few in one CTA a tile, one half, a pair of CTAs
FORMS = [(3, 700), (30, 300), (64, 3000), (40, 33), (100, 700), (200, 130), (1000, 5003)]


# ------------------------------------------------------------ 8-bit products: every bit of a sum
@pytest.mark.parametrize("M, N", FORMS)
@pytest.mark.parametrize("K", [1024, 1040, 2048, 5008])
def test_w8_odd_sums_next_to_the_limits(M, N, K):
    """Odd codes near 127: sums of 1024 k lie above 2^23, where an accumulator without one of fp32's 24 bits loses the
    lowest, and half of them are odd (one code of some rows is even)."""
    g = gen(M + N + K)
    x, w = (127 - 2 * torch.randint(0, 3, s, device=DEV, generator=g).to(torch.int8) for s in ((M, K), (N, K)))
    x[::2, K // 3] = 126
    w[::2, K // 2] = 125
    w[1::4] *= -1
    one = torch.ones(N, device=DEV), torch.ones(M, device=DEV)
    want = w8_reference(x, w, *one, F32)
    assert float(want.abs().max()) > 2 ** 23 and (K > 1040 or bool((want[0] % 2 != want[1] % 2).all()))
    assert torch.equal(m.w8_linear(x, w, *one, out_dtype=F32), want)


@pytest.mark.parametrize("M, N", FORMS)
@pytest.mark.parametrize("K", [2048, 4096, 3088])
def test_w8_odd_sums_that_cancel(M, N, K):
    """As above, every second 1024 k with the other sign: what two of them lose would be all that is left."""
    g = gen(M + N + K + 1)
    x, w = (127 - 2 * torch.randint(0, 3, s, device=DEV, generator=g).to(torch.int8) for s in ((M, K), (N, K)))
    x[::2, K // 3] = 126
    for k in range(1024, K, 2048):
        x[:, k:k + 1024] *= -1
    one = torch.ones(N, device=DEV), torch.ones(M, device=DEV)
    want = w8_reference(x, w, *one, F32)
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(m.w8_linear(x, w, *one, out_dtype=F32), want)


# ------------------------------------------------------------ 8-bit products: workspaces
def bytes_of(M, K):
    return 256 + 2 * M * K  # the status words, and the tokens in 16 bits


def timed_out(ws):
    """The words that a wait that gave up leaves, written by the host."""
    ws[:16].view(torch.int32)[1:3] = i32([1, 513])


def test_w8_workspace_sizes():
    assert m.w8_linear_workspace(64, 5000, 4096) is None and m.w8_linear_workspace(1, 1, 16, DEV) is None
    for M, N, K in ((65, 1, 16), (100, 700, 2048), (1000, 5003, 1040)):
        ws = m.w8_linear_workspace(M, N, K)
        assert ws.data_ptr() % 256 == 0 and ws.numel() == bytes_of(M, K) and ws.is_contiguous()


@pytest.mark.parametrize("M, N, K", [(65, 33, 16), (100, 700, 2048), (150, 4096, 1040), (1000, 5003, 1040)])
def test_w8_in_a_workspace_of_the_callers_own(M, N, K):
    """Whatever it held before: the same bits, a status of 0, and a status that an earlier call left is gone."""
    x, w, ws, xs = w8_inputs(M, N, K, gen(M + K))
    want = w8_reference(x, w, ws, xs, F32)
    space = m.w8_linear_workspace(M, N, K)
    for fill in (0xFF, 0x00, 0x7C):
        space.fill_(fill)
        timed_out(space)
        assert m.w8_linear_status(space) == m.MOE_ERR_DEVICE_TIMEOUT
        assert torch.equal(m.w8_linear(x, w, ws, xs, out_dtype=F32, workspace=space), want)
        assert m.w8_linear_status(space) == m.MOE_OK
    # any type, more room than needed, and nothing past what is needed is written
    wide = torch.full((bytes_of(M, K) // 4 + 200,), 7.0, device=DEV)
    assert torch.equal(m.w8_linear(x, w, ws, xs, out_dtype=F32, workspace=wide), want)
    assert bool((wide[bytes_of(M, K) // 4:] == 7).all())


def test_w8_calls_that_share_a_workspace():
    """A large call, smaller ones, one in the pair form and one that needs no workspace, in turn."""
    g = gen(21)
    sizes = [(1000, 5003, 2048), (100, 700, 1040), (65, 40, 16), (700, 6000, 1040), (20, 700, 1040), (300, 333, 2048)]
    ins = [w8_inputs(*s, g) for s in sizes]
    want = [w8_reference(*i, BF16) for i in ins]
    space = m.w8_linear_workspace(*sizes[0])
    space.fill_(0xFF)
    for order in (range(6), reversed(range(6)), (3, 1, 0, 2, 4, 0, 5)):
        order = list(order)
        got = [m.w8_linear(*ins[i], workspace=space) for i in order]
        assert m.w8_linear_status(space) == m.MOE_OK
        for i, y in zip(order, got):
            assert torch.equal(y, want[i]), sizes[i]


@pytest.mark.parametrize("M, N, K", [(100, 700, 2048), (1000, 5003, 1040)])
def test_w8_captured_with_a_workspace(M, N, K):
    """Captured calls that share one, replayed with other tokens and whatever else has been in it meanwhile."""
    g = gen(M)
    x, w, ws, xs = w8_inputs(M, N, K, g)
    space, out = m.w8_linear_workspace(M, N, K), [torch.empty(M, N, device=DEV) for _ in "ab"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        m.w8_linear(x, w, ws, xs, out=out[0], workspace=space)
        with torch.cuda.graph(graph, stream=side):
            m.w8_linear(x, w, ws, xs, out=out[0], workspace=space)
            m.w8_linear(x[:70], w, ws, xs[:70], out=out[1][:70], workspace=space)
    torch.cuda.synchronize()
    for turn in range(3):
        x.copy_(torch.randint(-128, 128, x.shape, device=DEV, generator=g, dtype=torch.int8))
        space.fill_(0xFF)
        timed_out(space)
        graph.replay()
        torch.cuda.synchronize()
        want = w8_reference(x, w, ws, xs, F32)
        assert torch.equal(out[0], want) and torch.equal(out[1][:70], want[:70])
        assert m.w8_linear_status(space) == m.MOE_OK


def test_w8_refuses_workspaces_that_do_not_fit():
    M, N, K = 100, 70, 256
    x, w, ws, xs = w8_inputs(M, N, K, gen(5))
    need, out = bytes_of(M, K), torch.full((M, N), 7.0, device=DEV)
    space = torch.empty(need + 512, dtype=torch.uint8, device=DEV)[:]
    space = space[(-space.data_ptr()) % 256:]
    for bad, code in ((space[:need - 1], m.MOE_ERR_WORKSPACE_TOO_SMALL), (space[:0], None), (space[16:], m.MOE_ERR_ALIGNMENT)):
        with pytest.raises(m.MoeError) as e:
            m.w8_linear(x, w, ws, xs, out=out, workspace=bad)
        assert code is None or e.value.code == code
    for bad in (torch.empty(need, dtype=torch.uint8), torch.empty(need, 2, dtype=torch.uint8, device=DEV)[:, 0]):
        with pytest.raises(ValueError):
            m.w8_linear(x, w, ws, xs, out=out, workspace=bad)
        with pytest.raises(ValueError):
            m.w8_linear_status(bad)
    torch.cuda.synchronize()
    assert bool((out == 7).all())
    assert torch.equal(m.w8_linear(x, w, ws, xs, out=out, workspace=space[:need]), w8_reference(x, w, ws, xs, F32))


# ------------------------------------------------------------ log probabilities of many rows
# vocabularies whose rows one warp takes (in one step, in some, in most that it can), CTAs of two and of four warps; a
# fp32 step has half as many elements
MANY = [(BF16, 900), (BF16, 4000), (BF16, 8191), (BF16, 9001), (BF16, 16000), (BF16, 20011), (FP16, 8200), (F32, 1003), (F32, 4096),
        (F32, 4500), (F32, 8200), (F32, 9001)]


def rows_for_every_sm():
    """Rows enough that each has few warps: eight an SM, and some more that end inside a CTA of four rows."""
    return 8 * torch.cuda.get_device_properties(0).multi_processor_count + 3


@pytest.mark.parametrize("dtype, V", MANY)
def test_logprobs_of_many_rows(dtype, V):
    """Ordinary rows, rows that rise, fall, repeat a few values or hold their largest at either end, masked rows."""
    rows, g = rows_for_every_sm(), gen(V)
    x = randn(rows, V, g=g) * rand(rows, 1, g=g, lo=0.2, hi=4.0)
    ramp = torch.linspace(-8, 8, V, device=DEV)
    x[1::16], x[2::16], x[3::16] = ramp, ramp.flip(0), 0.5
    x[4::16] = torch.randint(0, 3, x[4::16].shape, device=DEV, generator=g).float()
    x[5::16, 0], x[6::16, V - 1] = 30.0, 30.0
    x = x.to(dtype)
    keep = rand(*x[7::16].shape, g=g) < 0.01
    keep[:, V // 2] = True
    x[7::16] = x[7::16].masked_fill(~keep, float("-inf"))
    x[8::16] = x[8::16].masked_fill(rand(*x[8::16].shape, g=g) < 0.9, torch.finfo(dtype).min)
    tokens = torch.randint(0, V, (rows, 2), device=DEV, generator=g)
    tokens[::5, 1] = -1
    for top in (0, 3, 32):
        check_logprobs(x, tokens, top, m.token_logprobs(x, tokens, top))


@pytest.mark.parametrize("dtype, V", MANY)
def test_logprobs_of_many_rows_without_a_distribution(dtype, V):
    rows, g = rows_for_every_sm(), gen(V + 1)
    x = randn(rows, V, g=g).to(dtype)
    x[1::8] = float("-inf")
    x[2::8, V // 2], x[3::8, V - 1], x[4::8, 0], x[5::8, V - 1] = float("nan"), float("inf"), float("inf"), float("nan")
    tokens = torch.zeros(rows, dtype=torch.int32, device=DEV)
    lp, H, tlp, tid = m.token_logprobs(x, tokens, 4)
    kind = torch.arange(rows, device=DEV) % 8
    none, fine = (kind >= 1) & (kind <= 5), (kind == 0) | (kind > 5)
    for t in (lp[:, None], H[:, None], tlp):
        assert torch.isnan(t[none]).all() and torch.isfinite(t[fine]).all()
    assert bool((tid[kind == 1] == torch.arange(4, device=DEV)).all()) and bool((tid[none & (kind > 1)] == -1).all())
    check_logprobs(x[fine], tokens[fine], 4, tuple(t[fine] for t in (lp, H, tlp, tid)))


@pytest.mark.parametrize("dtype, V", [(BF16, 5001), (BF16, 9001), (BF16, 17001), (F32, 3001), (F32, 6001)])
def test_logprobs_of_many_strided_rows(dtype, V):
    """Rows inside wider ones, at offsets that differ from row to row, between elements that would change every result."""
    rows, g = rows_for_every_sm(), gen(V)
    for off, pad in ((1, 18), (5, 16)):
        wide = torch.full((rows, V + pad), float("nan"), device=DEV, dtype=dtype)
        wide[:, off:off + V] = randn(rows, V, g=g).to(dtype)
        x = wide[:, off:off + V]
        tokens = torch.randint(0, V, (rows,), device=DEV, generator=g)
        check_logprobs(x, tokens, 6, m.token_logprobs(x, tokens, 6))


@pytest.mark.parametrize("dtype, V", [(BF16, 1000), (BF16, 9001), (BF16, 50000), (F32, 9001)])
def test_logprobs_of_a_row_in_any_batch(dtype, V):
    """The ids of the likeliest tokens do not depend on the batch; sums are added up in an order that does, and stay
    within the operator's error."""
    rows, g = rows_for_every_sm(), gen(V)
    x = (randn(rows, V, g=g) * 3).to(dtype)
    tokens = torch.randint(0, V, (rows,), device=DEV, generator=g)
    whole = m.token_logprobs(x, tokens, 8)
    for lo, hi in ((0, 1), (5, 13), (100, 400)):
        part = m.token_logprobs(x[lo:hi], tokens[lo:hi], 8)
        check_logprobs(x[lo:hi], tokens[lo:hi], 8, part)
        assert torch.equal(part[3], whole[3][lo:hi])
    check_logprobs(x, tokens, 8, whole)


# ------------------------------------------------------------ norm pair
@pytest.mark.parametrize("h", [256, 1000, 4096, 5000])
def test_pair_gate_of_one_row_that_is_expanded(h):
    """A gate a token whose rows are one and the same memory is the gate that all tokens share."""
    x, r, pw, w, gt = pair_inputs(6, h, FP16, FP16, "channel", gen(h))
    want = m.norm_add_rmsnorm_quant(x, r, pw, w, gate=gt, want_y=True)
    for gate in (gt.expand(6, h), gt.repeat(6, 1)):
        for a, b in zip(m.norm_add_rmsnorm_quant(x, r, pw, w, gate=gate, want_y=True), want):
            assert torch.equal(a, b)


# ------------------------------------------------------------ numbers that do not fit the C structures
def test_numbers_past_32_bits_are_not_cut():
    one = i32([1])
    table = i32([[0, 1, 2, 3]])
    for size, pages, tokens in ((2 ** 32 + 16, 4, 1), (-2 ** 32 + 16, 4, 1), (16, 2 ** 32 + 4, 1), (16, -2 ** 32 + 4, 1), (16, 4, 2 ** 32 + 1),
                                (16, 4, -2 ** 32 + 1)):
        with pytest.raises(ValueError):
            m.page_plan(table, one, one, one, size, pages, tokens)
    for size, pages in ((-16, 4), (16, -4)):
        with pytest.raises(m.MoeError):
            m.page_plan(table, one, one, one, size, pages, 1)
    assert table.tolist() == [[0, 1, 2, 3]]
    logits = torch.zeros(2, 5, device=DEV)
    for n in (2 ** 32, 2 ** 32 + 1, 2 ** 31):
        with pytest.raises(ValueError):
            m.token_logprobs(logits, i32([[1], [2]]).expand(2, n))
    with pytest.raises(ValueError):
        m.token_logprobs(logits[:1].expand(2 ** 32 + 1, 5))
    with pytest.raises(ValueError):
        m.w8_linear_workspace(2 ** 32 + 100, 64, 64)
