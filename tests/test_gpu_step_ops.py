"""The operators of a serving step against their definitions in 64 bits: the
norm pair around a residual addition, 8-bit products, the plan of a step's pages,
log probabilities; and a step made of them.

8-bit products and plans are exact.  The other tolerances come from the
arithmetic: half a step of the output's type, fp32 sums whose error is bounded by
the additions that a term passes through times 2^-24 times the sum of magnitudes,
and what each test says beside it."""
import math

import pytest

torch = pytest.importorskip("torch")

import moe_expert_ffn_dispatch_gb300 as m  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32
U = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, F32: 2.0 ** -24}  # half a step, relative to the value
TINY = {BF16: 1e-38, FP16: 2.0 ** -25, F32: 1e-38}        # half a smallest step near zero
E = 2.0 ** -24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(*shape, g, std=1.0):
    return torch.randn(shape, device=DEV, generator=g) * std


def rand(*shape, g, lo=0.0, hi=1.0):
    return torch.rand(shape, device=DEV, generator=g) * (hi - lo) + lo


def codes(*shape, g):
    return torch.randint(-128, 128, shape, device=DEV, generator=g, dtype=torch.int8)


def close(got, ref, tol, what=""):
    """Elementwise |got - ref| <= tol (a tensor or a number), NaN nowhere."""
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    if bad.any():
        i = int(bad.flatten().nonzero()[0])
        t = tol.expand_as(err).flatten()[i] if torch.is_tensor(tol) else tol
        raise AssertionError("%s element %d of %d: got %r want %r, off %.3e > %.3e (%d bad)" % (
            what, i, err.numel(), float(got.flatten()[i]), float(ref.flatten()[i]), float(err.flatten()[i]), float(t),
            int(bad.sum())))


# ------------------------------------------------------------ norm pair
def check_pair(x, r, pw, w, gate, bs, smooth, eps, out):
    q, qs, res, y = out
    xd = x.double()
    p = xd / ((xd * xd).mean(1, keepdim=True) + eps).sqrt() * pw.double()
    if gate is not None:
        p = p * gate.double()
    bs = float(torch.tensor(bs, dtype=F32))
    s = r.double() + bs * p
    # a sum of squares passes at most 32 + 10 additions; then a division, a root and three products
    rel = 48 * E
    s_err = (bs * p).abs() * rel + s.abs() * E
    close(res, s, s.abs() * U[x.dtype] + 2 * s_err + TINY[x.dtype], "residual")
    r2 = 1 / ((s * s).mean(1, keepdim=True) + eps).sqrt()
    yr = s * r2 * w.double()
    # the sum of squares of s: its terms' own errors reach the root at most relative to the row's size
    row = (s_err ** 2).mean(1, keepdim=True).sqrt() * r2
    y_err = s_err * r2 * w.double().abs() + yr.abs() * (rel + row)
    if y is not None:
        close(y, yr, yr.abs() * U[x.dtype] + 2 * y_err + TINY[x.dtype], "y")
    if q is None:
        assert qs is None
        return
    z, z_err = (yr, y_err) if smooth is None else (yr * smooth.double(), y_err * smooth.double().abs())
    z_err = 2 * z_err + z.abs() * E
    sr = z.abs().amax(1).clamp(min=1e-4) / 127
    close(qs, sr, z_err.amax(1) / 127 + sr * 4 * E, "scale")
    code = (z / sr[:, None])
    close(q, code, 0.5 + z_err / sr[:, None] + code.abs() * (z_err.amax(1, keepdim=True) / (127 * sr[:, None]) + 4 * E), "codes")
    assert int(q.abs().max()) <= 127


def pair_inputs(rows, h, dtype, wdtype, gate, g):
    x, r = randn(rows, h, g=g).to(dtype), randn(rows, h, g=g, std=3).to(dtype)
    pw, w = (rand(h, g=g, lo=0.5, hi=1.5).to(wdtype) for _ in "pw")
    gt = None if gate is None else torch.sigmoid(randn(*((h,) if gate == "channel" else (rows, h)), g=g)).to(dtype)
    return x, r, pw, w, gt


@pytest.mark.parametrize("dtype, wdtype", [(BF16, BF16), (BF16, F32), (FP16, FP16), (FP16, F32)])
@pytest.mark.parametrize("rows, h", [(1, 1), (3, 7), (2, 8), (5, 64), (4, 100), (3, 257), (9, 512), (8, 1024), (8, 4096),
                                     (2, 4104), (300, 2048), (3, 8192), (2, 8200), (2, 16383), (2, 16384)])
def test_pair_sizes(dtype, wdtype, rows, h):
    g = gen(rows * 100003 + h)
    for gate in (None, "channel", "token"):
        x, r, pw, w, gt = pair_inputs(rows, h, dtype, wdtype, gate, g)
        sm = rand(h, g=g, lo=0.5, hi=1.5)
        check_pair(x, r, pw, w, gt, 0.3, sm, 1e-6, m.norm_add_rmsnorm_quant(
            x, r, pw, w, 1e-6, gate=gt, branch_scale=0.3, smooth=sm, want_y=True))
        check_pair(x, r, pw, w, gt, 1.0, None, 1e-5, m.norm_add_rmsnorm_quant(x, r, pw, w, 1e-5, gate=gt))
        check_pair(x, r, pw, w, gt, -2.0, None, 1e-5, m.norm_add_rmsnorm_quant(
            x, r, pw, w, 1e-5, gate=gt, branch_scale=-2.0, want_q=False, want_y=True))


@pytest.mark.parametrize("h", [1, 5, 8, 15, 16, 250, 513, 1023, 1024, 1031, 4095, 4104])
def test_pair_rows_at_any_offset(h):
    """Rows, and what is written, at odd places of larger buffers whose other bytes stay; the same bits as aligned ones."""
    g = gen(h)
    for rows, off in ((1, 1), (3, 3), (6, 0), (2, 6)):
        wide = [randn(rows, h + 24 + i, g=g).to(BF16) for i in (0, 1, 2)]
        x, r, gt = (t[:, off:off + h] for t in wide)
        pw, w = (rand(h + off, g=g, lo=0.5, hi=1.5).to(BF16)[off:] for _ in "pw")
        sm = rand(h + 1, g=g, lo=0.5, hi=1.5)[1:]
        q_all = torch.full((rows * h + 32,), 77, dtype=torch.int8, device=DEV)
        y_all, r_all = torch.full((rows * h + 32,), 7.0, dtype=BF16, device=DEV), torch.full((rows, h + 24), 7.0, dtype=BF16, device=DEV)
        q, y, ro = q_all[off:off + rows * h].view(rows, h), y_all[off:off + rows * h].view(rows, h), r_all[:, off + 1:off + 1 + h]
        scale = torch.empty(rows, device=DEV)
        want = m.norm_add_rmsnorm_quant(x.contiguous(), r.contiguous(), pw.clone(), w.clone(), 1e-6, gate=gt.contiguous(),
                                        branch_scale=0.5, smooth=sm.clone(), want_y=True)
        m.norm_add_rmsnorm_quant(x, r, pw, w, 1e-6, gate=gt, branch_scale=0.5, smooth=sm, q=q, q_scale=scale, residual_out=ro, y=y)
        check_pair(x, r, pw, w, gt, 0.5, sm, 1e-6, (q, scale, ro, y))
        for a, b in zip((q, scale, ro, y), want):
            assert torch.equal(a, b)
        assert (q_all[:off] == 77).all() and (q_all[off + rows * h:] == 77).all()
        assert (y_all[:off] == 7).all() and (y_all[off + rows * h:] == 7).all()
        assert (r_all[:, :off + 1] == 7).all() and (r_all[:, off + 1 + h:] == 7).all()


@pytest.mark.parametrize("h, off", [(256, 0), (256, 3), (4096, 0), (4097, 1), (9000, 0), (9001, 5)])
def test_pair_in_place(h, off):
    """The new residual over the old one, or over x, strided."""
    g = gen(h + off)
    wide = randn(5, 2 * h + 40, g=g).to(BF16)
    _, _, pw, w, gt = pair_inputs(5, h, BF16, BF16, "channel", g)
    for target in ("residual", "x"):
        t = wide.clone()
        x, r = t[:, off:off + h], t[:, h + 20 + off:2 * h + 20 + off]
        want = m.norm_add_rmsnorm_quant(x.clone(), r.clone(), pw, w, gate=gt, want_y=True)
        got = m.norm_add_rmsnorm_quant(x, r, pw, w, gate=gt, want_y=True, residual_out=r if target == "residual" else x)
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        keep = wide.clone()
        keep[:, h + 20 + off:2 * h + 20 + off] = want[2] if target == "residual" else r
        keep[:, off:off + h] = x if target == "residual" else want[2]
        assert torch.equal(t, keep)


@pytest.mark.parametrize("h", [64, 100, 4096])
def test_pair_extremes(h):
    x, r = (torch.ones(7, h, dtype=BF16, device=DEV) for _ in "xr")
    x[1] = 0
    x[2, h // 2] = float("nan")
    x[3, h - 1] = float("inf")
    r[4, 0] = float("-inf")
    x[5], r[5] = 0, 0
    x[6] = 1e-30
    w = torch.ones(h, dtype=BF16, device=DEV)
    q, s, ro, y = m.norm_add_rmsnorm_quant(x, r, w, w, want_y=True)
    for bad in (2, 3, 4):
        assert torch.isnan(s[bad]) and torch.isnan(y[bad]).any()
    assert torch.isnan(y[2:4]).all() and (y[4, 1:] == 0).all()  # an infinite residual: the others over an infinite root
    ok = [0, 1, 5, 6]
    assert torch.isfinite(s[ok]).all() and torch.isfinite(y[ok].float()).all() and torch.isfinite(ro[ok].float()).all()
    assert torch.equal(ro[1], r[1]) and (q[5] == 0).all() and (ro[5] == 0).all()
    close(ro[0], torch.full((h,), 2.0, device=DEV, dtype=torch.float64), 2 * U[BF16])
    # NaN in a gate reaches its row alone
    gt = torch.ones(7, h, dtype=BF16, device=DEV)
    gt[0, 1] = float("nan")
    _, s2, _, y2 = m.norm_add_rmsnorm_quant(x, r, w, w, gate=gt, want_y=True)
    assert torch.isnan(s2[0]) and torch.equal(y2[1], y[1])


def test_pair_agrees_with_the_two_norms_in_turn():
    g = gen(3)
    x, r, pw, w, _ = pair_inputs(33, 1024, BF16, F32, None, g)
    _, _, _, p = m.add_rmsnorm_quant(x, pw, want_y=True)
    _, _, s, y = m.add_rmsnorm_quant(p, w, residual=r, want_y=True)
    _, _, s2, y2 = m.norm_add_rmsnorm_quant(x, r, pw, w, want_y=True)
    close(s2, s.double(), s.double().abs() * 2 * U[BF16] + p.double().abs() * 2 * U[BF16] + 1e-30)  # p was rounded to bf16 there
    assert (y2.float() - y.float()).abs().max() < 0.1


# ------------------------------------------------------------ 8-bit products
def w8_reference(x, w, ws, xs, out):
    """The definition: the sum is exact in fp64 (below 2^53), then the stated fp32 roundings, which torch makes alike."""
    total = torch.empty(x.shape[0], w.shape[0], dtype=torch.float64, device=DEV)
    step = max(1, (1 << 26) // w.shape[1])
    for i in range(0, w.shape[0], step):
        total[:, i:i + step] = x.double() @ w[i:i + step].double().t()
    return ((total.float() * ws.float()) * xs[:, None]).to(out)


def w8_inputs(M, N, K, g, sdtype=F32):
    return codes(M, K, g=g), codes(N, K, g=g), rand(N, g=g, lo=0.5, hi=1.5).mul(1e-4).to(sdtype), rand(M, g=g, lo=0.01, hi=0.05)


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 100, 127, 128, 129, 200, 257, 300])
@pytest.mark.parametrize("N, K", [(1, 16), (7, 48), (32, 128), (33, 1008), (130, 1040), (257, 2064), (600, 4096)])
def test_w8_sizes(M, N, K):
    g = gen(M * 7919 + N * 31 + K)
    for sdtype, out in ((F32, F32), (BF16, BF16), (FP16, FP16)):
        x, w, ws, xs = w8_inputs(M, N, K, g, sdtype)
        assert torch.equal(m.w8_linear(x, w, ws, xs, out_dtype=out), w8_reference(x, w, ws, xs, out))


@pytest.mark.parametrize("M, N, K", [(1, 6144, 4096), (8, 4096, 4096), (16, 9001, 2048), (48, 4096, 14336), (64, 6144, 4096),
                                     (333, 6144, 4096), (1000, 4100, 1536), (4093, 640, 1024), (2048, 2048, 2048),
                                     (5, 3, 65536), (40, 5, 65536), (300, 300, 65536), (10000, 17, 64)])
def test_w8_large(M, N, K):
    g = gen(M + N + K)
    x, w, ws, xs = w8_inputs(M, N, K, g)
    assert torch.equal(m.w8_linear(x, w, ws, xs), w8_reference(x, w, ws, xs, BF16))


@pytest.mark.parametrize("M, N, K", [(4093, 6144, 4096), (2048, 6144, 4096), (1024, 6144, 4096), (300, 20000, 1024), (64, 60001, 2048),
                                     (33, 60001, 2048), (128, 40000, 2048), (8, 60001, 2048), (16, 3000, 4096), (32, 2000, 2048)])
def test_w8_many_tiles_a_cta_run_after_run(M, N, K):
    """Rings that go round many times, at full speed: every run has every bit."""
    g = gen(M + N)
    x, w, ws, xs = w8_inputs(M, N, K, g)
    want = w8_reference(x, w, ws, xs, F32)
    for _ in range(10):
        assert torch.equal(m.w8_linear(x, w, ws, xs, out_dtype=F32), want)


@pytest.mark.parametrize("M", [3, 20, 150, 600])
@pytest.mark.parametrize("K", [1024, 1040, 8192, 65536])
def test_w8_sums_are_exact_at_the_limits(M, K):
    """All codes as large as they come: sums up to 2^30, where fp32 sums would round."""
    N = 160
    x, w = (torch.full(s, -128, dtype=torch.int8, device=DEV) for s in ((M, K), (N, K)))
    x[M // 2] = 127
    w[1, ::2], w[1, 1::2] = 127, -128
    x[0, 0], w[2, K - 1] = 5, -7
    one = torch.ones(N, device=DEV), torch.ones(M, device=DEV)
    assert torch.equal(m.w8_linear(x, w, *one, out_dtype=F32), w8_reference(x, w, *one, F32))


PAIRS = [(1000, 5003, 4992), (700, 5100, 1040), (1500, 2000, 2192), (4093, 700, 1136), (2500, 2177, 1040), (1500, 5000, 1040),
         (1300, 3500, 4000), (300, 9000, 4096), (129, 20000, 2048)]


@pytest.mark.parametrize("M, N, K", PAIRS)
def test_w8_two_ctas_a_tile(M, N, K):
    """Sizes whose tiles are pairs of CTAs': tokens and weights that end in either half of a tile, or before its second
    half; steps of k that are odd in number, or end in zeros."""
    g = gen(M + N + K)
    x, w, ws, xs = w8_inputs(M, N, K, g)
    want = w8_reference(x, w, ws, xs, F32)
    for _ in range(3):
        y = torch.full((M + 1, N), 7.0, device=DEV)
        m.w8_linear(x, w, ws, xs, out=y[:M])
        assert torch.equal(y[:M], want) and bool((y[M] == 7).all())
    assert torch.equal(m.w8_linear(x, w, ws, xs), want.to(BF16))


@pytest.mark.parametrize("M, N, K", [(2500, 2177, 8192), (2000, 2100, 16384), (1500, 2177, 1040)])
def test_w8_two_ctas_a_tile_at_the_limits(M, N, K):
    x, w = (torch.full(s, -128, dtype=torch.int8, device=DEV) for s in ((M, K), (N, K)))
    x[M // 2] = 127
    x[::3, : K // 2] = 127  # sums that cross 2^24 and come back
    w[1, ::2], w[1, 1::2] = 127, -128
    x[0, 0], w[2, K - 1], w[N - 1, K - 3] = 5, -7, 9
    one = torch.ones(N, device=DEV), torch.ones(M, device=DEV)
    assert torch.equal(m.w8_linear(x, w, *one, out_dtype=F32), w8_reference(x, w, *one, F32))


def test_w8_two_ctas_a_tile_at_once_on_two_streams():
    g = gen(77)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    ins = [w8_inputs(1000, 5003, 2048, g), w8_inputs(700, 6000, 1040, g)]
    want = [w8_reference(*i, F32) for i in ins]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [m.w8_linear(*i, out_dtype=F32, stream=s) for i, s in zip(ins, sides)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_w8_strides_placement_and_what_is_not_written():
    g = gen(5)
    for M, N, K in ((5, 70, 256), (70, 70, 256), (300, 333, 512)):
        wide = codes(M, K + 272, g=g)
        x = wide[:, 256:256 + K]
        _, w, ws, xs = w8_inputs(M, N, K, g)
        for out in (F32, BF16):
            y_all = torch.full((M * N + 40,), 7.0, dtype=out, device=DEV)
            y = y_all[3:3 + M * N].view(M, N)
            assert m.w8_linear(x, w, ws, xs, out=y) is y
            assert torch.equal(y, w8_reference(x, w, ws, xs, out))
            assert (y_all[:3] == 7).all() and (y_all[3 + M * N:] == 7).all()


def test_w8_rows_do_not_depend_on_their_batch():
    g = gen(6)
    x, w, ws, xs = w8_inputs(700, 500, 3000 // 16 * 16, g)
    whole = m.w8_linear(x, w, ws, xs, out_dtype=F32)
    for lo, hi in ((0, 1), (3, 11), (100, 116), (5, 100), (200, 500)):
        assert torch.equal(m.w8_linear(x[lo:hi], w, ws, xs[lo:hi], out_dtype=F32), whole[lo:hi])


@pytest.mark.parametrize("M", [4, 40, 300])
def test_w8_scales_that_are_not_finite(M):
    g = gen(M)
    x, w, ws, xs = w8_inputs(M, 200, 256, g)
    clean = m.w8_linear(x, w, ws, xs, out_dtype=F32)
    ws[7], xs[2] = float("nan"), float("inf")
    y = m.w8_linear(x, w, ws, xs, out_dtype=F32)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[:, 7], hit[2] = True, True
    assert not torch.isfinite(y[hit]).any() and torch.equal(y[~hit], clean[~hit])
    assert m.w8_linear(x[:0], w, ws, xs[:0]).shape == (0, 200)


# ------------------------------------------------------------ page plan
def plan_reference(table, held, new, free, P, num_pages, tokens, taken):
    table = [list(r) for r in table]
    maxp = len(table[0]) if table else 0
    cu, lens, seq, pos, slot = [0], [], [], [], []
    at = max(0, taken)
    for b, (h, n) in enumerate(zip(held, new)):
        h, n = max(0, h), max(0, n)
        first, last = -(-h // P), min(maxp, -(-(h + n) // P))
        for i in range(first, last):
            table[b][i] = free[at] if at < len(free) else -1
            at += 1
        cu.append(min(cu[-1] + n, 2 ** 31 - 1))
        lens.append(min(h + n, 2 ** 31 - 1))
        for i in range(h, h + min(n, tokens)):
            page = table[b][i // P] if i // P < maxp else -1
            seq.append(b), pos.append(min(i, 2 ** 31 - 1)), slot.append(page * P + i % P if 0 <= page < num_pages else -1)
    live = min(len(seq), tokens)
    pad = [-1] * (tokens - live)
    return dict(table=table, cu_tokens=cu, seq_lens=lens, sequence=seq[:live] + pad, position=pos[:live] + pad,
                slot=slot[:live] + pad, taken=[min(at, len(free))], unplaced=[sum(s < 0 for s in slot[:live])])


def i32(v, shape=None):
    t = torch.tensor(v, dtype=torch.int32, device=DEV)
    return t if shape is None else t.view(shape)


def check_plan(held, new, P, maxp, free, num_pages, tokens, taken=None, seed=0, table=None):
    B = len(held)
    g = gen(seed)
    if table is None:
        table = torch.randint(0, max(1, num_pages), (B, maxp), device=DEV, generator=g, dtype=torch.int32)
    want = plan_reference(table.tolist(), held, new, free, P, num_pages, tokens, 0 if taken is None else taken)
    got = m.page_plan(table, i32(held, (B,)), i32(new, (B,)), i32(free, (len(free),)), P, num_pages, tokens,
                      taken=None if taken is None else i32([taken]))
    if B:
        assert table.tolist() == want["table"]
    for name in ("cu_tokens", "seq_lens", "sequence", "position", "slot", "taken", "unplaced"):
        assert getattr(got, name).tolist() == want[name], name
    return got


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("B, most, held", [(1, 1, 0), (1, 1, 63), (3, 1, 200), (64, 1, 500), (7, 300, 100), (1, 5000, 0),
                                           (2, 20000, 10), (513, 5, 90), (1025, 30, 40), (4096, 1, 130), (4096, 3, 10)])
def test_plan_sizes(P, B, most, held):
    import random
    r = random.Random(B * 131 + most + P)
    h, n = [r.randint(0, held) for _ in range(B)], [r.randint(0, most) for _ in range(B)]
    need = sum(-(-(a + b) // P) - -(-a // P) for a, b in zip(h, n))
    maxp = max(-(-(a + b) // P) for a, b in zip(h, n)) + 1
    free = list(range(5, 5 + need + 3))
    r.shuffle(free)
    got = check_plan(h, n, P, maxp, free, 5 + need + 3, sum(n) + r.randint(0, 70))
    assert int(got.unplaced) == 0 and int(got.taken) == need
    check_plan(h, n, P, maxp, [99] * 3 + free, 10 ** 6, sum(n), taken=3)


def test_plan_edges():
    # no sequences; none with new tokens; no tokens wanted
    check_plan([], [], 16, 0, [1, 2], 8, 5)
    check_plan([], [], 16, 0, [], 8, 0, taken=0)
    check_plan([5, 0], [0, 0], 16, 4, [3], 8, 4, taken=1)
    check_plan([5, 0], [3, 40], 16, 4, [3, 4, 5], 8, 0)
    # the list runs out inside a sequence, and before the call
    check_plan([10, 16, 0], [30, 16, 40], 16, 8, [7, 6, 5], 8, 100)
    check_plan([10, 16, 0], [30, 16, 40], 16, 8, [7, 6, 5], 8, 86, taken=3)
    check_plan([0], [40], 16, 8, [7, 6, 5], 8, 40, taken=9)
    check_plan([0], [40], 16, 8, [7, 6, 5], 8, 40, taken=-4)
    check_plan([1], [1], 16, 2, [], 8, 1)
    # sequences that outgrow their rows of the table, or already have
    check_plan([30, 0, 64, 100], [10, 100, 1, 3], 16, 4, list(range(20)), 20, 200)
    check_plan([0, 3], [5, 6], 16, 0, [1, 2], 8, 11)
    # pages outside the pool, in the list and in the table
    check_plan([8, 0], [20, 20], 16, 4, [50, -3, 2, 9], 10, 40, table=i32([[-1, 0, 0, 0], [0, 0, 0, 0]]))
    check_plan([8, 8], [4, 4], 16, 2, [1], 10, 8, table=i32([[10, 3], [9, 3]]))
    # fewer rows than tokens
    check_plan([0, 7], [100, 50], 32, 9, list(range(30)), 30, 99)
    check_plan([0, 7], [100, 50], 32, 9, list(range(30)), 30, 101)
    # negative lengths count as 0
    check_plan([-5, 3], [4, -2], 16, 3, [1, 2], 8, 6)


def test_plan_of_lengths_near_32_bits():
    top = 2 ** 31 - 1
    got = check_plan([top, top - 5, 0], [7, 5, 9], 16, 3, [4, 5, 6], 8, 21)
    assert got.seq_lens.tolist() == [top, top, 9] and got.position.tolist()[:7] == [top] * 7
    got = check_plan([0, 0, 0], [top, top, 3], 128, 2, [1, 2, 3, 4, 5], 8, 300)
    assert got.cu_tokens.tolist() == [0, top, top, top]


def test_plan_writes_only_new_entries_of_a_strided_table():
    wide = torch.full((6, 40), -7, dtype=torch.int32, device=DEV)
    table = wide[:, 5:25]
    held, new = [0, 17, 64, 5, 0, 31], [33, 1, 0, 11, 1, 2]
    m.page_plan(table, i32(held), i32(new), i32(list(range(50))), 16, 50, 48)
    fresh = torch.zeros_like(wide, dtype=torch.bool)
    for b, (h, n) in enumerate(zip(held, new)):
        fresh[b, 5 - (-h // 16):5 - (-(h + n) // 16)] = True
    assert (wide[~fresh] == -7).all()
    assert wide[fresh].tolist() == list(range(int(fresh.sum())))


def test_plan_moves_taken_on_in_place_and_replays():
    """A captured step: the same call again takes the next pages."""
    B, P = 3, 16
    table = torch.full((B, 8), -1, dtype=torch.int32, device=DEV)
    held, new, taken, free = i32([0, 0, 0]), i32([16, 32, 5]), i32([0]), i32(list(range(40)))
    p = m.page_plan(table, held, new, free, P, 40, 53, taken=taken, taken_out=taken)
    assert p.taken is taken and int(taken) == 4
    held = p.seq_lens.clone()
    new.fill_(16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        p = m.page_plan(table, held, new, free, P, 40, 48, taken=taken, taken_out=taken)
        held.copy_(p.seq_lens)
    for step in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert int(taken) == 10 and held.tolist() == [48, 64, 37]
    assert table[:, :4].tolist() == [[0, 4, 7, -1], [1, 2, 5, 8], [3, 6, 9, -1]]
    assert p.slot.view(3, 16)[:, 0].tolist() == [7 * 16, 8 * 16, 6 * 16 + 5]


# ------------------------------------------------------------ log probabilities
def check_logprobs(logits, tokens, top, out):
    rows, V = logits.shape
    lp, H, tlp, tid = out
    l = logits.double()
    p = torch.log_softmax(l, dim=1)
    big = l.amax(1)
    log_s = torch.logsumexp(l - big[:, None], dim=1)
    want_h = torch.special.entr(p.exp()).sum(1)
    # A term passes V / 256 additions of its thread where the row is long (64 and fewer else) and some 20 joins of 3
    # roundings; an exponential is good to 2^-22, its argument d to 2^-23 of it, and terms with |d| above 25 weigh nothing.
    base = (max(64, V // 256) + 64) * E + 2.0 ** -22 + 25 * 2 * E

    def tol(ref):
        """Beside the sums: the logarithm (at most 12, good to its last bit), and two roundings of the result's size, l - M and
        that less log S, each half a step."""
        return base + (12 + 3 * ref.abs()) * 2 * E
    if tokens is not None:
        idx = tokens.long().view(rows, -1)
        inside = (idx >= 0) & (idx < V)
        ref = torch.where(inside, p.gather(1, idx.clamp(0, V - 1)), float("-inf"))
        got = lp.view(rows, -1)
        inf = ref == float("-inf")
        assert torch.equal(inf, got == float("-inf"))
        ref = ref.masked_fill(inf, 0)
        close(got.masked_fill(inf, 0), ref, tol(ref), "logprob")
    mean = (log_s - want_h).abs()
    close(H, want_h, base * (1 + 2 * mean) + 16 * E * (1 + mean + want_h), "entropy")
    if top:
        order = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(tid.long(), order), "top_id"
        ref = p.gather(1, order)
        inf = ref == float("-inf")
        assert torch.equal(inf, tlp == float("-inf"))
        ref = ref.masked_fill(inf, 0)
        close(tlp.masked_fill(inf, 0), ref, tol(ref), "top_logprob")


@pytest.mark.parametrize("dtype", [BF16, FP16, F32])
@pytest.mark.parametrize("rows, V", [(1, 1), (3, 2), (2, 31), (5, 32), (4, 33), (3, 127), (7, 1000), (2, 4099), (1, 32001),
                                     (65, 9001), (700, 1025), (5, 65537), (2, 262144)])
def test_logprobs_sizes(dtype, rows, V):
    g = gen(rows * 1009 + V)
    logits = (randn(rows, V, g=g) * rand(rows, 1, g=g, lo=0.2, hi=4.0)).to(dtype)
    for top, n in ((0, 1), (1, 3), (min(5, V), 1), (min(20, V), 0), (min(32, V), 2)):
        tokens = torch.randint(0, V, (rows, n), device=DEV, generator=g)
        if n == 1:
            tokens = tokens[:, 0].int()
        check_logprobs(logits, tokens, top, m.token_logprobs(logits, tokens, top))
    assert m.token_logprobs(logits)[0] is None


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [40, 1000, 20011])
def test_logprobs_orders_and_ties(dtype, V):
    """Rows that rise, fall, repeat a few values, hold one value, or hide their largest at either end."""
    g = gen(V)
    ramp = torch.linspace(-8, 8, V, device=DEV)
    rows = [ramp, ramp.flip(0), torch.zeros(V, device=DEV), torch.randint(0, 3, (V,), device=DEV, generator=g).float(),
            torch.randint(0, 2, (V,), device=DEV, generator=g).float() * -0.0, ramp[torch.randperm(V, device=DEV, generator=g)],
            torch.where(torch.arange(V, device=DEV) == 0, 9.0, ramp), torch.where(torch.arange(V, device=DEV) == V - 1, 30.0, -ramp)]
    logits = torch.stack(rows).to(dtype)
    for top in (1, 7, 32):
        check_logprobs(logits, None, top, m.token_logprobs(logits, None, top))


@pytest.mark.parametrize("dtype", [BF16, FP16, F32])
def test_logprobs_masks(dtype):
    g = gen(9)
    V, low = 5000, torch.finfo(dtype).min
    logits = (randn(6, V, g=g) * 3).to(dtype)
    keep = rand(6, V, g=g) < 0.002
    keep[:, 77] = True
    for value in (float("-inf"), low):
        masked = logits.masked_fill(~keep, value)
        masked[0] = value
        masked[0, 4321] = 1.0                      # a single token is allowed
        masked[1] = value
        masked[1, 100:103] = low                   # the lowest numbers, among -inf or themselves
        tokens = torch.randint(0, V, (6, 4), device=DEV, generator=g)
        tokens[:, 0], tokens[0, 1] = 77, 4321
        got = m.token_logprobs(masked, tokens, 20)
        check_logprobs(masked, tokens, 20, got)
        assert float(got[0][0, 1]) == 0.0 and float(got[1][0]) == 0.0


def test_logprobs_rows_without_a_distribution():
    for V in (9, 3000, 70000):
        x = torch.randn(5, V, device=DEV)
        x[1] = float("-inf")
        x[2, V // 2] = float("nan")
        x[3, V - 1] = float("inf")
        tokens = torch.zeros(5, dtype=torch.int32, device=DEV)
        for dtype in (F32, BF16):
            lp, H, tlp, tid = m.token_logprobs(x.to(dtype), tokens, 4)
            for t in (lp[:, None], H[:, None], tlp):
                assert torch.isnan(t[1:4]).all() and torch.isfinite(t[[0, 4]]).all()
            assert tid[1].tolist() == [0, 1, 2, 3] and (tid[2:4] == -1).all()
            check_logprobs(x[[0, 4]].to(dtype), tokens[:2], 4, tuple(t[[0, 4]] for t in (lp, H, tlp, tid)))


def test_logprobs_tokens_outside_and_far_values():
    x = torch.randn(4, 300, device=DEV) * 2
    x[1] += 1000
    x[2] -= 30000
    x[3] *= 1e30
    tokens = torch.tensor([[-1, 300, 5], [0, 2 ** 31 - 1, 299], [1, -2 ** 31, 2], [3, 4, 5]], device=DEV)
    check_logprobs(x[:3], tokens[:3], 5, tuple(t[:3] for t in m.token_logprobs(x, tokens, 5)))
    lp, H, tlp, tid = m.token_logprobs(x, tokens, 5)
    assert float(H[3]) == 0.0 and float(tlp[3, 0]) == 0.0 and int(tid[3, 0]) == int(x[3].argmax())
    big = torch.tensor([[2 ** 40, 3]] * 4, device=DEV)
    assert (m.token_logprobs(x, big)[0][:, 0] == float("-inf")).all()
    assert torch.equal(m.token_logprobs(x, tokens.int())[0], lp)


@pytest.mark.parametrize("off", [0, 1, 3, 5, 8])
def test_logprobs_strided_rows_at_any_offset(off):
    """Rows inside wider ones whose other elements would change every result."""
    g = gen(off)
    for dtype in (BF16, F32):
        for V in (1, 6, 250, 4097):
            wide = torch.full((4, V + 19), float("nan"), device=DEV, dtype=dtype)
            wide[:, off:off + V] = randn(4, V, g=g).to(dtype)
            x = wide[:, off:off + V]
            a, b = m.token_logprobs(x, None, min(V, 6)), m.token_logprobs(x.clone(), None, min(V, 6))
            check_logprobs(x, None, min(V, 6), a)
            assert torch.equal(a[3], b[3])


# ------------------------------------------------------------ streams, graphs, devices
def every_call(seed):
    """One call of each operator, on inputs of the seed: (call, outputs expected)."""
    g = gen(seed)
    x, r, pw, w, gt = pair_inputs(37, 1000, BF16, BF16, "token", g)
    x8, w8, ws, xs = w8_inputs(150, 700, 2048, g)
    logits, tokens = randn(9, 30001, g=g).to(BF16), torch.randint(0, 30001, (9,), device=DEV, generator=g)
    held, new, free = i32([3, 100, 0]), i32([40, 1, 17]), i32(list(range(30)))
    table = torch.zeros(3, 9, dtype=torch.int32, device=DEV)
    return [lambda **k: m.norm_add_rmsnorm_quant(x, r, pw, w, gate=gt, want_y=True, **k),
            lambda **k: (m.w8_linear(x8, w8, ws, xs, **k),), lambda **k: (m.w8_linear(x8[:5], w8, ws, xs[:5], **k),),
            lambda **k: (m.w8_linear(x8[:40], w8, ws, xs[:40], **k),),
            lambda **k: m.token_logprobs(logits, tokens, 5, **k),
            lambda **k: tuple(m.page_plan(table, held, new, free, 16, 30, 64, **k))]


def same(a, b):
    return all(torch.equal(s, t) for s, t in zip(a, b))


def test_calls_on_another_stream():
    for call in every_call(1):
        want = call()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = [call(stream=side) for _ in range(3)]
        with torch.cuda.stream(side):
            got.append(call())
        torch.cuda.current_stream().wait_stream(side)
        assert all(same(want, o) for o in got)


def test_calls_at_once_on_two_streams():
    calls = every_call(2)
    want = [c() for c in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[c(stream=s) for c in calls for _ in range(2)] for s in streams]
    torch.cuda.synchronize()
    for outs in got:
        for i, o in enumerate(outs):
            assert same(want[i // 2], o)


def test_captured_calls_replay_with_new_inputs():
    for call in every_call(3):
        want = call()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            call()
            with torch.cuda.graph(graph, stream=side):
                first = call()
                second = call()
        for t in first + second:
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        assert same(want, first) and same(want, second)


def test_results_do_not_change_from_call_to_call():
    for call in every_call(4):
        want = call()
        assert all(same(want, call()) for _ in range(5))


# ------------------------------------------------------------ offsets past 32 bits
def test_w8_outputs_and_weights_past_32_bits():
    g = gen(11)
    M, N, K = 17000, 130001, 64
    x, w, ws, xs = w8_inputs(M, N, K, g)
    y = m.w8_linear(x, w, ws, xs)
    assert y.numel() > 2 ** 31
    for rows in (slice(0, 5), slice(16500, 16530), slice(M - 7, M)):
        assert torch.equal(y[rows], w8_reference(x[rows], w, ws, xs[rows], BF16))
    del y
    N, K = 600001, 4096
    w = torch.randint(-128, 128, (N, K), device=DEV, generator=g, dtype=torch.int8)
    assert w.numel() > 2 ** 31
    ws = rand(N, g=g)
    for M in (3, 20, 70, 200):
        x, xs = codes(M, K, g=g), rand(M, g=g)
        y = m.w8_linear(x, w, ws, xs)
        for cols in (slice(0, 300), slice(524200, 524400), slice(N - 200, N)):
            assert torch.equal(y[:, cols], w8_reference(x, w[cols], ws[cols], xs, BF16))


def test_pair_and_logprobs_past_32_bits():
    g = gen(12)
    rows, h = 140000, 16384
    x = torch.empty(rows, h, dtype=BF16, device=DEV).normal_(generator=g)
    r = torch.empty(rows, h, dtype=BF16, device=DEV).normal_(generator=g)
    assert x.numel() > 2 ** 31
    pw, w = (rand(h, g=g, lo=0.5, hi=1.5).to(BF16) for _ in "pw")
    whole = m.norm_add_rmsnorm_quant(x, r, pw, w, gate=r, want_y=True)
    for part in (slice(0, 3), slice(131071, 131074), slice(rows - 3, rows)):
        for a, b in zip(whole, m.norm_add_rmsnorm_quant(x[part], r[part], pw, w, gate=r[part], want_y=True)):
            assert torch.equal(a[part], b)
    del whole, r
    logits = x.view(-1)[:17000 * 130001].view(17000, 130001)
    whole = m.token_logprobs(logits, torch.zeros(17000, dtype=torch.int32, device=DEV), 3)
    for part in (slice(0, 2), slice(16515, 16520), slice(16998, 17000)):
        check_logprobs(logits[part], torch.zeros(logits[part].shape[0], dtype=torch.int32, device=DEV), 3,
                       tuple(t[part] for t in whole))
