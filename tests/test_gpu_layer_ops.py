"""The decoder-layer operators against their definitions in 64 bits.

Tolerances come from the arithmetic: the unit roundoff of the output type,
fp32 sums whose error is bounded by the number of additions a term passes
through times 2^-23 times the sum of magnitudes, and, for the attention, the
rounding of the softmax weights to fp16 (2^-11 of sum p |v|)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_expert_ffn_dispatch_gb300 as m  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 1e-38, torch.float16: 2.0 ** -25, torch.float32: 1e-38}  # half a smallest step near zero
BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(*shape, g, std=1.0):
    return torch.randn(shape, device=DEV, generator=g) * std


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


# ------------------------------------------------------------ norm
def check_norm(x, w, residual, smooth, out, eps):
    q, qs, res, y = out
    s = x.double() if residual is None else x.double() + residual.double()
    if residual is not None:
        assert torch.equal(res, (x.float() + residual.float()).to(x.dtype))
    yr = s / ((s * s).mean(1, keepdim=True) + eps).sqrt() * w.double()
    # at most 16 + 10 additions a thread and warp tree, and a few roundings
    rel = 48 * 2.0 ** -24
    if y is not None:
        close(y, yr, yr.abs() * (U[x.dtype] + rel) + TINY[x.dtype], "y")
    z = yr if smooth is None else yr * smooth.double()
    sr = z.abs().amax(1).clamp(min=1e-4) / 127
    close(qs, sr, sr * (rel + 4 * 2.0 ** -24), "scale")
    code = z / sr[:, None]
    close(q, code, 0.5 + 127 * 2 * (rel + 4 * 2.0 ** -24), "codes")
    assert int(q.abs().max()) <= 127


@pytest.mark.parametrize("dtype, wdtype", [(BF16, BF16), (BF16, F32), (FP16, FP16), (FP16, F32)])
@pytest.mark.parametrize("rows, h", [(1, 1), (3, 7), (2, 8), (5, 64), (4, 100), (3, 257), (8, 4096), (2, 4104), (300, 2048),
                                     (3, 8192), (2, 8200), (2, 16383), (2, 16384)])
def test_norm_sizes(dtype, wdtype, rows, h):
    g = gen(rows * 100003 + h)
    x, r = randn(rows, h, g=g).to(dtype), randn(rows, h, g=g, std=3).to(dtype)
    w = (torch.rand(h, device=DEV, generator=g) + 0.5).to(wdtype)
    sm = torch.rand(h, device=DEV, generator=g) + 0.5
    check_norm(x, w, r, sm, m.add_rmsnorm_quant(x, w, 1e-6, residual=r, smooth=sm, want_y=True), 1e-6)
    check_norm(x, w, None, None, m.add_rmsnorm_quant(x, w, 1e-5), 1e-5)


@pytest.mark.parametrize("h", [1, 5, 8, 15, 16, 250, 513, 1023, 1024, 1031, 4095, 4104])
def test_norm_rows_at_any_offset(h):
    """Rows, and what is written, at odd places of larger buffers whose other bytes stay."""
    g = gen(h)
    for rows, off in ((1, 1), (3, 3), (6, 0), (2, 6)):
        wide_x, wide_r = randn(rows, h + 24, g=g).to(BF16), randn(rows, h + 9, g=g).to(BF16)
        x, r = wide_x[:, off:off + h], wide_r[:, off:off + h]
        w, sm = (torch.rand(h + off, device=DEV, generator=g) + 0.5)[off:], torch.rand(h + 1, device=DEV, generator=g)[1:] + 0.5
        w = w.to(BF16)
        q_all = torch.full((rows * h + 32,), 77, dtype=torch.int8, device=DEV)
        y_all, r_all = torch.full((rows * h + 32,), 7.0, dtype=BF16, device=DEV), torch.full((rows, h + 24), 7.0, dtype=BF16, device=DEV)
        q, y, ro = q_all[off:off + rows * h].view(rows, h), y_all[off:off + rows * h].view(rows, h), r_all[:, off + 1:off + 1 + h]
        scale = torch.empty(rows, device=DEV)
        want = m.add_rmsnorm_quant(x.contiguous(), w, 1e-6, residual=r.contiguous(), smooth=sm, want_y=True)
        m.add_rmsnorm_quant(x, w, 1e-6, residual=r, smooth=sm, q=q, q_scale=scale, residual_out=ro, y=y)
        check_norm(x, w, r, sm, (q, scale, ro, y), 1e-6)
        for a, b in zip((q, scale, ro, y), want):
            assert torch.equal(a, b)
        assert (q_all[:off] == 77).all() and (q_all[off + rows * h:] == 77).all()
        assert (y_all[:off] == 7).all() and (y_all[off + rows * h:] == 7).all()
        assert (r_all[:, :off + 1] == 7).all() and (r_all[:, off + 1 + h:] == 7).all()


def test_norm_strides_alignment_and_in_place():
    g = gen(1)
    wide = randn(6, 600, g=g).to(BF16)
    w = torch.ones(256, dtype=BF16, device=DEV)
    for off in (0, 8, 1, 3):  # 16-byte aligned rows, and rows that are not
        x, r = wide[:, off:off + 256], wide[:, off + 260:off + 516]
        check_norm(x, w, r, None, m.add_rmsnorm_quant(x, w, residual=r, want_y=True), 1e-6)
    # the sum replaces the residual, strided, and y replaces x
    x, r = wide[:, :256].contiguous(), wide[:, 300:556]
    want = m.add_rmsnorm_quant(x, w, residual=r.clone(), want_y=True)
    keep = wide.clone()
    got = m.add_rmsnorm_quant(x, w, residual=r, residual_out=r, y=x)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert torch.equal(wide[:, :300], keep[:, :300]) and torch.equal(wide[:, 556:], keep[:, 556:])


@pytest.mark.parametrize("h", [64, 100, 4096])
def test_norm_extremes(h):
    x = torch.ones(6, h, dtype=BF16, device=DEV)
    x[1] = 0
    x[2, h // 2] = float("nan")
    x[3, h - 1] = float("inf")
    x[4] = 1e-30
    w = torch.ones(h, dtype=F32, device=DEV)
    q, qs, _, y = m.add_rmsnorm_quant(x, w, 1e-6, want_y=True)
    assert (q[1] == 0).all() and (y[1] == 0).all()
    close(qs[[1, 4]], torch.full((2,), 1e-4 / 127, dtype=torch.float64, device=DEV), 1e-12)
    assert torch.isnan(qs[2]) and torch.isnan(qs[3])
    assert (q[0] == 127).all() and (q[5] == 127).all() and torch.isfinite(qs[[0, 5]]).all()


def test_norm_refusals_and_empty():
    x, w = torch.ones(4, 64, dtype=BF16, device=DEV), torch.ones(64, dtype=BF16, device=DEV)
    q, qs, r, y = m.add_rmsnorm_quant(x[:0], w)
    assert q.shape == (0, 64) and qs.shape == (0,) and r is None and y is None
    for bad in (lambda: m.add_rmsnorm_quant(x.float(), w), lambda: m.add_rmsnorm_quant(x, w.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: m.add_rmsnorm_quant(x[0], w), lambda: m.add_rmsnorm_quant(x, w[:32]),
                lambda: m.add_rmsnorm_quant(x, w, residual=x[:2]), lambda: m.add_rmsnorm_quant(x, w, residual_out=x),
                lambda: m.add_rmsnorm_quant(x.t().contiguous().t(), w), lambda: m.add_rmsnorm_quant(x, w.cpu())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(m.MoeError):
        m.add_rmsnorm_quant(torch.ones(1, 16385, dtype=BF16, device=DEV), torch.ones(16385, dtype=BF16, device=DEV))


# ------------------------------------------------------------ 4-bit products
def w4_case(M, N, K, group, dtype, seed, x8=False, zero=False, sdtype=None):
    g = gen(seed)
    code = torch.randint(0, 16, (N, K), device=DEV, generator=g, dtype=torch.uint8)
    w = code[:, 0::2] | (code[:, 1::2] << 4)
    ws = (torch.rand(N, K // group, device=DEV, generator=g) + 0.5).to(sdtype or dtype)
    z = torch.randint(0, 16, (N, K // group), device=DEV, generator=g, dtype=torch.uint8) if zero else None
    if x8:
        x, xs = torch.randint(-127, 128, (M, K), device=DEV, generator=g, dtype=torch.int8), torch.rand(M, device=DEV, generator=g)
    else:
        x, xs = randn(M, K, g=g).to(dtype), None
    return code, w, ws, z, x, xs


def check_w4(code, ws, z, x, xs, got):
    K = code.shape[1]
    group = K // ws.shape[1]
    wd = code.double() - (8 if z is None else z.double().repeat_interleave(group, 1))
    wd = wd * ws.double().repeat_interleave(group, 1)
    xd = x.double() if xs is None else x.double() * xs.double()[:, None]
    ref, mag = xd @ wd.t(), xd.abs() @ wd.abs().t()
    # a term passes through the 16 of a product, the products of its group, the groups and parts of K
    close(got, ref, ref.abs() * U[got.dtype] + (K / 16 + K / group + 48) * 2.0 ** -23 * mag + TINY[got.dtype])


@pytest.mark.parametrize("M, N, K, group", [
    (1, 1, 32, 32), (1, 17, 64, 64), (2, 16, 96, 32), (3, 15, 128, 128), (7, 100, 160, 32), (8, 33, 256, 64),
    (9, 64, 256, 256), (16, 100, 512, 128), (17, 1000, 1024, 128), (32, 48, 320, 64), (33, 70, 512, 32), (64, 500, 4096, 128),
    (100, 40, 384, 128), (1, 5000, 4096, 128), (8, 40000, 256, 64), (20, 80000, 128, 128), (16, 90000, 192, 32),
    (1, 64, 16384, 128), (8, 300, 12800, 64), (16, 50, 11008, 32), (64, 33, 16384, 16384), (4, 16, 65536, 128)])
@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_w4_sizes(M, N, K, group, dtype):
    code, w, ws, z, x, xs = w4_case(M, N, K, group, dtype, M + N + K, zero=(M + N) % 2 == 0)
    got = m.w4_linear(x, w, ws, zero=z, out_dtype=F32)
    assert got.dtype == F32 and got.shape == (M, N)
    check_w4(code, ws, z, x, xs, got)
    out = torch.full((M, N), float("nan"), dtype=dtype, device=DEV)
    assert m.w4_linear(x, w, ws, zero=z, out=out) is out
    assert torch.equal(out, got.to(dtype))  # one rounding of the same sums, and every element written


@pytest.mark.parametrize("M, N, K, group", [
    (16, 20000, 8352, 32), (8, 30001, 8224, 32), (16, 41, 65536, 64), (30, 9000, 12832, 32), (8, 700, 40960, 128)])
@pytest.mark.parametrize("x8", [False, True])
def test_w4_rows_longer_than_shared_memory(M, N, K, group, x8):
    """Clusters that share K, over several rounds of tiles and several pieces."""
    code, w, ws, z, x, xs = w4_case(M, N, K, group, BF16, N + K, x8=x8, zero=True)
    got = m.w4_linear(x, w, ws, zero=z, x_scale=xs, out_dtype=F32)
    check_w4(code, ws, z, x, xs, got)
    assert torch.equal(got, m.w4_linear(x, w, ws, zero=z, x_scale=xs, out_dtype=F32))


@pytest.mark.parametrize("M, N, K, group", [(1, 40, 64, 32), (8, 200, 4096, 64), (13, 77, 1024, 128), (40, 30, 8320, 64)])
@pytest.mark.parametrize("sdtype", [BF16, FP16, F32])
def test_w4_int8_rows_and_scale_types(M, N, K, group, sdtype):
    code, w, ws, z, x, xs = w4_case(M, N, K, group, BF16, 7 * M + N, x8=True, zero=True, sdtype=sdtype)
    got = m.w4_linear(x, w, ws, zero=z, x_scale=xs)
    assert got.dtype == BF16
    check_w4(code, ws, z, x, xs, got)
    check_w4(code, ws, z, x, xs, m.w4_linear(x, w, ws, zero=z, x_scale=xs, out_dtype=FP16 if sdtype != BF16 else F32)
             if float(ws.float().max()) < 1e3 and K * 127 * 15 < 6e4 else got)


def test_w4_strided_rows_repeat_and_nan_rows():
    code, w, ws, z, wide, _ = w4_case(9, 130, 512, 128, BF16, 5)
    wide = torch.cat([wide, wide + 1, wide], dim=1)
    x = wide[:, 512:1024]
    a, b = m.w4_linear(x, w, ws), m.w4_linear(x.contiguous(), w, ws)
    assert torch.equal(a, b)
    x = x.clone()
    x[4, 100] = float("nan")
    x[7, 3] = float("inf")
    c = m.w4_linear(x, w, ws)
    rows = [0, 1, 2, 3, 5, 6, 8]
    assert torch.equal(c[rows], a[rows])  # a row of x meets no other row
    assert torch.isnan(c[4]).all() and not torch.isfinite(c[7]).any()


def test_w4_refusals_and_empty():
    code, w, ws, z, x, _ = w4_case(2, 32, 256, 128, BF16, 6)
    assert m.w4_linear(x[:0], w, ws).shape == (0, 32)
    for bad in (lambda: m.w4_linear(x.float(), w, ws), lambda: m.w4_linear(x, w.to(torch.int8), ws),
                lambda: m.w4_linear(x, w, ws, zero=ws), lambda: m.w4_linear(x, w, ws, out_dtype=torch.float64)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: m.w4_linear(x, w[:, :64], ws), lambda: m.w4_linear(x, w[:16], ws),
                lambda: m.w4_linear(x.to(torch.int8), w, ws), lambda: m.w4_linear(x, w, ws, x_scale=ws[0].float()),
                lambda: m.w4_linear(x, w.t().contiguous().t(), ws), lambda: m.w4_linear(x, w, ws.cpu()),
                lambda: m.w4_linear(x, w, ws, out=torch.empty(3, 32, dtype=BF16, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(m.MoeError):  # groups of 16
        m.w4_linear(x, w, torch.ones(32, 16, dtype=BF16, device=DEV))
    with pytest.raises(m.MoeError):  # rows that are not 16-byte aligned
        m.w4_linear(torch.ones(2, 300, dtype=BF16, device=DEV)[:, 3:259], w, ws)


# ------------------------------------------------------------ cache append
def new_cache(pages, heads, page, dim, seed=0, fused=False):
    """Codes and scales that a call must not take for new ones; `fused`: K and V interleaved in one tensor."""
    g = gen(seed)
    both = torch.randint(-127, 128, (pages, 2, heads, page, dim), device=DEV, generator=g, dtype=torch.int8)
    sc = torch.rand(pages, 2, heads, device=DEV, generator=g) * 0.02 + 0.005
    if fused:
        return m.KvCache(both[:, 0], both[:, 1], sc[:, 0], sc[:, 1])
    return m.KvCache(*(t.contiguous() for t in (both[:, 0], both[:, 1], sc[:, 0], sc[:, 1])))


def page_table(need, pool, seed=0, pad=2):
    ids = np.random.default_rng(seed).permutation(pool)
    t = np.full((len(need), max(max(need), 1) + pad), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = ids[at:at + k]
        at += k
    return torch.from_numpy(t)


def append_reference(code, scale, new, table, start, counts, page):
    """The definition, in fp32 operations that round once each (numpy, on the host)."""
    f = np.float32
    code, scale = code.copy(), scale.copy()
    at = 0
    for b, n in enumerate(counts):
        x = new[at:at + n]
        at += n
        for p in range(start[b] // page, (start[b] + n - 1) // page + 1 if n else 0):
            lo, hi = max(start[b] - p * page, 0), min(start[b] + n - p * page, page)
            rows = x[p * page + lo - start[b]:p * page + hi - start[b]]
            pg = table[b][p] if p < table.shape[1] else -1
            if pg < 0 or pg >= code.shape[0]:
                continue
            for h in range(code.shape[1]):
                top = f(np.abs(rows[:, h]).max())
                old = scale[pg, h]
                to = max(top, f(1e-4)) / f(127) if lo == 0 else max(old, top / f(127))
                if lo > 0 and to > old:
                    code[pg, h, :lo] = np.clip(np.rint(code[pg, h, :lo].astype(f) * (old / to)), -127, 127)
                scale[pg, h] = to
                code[pg, h, lo:hi] = np.clip(np.rint(rows[:, h] * (f(1) / to)), -127, 127)
    return code, scale


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page, heads", [(16, 1), (32, 3), (64, 8), (128, 2)])
@pytest.mark.parametrize("lens", [
    [(0, 1)], [(0, 1), (15, 1), (16, 1), (63, 1), (64, 1), (127, 1), (200, 1)],
    [(0, 300), (5, 0), (31, 1), (16, 16), (100, 129), (64, 64), (7, 2)], [(130, 1000)]])
def test_append(dim, page, heads, lens):
    start, counts = [a for a, _ in lens], [n for _, n in lens]
    need = [-(-(a + n) // page) for a, n in lens]
    pool = sum(need) + 4
    cache = new_cache(pool, heads, page, dim, seed=page + heads, fused=heads == 3)
    table = page_table(need, pool, seed=dim)
    g = gen(11)
    T = sum(counts)
    dtype = BF16 if heads != 2 else FP16
    wide = (randn(T, 4 * heads * dim, g=g) * torch.rand(T, 1, device=DEV, generator=g) * 4).to(dtype)
    k, v = (wide[:, i * heads * dim:(i + 1) * heads * dim].view(T, heads, dim) for i in (1, 3))
    want = [append_reference(c.cpu().numpy(), s.cpu().numpy(), x.float().cpu().numpy(), table.numpy(), start, counts, page)
            for c, s, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v))]
    cu = None if counts == [1] * len(counts) else torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device=DEV)
    st = torch.tensor(start, dtype=torch.int32, device=DEV)
    for _ in range(2):  # the second call writes the same again: no scale grows, no code moves
        cache.append(k, v, table.to(DEV), st, cu_tokens=cu)
        for (c, s), got_c, got_s in zip(want, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
            assert np.array_equal(s, got_s.cpu().numpy())
            assert np.array_equal(c, got_c.cpu().numpy())


def test_append_skips_what_has_no_page_and_keeps_nan_to_its_page():
    cache = new_cache(6, 2, 16, 64, seed=1)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    g = gen(2)
    k, v = randn(4, 2, 64, g=g).to(BF16), randn(4, 2, 64, g=g).to(BF16)
    table = torch.tensor([[-1, 0], [6, 1], [2, 2], [3, 4]], dtype=torch.int32, device=DEV)
    cache.append(k, v, table, torch.tensor([3, 0, 32, -1], dtype=torch.int32, device=DEV))
    for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)):
        assert torch.equal(a, b)
    k[1, 0, 5] = float("nan")
    v[2, 1, 3] = float("inf")
    table = torch.tensor([[0], [1], [2], [3]], dtype=torch.int32, device=DEV)
    cache.append(k, v, table, torch.zeros(4, dtype=torch.int32, device=DEV))
    assert torch.isnan(cache.k_scale[1, 0]) and not torch.isfinite(cache.v_scale[2, 1])
    bad_k, bad_v = torch.zeros(4, 2, dtype=torch.bool, device=DEV), torch.zeros(4, 2, dtype=torch.bool, device=DEV)
    bad_k[1, 0] = bad_v[2, 1] = True
    assert torch.isfinite(cache.k_scale[:4][~bad_k]).all() and torch.isfinite(cache.v_scale[:4][~bad_v]).all()
    cache.append(k[:0], v[:0], table[:0], torch.zeros(0, dtype=torch.int32, device=DEV))


# ------------------------------------------------------------ attention
def attention_reference(q, k, v, ks, vs, table, kv, qlen, window, scale):
    """(out, tolerance without the output's rounding) in 64 bits, sequence by sequence."""
    P, H, D = k.shape[2], k.shape[1], k.shape[3]
    G = q.shape[1] // H
    out, tol = torch.zeros(q.shape, dtype=torch.float64, device=DEV), torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, c) in enumerate(zip(kv, qlen)):
        rows = slice(at, at + c)
        at += c
        if n <= 0 or c == 0:
            continue
        pages = table[b, :-(-n // P)].long()
        good = ((pages >= 0) & (pages < k.shape[0])).repeat_interleave(P)[:n].to(DEV)
        pages = pages.clamp(0, k.shape[0] - 1).to(DEV)
        i = torch.arange(n, device=DEV)
        p = torch.arange(n - c, n, device=DEV)[:, None]
        seen = (i <= p) & good & (i > p - (window or n + c + 1))
        for h in range(H):
            kd = (k[pages, h].double() * ks[pages, h].double()[:, None, None]).reshape(-1, D)[:n]
            vd = (v[pages, h].double() * vs[pages, h].double()[:, None, None]).reshape(-1, D)[:n]
            kd, vd = kd.masked_fill(~good[:, None], 0), vd.masked_fill(~good[:, None], 0)
            heads = slice(h * G, (h + 1) * G)
            qd = q[rows, heads].double()
            a = (torch.einsum("cgd,nd->cgn", qd, kd) * scale).masked_fill(~seen[:, None], -math.inf)
            w = torch.softmax(a, -1).nan_to_num(0.0)
            out[rows, heads] = torch.einsum("cgn,nd->cgd", w, vd)
            # scores: D / 16 + 16 additions of |q k| at 2^-23 each, seen twice (weight and sum), with the
            # scales' and the exponential's roundings of the score itself
            mag = (torch.einsum("cgd,nd->cgn", qd.abs(), kd.abs()) * abs(scale)).masked_fill(~seen[:, None], 0)
            e = 2 * ((D / 16 + 24) * 2.0 ** -23 * mag.amax(-1) + 2.0 ** -20)
            rel = (2.0 ** -11 + e + n * 2.0 ** -24)[..., None]
            small = n * 2.0 ** -25 * vd.abs().max()  # weights below fp16's normal numbers
            tol[rows, heads] = rel * torch.einsum("cgn,nd->cgd", w, vd.abs()) + small * 2.0 ** -0
    return out, tol


def run_attention(kv, qlen, H, G, D, page, dtype=BF16, window=0, seed=0, fused=False, qstd=2.0, scale=None, edit=None,
                  max_q=None, batch_pad=0):
    need = [-(-max(n, 0) // page) for n in kv]
    pool = sum(need) + 3
    cache = new_cache(pool, H, page, D, seed=seed, fused=fused)
    table = page_table(need, pool, seed=seed)
    g = gen(seed + 1)
    T = sum(qlen)
    wide = randn(T, (G + 1) * H * D, g=g, std=qstd).to(dtype)
    q = wide[:, :G * H * D].view(T, G * H, D)
    # what no key lies on may hold anything
    used = torch.zeros(pool, dtype=torch.bool)
    used[table[table >= 0].long()] = True
    cache.k_scale[~used.to(DEV)] = float("nan")
    cache.v_scale[~used.to(DEV)] = float("nan")
    if edit is not None:
        edit(cache, table, q)
    cu = None if qlen == [1] * len(kv) else torch.tensor(np.cumsum([0] + qlen), dtype=torch.int32, device=DEV)
    lens = torch.tensor(kv, dtype=torch.int32, device=DEV)
    sc = D ** -0.5 if scale is None else scale
    out = torch.full(q.shape, float("nan"), dtype=dtype, device=DEV)
    got = cache.attention(q, table.to(DEV), lens, cu_q=cu, max_q=max_q or max(qlen + [1]), scale=sc, window=window, out=out)
    assert got is out
    again = cache.attention(q.contiguous(), table.to(DEV), lens, cu_q=cu, max_q=max_q or max(qlen + [1]), scale=sc,
                            window=window)
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))
    ref, tol = attention_reference(q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, kv, qlen, window, sc)
    close(got, ref, tol + ref.abs() * U[dtype] + TINY[dtype])
    return got


@pytest.mark.parametrize("H, G", [(1, 1), (2, 3), (8, 4), (1, 8), (2, 9), (4, 16), (1, 40), (1, 128)])
@pytest.mark.parametrize("D, page", [(64, 16), (64, 128), (128, 32), (128, 64)])
def test_attention_single_tokens(H, G, D, page):
    kv = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 1023, 2000]
    run_attention(kv, [1] * len(kv), H, G, D, page, seed=H * G + D)


@pytest.mark.parametrize("kv, qlen", [
    ([7], [7]), ([1, 40, 90], [1, 2, 3]), ([300, 0, 64, 1000, 5], [4, 2, 0, 8, 9]), ([513], [130]), ([200, 777], [200, 65]),
    ([1500, 33], [300, 33]), ([600], [600])])
@pytest.mark.parametrize("G, D, dtype", [(1, 64, FP16), (4, 128, BF16), (5, 128, FP16), (8, 64, BF16)])
def test_attention_several_tokens(kv, qlen, G, D, dtype):
    run_attention(kv, qlen, 2, G, D, 32, dtype=dtype, seed=len(kv) + G)


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("qlen", [[1] * 6, [3, 1, 5, 40, 2, 1], [150, 64, 70, 16, 300, 1]])
def test_attention_window(window, qlen):
    run_attention([400, 16, 90, 1000, 333, 2], qlen, 2, 4, 128, 16, window=window, seed=window % 97)


@pytest.mark.parametrize("G, D", [(4, 128), (6, 64)])
@pytest.mark.parametrize("B", [9, 15, 30, 70, 160])
def test_attention_any_number_of_short_sequences(B, G, D):
    """Units from a few, which several CTAs share, to more than run at once; and one context far longer than the table's others."""
    kv = [(37 * i) % 301 for i in range(B)]
    run_attention(kv, [1] * B, 8, G, D, 16, seed=B)
    qlen = [min(n, 1 + i % 3) for i, n in enumerate(kv)]
    run_attention(kv, qlen, 4, G, D, 32, seed=B + 1, dtype=FP16)
    run_attention([7001] + kv[1:], [1] * B, 2, G, D, 64, seed=B + 2)


def test_attention_window_at_the_end_of_long_contexts():
    run_attention([20000, 9000, 33], [1, 1, 1], 2, 4, 128, 64, window=500, seed=51)
    run_attention([20000, 9000, 33], [3, 5, 2], 2, 4, 128, 64, window=700, seed=52)
    run_attention([30000], [1], 1, 8, 64, 16, window=6130, seed=53)
    run_attention([12000] * 30, [1] * 30, 8, 2, 128, 128, window=900, seed=54)


@pytest.mark.parametrize("fused", [False, True])
def test_attention_long_and_uneven(fused):
    """Many CTAs share a unit, beside units of a few keys; strided caches."""
    run_attention([30000, 1, 50, 17001, 0, 130], [1] * 6, 2, 8, 128, 64, seed=3, fused=fused)
    run_attention([20000], [1], 1, 1, 64, 16, seed=4, fused=fused)
    run_attention([9000, 8], [20, 3], 1, 6, 128, 128, seed=5, fused=fused)


def test_attention_large_scores_scales_and_zero_scale():
    def spread(cache, table, q):  # page scales over many powers of two, some zero; one row one-hot
        g = gen(9)
        cache.v_scale *= torch.exp2(torch.randint(-20, 6, cache.v_scale.shape, device=DEV, generator=g).float())
        cache.v_scale[::5] = 0
        cache.k_scale *= torch.exp2(torch.randint(-6, 3, cache.k_scale.shape, device=DEV, generator=g).float())
        q[0] *= 8
    run_attention([700, 64, 1500], [1, 1, 1], 2, 8, 128, 16, seed=12, edit=spread)
    run_attention([700, 64, 1500], [90, 3, 200], 2, 4, 128, 16, seed=13, edit=spread)
    run_attention([300, 40], [1, 1], 2, 2, 64, 32, seed=14, scale=0.0)
    run_attention([300, 40], [1, 1], 2, 2, 64, 32, seed=15, scale=-0.3)

    def zero(cache, table, q):
        q.zero_()
    run_attention([300, 40], [1, 1], 2, 2, 64, 32, seed=16, edit=zero)


@pytest.mark.parametrize("qlen", [[1, 1, 1], [40, 3, 100]])
def test_attention_skips_pages_that_do_not_exist(qlen):
    def holes(cache, table, q):
        table[0, 1] = -1
        table[1, :] = 10 ** 6  # nothing left to see
        table[2, 3] = cache.k.shape[0]
    got = run_attention([100, 50, 200], qlen, 2, 4, 128, 32, seed=21, edit=holes)
    assert (got[qlen[0]:qlen[0] + qlen[1]] == 0).all()


@pytest.mark.parametrize("qlen", [[1, 1, 1], [70, 20, 90]])
def test_attention_keeps_nan_to_its_sequence_and_head(qlen):
    kv, H, G = [200, 100, 150], 2, 4
    base = run_attention(kv, qlen, H, G, 128, 16, seed=31)
    need = [-(-n // 16) for n in kv]
    cache, table = new_cache(sum(need) + 3, H, 16, 128, seed=31), page_table(need, sum(need) + 3, seed=31)
    wide = randn(sum(qlen), (G + 1) * H * 128, g=gen(32), std=2.0).to(BF16)
    q = wide[:, :G * H * 128].view(-1, G * H, 128)
    cache.v_scale[table[1, 2], 1] = float("nan")
    cu = None if qlen == [1] * 3 else torch.tensor(np.cumsum([0] + qlen), dtype=torch.int32, device=DEV)
    got = cache.attention(q, table.to(DEV), torch.tensor(kv, dtype=torch.int32, device=DEV), cu_q=cu, max_q=max(qlen))
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    hit[qlen[0]:qlen[0] + qlen[1], G:] = True
    assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], base[~hit])


@pytest.mark.parametrize("what, value", [("v_scale", math.nan), ("v_scale", math.inf), ("v_scale", -math.inf),
                                         ("k_scale", math.nan), ("k_scale", math.inf)])
@pytest.mark.parametrize("kv, qlen, G, page, bad, window", [
    (52, 8, 1, 16, 3, 0), (52, 8, 2, 16, 3, 0), (68, 8, 1, 16, 3, 3), (68, 8, 2, 16, 3, 3), (100, 100, 2, 16, 3, 20),
    (700, 300, 2, 32, 15, 0), (700, 300, 2, 32, 15, 100), (300, 200, 4, 128, 1, 0), (40, 40, 5, 16, 0, 7)])
def test_attention_keeps_a_scale_that_is_not_finite_to_the_tokens_that_see_it(kv, qlen, G, page, bad, window, what, value):
    H, D, need = 2, 128, -(-kv // page)
    cache, table = new_cache(need + 1, H, page, D, seed=kv), page_table([need], need + 1, seed=kv)
    q = randn(qlen, G * H, D, g=gen(kv), std=2.0).to(BF16)
    ref, tol = attention_reference(q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, [kv], [qlen], window, D ** -0.5)
    getattr(cache, what)[table[0, bad], 1] = value
    cu = torch.tensor([0, qlen], dtype=torch.int32, device=DEV)
    got = cache.attention(q, table.to(DEV), torch.tensor([kv], dtype=torch.int32, device=DEV), cu_q=cu, max_q=qlen,
                          window=window)
    p = torch.arange(kv - qlen, kv, device=DEV)
    sees = (p >= bad * page) & ((p - (window or kv + 1)) < (bad + 1) * page - 1)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    hit[sees, G:] = True
    assert hit.any()
    close(got[~hit], ref[~hit], (tol + ref.abs() * U[BF16] + TINY[BF16])[~hit])
    if what == "v_scale" or math.isnan(value):  # (an infinite scale of K makes a score of minus infinity a weight of 0)
        assert not torch.isfinite(got[hit]).any()


def test_attention_lengths_beyond_the_table_and_tokens_beyond_max_q():
    cache, table = new_cache(4, 1, 16, 64, seed=41), torch.tensor([[2, 0]], dtype=torch.int32, device=DEV)
    q = randn(1, 2, 64, g=gen(42)).to(BF16)
    a = cache.attention(q, table, torch.tensor([32], dtype=torch.int32, device=DEV))
    b = cache.attention(q, table, torch.tensor([1 << 30], dtype=torch.int32, device=DEV))
    c = cache.attention(q, table, torch.tensor([-5], dtype=torch.int32, device=DEV))
    assert torch.equal(a, b) and (c == 0).all()
    empty = cache.attention(q[:0], table[:0], torch.zeros(0, dtype=torch.int32, device=DEV))
    assert empty.shape == (0, 2, 64)


def test_attention_offsets_past_32_bits():
    """Pages whose byte offsets pass 2^32: the last ones of a pool of 4.3 GB each for K and V."""
    H, page, D = 8, 128, 128
    pool = (1 << 32) // (H * page * D) + 40
    k, v = (torch.empty(pool, H, page, D, dtype=torch.int8, device=DEV) for _ in "kv")
    sc = torch.full((pool, H), 0.02, device=DEV)
    cache = m.KvCache(k, v, sc, sc.clone())
    g = gen(51)
    n = 1000
    table = torch.arange(pool - 1, pool - 9, -1, dtype=torch.int32)[None]
    kn, vn = randn(n, H, D, g=g).to(BF16), randn(n, H, D, g=g).to(BF16)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    cache.append(kn, vn, table.to(DEV), torch.zeros(1, dtype=torch.int32, device=DEV), cu_tokens=cu)
    for c in (1, 64):
        q = randn(c, H * 2, D, g=g).to(BF16)
        got = cache.attention(q, table.to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV),
                              cu_q=None if c == 1 else torch.tensor([0, c], dtype=torch.int32, device=DEV), max_q=c)
        at = table[0].long().to(DEV)
        ref, tol = attention_reference(q, k[at], v[at], cache.k_scale[at], cache.v_scale[at],
                                       torch.arange(8, dtype=torch.int32)[None], [n], [c], 0, D ** -0.5)
        close(got, ref, tol + ref.abs() * U[BF16])
    assert float((k[at[0], 0, 0].float() * cache.k_scale[at[0], 0] - kn[0, 0].float()).abs().max()) < 0.05


def test_cache_refusals():
    cache = new_cache(4, 2, 16, 64)
    q = torch.zeros(2, 4, 64, dtype=BF16, device=DEV)
    table, lens = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    for bad in (lambda: cache.attention(q.float(), table, lens), lambda: cache.attention(q, table.long(), lens),
                lambda: cache.attention(q, table, lens.long())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: cache.attention(q[:, :3], table, lens), lambda: cache.attention(q[..., :32], table, lens),
                lambda: cache.attention(q[:1], table, lens), lambda: cache.attention(q, table, lens[:1]),
                lambda: cache.attention(q, table, lens, max_q=2), lambda: cache.attention(q, table[0], lens),
                lambda: cache.attention(q, table, lens, out=q[:1]), lambda: cache.append(q, q, table, lens),
                lambda: cache.append(q[:, :2], q, table, lens), lambda: cache.append(q[:1, :2], q[:1, :2], table, lens),
                lambda: m.KvCache(cache.k, cache.v[:2], cache.k_scale, cache.v_scale),
                lambda: m.KvCache(cache.k.transpose(2, 3), cache.v.transpose(2, 3), cache.k_scale, cache.v_scale),
                lambda: m.KvCache(cache.k, cache.v, cache.k_scale[:2], cache.v_scale)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(m.MoeError) as e:
        cache.attention(q, table, lens, workspace=cache.workspace()[:1024])
    assert e.value.code == m.MOE_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(m.MoeError):
        cache.attention(q, table, lens, window=-1)


# ------------------------------------------------------------ streams and graphs
def test_other_streams_and_graphs_give_the_same():
    g = gen(61)
    H, G, D, page, B, h = 2, 4, 64, 16, 3, 512
    x, w = randn(B, h, g=g).to(BF16), torch.ones(h, dtype=BF16, device=DEV)
    code, wq, ws, _, _, _ = w4_case(1, (G + 2) * H * D, h, 128, BF16, 62)
    table = page_table([2, 2, 2], 8).to(DEV)
    start = torch.tensor([0, 5, 20], dtype=torch.int32, device=DEV)

    def step(cache, **kw):
        q8, qs, _, _ = m.add_rmsnorm_quant(x, w, **kw)
        qkv = m.w4_linear(q8, wq, ws, x_scale=qs, **kw)
        hd = H * D
        cache.append(qkv[:, G * hd:(G + 1) * hd].view(B, H, D), qkv[:, (G + 1) * hd:].view(B, H, D), table, start, **kw)
        return cache.attention(qkv[:, :G * hd].view(B, G * H, D), table, start + 1, **kw)

    def fresh():
        c = new_cache(8, H, page, D, seed=63)
        return c

    want = step(fresh())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    cache = fresh()
    side.wait_stream(torch.cuda.current_stream())
    got = step(cache, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    cache = fresh()
    cache.workspace().fill_(0xFF)  # the workspace needs no initial content
    lens = start + 1
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache)
    side.synchronize()
    cache2 = fresh()
    cache2.workspace()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(cache2)
    for a, b in zip((cache2.k, cache2.v, cache2.k_scale, cache2.v_scale), (lambda c: (c.k, c.v, c.k_scale, c.v_scale))(fresh())):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    del lens
