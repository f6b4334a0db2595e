"""The decoder-layer operators where their definitions are easily missed: query
tokens past what a call computes, page scales far apart or not finite, empty
tables, workspaces of the caller's own.  References and tolerances are those of
the operators' other tests unless a test derives its own."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_expert_ffn_dispatch_gb300 as m  # noqa: E402
from test_gpu_layer_ops import (BF16, DEV, F32, FP16, TINY, U, attention_reference, check_w4, close, gen,  # noqa: E402
                                new_cache, page_table, randn, w4_case)

pytestmark = pytest.mark.gpu


def cum(v):
    return torch.tensor(np.cumsum([0] + list(v)), dtype=torch.int32, device=DEV)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------ query tokens past max_q or past the tensor
@pytest.mark.parametrize("window", [0, 5])
@pytest.mark.parametrize("kv, qlen, max_q, G", [
    ([10], [8], 4, 2), ([10, 300, 7], [8, 2, 7], 4, 2), ([40, 500, 3], [30, 3, 9], 5, 3), ([70, 2000], [70, 1], 1, 4),
    ([400, 900, 20], [300, 64, 20], 100, 4), ([1300], [700], 130, 2), ([5, 40], [20, 11], 6, 4)])
def test_attention_leaves_tokens_past_max_q_and_keeps_the_others_where_they_stand(kv, qlen, max_q, G, window):
    """The first max_q query tokens of a longer sequence stand where they would with all of them."""
    H, D, page = 2, 128, 16
    need = [-(-n // page) for n in kv]
    cache, table = new_cache(sum(need) + 1, H, page, D, seed=kv[0]), page_table(need, sum(need) + 1, seed=kv[0])
    q = randn(sum(qlen), G * H, D, g=gen(kv[0]), std=2.0).to(BF16)
    out = torch.full(q.shape, 7.0, dtype=BF16, device=DEV)
    cache.attention(q, table.to(DEV), i32(kv), cu_q=cum(qlen), max_q=max_q, window=window, out=out)
    ref, tol = attention_reference(q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, kv, qlen, window, D ** -0.5)
    done = torch.cat([torch.arange(n, device=DEV) < max_q for n in qlen])
    close(out[done], ref[done], (tol + ref.abs() * U[BF16] + TINY[BF16])[done])
    assert not done.all() and (out[~done] == 7).all()


@pytest.mark.parametrize("tokens", [3, 90])
def test_attention_of_the_leading_query_tokens_of_a_call(tokens):
    """cu_q goes past the rows of q: those that are there stay where they stand."""
    H, G, D, page, kv, qlen = 2, 4, 64, 32, 200, 150
    cache, table = new_cache(8, H, page, D, seed=5), page_table([7], 8, seed=5)
    q = randn(qlen, G * H, D, g=gen(6), std=2.0).to(FP16)
    ref, tol = attention_reference(q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, [kv], [qlen], 0, D ** -0.5)
    got = cache.attention(q[:tokens], table.to(DEV), i32([kv]), cu_q=i32([0, qlen]), max_q=qlen)
    close(got, ref[:tokens], (tol + ref.abs() * U[FP16] + TINY[FP16])[:tokens])


def test_attention_wants_max_q_with_cu_q():
    cache, table = new_cache(4, 1, 16, 64), i32([[0, 1]])
    q = torch.zeros(3, 2, 64, dtype=BF16, device=DEV)
    with pytest.raises(ValueError):
        cache.attention(q, table, i32([20]), cu_q=i32([0, 3]))
    cache.attention(q, table, i32([20]), cu_q=i32([0, 3]), max_q=3)
    cache.attention(q[:1], table, i32([20]))
    cache.attention(q[:1], table, i32([20]), max_q=1)


# ------------------------------------------------------------ prompt chunks: one piece that scales the output twice
@pytest.mark.parametrize("odd", [0.0, -0.02, 1e-9, -1e-30])
@pytest.mark.parametrize("D, page", [(128, 16), (64, 16), (128, 32)])
def test_attention_chunk_where_scale_and_row_reference_grow_in_one_piece(D, page, odd):
    """In pieces past the first: a page whose scale of V is many times those before it, beside one with an odd
    scale, and keys that score far above all earlier ones.  All rows see them."""
    H, G, kv, qlen = 2, 4, 1100, 70
    need = -(-kv // page)
    cache, table = new_cache(need + 1, H, page, D, seed=71), page_table([need], need + 1, seed=71)
    for at, v_times, k_times in ((256, 20, 1), (512, 300, 6), (768, 3000, 12)):
        p = table[0, at // page:at // page + 4].long().to(DEV)
        cache.v_scale[p[0]] *= v_times
        cache.v_scale[p[1]] = odd
        cache.k_scale[p[2:]] *= k_times
    q = randn(qlen, G * H, D, g=gen(72), std=2.0).to(BF16)
    got = cache.attention(q, table.to(DEV), i32([kv]), cu_q=i32([0, qlen]), max_q=qlen)
    ref, tol = attention_reference(q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, [kv], [qlen], 0, D ** -0.5)
    close(got, ref, tol + ref.abs() * U[BF16] + TINY[BF16])


# ------------------------------------------------------------ what is not finite
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("kv, qlen, G, page, bad, window", [
    (52, 1, 4, 16, 2, 0), (52, 1, 16, 16, 2, 0), (3000, 1, 4, 64, 5, 0), (52, 8, 2, 16, 3, 0), (68, 8, 2, 16, 3, 3),
    (100, 100, 2, 16, 3, 20), (700, 300, 2, 32, 15, 0), (700, 300, 2, 32, 15, 100), (300, 200, 4, 128, 1, 0)])
def test_attention_is_not_finite_where_a_scale_of_k_is_not(kv, qlen, G, page, bad, window, value):
    """Also where it would make scores of minus infinity; the tokens and heads that do not see the page stay."""
    H, D, need = 2, 128, -(-kv // page)
    cache, table = new_cache(need + 1, H, page, D, seed=kv), page_table([need], need + 1, seed=kv)
    q = randn(qlen, G * H, D, g=gen(kv), std=2.0).to(BF16)
    ref, tol = attention_reference(q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, [kv], [qlen], window, D ** -0.5)
    cache.k_scale[table[0, bad], 1] = value
    got = cache.attention(q, table.to(DEV), i32([kv]), cu_q=None if qlen == 1 else i32([0, qlen]), max_q=qlen, window=window)
    p = torch.arange(kv - qlen, kv, device=DEV)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    hit[(p >= bad * page) & ((p - (window or kv + 1)) < (bad + 1) * page - 1), G:] = True
    assert hit.any() and not torch.isfinite(got[hit]).any()
    close(got[~hit], ref[~hit], (tol + ref.abs() * U[BF16] + TINY[BF16])[~hit])


@pytest.mark.parametrize("kv, qlen, G, page", [(1, 1, 4, 16), (40, 1, 4, 16), (3000, 1, 12, 64), (50, 9, 4, 32), (300, 100, 4, 32),
                                               (20, 40, 4, 16)])
@pytest.mark.parametrize("value", [-math.inf, math.inf, math.nan])
def test_attention_is_not_finite_where_a_query_is_not(kv, qlen, G, page, value):
    """Also where all scores of the row are minus infinity; a row that sees no key stays 0."""
    H, D, need = 2, 128, -(-kv // page)
    cache, table = new_cache(need + 1, H, page, D, seed=kv), page_table([need], need + 1, seed=kv)
    cache.k[..., 3] = 5
    q = randn(qlen, G * H, D, g=gen(kv), std=2.0).to(BF16)
    ref, tol = attention_reference(q, cache.k, cache.v, cache.k_scale, cache.v_scale, table, [kv], [qlen], 0, D ** -0.5)
    q[::3, 1, 3] = value
    got = cache.attention(q, table.to(DEV), i32([kv]), cu_q=None if qlen == 1 else i32([0, qlen]), max_q=qlen)
    hit = torch.zeros(q.shape[:2], dtype=torch.bool, device=DEV)
    hit[::3, 1] = True
    hit &= (torch.arange(kv - qlen, kv, device=DEV) >= 0)[:, None]
    assert hit.any() and not torch.isfinite(got[hit]).any()
    close(got[~hit], ref[~hit], (tol + ref.abs() * U[BF16] + TINY[BF16])[~hit])


# ------------------------------------------------------------ weights and page scales far apart
def far_reference(q, cache, table, kv, qlen, window, scale):
    """(out, tolerance) in 64 bits.  Beside the terms of attention_reference a weight times its page's scale of V
    may be off by half a step of 2^-31 of the row's largest such product.  The codes that these errors meet are
    independent and of either sign (and at most 127), so their sum stays within 8 sqrt(keys) of one."""
    P, H, D = cache.k.shape[2], cache.k.shape[1], cache.k.shape[3]
    G = q.shape[1] // H
    out, tol = torch.zeros(q.shape, dtype=torch.float64, device=DEV), torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    pages = table[0, :-(-kv // P)].long().to(DEV)
    i, p = torch.arange(kv, device=DEV), torch.arange(kv - qlen, kv, device=DEV)[:, None]
    seen = (i <= p) & (i > p - (window or kv + qlen + 1))
    for h in range(H):
        vs = cache.v_scale[pages, h].double().repeat_interleave(P)[:kv]
        kd = (cache.k[pages, h].double() * cache.k_scale[pages, h].double()[:, None, None]).reshape(-1, D)[:kv]
        vd = cache.v[pages, h].double().reshape(-1, D)[:kv] * vs[:, None]
        heads = slice(h * G, (h + 1) * G)
        qd = q[:, heads].double()
        w = torch.softmax((torch.einsum("cgd,nd->cgn", qd, kd) * scale).masked_fill(~seen[:, None], -math.inf), -1).nan_to_num(0.0)
        out[:, heads] = torch.einsum("cgn,nd->cgd", w, vd)
        mag = (torch.einsum("cgd,nd->cgn", qd.abs(), kd.abs()) * abs(scale)).masked_fill(~seen[:, None], 0)
        # rounding of the score, of the exponential and the logarithm (2^-21 together), and of what is added to it
        rel = 2.0 ** -11 + 2 * ((D / 16 + 24) * 2.0 ** -23 * mag.amax(-1) + 2.0 ** -20) + kv * 2.0 ** -24 + 2.0 ** -16
        step = 8 * kv ** 0.5 * 127 * 2.0 ** -32 * (w * vs.abs()).amax(-1)
        tol[:, heads] = rel[..., None] * torch.einsum("cgn,nd->cgd", w, vd.abs()) + step[..., None]
    return out, tol


def check_far(kv, qlen, G, D, page, edit, window=0, dtype=FP16):
    H, need = 2, -(-kv // page)
    cache, table = new_cache(need + 1, H, page, D, seed=kv + G), page_table([need], need + 1, seed=kv + G)
    q = randn(qlen, G * H, D, g=gen(kv + G), std=1.0).to(dtype)
    edit(cache, table[0].long().to(DEV), q)
    got = cache.attention(q, table.to(DEV), i32([kv]), cu_q=None if qlen == 1 else i32([0, qlen]), max_q=qlen, window=window)
    ref, tol = far_reference(q, cache, table, kv, qlen, window, D ** -0.5)
    close(got, ref, tol + ref.abs() * U[dtype] + TINY[dtype])


FAR_SHAPES = [(8192, 1, 4, 128, 64, 0), (500, 1, 8, 64, 16, 0), (8192, 1, 16, 128, 64, 0), (3000, 4, 4, 128, 16, 0),
              (3000, 40, 4, 128, 64, 0), (8192, 100, 4, 128, 64, 0), (900, 300, 2, 64, 128, 0), (2000, 8, 2, 128, 16, 300),
              (2000, 200, 4, 128, 16, 300), (4000, 30, 8, 64, 32, 700)]


@pytest.mark.parametrize("log2", [16, 20, 24, 45, 70])
@pytest.mark.parametrize("kv, qlen, G, D, page, window", FAR_SHAPES)
def test_attention_keeps_its_precision_beside_a_page_with_a_large_scale(kv, qlen, G, D, page, window, log2):
    """One page has a scale of V 2^log2 times the others' and weights that leave it next to no share in any row."""
    def edit(cache, pages, q):
        q[..., 0] = 12.0 * 2.0 ** 6
        cache.k[..., 0] = 0
        at = pages[min(len(pages) - 1, (kv - qlen) // page - 1)]  # before the last query tokens; the window leaves it to some
        cache.k[at, :, :, 0] = -100  # scores about 100 octaves below the others'
        cache.k_scale[at] = 0.02
        cache.v_scale[at] *= 2.0 ** log2
        cache.v_scale /= 64
    check_far(kv, qlen, G, D, page, edit, window=window)


@pytest.mark.parametrize("scale", [0.0, -0.01, 1e-8])
@pytest.mark.parametrize("log2", [16, 24, 70])
@pytest.mark.parametrize("kv, qlen, G, D, page, window", FAR_SHAPES)
def test_attention_keeps_its_precision_beside_large_zero_and_negative_scales(kv, qlen, G, D, page, window, log2, scale):
    def edit(cache, pages, q):
        q[..., 0] = 12.0 * 2.0 ** 6
        cache.k[..., 0] = 0
        cache.k[pages[1], :, :, 0] = -100
        cache.k_scale[pages[1]] = 0.02
        cache.v_scale[pages[1]] *= 2.0 ** log2
        cache.v_scale[pages[2::5]] = scale
        cache.v_scale /= 64
    check_far(kv, qlen, G, D, page, edit, window=window)


@pytest.mark.parametrize("nats", [16, 18, 22])
@pytest.mark.parametrize("kv, qlen, G, D, page, window", FAR_SHAPES)
def test_attention_keeps_its_precision_beside_a_dominant_key_of_zero_value(kv, qlen, G, D, page, window, nats):
    """What remains of such a row comes from weights of 2^-23 to 2^-32 of the largest, where fp16 still has steps."""
    def edit(cache, pages, q):
        q[:] = q / 4
        q[..., 0] = 2.0
        cache.k[..., 0] = 0
        cache.k_scale.fill_(0.01)
        cache.k_scale[pages[0]] = nats * D ** 0.5 / 2.0 / 100
        cache.k[pages[0], :, 3:] = 0
        cache.k[pages[0], :, 3] = 0
        cache.k[pages[0], :, 3, 0] = 100
        cache.v[pages[0], :, 3] = 0
    check_far(kv, qlen, G, D, page, edit, window=window)


def test_attention_of_scales_at_the_ends_of_fp32():
    """Large scales in some pages, small ones in others, for both kernels: outputs as in fp32."""
    for kv, qlen, G in ((700, 1, 4), (700, 90, 4), (40000, 1, 4), (9000, 100, 2)):
        for lo, hi in ((-70, 60), (-20, 100), (-100, -80)):
            def edit(cache, pages, q):
                r = torch.randint(lo, hi, cache.v_scale.shape, device=DEV, generator=gen(kv + hi)).float()
                cache.v_scale *= torch.exp2(r)
            check_far(kv, qlen, G, 128, 64, edit, dtype=BF16)


# ------------------------------------------------------------ workspaces
def small_attention(cache, **kw):
    return cache.attention(torch.ones(1, 2, 64, dtype=BF16, device=DEV), i32([[0, 1]]), i32([20]), **kw)


def test_status_of_a_handle_that_has_run_nothing():
    full = torch.full((1 << 26,), 0xFF, dtype=torch.uint8, device=DEV)  # what the handle's memory held before
    del full
    cache = new_cache(4, 1, 16, 64)
    assert cache.status() == m.MOE_OK
    cache = new_cache(4, 1, 16, 64)
    cache.attention(torch.ones(0, 2, 64, dtype=BF16, device=DEV), i32([[0, 1]])[:0], i32([]))
    assert cache.status() == m.MOE_OK


def test_status_says_that_a_wait_gave_up_until_the_next_attention():
    """The words that a kernel leaves when a wait runs out, written by the host."""
    for qlen, kw in ((1, {}), (40, {"cu_q": i32([0, 40]), "max_q": 40})):
        cache = new_cache(4, 1, 16, 64)
        ws = cache.workspace()
        ws[:16].view(torch.int32)[1:3] = i32([1, 256])
        assert cache.status() == m.MOE_ERR_DEVICE_TIMEOUT and cache.status(ws) == m.MOE_ERR_DEVICE_TIMEOUT
        cache.attention(torch.ones(qlen, 2, 64, dtype=BF16, device=DEV), i32([[0, 1, 2]]), i32([45]), **kw)
        assert cache.status() == m.MOE_OK


def test_a_workspace_of_the_callers_own():
    cache = new_cache(4, 1, 16, 64)
    want, ws = small_attention(cache), torch.empty_like(cache.workspace())
    assert torch.equal(small_attention(cache, workspace=ws), want) and cache.status(ws) == m.MOE_OK
    assert torch.equal(small_attention(cache, workspace=ws[:ws.numel() // 4 * 4].view(torch.float32)), want)
    for bad in (torch.empty(ws.numel(), dtype=torch.uint8), torch.empty(ws.numel(), 2, dtype=torch.uint8, device=DEV)[:, 0]):
        with pytest.raises(ValueError):
            small_attention(cache, workspace=bad)
        with pytest.raises(ValueError):
            cache.status(bad)


def test_the_handles_workspace_outlives_it_on_a_stream_that_still_uses_it():
    cache = new_cache(4, 1, 16, 64)
    torch.cuda.empty_cache()  # nothing else of its size is free
    args = torch.ones(1, 2, 64, dtype=BF16, device=DEV), i32([[0, 1]]), i32([20])
    cache.attention(*args)  # allocates the workspace for the current stream
    at, size, side = cache.workspace().data_ptr(), cache.workspace().numel(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # a few tenths of a second
        out = cache.attention(*args)
    assert not side.query()
    del cache
    taken = torch.empty(size, dtype=torch.uint8, device=DEV)
    assert taken.data_ptr() + size <= at or taken.data_ptr() >= at + size
    side.synchronize()
    assert torch.isfinite(out).all()


# ------------------------------------------------------------ numbers that do not fit the C structures
def test_numbers_past_32_bits_are_not_cut():
    cache, table = new_cache(8, 1, 16, 64, seed=3), i32([[0, 1, 2, 3, 4, 5, 6]])
    q = randn(30, 2, 64, g=gen(4)).to(BF16)
    want = cache.attention(q, table, i32([100]), cu_q=i32([0, 30]), max_q=30)
    for window in (2 ** 31, 2 ** 32 + 5, 2 ** 40):
        assert torch.equal(cache.attention(q, table, i32([100]), cu_q=i32([0, 30]), max_q=30, window=window), want)
    for window in (-1, -2 ** 32, -2 ** 32 + 5):
        with pytest.raises(m.MoeError):
            cache.attention(q, table, i32([100]), cu_q=i32([0, 30]), max_q=30, window=window)
    with pytest.raises(ValueError):
        cache.attention(q, table, i32([100]), cu_q=i32([0, 30]), max_q=2 ** 32 + 1)
    with pytest.raises(m.MoeError):
        cache.attention(q, table, i32([100]), cu_q=i32([0, 30]), max_q=-2 ** 32 + 1)
    one = torch.ones(1, 1, dtype=BF16, device=DEV)
    with pytest.raises(ValueError):
        m.add_rmsnorm_quant(one.expand(2 ** 32 + 5, 1), one[0])
    with pytest.raises(ValueError):
        m.w4_linear(one.expand(2 ** 32 + 5, 64), torch.zeros(16, 32, dtype=torch.uint8, device=DEV), one.expand(16, 1).contiguous())
    with pytest.raises(ValueError):
        cache.attention(q[:1], table[:, :1].expand(1, 2 ** 32 + 5), i32([16]))


@pytest.mark.parametrize("qlen, G", [([1, 1, 1], 4), ([1, 1, 1], 16), ([3, 0, 40], 4), ([2, 1, 5], 1)])
def test_a_page_table_without_pages(qlen, G):
    """No sequence of the batch has a key yet: nothing is written, and attention gives zeros."""
    cache, table = new_cache(4, 2, 16, 64, seed=8), torch.empty(3, 0, dtype=torch.int32, device=DEV)
    before = [t.clone() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    q = randn(sum(qlen), 2 * G, 64, g=gen(9)).to(BF16)
    cu = None if qlen == [1, 1, 1] else cum(qlen)
    out = cache.attention(q, table, i32([0, 0, 7]), cu_q=cu, max_q=max(qlen), out=torch.full(q.shape, 7.0, dtype=BF16, device=DEV))
    assert (out == 0).all()
    cache.append(q[:, :2], q[:, :2], table, i32([0, 0, 0]), cu_tokens=cu)
    for a, b in zip(before, (cache.k, cache.v, cache.k_scale, cache.v_scale)):
        assert torch.equal(a, b)


# ------------------------------------------------------------ codes
@pytest.mark.parametrize("size", [1e-36, 3e-37, 1e-38, 2e-40])
def test_append_of_the_smallest_numbers_to_a_held_page_gives_codes_of_127_at_most(size):
    """A page that holds tokens of zeros only has a scale of 0, and takes the new tokens' scale without a floor."""
    cache = m.KvCache.empty(2, 1, 16, 64)
    g = gen(10)
    k, v = ((torch.rand(5, 1, 64, device=DEV, generator=g) - 0.5).sign() * size for _ in "kv")
    k, v = k.to(BF16), v.to(BF16)
    cache.append(k, v, i32([[1]]), i32([4]), cu_tokens=i32([0, 5]))
    for code, x in ((cache.k, k), (cache.v, v)):
        new = code[1, 0, 4:9].int()
        assert int(code.min()) >= -127 and (new.sign() == x[:, 0].sign()).all() and (code[1, 0, :4] == 0).all()


# ------------------------------------------------------------ 4-bit products of large and small rows
@pytest.mark.parametrize("size", [1e30, 1e36, 3e37, 1e-25])
@pytest.mark.parametrize("M, N, K, group, zero", [(1, 40, 128, 32, True), (8, 200, 1024, 64, False), (16, 64, 4096, 128, True),
                                                  (20, 33, 16384, 128, False)])
def test_w4_rows_of_any_size_that_fp32_holds(M, N, K, group, zero, size):
    """Sums of x times scale that fp32 holds are found, though x alone, or x times its power of two, passes it."""
    code, w, ws, z, x, _ = w4_case(M, N, K, group, BF16, M + K, zero=zero)
    x = (x.float() * size).to(BF16)
    x[0, ::7] *= 2.0 ** -6
    ws = (ws.float() * 2.0 ** -14).to(BF16)
    check_w4(code, ws, z, x, None, m.w4_linear(x, w, ws, zero=z, out_dtype=F32))
    check_w4(code, ws, z, x, None, m.w4_linear(x, w, ws, zero=z))


@pytest.mark.parametrize("sdtype", [BF16, FP16, F32])
@pytest.mark.parametrize("M, N, K, group", [(1, 40, 64, 32), (8, 200, 4096, 64), (13, 77, 1024, 128), (40, 30, 8320, 64)])
def test_w4_int8_rows_in_every_output_type(M, N, K, group, sdtype):
    code, w, ws, z, x, xs = w4_case(M, N, K, group, BF16, 7 * M + N, x8=True, zero=True, sdtype=sdtype)
    xs = xs * 2.0 ** -10  # outputs of a few hundred, which fp16 holds
    for out in (BF16, FP16, F32):
        got = m.w4_linear(x, w, ws, zero=z, x_scale=xs, out_dtype=out)
        assert got.dtype == out
        check_w4(code, ws, z, x, xs, got)


@pytest.mark.parametrize("nats", [10, 17, 18, 20])
@pytest.mark.parametrize("kv, qlen, G, D, page, window", FAR_SHAPES)
def test_attention_keeps_the_weights_of_keys_before_a_dominant_one(kv, qlen, G, D, page, window, nats):
    """The dominant key, of no value, comes late in its 128 keys: what lies before it moves with the reference."""
    def edit(cache, pages, q):
        at = (kv - qlen) // 128 * 128 - 28
        page_at, slot = pages[at // page], at % page
        q[:] = q / 4
        q[..., 0] = 2.0
        cache.k[..., 0] = 0
        cache.k_scale.fill_(0.01)
        cache.k_scale[page_at] = nats * D ** 0.5 / 2.0 / 100
        cache.k[page_at, :, :, 1:] = 0
        cache.k[page_at, :, slot, 0] = 100
        cache.v[page_at, :, slot] = 0
    check_far(kv, qlen, G, D, page, edit, window=window)
