"""The decoder-layer operators where their definitions are easily missed: query
tokens past what a call computes, page scales far apart or not finite, empty
tables, workspaces of the caller's own.  References and tolerances are those of
the operators' other tests unless a test derives its own."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_expert_ffn_dispatch_gb300 as m  # noqa: E402
from test_gpu_layer_ops import (BF16, DEV, FP16, TINY, U, attention_reference, close, gen, new_cache, page_table,  # noqa: E402
                                randn)

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
