"""Rows that are NaN, empty or far below: their weights are NaN, zero and zero in every column of a
tile, whichever unit takes the column's exponential."""
import math

import pytest

import prompt_helpers as P
from bit_kv_cache_17_b200 import kvq

pytestmark = pytest.mark.gpu


def weigh(c, q, lse, causal=False, **kw):
    m = c.attn_mass(0, [0], [q.shape[0]], q, lse, causal=causal, **kw)
    assert c.status() == 0
    return m


@pytest.mark.parametrize("type_,n,m,G", [("bf16", 200, 128, 1), ("bf16", 130, 25, 5), ("q8_0", 130, 40, 3)])
def test_a_nan_row_shows_from_every_column(type_, n, m, G):
    """One NaN row (its lse, as a NaN query gives it) at each place of a tile in turn."""
    t = P.torch()
    k, v = P.kv(1, [n], 1)
    c = P.cache(type_, [n], 1, k, v)
    q = P.queries(1, m, G, t.bfloat16)
    _, lse = c.batch_attn(0, [0], [m], q, return_lse=True)
    want = weigh(c, q, lse)
    assert bool(t.isfinite(want).all())
    for i in range(m):
        for h in range(G):
            bad = lse.clone()
            bad[i, h] = math.nan
            assert bool(t.isnan(weigh(c, q, bad)).all()), (i, h)
    # and with the query itself NaN
    for i in range(m):
        x = q.clone()
        x[i, 0] = math.nan
        out, ls = c.batch_attn(0, [0], [m], x, return_lse=True)
        ok = t.ones(m, G, dtype=t.bool, device="cuda")
        ok[i, 0] = False
        assert bool(t.isnan(out[i, 0]).all()) and bool(t.isnan(ls[i, 0])) and bool(t.isfinite(out[ok]).all())
        assert bool(t.isnan(weigh(c, x, ls)).all()), i


@pytest.mark.parametrize("type_", ["bf16", "q8_0"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("low", [math.inf, 400.0])
def test_rows_that_weigh_nothing_add_exactly_zero(type_, causal, low):
    """lse = -inf (a row that saw nothing), and scores so far below their lse that fp32 holds no weight."""
    t = P.torch()
    n, m, G = 300, 300, 3
    k, v = P.kv(2, [n], 2)
    c = P.cache(type_, [n], 2, k, v)
    q = P.queries(2, m, 2 * G, t.bfloat16)
    lse = t.full((m, 2 * G), -math.inf if low == math.inf else low, device="cuda")
    assert bool((weigh(c, q, lse, causal) == 0).all())
    prev = t.rand(1, 2, n, device="cuda")
    assert t.equal(weigh(c, q, lse, causal, decay=1.0, mass_in=prev), prev)


def test_a_weight_past_the_range_is_infinite_in_every_column():
    """Rows whose lse does not belong to their scores, at each place of a tile in turn."""
    t = P.torch()
    k, v = P.kv(6, [130], 1)
    c = P.cache("bf16", [130], 1, k, v)
    q = P.queries(6, 25, 5, t.bfloat16)
    for low in (-200.0, -3e38):
        for i in range(25):
            lse = t.full((25, 5), -math.inf, device="cuda")
            lse[i, i % 5] = low
            assert bool((weigh(c, q, lse) == math.inf).all()), (low, i)


def test_tokens_a_row_does_not_see_get_exactly_zero():
    """Causal, one row with weight: the tokens behind it get nothing from it, and keep their order of index
    where an eviction has to choose among them."""
    t = P.torch()
    n = 300
    k, v = P.kv(3, [n], 1)
    c = P.cache("bf16", [n], 1, k, v)
    q = P.queries(3, n, 1, t.bfloat16)
    _, lse = c.batch_attn(0, [0], [n], q, causal=True, return_lse=True)
    for row in (0, 7, 64, 127, 128, 200):
        only = t.full_like(lse, -math.inf)
        only[row] = lse[row]
        w = weigh(c, q, only, True)[0, 0]
        assert bool((w[row + 1:] == 0).all()) and bool((w[: row + 1] > 0).all()), row
        dst = kvq.KVCache(n_kv_heads=1, max_ctx=n, type_k="bf16", type_v="bf16", tail=0)
        keep = min(row + 20, n)
        kept, _ = c.evict(dst, 0, 0, [0], [0], w.view(1, 1, n), keep)
        assert t.equal(kept[0, 0].long().cpu(), t.arange(keep)), row


def test_a_nan_row_does_not_reach_the_tokens_it_does_not_see():
    t = P.torch()
    n, G = 300, 2
    k, v = P.kv(4, [n], 1)
    c = P.cache("bf16", [n], 1, k, v)
    q = P.queries(4, n, G, t.bfloat16)
    _, lse = c.batch_attn(0, [0], [n], q, causal=True, return_lse=True)
    want = weigh(c, q, lse, True)
    for row in (0, 5, 63, 64, 100, 127, 128, 191, 250, 298):
        bad = lse.clone()
        bad[row, 1] = math.nan
        got = weigh(c, q, bad, True)
        assert bool(t.isnan(got[..., : row + 1]).all()), row
        assert t.equal(got[..., row + 1:], want[..., row + 1:]), row


@pytest.mark.parametrize("m,G", [(200, 1), (60, 5)])
def test_masked_values_add_nothing_however_large(m, G):
    """Values near the largest BF16 number in tokens that the first rows of a prompt do not see."""
    t = P.torch()
    n = m
    k, v = P.kv(5, [n], 1)
    far = m // 2
    v2 = v.clone()
    v[far:], v2[far:] = 3e38, 0.0
    q = P.queries(5, m, G, t.bfloat16)
    a, b = (P.cache("bf16", [n], 1, k, x).batch_attn(0, [0], [m], q, causal=True) for x in (v, v2))
    assert t.equal(a[:far], b[:far])


def test_keys_and_queries_up_to_the_f16_range_of_a_rebuilt_cache():
    """The last values that F16 holds, in a key and in a query of a quantized cache's 16-bit tail."""
    t = P.torch()
    n = 40
    k, v = P.kv(7, [n], 1)
    k[3, 0, 5] = 65280.0  # the largest BF16 number below 65520
    k[4, 0, 5] = -65280.0
    c = P.cache("q8_0", [n], 1, k, v, tail=64)
    q = P.queries(7, 4, 2, t.bfloat16)
    q[..., 5] = 0.0
    q[1, 1, 6] = 65280.0
    out, lse = c.batch_attn(0, [0], [4], q, return_lse=True, softmax_scale=1e-4)
    assert bool(t.isfinite(out).all()) and bool(t.isfinite(lse).all())
    ref = P.attention(q, *P.cached(c, 0, 0), False, 1e-4)
    P.check_attention(out, lse, ref, n, P.U16, True)
