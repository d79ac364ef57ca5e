"""Attention weights per cached token against sums of exp(x - lse) in 64 bits."""
import math

import pytest

import prompt_helpers as P
from bit_kv_cache_17_b200 import kvq

pytestmark = pytest.mark.gpu


def check(type_, lens, n_q, hkv, G, causal, tail=0, tail_f16=0, decay=0.7, seed=0, ids=None, inplace=False):
    t = P.torch()
    ids = list(range(len(lens))) if ids is None else ids
    k, v = P.kv(seed, lens, hkv)
    c = P.cache(type_, lens, hkv, k, v, tail, tail_f16)
    q = P.queries(seed, sum(n_q), hkv * G, t.float16 if tail_f16 else t.bfloat16)
    refs, lse, row = [], t.empty(sum(n_q), hkv * G, device="cuda"), 0
    for s, m in zip(ids, n_q):
        refs.append(P.attention(q[row:row + m], *P.cached(c, 0, s), causal))
        lse[row:row + m] = refs[-1][3]
        row += m
    ld = max(lens) + 3
    g = t.Generator().manual_seed(seed)
    prev = t.rand(len(ids), hkv, ld, generator=g).cuda()
    start = prev.clone()
    out = prev if inplace else t.full_like(prev, 5.0)
    c.attn_mass(0, ids, n_q, q, lse, causal=causal, decay=decay, mass_in=prev, mass_out=out)
    assert c.status() == 0
    row = 0
    for i, (s, m) in enumerate(zip(ids, n_q)):
        n = lens[s]
        x, _, _, want_lse, spread = refs[i]
        l32 = lse[row:row + m].double().T[..., None]
        p = t.where(l32 == -math.inf, 0.0, t.exp(x - l32)) if n else x
        add = p.view(hkv, G, m, n).sum((1, 2))
        # a weight is off by its score's error, the scaled lse's rounding and exp's own steps; the sum
        # by one step a term; then the decay's product and sum
        e = P.score_error(spread, P.U16 if type_ != "bf16" else 0.0).amax() if m and n else 0.0
        le = 4 * P.U32 * float(want_lse[want_lse > -math.inf].abs().amax()) if m and n else 0.0
        rel = e + le + 8 * P.U32 + m * G * P.U32
        want = decay * start[i, :, :n].double() + add
        err = (out[i, :, :n].double() - want).abs()
        tol = rel * add + 2 * P.U32 * want + 1e-30
        assert bool((err <= tol).all()), (i, float((err - tol).max()), float(err.max()))
        keep = start if inplace else t.full_like(start, 5.0)
        assert t.equal(out[i, :, n:], keep[i, :, n:])  # places behind the sequence stay
        row += m


@pytest.mark.parametrize("f16", [0, 1])
@pytest.mark.parametrize("G", [1, 3, 5, 8])
def test_lengths(G, f16):
    check("bf16", [1, 0, 127, 128, 129, 300, 513], [3, 5, 1, 0, 52, 26, 257], 2, G, False, tail_f16=f16, seed=G)
    check("bf16", [1, 130, 257, 400, 640, 127], [1, 130, 1, 37, 640, 126], 2, G, True, tail_f16=f16, seed=20 + G)


def test_long_context_and_in_place():
    check("bf16", [20011], [32], 2, 5, True, seed=2, inplace=True)
    check("bf16", [9000, 77, 4097], [1, 1, 3], 1, 8, False, seed=3, decay=1.0)


@pytest.mark.parametrize("type_", ["q4_0", "q4_1", "kvarn4", "q8_0"])
def test_quantized(type_):
    check(type_, [700, 0, 300], [9, 2, 70], 2, 5, False, tail=100, seed=4)
    check(type_, [300, 150], [4, 1, 7], 2, 4, True, ids=[1, 0, 1], seed=7)


def test_decay_zero_reads_nothing_and_default_output():
    t = P.torch()
    lens = [90, 40]
    k, v = P.kv(1, lens, 2)
    c = P.cache("bf16", lens, 2, k, v)
    q = P.queries(1, 12, 4, t.bfloat16)
    out, lse = c.batch_attn(0, [0, 1], [5, 7], q, return_lse=True)
    a = c.attn_mass(0, [0, 1], [5, 7], q, lse)
    assert a.shape == (2, 2, 90) and bool((a[1, :, 40:] == 0).all())
    junk = t.full_like(a, math.nan)
    b = c.attn_mass(0, [0, 1], [5, 7], q, lse, decay=0.0, mass_in=junk, mass_out=t.zeros_like(a))
    assert t.equal(a, b)
    # every row's weights sum to one, so a KV head gathers its query heads times rows
    total = a.double().sum(-1)
    want = t.tensor([[10.0, 10.0], [14.0, 14.0]], device="cuda", dtype=t.float64)
    assert bool(((total - want).abs() < 1e-4 * want).all())
    # a row that saw nothing weighs nothing
    lse2 = lse.clone()
    lse2[0] = -math.inf
    d = c.attn_mass(0, [0, 1], [5, 7], q, lse2)
    e = c.attn_mass(0, [0, 1], [4, 7], q[1:], lse[1:])
    assert bool(((d - e).abs() <= 1e-5 * (1 + e)).all()) and bool(t.isfinite(d).all())


@pytest.mark.parametrize("m", [1, 3, 26, 30])
def test_an_entry_does_not_see_the_queries_behind_its_own(m):
    """NaN queries of the next entry share a tile's copy with this entry's last ones."""
    t = P.torch()
    lens = [300, 300]
    k, v = P.kv(5, lens, 1)
    c = P.cache("bf16", lens, 1, k, v)
    q = P.queries(5, m + 40, 5, t.bfloat16)
    out, lse = c.batch_attn(0, [0, 1], [m, 40], q, return_lse=True)
    want = c.attn_mass(0, [0, 1], [m, 40], q, lse)
    q[m:] = math.nan
    out2 = c.batch_attn(0, [0, 1], [m, 40], q)
    got = c.attn_mass(0, [0, 1], [m, 40], q, lse)
    assert t.equal(out2[:m], out[:m]) and t.equal(got[0], want[0])
    assert bool(t.isnan(got[1]).all()) and bool(t.isnan(out2[m:]).all())


def test_no_queries_only_decays():
    t = P.torch()
    k, v = P.kv(1, [50], 2)
    c = P.cache("bf16", [50], 2, k, v)
    q = P.queries(1, 1, 4, t.bfloat16)[:0]
    prev = t.rand(1, 2, 50, device="cuda")
    got = c.attn_mass(0, [0], [0], q, t.empty(0, 4, device="cuda"), decay=0.5, mass_in=prev)
    assert t.equal(got, prev * 0.5)


def test_same_bits_in_a_graph():
    t = P.torch()
    lens = [1500]
    k, v = P.kv(2, lens, 2)
    c = P.cache("bf16", lens, 2, k, v)
    q = P.queries(2, 16, 10, t.bfloat16)
    _, lse = c.batch_attn(0, [0], [16], q, causal=True, return_lse=True)
    want = c.attn_mass(0, [0], [16], q, lse, causal=True)
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        got = c.attn_mass(0, [0], [16], q, lse, causal=True)
    for _ in range(3):
        g.replay()
        assert t.equal(got, want)


def test_refusals():
    t = P.torch()
    k, v = P.kv(3, [100], 2)
    c = P.cache("bf16", [100], 2, k, v)
    q = P.queries(3, 8, 4, t.bfloat16)
    lse = t.zeros(8, 4, device="cuda")

    def code(*a, **kw):
        with pytest.raises(kvq.KVQError) as e:
            c.attn_mass(*a, **kw)
        return e.value.code

    m = t.zeros(1, 2, 100, device="cuda")
    assert code(0, [0], [8], q, lse, mass_in=m[:, :, :99].contiguous()) == kvq.KVQ_E_INVAL
    assert code(0, [0], [8], q, lse, mass_in=m, decay=1.5) == kvq.KVQ_E_INVAL
    assert code(0, [0], [8], q, lse, mass_in=m, decay=-0.5) == kvq.KVQ_E_INVAL
    assert code(0, [0], [8], q, lse, mass_in=m, decay=math.nan) == kvq.KVQ_E_INVAL
    assert code(0, [0], [8], q, lse[:7], mass_in=m) == kvq.KVQ_E_INVAL
    assert code(0, [0], [8], q, lse, mass_in=m.double()) == kvq.KVQ_E_INVAL
    assert code(0, [0], [8], q, lse, mass_in=m.expand(1, 2, 100)[:, :1]) == kvq.KVQ_E_INVAL
    assert code(0, [0], [101], q, lse, causal=True) == kvq.KVQ_E_INVAL


def test_weights_that_overlap_without_being_one_are_refused():
    t = P.torch()
    k, v = P.kv(3, [100], 2)
    c = P.cache("bf16", [100], 2, k, v)
    q = P.queries(3, 8, 4, t.bfloat16)
    lse = t.zeros(8, 4, device="cuda")
    m = t.zeros(3, 2, 100, device="cuda").view(-1)
    at = lambda i: m[i:i + 200].view(1, 2, 100)  # noqa: E731
    for a, b in ((0, 100), (100, 0), (0, 196)):
        with pytest.raises(kvq.KVQError) as e:
            c.attn_mass(0, [0], [8], q, lse, mass_in=at(a), mass_out=at(b))
        assert e.value.code == kvq.KVQ_E_INVAL
    assert not m.any()
    c.attn_mass(0, [0], [8], q, lse, mass_in=at(0), mass_out=at(200))
    c.attn_mass(0, [0], [8], q, lse, decay=0.0, mass_in=at(0), mass_out=at(100))  # not read
