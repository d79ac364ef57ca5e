"""Batch attention held to bounds that see one wrong tile and one rounding too many."""
import math

import pytest

import attn_bounds as B
import prompt_helpers as P

pytestmark = pytest.mark.gpu


def run(type_, lens, n_q, hkv, G, causal, f16=0, seed=0, tail=0):
    t = P.torch()
    dt = t.float16 if f16 else t.bfloat16
    ks, vs, qs = [], [], []
    for i, (n, m) in enumerate(zip(lens, n_q)):
        q, k = B.inputs(seed + i, n, m, hkv, G)
        qs.append(q), ks.append(k), vs.append(B.marked_values(n, hkv))
    c = P.cache(type_, lens, hkv, t.cat(ks).cuda(), t.cat(vs).cuda(), tail, f16)
    q = t.cat(qs).to(dt).cuda()
    out, lse = c.batch_attn(0, list(range(len(lens))), n_q, q, causal=causal, return_lse=True)
    assert c.status() == 0
    quant, row = type_ != "bf16", 0
    for i, (n, m) in enumerate(zip(lens, n_q)):
        kk, vv = P.cached(c, 0, i)
        ref = P.attention(q[row:row + m], kk, vv, causal)
        B.check(out[row:row + m], lse[row:row + m], ref, n, B.weight_step(m, G, f16 or quant), bool(f16) or quant, quant)
        row += m


@pytest.mark.parametrize("f16", [0, 1])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n,m", [(20011, 1), (20011, 17), (9000, 40), (4097, 2), (1300, 130), (512, 1)])
def test_every_tile_is_where_it_belongs(n, m, causal, f16):
    run("bf16", [n], [m], 2, 5, causal, f16, seed=n + m)


@pytest.mark.parametrize("type_", ["q8_0", "kvarn4", "q4_1"])
def test_every_tile_of_a_rebuilt_cache(type_):
    run(type_, [5001, 300], [3, 60], 2, 5, False, seed=3, tail=128)
    run(type_, [2100], [140], 1, 5, True, seed=4)


def faint(n, count, f16):
    """A flat background below one peak in every 128 tokens (so that no part of the row's weights is relative to
    the background): count rows x 5 heads whose background's scores lie (row * 5 + head) / 32 below the
    peaks'.  -> q, k, v of one KV head, exact out"""
    t = P.torch()
    q = t.zeros(count, 5, 128)
    q[..., 0] = t.arange(1, 5 * count + 1).view(count, 5) / 32
    k, v = t.zeros(n, 1, 128), t.full((n, 1, 128), 1.25)
    k[::128, 0, 0] = 1.0
    v[::128] = 0.0
    peaks = -(-n // 128)
    w = (n - peaks) * t.exp(-q[..., 0].double())
    out = 1.25 * w / (peaks + w)
    return q.to(t.float16 if f16 else t.bfloat16).cuda(), k.bfloat16().cuda(), v.bfloat16().cuda(), out.cuda()


@pytest.mark.parametrize("f16", [0, 1])
@pytest.mark.parametrize("company", ["none", "rows", "tokens", "both"])
def test_few_rows_are_as_exact_as_their_type_whatever_else_is_in_the_call(company, f16):
    t = P.torch()
    n = 1000
    q, k, v, want = faint(n, 25, f16)
    lens, n_q, extra = [n], [25], 0
    if company in ("tokens", "both"):
        lens, n_q, extra = lens + [20000], n_q + [1], extra + 1
    if company in ("rows", "both"):
        lens, n_q, extra = lens + [400], n_q + [90], extra + 90
    k2, v2 = P.kv(1, [max(sum(lens[1:]), 1)], 1)
    c = P.cache("bf16", lens, 1, t.cat([k, k2])[:sum(lens)], t.cat([v, v2])[:sum(lens)], tail_f16=f16)
    qs = t.cat([q, P.queries(2, extra, 5, q.dtype)]) if extra else q
    out = c.batch_attn(0, list(range(len(lens))), n_q, qs, softmax_scale=1.0)[:25].double()
    assert c.status() == 0
    # the scores are exact; exp's few steps, one step a sum, the remainders' rounding; then the output's half step
    rel = 16 * P.U32 + (n + 16) * 2 * P.U32 + (P.U16 if f16 else P.UB16) ** 2
    want = want[..., None]
    tol = rel * want + P.half_step(q.dtype) * want * (1 + rel)
    err = (out - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("type_", ["f16", "q8_0"])
@pytest.mark.parametrize("n_q", [[25] * 20, [1000]])
def test_many_faint_tokens_add_up(n_q, type_):
    """65 536 tokens 17.5 below a peak in front of them: each weight is under half of the least F16 number.  As
    many rows as leave the context in one piece (a piece without the peak has no small weights)."""
    t = P.torch()
    n, m, f16 = 65536, sum(n_q), int(type_ == "f16")
    q = t.zeros(m, 40, 128)
    q[..., 0] = 17.5
    k, v = t.zeros(n, 8, 128), t.ones(n, 8, 128)
    peaks = 2  # in the first two tiles, which calls of few rows take separately
    k[0, :, 0] = k[128, :, 0] = 1.0
    v[0] = v[128] = 0.0
    c = P.cache("bf16" if f16 else type_, [n], 8, k.bfloat16().cuda(), v.bfloat16().cuda(), tail_f16=f16)
    q = q.to(t.float16 if f16 else t.bfloat16).cuda()
    out = c.batch_attn(0, [0] * len(n_q), n_q, q, softmax_scale=1.0)
    assert c.status() == 0
    key, value = (float(x[i, 0, 0]) for x, i in zip(P.cached(c, 0, 0), (0, 1)))
    w = (n - peaks) * math.exp(-17.5 * key)
    want = value * w / (peaks + w)
    # the score is one product (and, rebuilt, a key of 22 bits); a weight below the normal range is off by 2^-25
    # of 2^7 or more; a step of fp32 for every addition; the value's rounding
    rel = 2 * 17.5 * (4 * P.U32 + (0.0 if f16 else 2.0 ** -22)) + (n + 16) * 2 * P.U32 + (0.0 if f16 else P.U16)
    tol = rel * want + n * 2.0 ** -32
    tol = tol + P.half_step(q.dtype) * (want + tol) + 2.0 ** -25
    assert want > 8 * tol
    err = (out.double() - want).abs().amax()
    assert float(err) <= tol, (want, float(err), tol)
