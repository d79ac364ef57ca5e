"""Batch attention held to bounds that see one wrong tile and one rounding too many."""
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
