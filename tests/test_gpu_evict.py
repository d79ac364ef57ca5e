"""Eviction: the kept indices equal a sort in 64 bits, the destination equals a cache the kept rows
were appended to."""
import math

import numpy as np
import pytest

import prompt_helpers as P
from bit_kv_cache_17_b200 import kvq

pytestmark = pytest.mark.gpu


def weights(seed, shape, kind):
    rng = np.random.default_rng(seed)
    w = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        w = np.where(w < 3, 0, np.round(w)).astype(np.float32)
    if kind == "equal":
        w[:] = 0.25
    if kind == "odd":  # signed zeros, infinities, NaN, negative and tiny numbers
        w = rng.choice(np.array([0.0, -0.0, np.inf, -np.inf, np.nan, -1.0, 1e-45, 1.0, 3e38], np.float32), shape)
    return w


def check(lens, budget, sink, recent, hkv=2, kind="plain", dst_type="bf16", tail=0, f16=0, dst_f16=0, seed=0, ids=None):
    t = P.torch()
    ids = list(range(len(lens))) if ids is None else ids
    k, v = P.kv(seed, lens, hkv)
    src = P.cache("bf16", lens, hkv, k, v, tail_f16=f16)
    cap = max(budget, 1) + 5
    dst = kvq.KVCache(n_layers=2, n_seqs=len(ids) + 1, n_kv_heads=hkv, max_ctx=cap, type_k=dst_type, type_v=dst_type,
                      tail=tail, tail_f16=dst_f16)
    dst_ids = [(i + 1) % (len(ids) + 1) for i in range(len(ids))]
    ld = max(lens) + 2
    w = weights(seed, (len(ids), hkv, ld), kind)
    kept, mass = src.evict(dst, 0, 1, ids, dst_ids, t.from_numpy(w).cuda(), budget, sink=sink, recent=recent)
    assert src.status() == 0 and dst.status() == 0
    starts = np.concatenate([[0], np.cumsum(lens)])
    ref = kvq.KVCache(n_layers=2, n_seqs=len(ids) + 1, n_kv_heads=hkv, max_ctx=cap, type_k=dst_type, type_v=dst_type,
                      tail=tail, tail_f16=dst_f16)
    kept, mass = kept.cpu().numpy(), mass.cpu().numpy()
    for i, (s, d) in enumerate(zip(ids, dst_ids)):
        n = lens[s]
        count = min(n, budget)
        assert dst.seq_len(1, d) == count and dst.seq_len(0, d) == 0
        rows_k, rows_v = t.empty(count, hkv, 128, dtype=t.bfloat16, device="cuda"), t.empty(count, hkv, 128, dtype=t.bfloat16, device="cuda")
        for h in range(hkv):
            want = P.evict_ref(w[i, h], n, budget, sink, recent)
            assert np.array_equal(kept[i, h, :count], want), (i, h)
            assert (kept[i, h, count:] == -1).all()
            assert np.array_equal(mass[i, h, :count].view(np.int32), w[i, h, want].view(np.int32))
            assert (mass[i, h, count:] == 0).all()
            at = t.from_numpy(want + starts[s]).cuda()
            rows_k[:, h], rows_v[:, h] = k[at, h], v[at, h]
        if count:
            if f16:
                rows_k, rows_v = rows_k.half().bfloat16(), rows_v.half().bfloat16()
            ref.append(1, [d], [count], rows_k, rows_v)
            for which in (0, 1):
                a, b = (x.dequant(1, d, which, 0, count, basis=0) for x in (dst, ref))
                assert t.equal(a, b)
    return src, dst


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
def test_selection(kind):
    check([1, 0, 64, 65, 700, 1024, 1025, 5000], 64, 4, 16, kind=kind, seed=1)
    check([300, 40], 63, 0, 0, kind=kind, seed=2)


@pytest.mark.parametrize("budget,sink,recent", [(50, 50, 0), (50, 0, 50), (50, 20, 30), (1, 0, 0), (1, 1, 0), (49, 0, 1),
                                                (0, 0, 0), (499, 3, 7), (500, 3, 7), (501, 3, 7)])
def test_budgets(budget, sink, recent):
    check([500, 7], budget, sink, recent, kind="ties", seed=3)


def test_long_rows():
    """Rows longer than one block's shared memory holds."""
    check([70001, 131], 9000, 4, 333, hkv=1, kind="ties", seed=4)
    check([150000], 140000, 4, 333, hkv=1, seed=5)


def test_rows_longer_than_a_cluster_holds():
    """450 000 tokens: the weights are read again in each pass."""
    check([450000], 1000, 4, 333, hkv=1, kind="ties", seed=16)


@pytest.mark.parametrize("dst_type", ["q4_0", "q8_0", "q5_1", "kvarn4", "kvarn3"])
def test_quantized_destination(dst_type):
    check([900, 300, 20], 600, 4, 100, dst_type=dst_type, tail=128, seed=6)
    check([900], 520, 4, 100, dst_type=dst_type, tail=0, seed=7)


@pytest.mark.parametrize("f16,dst_f16", [(1, 1), (1, 0), (0, 1)])
def test_tail_formats(f16, dst_f16):
    check([300], 100, 4, 10, f16=f16, dst_f16=dst_f16, seed=8)
    check([600], 400, 4, 10, f16=f16, dst_f16=dst_f16, dst_type="kvarn4", tail=64, seed=9)


def test_many_entries_and_a_source_used_twice():
    check([(53 * i) % 400 for i in range(70)], 100, 2, 9, hkv=1, kind="ties", seed=10)
    check([300, 200], 90, 2, 9, ids=[1, 0, 1], seed=11)


def test_within_one_cache_and_again():
    """Between sequences of one cache, ping-pong: the second cut sees the first one's result."""
    t = P.torch()
    k, v = P.kv(12, [400], 2)
    c = kvq.KVCache(n_seqs=2, n_kv_heads=2, max_ctx=400, type_k="bf16", type_v="bf16", tail=0)
    c.append(0, [0], [400], k, v)
    w = weights(12, (1, 2, 400), "plain")
    kept, mass = c.evict(c, 0, 0, [0], [1], t.from_numpy(w).cuda(), 200, sink=4, recent=8)
    kept2, mass2 = c.evict(c, 0, 0, [1], [0], mass, 100, sink=4, recent=8)
    assert c.seq_len(0, 1) == 200 and c.seq_len(0, 0) == 100
    for h in range(2):
        a = P.evict_ref(w[0, h], 400, 200, 4, 8)
        b = a[P.evict_ref(w[0, h][a], 200, 100, 4, 8)]
        at = t.from_numpy(b).cuda()
        assert t.equal(c.rows16(0)[0, h, 0, :100], k[at, h]) and t.equal(c.rows16(0)[0, h, 1, :100], v[at, h])


def test_destination_rows_behind_stay():
    t = P.torch()
    k, v = P.kv(13, [100], 2)
    src = P.cache("bf16", [100], 2, k, v)
    dst = kvq.KVCache(n_seqs=2, n_kv_heads=2, max_ctx=80, type_k="bf16", type_v="bf16", tail=0)
    dst.rows16(0).fill_(3.0)
    src.evict(dst, 0, 0, [0], [1], t.rand(1, 2, 100, device="cuda"), 30)
    assert bool((dst.rows16(0)[0] == 3.0).all()) and bool((dst.rows16(0)[1, :, :, 30:] == 3.0).all())


def test_streams_and_graph():
    t = P.torch()
    k, v = P.kv(14, [3000], 2)
    src = P.cache("bf16", [3000], 2, k, v)
    new = lambda: kvq.KVCache(n_kv_heads=2, max_ctx=600, type_k="bf16", type_v="bf16", tail=0)  # noqa: E731
    w = t.rand(1, 2, 3000, device="cuda")
    a = new()
    want = src.evict(a, 0, 0, [0], [0], w, 600, recent=30)
    s, b = t.cuda.Stream(), new()
    s.wait_stream(t.cuda.current_stream())
    got = src.evict(b, 0, 0, [0], [0], w, 600, recent=30, stream=s)
    s.synchronize()
    assert t.equal(want[0], got[0]) and t.equal(a.rows16(0), b.rows16(0))
    g, c = t.cuda.CUDAGraph(), new()
    with t.cuda.graph(g):
        got = src.evict(c, 0, 0, [0], [0], w, 600, recent=30)
    w2 = t.rand(1, 2, 3000, device="cuda")
    w.copy_(w2)
    g.replay()
    want = src.evict(a, 0, 0, [0], [0], w2, 600, recent=30)
    assert t.equal(want[0], got[0]) and t.equal(want[1], got[1]) and t.equal(a.rows16(0), c.rows16(0))


def test_indices_in_the_workspace():
    """Without `kept` and `mass_out` the indices live in the workspace, which then has to be there."""
    t = P.torch()
    k, v = P.kv(17, [300], 2)
    src = P.cache("bf16", [300], 2, k, v)
    st = t.cuda.current_stream().cuda_stream
    w = t.rand(1, 2, 300, device="cuda")
    for type_ in ("bf16", "q8_0"):
        a, b = (kvq.KVCache(n_kv_heads=2, max_ctx=120, type_k=type_, type_v=type_, tail=16) for _ in range(2))
        src.evict(a, 0, 0, [0], [0], w, 120, recent=20)
        need = kvq.kvq_evict_workspace_bytes(src.handle, b.handle, 1, 120)
        ws = t.empty(need, dtype=t.uint8, device="cuda")
        args = (src.handle, 0, b.handle, 0, [0], [0], w.data_ptr(), 300, 120, 0, 20, 0, 0, 0)
        with pytest.raises(kvq.KVQError) as e:
            kvq.kvq_evict(*args, 0, need, st)
        assert e.value.code == kvq.KVQ_E_INVAL
        with pytest.raises(kvq.KVQError) as e:
            kvq.kvq_evict(*args, ws.data_ptr(), need - 1, st)
        assert e.value.code == kvq.KVQ_E_SIZE
        kvq.kvq_evict(*args, ws.data_ptr(), need, st)
        for which in (0, 1):
            assert t.equal(a.dequant(0, 0, which, 0, 120), b.dequant(0, 0, which, 0, 120))


def test_refusals_change_nothing():
    t = P.torch()
    k, v = P.kv(15, [100, 30], 2)
    src = P.cache("bf16", [100, 30], 2, k, v)
    dst = kvq.KVCache(n_seqs=2, n_kv_heads=2, max_ctx=50, type_k="bf16", type_v="bf16", tail=0)
    w = t.rand(2, 2, 100, device="cuda")

    def code(f, *a, **kw):
        n0 = kvq.kvq_launch_count()
        with pytest.raises(kvq.KVQError) as e:
            f(*a, **kw)
        assert kvq.kvq_launch_count() == n0
        return e.value.code

    E = src.evict
    assert code(E, dst, 0, 0, [0, 1], [0, 1], w, 51) == kvq.KVQ_E_CAPACITY
    assert code(E, dst, 0, 0, [0, 1], [1, 1], w, 40) == kvq.KVQ_E_INVAL
    assert code(E, dst, 0, 0, [0], [0, 1], w, 40) == kvq.KVQ_E_INVAL
    assert code(E, dst, 0, 0, [0, 2], [0, 1], w, 40) == kvq.KVQ_E_INVAL
    assert code(E, dst, 0, 0, [0, 1], [0, 1], w, 40, sink=20, recent=21) == kvq.KVQ_E_INVAL
    assert code(E, dst, 0, 0, [0, 1], [0, 1], w, 40, sink=-1) == kvq.KVQ_E_INVAL
    assert code(E, dst, 0, 0, [0, 1], [0, 1], w, -1) == kvq.KVQ_E_INVAL
    assert code(E, dst, 0, 0, [0, 1], [0, 1], w[:, :, :99].contiguous(), 40) == kvq.KVQ_E_INVAL
    assert code(E, dst, 0, 1, [0, 1], [0, 1], w, 40) == kvq.KVQ_E_INVAL
    assert code(E, src, 0, 0, [0], [0], w[:1], 40) == kvq.KVQ_E_INVAL   # onto itself
    assert code(E, src, 0, 0, [0, 1], [1, 0], w, 40) == kvq.KVQ_E_INVAL
    other = kvq.KVCache(n_seqs=2, n_kv_heads=1, max_ctx=50, type_k="bf16", type_v="bf16", tail=0)
    assert code(E, other, 0, 0, [0], [0], w[:1], 40) == kvq.KVQ_E_UNSUPPORTED
    q = P.cache("q8_0", [100, 30], 2, k, v)
    assert code(q.evict, dst, 0, 0, [0], [0], w[:1], 40) == kvq.KVQ_E_UNSUPPORTED
    assert dst.seq_len(0, 0) == 0 and dst.seq_len(0, 1) == 0 and src.seq_len(0, 0) == 100


def test_outputs_over_the_weights_are_refused():
    t = P.torch()
    k, v = P.kv(15, [100], 2)
    src = P.cache("bf16", [100], 2, k, v)
    dst = kvq.KVCache(n_seqs=1, n_kv_heads=2, max_ctx=50, type_k="bf16", type_v="bf16", tail=0)
    w = t.rand(1, 2, 100, device="cuda")
    before = w.clone()
    part = w.view(-1)[40:120].view(1, 2, 40)
    rows = t.zeros(1, 2, 40, dtype=t.int32, device="cuda")
    n0 = kvq.kvq_launch_count()
    for kw in (dict(mass_out=part), dict(kept=part.view(t.int32)), dict(kept=rows, mass_out=rows.view(t.float32)),
               dict(mass_out=w)):
        with pytest.raises(kvq.KVQError) as e:
            src.evict(dst, 0, 0, [0], [0], w, 40, **kw)
        assert e.value.code == kvq.KVQ_E_INVAL
    assert kvq.kvq_launch_count() == n0 and t.equal(w, before) and dst.seq_len(0, 0) == 0
