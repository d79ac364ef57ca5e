"""Batch attention (cross attention and causal chunks) against attention in 64 bits over the values
the cache holds: every output element within the bound of its roundings."""
import math

import pytest

import prompt_helpers as P
from bit_kv_cache_17_b200 import kvq

pytestmark = pytest.mark.gpu


def run_case(type_, lens, n_q, hkv, G, causal, tail=0, tail_f16=0, type_v=None, seed=0, ids=None, scale=0.0, qscale=1.0):
    t = P.torch()
    ids = list(range(len(lens))) if ids is None else ids
    k, v = P.kv(seed, lens, hkv)
    c = P.cache(type_, lens, hkv, k, v, tail, tail_f16, type_v)
    dt = t.float16 if tail_f16 else t.bfloat16
    q = P.queries(seed, sum(n_q), hkv * G, dt) * qscale
    out, lse = c.batch_attn(0, ids, n_q, q, causal=causal, return_lse=True, softmax_scale=scale)
    assert c.status() == 0
    u = P.UB16 if (type_ == "bf16" and not tail_f16) else P.U16
    row = 0
    for s, m in zip(ids, n_q):
        kk, vv = P.cached(c, 0, s)
        ref = P.attention(q[row:row + m], kk, vv, causal, scale or None)
        P.check_attention(out[row:row + m], lse[row:row + m], ref, lens[s], u, type_ != "bf16")
        row += m
    return c, q, out, lse


# tokens and queries around the tile edges: a tile is 128 rows or tokens
@pytest.mark.parametrize("f16", [0, 1])
@pytest.mark.parametrize("G", [1, 3, 5, 8])
def test_cross_lengths(G, f16):
    run_case("bf16", [1, 0, 127, 128, 129, 300, 513], [3, 5, 1, 0, 52, 26, 257], 2, G, False, tail_f16=f16, seed=G)


@pytest.mark.parametrize("f16", [0, 1])
@pytest.mark.parametrize("G", [1, 2, 7])
def test_causal_lengths(G, f16):
    # the whole prompt, its last tokens, one token, one of one
    run_case("bf16", [1, 130, 257, 400, 640, 127], [1, 130, 1, 37, 640, 126], 2, G, True, tail_f16=f16, seed=10 + G)


@pytest.mark.parametrize("m", [1, 2, 17])
def test_long_context_few_rows(m):
    """The context split over the SMs and joined."""
    run_case("bf16", [20011], [m], 8, 5, False, seed=m)
    run_case("bf16", [9000, 77, 4097], [m, 1, m], 1, 8, True, seed=m, tail_f16=1)


@pytest.mark.parametrize("t", ["q2_0", "q3_0", "q4_0", "q5_0", "q6_0", "q8_0", "q4_1", "q2_1", "q3_1", "q5_1", "q6_1",
                               "kvarn2", "kvarn3", "kvarn4", "kvarn5", "kvarn6", "kvarn8"])
def test_quantized_types(t):
    run_case(t, [700, 0, 300], [9, 2, 70], 2, 5, False, tail=100, seed=4)
    run_case(t, [333], [60], 1, 3, True, tail=0, seed=5)


def test_mixed_types_and_f16_tail():
    run_case("kvarn4", [600, 50], [20, 3], 2, 2, False, tail=256, tail_f16=1, type_v="q8_0", seed=6)


def test_one_sequence_listed_several_times_and_scale():
    run_case("bf16", [200, 150], [4, 1, 7, 2], 2, 4, False, ids=[1, 0, 1, 1], scale=0.3, seed=7)
    run_case("q8_0", [200, 150], [4, 1, 7, 2], 2, 4, False, ids=[1, 0, 1, 1], scale=0.3, seed=7)


def test_more_entries_than_a_launch_takes():
    lens = [(37 * i) % 200 for i in range(70)]
    run_case("bf16", lens, [1 + i % 3 for i in range(70)], 1, 2, False, seed=8)


def test_empty_sequences_give_zeros_every_time():
    """Rows of empty sequences beside others, many at once and again and again: exactly zero (their
    query rows must never show through)."""
    t = P.torch()
    lens = [0] * 12 + [300]
    k, v = P.kv(4, lens, 2)
    c = P.cache("bf16", lens, 2, k, v)
    n_q = [100] * 13
    q = P.queries(4, 1300, 10, t.bfloat16)
    for _ in range(20):
        out, lse = c.batch_attn(0, list(range(13)), n_q, q, return_lse=True)
        assert bool((out[:1200] == 0).all()) and bool((lse[:1200] == -math.inf).all())
        assert bool((out[1200:] != 0).any())


def test_sharp_and_shifted_scores():
    """Scores far apart (the weights of all but a few tokens vanish) and far from zero."""
    run_case("bf16", [1000], [33], 2, 5, False, seed=9, qscale=16.0)
    run_case("bf16", [1000], [200], 2, 5, True, seed=9, qscale=16.0, tail_f16=1)


def test_rows_of_other_calls_stay():
    """Output and lse rows behind the last query are not touched; an empty list does nothing."""
    t = P.torch()
    lens = [140]
    k, v = P.kv(1, lens, 2)
    c = P.cache("bf16", lens, 2, k, v)
    q = P.queries(1, 40, 4, t.bfloat16)
    out, lse = t.full_like(q, 7.0), t.full((40, 4), 7.0, device="cuda")
    ws = t.empty(1 << 20, dtype=t.uint8, device="cuda")
    kvq.kvq_batch_attn(c.handle, 0, [0], [29], 4, 0, q.data_ptr(), 0.0, out.data_ptr(), lse.data_ptr(), ws.data_ptr(),
                       ws.numel(), t.cuda.current_stream().cuda_stream)
    assert bool((out[29:] == 7.0).all()) and bool((lse[29:] == 7.0).all())
    want, wl = c.batch_attn(0, [0], [29], q[:29], return_lse=True)
    assert t.equal(out[:29], want) and t.equal(lse[:29], wl)
    e = c.batch_attn(0, [], [], q[:0])
    assert e.shape == (0, 4, 128)
    # an infinite query makes its own row NaN and no other
    q2 = q[:29].clone()
    q2[3, 1] = math.inf
    got = c.batch_attn(0, [0], [29], q2)
    bad = t.zeros(29, 4, dtype=t.bool, device="cuda")
    bad[3, 1] = True
    assert t.equal(got[~bad], want[~bad])


def test_same_bits_every_time_on_streams_and_in_graphs():
    t = P.torch()
    lens = [3000, 200]
    k, v = P.kv(2, lens, 2)
    c = P.cache("bf16", lens, 2, k, v)
    q = P.queries(2, 9, 10, t.bfloat16)
    q2 = P.queries(3, 9, 10, t.bfloat16)
    want, want2 = c.batch_attn(0, [0, 1], [4, 5], q), c.batch_attn(0, [0, 1], [4, 5], q2)
    streams = [t.cuda.Stream() for _ in range(2)]
    t.cuda.synchronize()
    got = [[c.batch_attn(0, [0, 1], [4, 5], x, stream=s) for s, x in zip(streams, (q, q2))] for _ in range(10)]
    t.cuda.synchronize()
    assert all(t.equal(a, want) and t.equal(b, want2) for a, b in got)
    graphs = []
    for x in (q, q2):
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            graphs.append((g, c.batch_attn(0, [0, 1], [4, 5], x)))
    for g, _ in graphs:
        g.replay()
    assert t.equal(graphs[0][1], want) and t.equal(graphs[1][1], want2)
    assert c.status() == 0


def test_refusals():
    t = P.torch()
    lens = [100, 50]
    k, v = P.kv(3, lens, 2)
    c = P.cache("bf16", lens, 2, k, v)
    q = P.queries(3, 60, 4, t.bfloat16)

    def code(f, *a, **kw):
        n0 = kvq.kvq_launch_count()
        with pytest.raises(kvq.KVQError) as e:
            f(*a, **kw)
        assert kvq.kvq_launch_count() == n0
        return e.value.code

    assert code(c.batch_attn, 0, [0], [60], q.half()) == kvq.KVQ_E_UNSUPPORTED
    assert code(c.batch_attn, 0, [0], [59], q) == kvq.KVQ_E_INVAL
    assert code(c.batch_attn, 0, [0, 1], [60], q) == kvq.KVQ_E_INVAL
    assert code(c.batch_attn, 0, [2], [60], q) == kvq.KVQ_E_INVAL
    assert code(c.batch_attn, 1, [0], [60], q) == kvq.KVQ_E_INVAL
    assert code(c.batch_attn, 0, [1], [60], q, causal=True) == kvq.KVQ_E_INVAL   # more queries than tokens
    assert code(c.batch_attn, 0, [0], [60], q[:, :3].contiguous()) == kvq.KVQ_E_INVAL  # heads per KV head
    assert code(c.batch_attn, 0, [0], [60], q.repeat(1, 5, 1)) == kvq.KVQ_E_UNSUPPORTED  # G = 10
    assert code(c.batch_attn, 0, [0], [60], q, out=q[:, :2]) == kvq.KVQ_E_INVAL
    assert code(c.batch_attn, 0, [0], [60], q.cpu()) == kvq.KVQ_E_INVAL
    assert code(c.batch_attn, 0, [0], [60], q, lse=t.zeros(60, 3, device="cuda")) == kvq.KVQ_E_INVAL
    d = P.cache("q8_0", lens, 2, k, v)
    st = t.cuda.current_stream().cuda_stream
    args = (d.handle, 0, [0], [60], 4)
    need = kvq.kvq_batch_workspace_bytes(*args)
    ws = t.empty(need, dtype=t.uint8, device="cuda")
    out = t.empty_like(q)
    assert code(kvq.kvq_batch_attn, *args, 0, q.data_ptr(), 0.0, out.data_ptr(), 0, ws.data_ptr(), need - 1,
                st) == kvq.KVQ_E_SIZE
    assert code(kvq.kvq_batch_attn, *args, 0, q.data_ptr() + 2, 0.0, out.data_ptr(), 0, ws.data_ptr(), need,
                st) == kvq.KVQ_E_ALIGN
    assert code(kvq.kvq_batch_attn, *args, 2, q.data_ptr(), 0.0, out.data_ptr(), 0, ws.data_ptr(), need,
                st) == kvq.KVQ_E_INVAL


def test_an_output_over_its_queries_is_refused():
    t = P.torch()
    k, v = P.kv(3, [100], 2)
    c = P.cache("bf16", [100], 2, k, v)
    both = t.zeros(120, 4, 128, dtype=t.bfloat16, device="cuda")
    n0 = kvq.kvq_launch_count()
    for a, b in ((0, 0), (0, 59), (59, 0)):
        with pytest.raises(kvq.KVQError) as e:
            c.batch_attn(0, [0], [60], both[a:a + 60], out=both[b:b + 60])
        assert e.value.code == kvq.KVQ_E_INVAL
    assert kvq.kvq_launch_count() == n0
    c.batch_attn(0, [0], [60], both[:60], out=both[60:])  # neighbours
    assert kvq.kvq_launch_count() > n0


@pytest.mark.parametrize("m", [3, 200])
def test_rebuilt_calls_one_after_another_and_in_a_graph(m):
    """The attention is set up behind the launch that rebuilds the cache and converts the queries:
    calls in a row, which take the same workspace, and replays give what single calls give."""
    t = P.torch()
    lens = [700, 0, 3000]
    k, v = P.kv(8, lens, 2)
    c = P.cache("q8_0", lens, 2, k, v, tail=128)
    n_q = [m, 2, m]
    qs = [P.queries(40 + i, sum(n_q), 10, t.bfloat16) for i in range(8)]
    want = []
    for q in qs:
        want.append(c.batch_attn(0, [0, 1, 2], n_q, q, return_lse=True))
        t.cuda.synchronize()
    for _ in range(3):
        got = [c.batch_attn(0, [0, 1, 2], n_q, q, return_lse=True) for q in qs]
        for (a, la), (b, lb) in zip(want, got):
            assert t.equal(a, b) and t.equal(la, lb)
    q = qs[0].clone()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        out, lse = c.batch_attn(0, [0, 1, 2], n_q, q, return_lse=True)
    for x, (a, la) in zip(qs, want):
        q.copy_(x)
        g.replay()
        assert t.equal(out, a) and t.equal(lse, la)
