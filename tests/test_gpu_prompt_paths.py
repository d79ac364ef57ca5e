"""Ways through the batch attention and weight kernels that the sizes of the other tests do not take: query
tiles that stream past several key pairs, splits of them over rebuilt keys, many rebuilt sequences and
launches in a row."""
import pytest

import prompt_helpers as P
import test_gpu_attn_bounds as bounds
import test_gpu_attn_mass as mass
import test_gpu_batch_attn as attn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("type_,f16", [("bf16", 0), ("bf16", 1), ("q8_0", 0), ("kvarn4", 0)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("n", [1024, 1300, 4096])
def test_streamed_query_tiles_past_several_key_pairs(n, causal, type_, f16):
    """More than three query tiles, and more than one pair of key tiles per block: the ring of query tiles
    goes on from pair to pair."""
    mass.check(type_, [n], [100], 8, 5, causal, tail=0 if type_ == "bf16" else 128, tail_f16=f16, seed=n)


@pytest.mark.parametrize("type_", ["bf16", "q8_0", "q4_1", "kvarn4"])
@pytest.mark.parametrize("causal", [False, True])
def test_splits_of_the_query_tiles(causal, type_):
    """Query tiles split over blocks whose sums a second kernel adds, alone and beside entries without splits."""
    mass.check(type_, [2000], [500], 2, 5, causal, tail=0 if type_ == "bf16" else 100, seed=5)
    mass.check(type_, [1500, 0, 300, 2049], [450, 1 - causal, 30, 7], 2, 3, causal,
               tail=0 if type_ == "bf16" else 64, seed=6)


def test_every_query_of_a_long_prompt():
    mass.check("bf16", [4500], [1100], 2, 5, True, seed=7, inplace=True)


def many(seed, long_):
    """140 short sequences, some of them empty, and with `long_` two whose contexts are split"""
    lens = [(29 * i + seed) % 90 for i in range(140)] + ([3000, 2500] if long_ else [])
    n_q = [1 + i % 3 for i in range(140)] + ([2, 1] if long_ else [])
    return lens, n_q


@pytest.mark.parametrize("type_,type_v", [("q8_0", None), ("kvarn4", "q5_1")])
@pytest.mark.parametrize("long_", [False, True])
def test_many_rebuilt_sequences(long_, type_, type_v):
    """More sequences than one launch rebuilds, more entries than one attends: attention launches set up behind
    one another, and behind a join."""
    lens, n_q = many(1, long_)
    attn.run_case(type_, lens, n_q, 1, 2, False, tail=20, type_v=type_v, seed=11)
    mass.check(type_, lens, n_q, 1, 2, False, tail=20, seed=12)


def test_many_rebuilt_sequences_within_tight_bounds():
    lens = [40 + (29 * i) % 300 for i in range(140)] + [3000, 2500]
    bounds.run("q8_0", lens, [1 + i % 3 for i in range(140)] + [2, 130], 1, 2, False, seed=50, tail=20)


def test_many_rebuilt_sequences_in_a_row_and_replayed():
    """The same call again behind itself, and as a graph: each waits for what it reads."""
    t = P.torch()
    lens, n_q = many(3, True)
    k, v = P.kv(13, lens, 1)
    c = P.cache("q8_0", lens, 1, k, v, tail=20)
    ids = list(range(len(lens)))
    qs = [P.queries(60 + i, sum(n_q), 2, t.bfloat16) for i in range(3)]
    want = []
    for q in qs:
        want.append(c.batch_attn(0, ids, n_q, q, return_lse=True))
        t.cuda.synchronize()
    for _ in range(3):
        for q, (a, la) in zip(qs, want):
            b, lb = c.batch_attn(0, ids, n_q, q, return_lse=True)
            assert t.equal(a, b) and t.equal(la, lb)
    q = qs[0].clone()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        out, lse = c.batch_attn(0, ids, n_q, q, return_lse=True)
    for x, (a, la) in zip(qs, want):
        q.copy_(x)
        g.replay()
        assert t.equal(out, a) and t.equal(lse, la)
    assert c.status() == 0
