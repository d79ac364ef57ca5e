"""Rotary positions with several axes against complex multiplication in 64 bits, every element within
the bound that fp32 sines, products and one output rounding allow."""
import numpy as np
import pytest

import prompt_helpers as P
from bit_kv_cache_17_b200 import kvq

pytestmark = pytest.mark.gpu


def axes(sections, turns):
    left, out, a = list(sections), [], 0
    while sum(left):
        if left[a] and not turns:
            out += [a] * left[a]
            left[a] = 0
        elif left[a]:
            out.append(a)
            left[a] -= 1
        a = (a + 1) % len(left)
    return out


def reference(x, pos, sections, rot, turns, adjacent, inverse, freq):
    """x [n, h, 128] -> (rotated fp64, bound of the fp32 result's error)"""
    t = P.torch()
    half = rot // 2
    ang = t.stack([pos[a].double() * f for a, f in zip(axes(sections, turns), freq)], 1)[:, None]
    y = x.double().cpu().clone()
    i = t.arange(half)
    a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
    z = t.complex(y[..., a], y[..., b]) * t.polar(t.ones_like(ang), -ang if inverse else ang)
    mag = y.abs()
    tol = t.zeros_like(y)
    both = mag[..., a] + mag[..., b]
    # sine and cosine: the angle's cast (2^-25 of half a turn, times pi), their own 2 steps, and the
    # rounding of two products and a sum
    tol[..., a] = tol[..., b] = both * (np.pi * P.U32 + 4 * P.U32 + 2 * P.U32)
    y[..., a], y[..., b] = z.real, z.imag
    return y, tol


def check(got, want, tol, dtype):
    err = (got.double().cpu() - want).abs()
    full = tol + (0.0 if dtype == P.torch().float32 else P.half_step(dtype)) * (want.abs() + tol) + \
        (2.0 ** -25 if dtype == P.torch().float16 else 0.0)
    assert bool((err <= full).all()), float((err - full).max())


def positions(seed, n_axes, n, far):
    return P.torch().from_numpy(np.random.default_rng(seed).integers(-far, far, (n_axes, n)).astype(np.int32))


CASES = [
    # n, hq, hk, q type, out type, sections, rot, turns, adjacent
    (1, 40, 8, "bfloat16", "float32", (16, 24, 24), 128, False, False),
    (37, 40, 8, "float32", "float32", (24, 20, 20), 128, True, False),
    (4099, 3, 1, "bfloat16", "bfloat16", (64,), 128, False, True),
    (130, 10, 2, "float16", "float16", (24, 24), 96, True, True),
    (77, 5, 5, "float16", "float32", (11, 0, 20), 62, True, False),   # rot_dim no multiple of 16, an empty axis
    (5, 2, 1, "float32", "bfloat16", (1,), 2, False, False),
    (9, 1, 2, "bfloat16", "float16", (8, 8, 8, 9), 66, False, True),
]


@pytest.mark.parametrize("n,hq,hk,ti,to,sections,rot,turns,adjacent", CASES)
@pytest.mark.parametrize("inverse", [False, True])
def test_matches_the_definition(n, hq, hk, ti, to, sections, rot, turns, adjacent, inverse):
    t = P.torch()
    ti, to = getattr(t, ti), getattr(t, to)
    g = t.Generator().manual_seed(n)
    q, k = t.randn(n, hq, 128, generator=g).to(ti), t.randn(n, hk, 128, generator=g).bfloat16()
    pos = positions(n, len(sections), n, 1 << 30)
    r = kvq.Rope(sections, theta=1e6, rot_dim=rot, turns=turns, adjacent=adjacent)
    qo, ko = r.apply(pos.cuda(), q.cuda(), k.cuda(), q_dtype=to, inverse=inverse)
    freq = [1e6 ** (-2.0 * i / rot) for i in range(rot // 2)]
    for x, got, dt in ((q, qo, to), (k, ko, t.bfloat16)):
        want, tol = reference(x, pos, sections, rot, turns, adjacent, inverse, freq)
        check(got, want, tol, dt)
        # channels that do not turn are converted only
        assert t.equal(got[..., rot:].cpu(), x[..., rot:].to(dt))


def test_packed_rows_in_place_and_given_frequencies():
    """q and k as slices of packed q|k|v rows, rotated in place; the v part and the passing channels,
    NaN and infinity among them, stay as they were."""
    t = P.torch()
    n, hq, hk = 19, 6, 2
    rows = t.randn(n, (hq + 2 * hk) * 128, generator=t.Generator().manual_seed(3)).bfloat16()
    rows.view(n, -1, 128)[:, :, 100] = float("nan")
    rows.view(n, -1, 128)[:, :, 101] = float("inf")
    pos = positions(3, 2, n, 5000)
    freq = [0.5 ** (i / 7) for i in range(32)]
    dev = rows.cuda()
    q, k = dev[:, : hq * 128].view(n, hq, 128), dev[:, hq * 128:(hq + hk) * 128].view(n, hk, 128)
    r = kvq.Rope((20, 12), rot_dim=64, inv_freq=freq)
    qo, ko = r.apply(pos.cuda(), q, k, q_out=q, k_out=k)
    assert qo.data_ptr() == q.data_ptr()
    x = rows.view(n, -1, 128)
    want, tol = reference(x[:, : hq + hk], pos, (20, 12), 64, False, False, False, freq)
    got = dev.cpu().view(n, -1, 128)
    check(got[:, : hq + hk, :64], want[..., :64], tol[..., :64], t.bfloat16)
    assert t.equal(got.view(t.int16)[:, : hq + hk, 64:], x.view(t.int16)[:, : hq + hk, 64:])
    assert t.equal(got.view(t.int16)[:, hq + hk:], x.view(t.int16)[:, hq + hk:])


def test_only_q_only_k_and_no_tokens():
    t = P.torch()
    r = kvq.Rope((64,))
    pos = t.arange(4, dtype=t.int32).cuda()
    x = t.randn(4, 2, 128).bfloat16().cuda()
    a, none = r.apply(pos, q=x)
    assert none is None
    _, b = r.apply(pos, k=x)
    assert t.equal(a, b)
    e, _ = r.apply(pos[:0], q=x[:0])
    assert e.shape == (0, 2, 128)
    # one token of a packed buffer keeps its row stride
    a1, _ = r.apply(pos[1:2], q=x[1:2])
    assert t.equal(a1, a[1:2])


@pytest.mark.parametrize("n", [1, 300])
def test_one_row_of_positions_for_all_axes(n):
    t = P.torch()
    r = kvq.Rope((16, 24, 24), turns=True)
    x = t.randn(n, 3, 128, generator=t.Generator().manual_seed(n)).bfloat16().cuda()
    row = positions(n, 1, n, 5000)[0].cuda()
    want, _ = r.apply(row.repeat(3, 1), q=x)
    assert t.equal(r.apply(row.expand(3, n), q=x)[0], want)
    if n > 2:  # rows that overlap
        with pytest.raises(kvq.KVQError):
            r.apply(row.as_strided((3, n - 2), (1, 1)), q=x[:n - 2])


def test_inverse_is_the_gradient():
    """The gradient of sum(w . rope(x)) by x is rope_inverse(w): against differences of the fp32 result."""
    t = P.torch()
    r = kvq.Rope((10, 22), theta=100.0, turns=True)
    pos = positions(9, 2, 3, 50).cuda()
    g = t.Generator().manual_seed(5)
    x, w = (t.randn(3, 2, 128, generator=g).cuda() for _ in range(2))
    grad, _ = r.apply(pos, q=w, inverse=True)
    f = lambda y: (r.apply(pos, q=y)[0].double() * w.double()).sum()  # noqa: E731
    # a linear map: a step of 1 has no truncation error, only the fp32 roundings of two results of
    # size up to |x| + 1 over 256 channels' terms
    for at in ((0, 0, 3), (1, 1, 64), (2, 0, 127)):
        d = t.zeros_like(x)
        d[at] = 1.0
        diff = float(f(x + d) - f(x))
        size = float((x.abs().amax() + 1) * w.abs().amax())
        assert abs(diff - float(grad[at])) <= 2 * 4 * 8 * P.U32 * size * 2


def test_stream_and_graph():
    t = P.torch()
    r = kvq.Rope((32, 32), turns=True)
    pos = positions(1, 2, 33, 1000).cuda()
    q, k = t.randn(33, 4, 128).bfloat16().cuda(), t.randn(33, 2, 128).bfloat16().cuda()
    want = r.apply(pos, q, k)
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    got = r.apply(pos, q, k, stream=s)
    s.synchronize()
    assert t.equal(want[0], got[0]) and t.equal(want[1], got[1])
    gr = t.cuda.CUDAGraph()
    with t.cuda.graph(gr):
        out = r.apply(pos, q, k)
    q2 = t.randn(33, 4, 128).bfloat16().cuda()
    q.copy_(q2)
    gr.replay()
    assert t.equal(out[0], r.apply(pos, q2, k)[0])
