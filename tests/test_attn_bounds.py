"""The bounds batch attention is held to reject results with one tile of values or keys wrong (no device
needed)."""
import pytest

import attn_bounds as B
import prompt_helpers as P


def swapped(x, a, b):
    y = x.clone()
    y[a * 128:(a + 1) * 128], y[b * 128:(b + 1) * 128] = x[b * 128:(b + 1) * 128], x[a * 128:(a + 1) * 128]
    return y


@pytest.mark.parametrize("n,m,dtype,causal", [(20011, 1, "bfloat16", False), (20011, 17, "bfloat16", False),
                                              (4097, 2, "float16", True), (9000, 40, "float16", True)])
def test_a_wrong_tile_is_rejected(n, m, dtype, causal):
    t = P.torch()
    dtype, G = getattr(t, dtype), 5
    f16 = dtype == t.float16
    q, k = B.inputs(n + m, n, m, 1, G)
    k, v = k.double(), B.marked_values(n, 1).double()
    ref = P.attention(q.to(dtype), k, v, causal)
    u = B.weight_step(m, G, f16)
    out, lse = B.rounded(ref, dtype)
    B.check(out, lse, ref, n, u, f16)
    last = (n - 1) // 128
    zeroed, dropped = v.clone(), v.clone()
    zeroed[128 * 3:128 * 4] = 0
    dropped[128 * last:] = 0
    for wrong in (P.attention(q, k, swapped(v, 2, 9), causal), P.attention(q, k, swapped(v, 0, last - 1), causal),
                  P.attention(q, k, zeroed, causal), P.attention(q, swapped(k, 2, 9), v, causal),
                  P.attention(q, k, dropped, causal)):
        with pytest.raises(AssertionError):
            B.check(B.rounded(wrong, dtype)[0], None, ref, n, u, f16)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
def test_rounded_weights_are_rejected_where_their_remainders_count(dtype):
    """A flat background below one peak: its weights all round the same way."""
    t = P.torch()
    dtype = getattr(t, dtype)
    x = t.arange(1, 26, dtype=t.float64)[:, None] / 8  # the background's scores below the peak's
    w = t.exp(-x)
    n, v = 1000, 1.25
    exact = (n - 1) * w * v / (1 + (n - 1) * w)
    taken = (n - 1) * w.to(dtype).double() * v / (1 + (n - 1) * w)
    step = P.half_step(dtype)
    slack = 1e-4 * exact
    assert not bool(((taken.to(dtype).double() - exact).abs() <= step * exact + slack).all())
    assert bool(((exact.to(dtype).double() - exact).abs() <= step * exact + slack).all())
