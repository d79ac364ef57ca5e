"""Outputs over what other blocks still read are refused before anything is launched; neighbours are not."""
import math

import pytest

import prompt_helpers as P
from bit_kv_cache_17_b200 import kvq

pytestmark = pytest.mark.gpu

M, HQ = 60, 4


def setup():
    """A cache of 100 tokens, and one buffer to cut overlapping views from"""
    t = P.torch()
    k, v = P.kv(3, [100], 2)
    c = P.cache("bf16", [100], 2, k, v)
    buf = t.zeros(1 << 18, dtype=t.uint8, device="cuda")
    at = lambda dtype, off, *shape: buf[off:off + math.prod(shape) * dtype.itemsize].view(dtype).view(*shape)  # noqa: E731
    return t, c, buf, at


def refused(f):
    n0 = kvq.kvq_launch_count()
    with pytest.raises(kvq.KVQError) as e:
        f()
    assert e.value.code == kvq.KVQ_E_INVAL and kvq.kvq_launch_count() == n0


def test_lse_over_the_queries_or_the_output():
    t, c, buf, at = setup()
    rows, lses = M * HQ * 256, M * HQ * 4
    far = 1 << 17
    q, lse = at(t.bfloat16, far, M, HQ, 128), lambda off: at(t.float32, off, M, HQ)
    out = at(t.bfloat16, 4096, M, HQ, 128)
    for off in (4096, 4096 + rows - 16, 4096 - lses + 16, far, far + rows - 16, far - lses + 16):
        refused(lambda: c.batch_attn(0, [0], [M], q, out=out, lse=lse(off)))  # noqa: B023
    assert not buf.any()
    for off in (4096 + rows, 4096 - lses, far - lses, far + rows):
        c.batch_attn(0, [0], [M], q, out=out, lse=lse(off))
    assert c.status() == 0


def test_weights_over_the_queries_or_their_lse():
    t, c, buf, at = setup()
    rows, lses, mass = M * HQ * 256, M * HQ * 4, 2 * 100 * 4
    a, b = 8192, 1 << 17
    q, lse = at(t.bfloat16, a, M, HQ, 128), at(t.float32, b, M, HQ)
    for off in (a, a + rows - 16, a - mass + 16, b, b + lses - 16, b - mass + 16):
        refused(lambda: c.attn_mass(0, [0], [M], q, lse, mass_out=at(t.float32, off, 1, 2, 100)))  # noqa: B023
        refused(lambda: c.attn_mass(0, [0], [M], q, lse, mass_in=at(t.float32, off, 1, 2, 100),  # noqa: B023
                                    mass_out=at(t.float32, off, 1, 2, 100)))  # noqa: B023
    assert not buf.any()
    for off in (a + rows, a - mass, b + lses, b - mass):
        c.attn_mass(0, [0], [M], q, lse, mass_out=at(t.float32, off, 1, 2, 100))
    # without query rows nothing of theirs is read
    none = at(t.bfloat16, a, M, HQ, 128)[:0]
    c.attn_mass(0, [0], [0], none, at(t.float32, a, M, HQ)[:0], mass_out=at(t.float32, a, 1, 2, 100))
    assert c.status() == 0
