"""Outputs of kvq_rope over rows that other blocks still read or write are refused on the host (no device
needed); slices of a packed row are not."""
import itertools

import pytest
import torch

from bit_kv_cache_17_b200 import kvq

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")

BASE = 1 << 30


def code(n, q, q_out, k, k_out, pos=1 << 20, types=(1, 1), heads=(2, 1), axes=1, pos_ld=None):
    """q, q_out, k, k_out: (address, row stride in elements)"""
    p = kvq.kvq_rope_default_params(n_axes=axes, sections=[64, 0, 0, 0])
    return kvq._lib.kvq_rope(kvq.C.byref(p), None, n, pos, n if pos_ld is None else pos_ld, heads[0], q[0], types[0],
                             q[1], q_out[0], types[1], q_out[1], heads[1], k[0], k[1], k_out[0], k_out[1], None)


def refused(*a, **kw):
    return code(*a, **kw) == kvq.KVQ_E_INVAL


FAR = [(BASE + (i << 24), 256) for i in range(4)]
KFAR = (BASE + (5 << 24), 128)


@pytest.mark.parametrize("n", [1, 2, 9])
def test_an_output_over_the_other_tensor(n):
    q, qo = FAR[0], FAR[1]
    k, ko = (FAR[2][0], 128), (FAR[3][0], 128)
    assert refused(n, q, (k[0], 256), k, ko)          # q_out over k
    assert refused(n, q, qo, k, (q[0], 128))          # k_out over q
    assert refused(n, q, qo, k, (qo[0], 128))         # one buffer for both
    assert refused(n, q, qo, k, (qo[0] + 256 * n, 128))
    assert refused(n, q, (k[0] + 16, 256), k, ko)
    # an output in place, and the other tensor's output over it
    assert refused(n, q, q, k, (q[0] + 256, 128))
    assert refused(n, q, qo, k, ko, pos=qo[0])
    assert refused(n, q, qo, k, ko, pos=ko[0] + 256 * n - 4)
    assert refused(n, q, qo, k, ko, pos=qo[0] - 4 * n, axes=2, pos_ld=n)
    assert refused(n, q, q, k, k, pos=q[0] + 4)


def test_slices_of_a_packed_row_are_taken():
    """q|k|v rows of (2 + 1 + 1) x 128 BF16 channels, rotated in place: nothing is refused up to the launch
    (which fails without a device)."""
    ok = [kvq.KVQ_OK, kvq.KVQ_E_CUDA]
    q, k = (BASE, 512), (BASE + 512, 512)
    assert code(7, q, q, k, k) in ok
    assert code(7, q, q, k, (BASE + 768, 512)) == kvq.KVQ_E_INVAL  # (the span of k and k_out)
    assert code(7, FAR[0], (BASE + (3 << 24), 512), KFAR, (BASE + (3 << 24) + 512, 512)) in ok
    assert code(7, FAR[0], (BASE + (3 << 24), 512), KFAR, (BASE + (3 << 24) + 496, 512)) == kvq.KVQ_E_INVAL
    assert code(7, FAR[0], (BASE + (3 << 24), 512), KFAR, (BASE + (3 << 24) + 784, 512)) == kvq.KVQ_E_INVAL
    assert code(1, FAR[0], FAR[1], KFAR, (FAR[1][0] + 512, 128)) in ok      # neighbours
    assert code(1, FAR[0], FAR[1], KFAR, (FAR[1][0] - 256, 128)) in ok


def test_against_every_byte():
    """The rule against the bytes themselves, for small rows of one stride and of several."""
    at = BASE + (1 << 26)
    for n, stride, shift in itertools.product((1, 2, 3), (256, 384, 512), range(-1200, 1216, 48)):
        qo, ko = (at, stride), (at + 16 * (shift // 16) * 2, stride)
        a = {qo[0] + 2 * stride * i + j for i in range(n) for j in range(512)}
        b = {ko[0] + 2 * stride * i + j for i in range(n) for j in range(256)}
        got = code(n, FAR[0], qo, KFAR, ko)
        assert (got == kvq.KVQ_E_INVAL) == bool(a & b), (n, stride, shift)
