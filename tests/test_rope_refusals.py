"""What kvq_rope refuses, checked on the host before any launch (no device needed)."""
import ctypes as C

import pytest

from bit_kv_cache_17_b200 import kvq

GOOD = dict(rot_dim=128, n_axes=2, sections=[32, 32, 0, 0], theta=1e4)


def call(params, n=4, pos=16, pos_ld=4, hq=2, q=256, qt=1, q_ld=256, qo=1 << 20, qot=1, qo_ld=256, hk=0, k=0, k_ld=0,
         ko=0, ko_ld=0, freq=None):
    kvq.kvq_rope(kvq.kvq_rope_default_params(**params), freq, n, pos, pos_ld, hq, q, qt, q_ld, qo, qot, qo_ld, hk, k,
                 k_ld, ko, ko_ld, 0)


@pytest.mark.parametrize("change", [
    dict(rot_dim=127), dict(rot_dim=130), dict(rot_dim=0), dict(n_axes=0), dict(n_axes=5), dict(sections=[32, 31, 0, 0]),
    dict(sections=[65, -1, 0, 0]), dict(turns=2), dict(adjacent=-1), dict(inverse=3), dict(theta=0.0),
    dict(theta=float("nan")), dict(theta=float("inf")),
])
def test_parameters(change):
    with pytest.raises(kvq.KVQError) as e:
        call({**GOOD, **change})
    assert e.value.code == kvq.KVQ_E_INVAL


@pytest.mark.parametrize("change,code", [
    (dict(n=-1), kvq.KVQ_E_INVAL), (dict(hq=-1), kvq.KVQ_E_INVAL), (dict(pos=0), kvq.KVQ_E_INVAL),
    (dict(pos_ld=3), kvq.KVQ_E_INVAL), (dict(pos=18), kvq.KVQ_E_ALIGN), (dict(q=0), kvq.KVQ_E_INVAL),
    (dict(qo=0), kvq.KVQ_E_INVAL), (dict(q=264), kvq.KVQ_E_ALIGN), (dict(q_ld=255), kvq.KVQ_E_INVAL),
    (dict(q_ld=257), kvq.KVQ_E_ALIGN), (dict(qo_ld=128), kvq.KVQ_E_INVAL), (dict(qt=3), kvq.KVQ_E_UNSUPPORTED),
    (dict(qot=-1), kvq.KVQ_E_UNSUPPORTED),
    (dict(qo=512), kvq.KVQ_E_INVAL),                 # overlaps the input without being it
    (dict(qo=256, qot=0), kvq.KVQ_E_INVAL),          # the same place in another type
    (dict(qo=256, qo_ld=512), kvq.KVQ_E_INVAL),      # the same place at another stride
    (dict(hk=1, k=0, ko=16, k_ld=128, ko_ld=128), kvq.KVQ_E_INVAL),
    (dict(hk=1, k=1 << 24, ko=(1 << 25) + 8, k_ld=128, ko_ld=128), kvq.KVQ_E_ALIGN),
    (dict(q_ld=1 << 61), kvq.KVQ_E_INVAL), (dict(n=1 << 31, pos_ld=1 << 31), kvq.KVQ_E_INVAL),
])
def test_rows(change, code):
    with pytest.raises(kvq.KVQError) as e:
        call(GOOD, **change)
    assert e.value.code == code


def test_nothing_to_do_looks_at_no_pointer():
    call(GOOD, n=0, pos=0, q=0, qo=0)
    call(GOOD, hq=0, pos=0, q=0, qo=0)
    freq = (C.c_double * 64)(*([1.0] * 64))
    call({**GOOD, "theta": 0.0}, n=0, freq=freq)  # theta is not looked at beside given frequencies


def test_binding_refuses():
    import torch as t

    with pytest.raises(kvq.KVQError):
        kvq.Rope((32, 31), rot_dim=128)
    with pytest.raises(kvq.KVQError):
        kvq.Rope((8, 8, 8, 8, 8))
    with pytest.raises(kvq.KVQError):
        kvq.Rope((64,), inv_freq=[1.0] * 63)
    r = kvq.Rope((64,))
    pos = t.arange(3, dtype=t.int32)
    for bad in (pos.long(), pos[None].expand(2, 3), pos):  # type, axes, a host tensor
        with pytest.raises(kvq.KVQError):
            r.apply(bad, q=t.zeros(3, 1, 128))


@pytest.mark.parametrize("n", [1, 5])
@pytest.mark.parametrize("expanded", [False, True])
def test_the_stride_of_the_positions_is_passed_as_it_is(monkeypatch, n, expanded):
    """One row expanded over the axes has stride 0: any other number would be read past its end."""
    import types

    import torch as t

    class OnDevice(t.Tensor):
        def get_device(self):
            return 0

    rope, calls = kvq.Rope((16, 24, 24)), []
    rope.torch = types.SimpleNamespace(cuda=types.SimpleNamespace(current_device=lambda: 0), int32=t.int32,
                                       empty_like=t.empty_like, contiguous_format=t.contiguous_format)
    rope._raw_stream = lambda index: 0
    monkeypatch.setattr(kvq, "_lib", types.SimpleNamespace(kvq_rope=lambda *a: calls.append(a) or 0))
    row = t.arange(n, dtype=t.int32)
    pos = (row.expand(3, n) if expanded else row.repeat(3, 1)).as_subclass(OnDevice)
    rope.apply(pos, q=t.zeros(n, 2, 128).as_subclass(OnDevice))
    assert calls[0][3] == pos.data_ptr() and calls[0][4] == (0 if expanded else n)


def test_null_handles_are_refused():
    L = kvq._lib
    n = C.c_size_t()
    ids = (C.c_int32 * 1)(0)
    assert L.kvq_batch_workspace_bytes(None, 0, 1, ids, ids, 8, C.byref(n)) == kvq.KVQ_E_INVAL
    assert L.kvq_batch_attn(None, 0, 1, ids, ids, 8, 0, None, 0.0, None, None, None, 0, None) == kvq.KVQ_E_INVAL
    assert L.kvq_attn_mass(None, 0, 1, ids, ids, 8, 0, None, 0.0, None, 1.0, None, None, 0, None, 0,
                           None) == kvq.KVQ_E_INVAL
    assert L.kvq_evict_workspace_bytes(None, None, 1, 8, C.byref(n)) == kvq.KVQ_E_INVAL
    assert L.kvq_evict(None, 0, None, 0, 1, ids, ids, None, 0, 8, 0, 0, None, None, 0, None, 0,
                       None) == kvq.KVQ_E_INVAL
