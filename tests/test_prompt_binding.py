"""The binding of the prompt operators on the host: what it passes on and refuses (no device needed)."""
import types

import pytest

from bit_kv_cache_17_b200 import kvq


def bare_cache():
    """A KVCache without its handle and storage"""
    import torch as t

    c = object.__new__(kvq.KVCache)
    c.torch, c.handle, c._index = t, None, 0
    c.storage = t.zeros(1, dtype=t.uint8)
    c._size = kvq._sz()  # one cell for all calls, which none may use
    c._size_ref = kvq.C.byref(c._size)
    return c


def test_calls_that_overlap_size_their_own_workspaces(monkeypatch):
    """The library runs without the interpreter's lock, so another thread's call may come between
    the size and its use: here it comes from inside the first one."""
    c, sizes = bare_cache(), [(128, True), (4096, False)]

    def workspace_bytes(h, layer, n, ids, nq, hq, out):
        size, again = sizes.pop(0)
        out._obj.value = size
        if again:
            assert c._batch_workspace(0, 1, None, None, 8)[2] == 4096
        return 0

    monkeypatch.setattr(kvq, "_lib", types.SimpleNamespace(kvq_batch_workspace_bytes=workspace_bytes))
    ws, ptr, nb = c._batch_workspace(0, 1, None, None, 8)
    assert nb == 128 and ws.numel() == 128 and ptr == ws.data_ptr()


def test_a_stream_of_another_device_is_refused():
    import torch as t

    stream = types.SimpleNamespace(device=t.device("cuda", 1))
    with pytest.raises(kvq.KVQError):
        kvq._On(t, t.device("cuda", 0), stream)
    assert len(kvq._On(t, t.device("cuda", 1), None).both) == 1
