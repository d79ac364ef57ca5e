"""A cache that lives until the interpreter ends is destroyed without an error message."""
import os
import subprocess
import sys

import pytest

from bit_kv_cache_17_b200 import kvq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_destroyed_without_the_modules_names(monkeypatch):
    c = object.__new__(kvq.KVCache)
    c.handle = 16  # no cache: only handed on
    calls = []
    for name in ("kvq_cache_destroy", "_lib"):
        monkeypatch.setattr(kvq, name, None)
    kvq.KVCache.__del__(c, calls.append)
    assert calls == [16] and c.handle is None


@pytest.mark.gpu
def test_a_program_ends_quietly():
    code = "from bit_kv_cache_17_b200 import kvq\nc = kvq.KVCache(n_kv_heads=1, max_ctx=64)\nd = [c]; d.append(d)\nprint('ok')\n"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok" and "Exception ignored" not in r.stderr, r.stderr
