"""The smoke entry reaches the library's operators (one that it leaves out could
be broken by a build without its noticing)."""
import pytest

import __graft_entry__ as entry
import paged_kv_cache_67_gb300 as pkv

pytestmark = pytest.mark.gpu


def test_smoke_reaches_every_operator(monkeypatch):
    names = ("pkv_write", "pkv_decode_attention", "pkv_write_decode_attention", "pkv_build_step", "pkv_rope_write",
             "pkv_chunk_attention")
    calls = dict.fromkeys(names, 0)

    def counted(name, fn):
        def call(*args, **kwargs):
            calls[name] += 1
            return fn(*args, **kwargs)
        return call

    for name in names:
        monkeypatch.setattr(pkv, name, counted(name, getattr(pkv, name)))
    entry.smoke()
    assert all(calls.values()), calls
