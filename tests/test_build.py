"""The build where there is no torch: the library alone, for C programs."""
import importlib.util
import subprocess

from kv_cache_compression_cas_b200 import build


def test_without_torch_the_library_alone_is_built(monkeypatch, tmp_path):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(build, "CALL", str(tmp_path / "_paged_call.so"))
    monkeypatch.setattr(subprocess, "run", lambda *a, **k: (_ for _ in ()).throw(AssertionError("no compiler is called")))
    assert build.build_call() is None
    assert not (tmp_path / "_paged_call.so").exists()
