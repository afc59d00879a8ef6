"""When build() makes `_operators.so` anew: besides newer sources, after a change of Python or torch, whose binary
interfaces the module is built against (it would fail to load, or worse)."""
import os

import self_speculation_b200 as nb
from self_speculation_b200 import build as b


def test_operators_module_says_what_it_was_built_for():
    assert nb._native().__doc__ == b.operators_built_for()


def test_operators_are_rebuilt_for_another_torch_or_python(tmp_path, monkeypatch):
    source, built = tmp_path / "source", tmp_path / "built"
    source.write_text("")
    assert b._operators_stale(str(built), [str(source)])
    built.write_bytes(b"\x7fELF" + b.operators_built_for().encode() + b"\0")
    os.utime(source, (1, 1))
    assert not b._operators_stale(str(built), [str(source)])
    now = b.operators_built_for()
    monkeypatch.setattr(b.importlib.metadata, "version", lambda name: "1.0")
    assert b.operators_built_for() != now and b._operators_stale(str(built), [str(source)])
    monkeypatch.undo()
    monkeypatch.setattr(b.sysconfig, "get_config_var", lambda name: "cpython-399")
    assert b._operators_stale(str(built), [str(source)])
