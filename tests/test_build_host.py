"""CPU test of the build: the C ABI's library does not depend on the binding's."""
import types

import pytest

from rotation_then_quantize_amd import _build


def test_library_is_built_where_the_binding_is_not(tmp_path, monkeypatch):
    def link(cmd, **_):
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    def no_binding():
        raise RuntimeError("host compiler failed for bind.cpp")

    monkeypatch.setattr(_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "librtq.so"))
    monkeypatch.setattr(_build, "_compile", lambda src: src)
    monkeypatch.setattr(_build, "_build_native", no_binding)
    monkeypatch.setattr(_build.subprocess, "run", link)
    with pytest.raises(RuntimeError, match="bind.cpp"):          # it is still an error ...
        _build.build()
    assert (tmp_path / "librtq.so").exists()                     # ... but the library is there
