"""The build's order (CPU, no compiler is run): the C library does not wait for the binding,
which needs torch, its headers and a host compiler."""
import os

import pytest

from fp8_rowwise_scaled_amd import build as B


@pytest.fixture
def place(tmp_path, monkeypatch):
    """Outputs under tmp_path, sources without content, and a compiler that only writes its output."""
    for name in ("LIB", "BINDING"):
        monkeypatch.setattr(B, name, str(tmp_path / os.path.basename(getattr(B, name))))
    monkeypatch.setattr(B, "PKG", str(tmp_path))
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(B, "_hipcc", lambda: "hipcc")
    calls = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return Done()
    monkeypatch.setattr(B.subprocess, "run", run)
    return calls


def test_library_is_linked_when_the_binding_cannot_be_compiled(place, monkeypatch):
    def no_torch(obj):
        raise ImportError("No module named 'torch'")
    monkeypatch.setattr(B, "compile_binding", no_torch)
    with pytest.raises(RuntimeError, match="binding.*torch"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.BINDING)


def test_both_are_built(place):
    assert B.build() == B.LIB
    assert os.path.exists(B.LIB) and os.path.exists(B.BINDING)
    outputs = [os.path.basename(c[c.index("-o") + 1]) for c in place]
    assert outputs.index("libfp8gg.so.tmp") < outputs.index("_layer_binding.so.tmp")
    assert {os.path.basename(s) + ".o" for s in B.sources()} <= set(outputs)
