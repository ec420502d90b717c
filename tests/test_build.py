"""The C library is built with or without a torch to bind it to (no GPU needed)."""
import os

import pytest

from compensated_fp32_projection_gb300 import build as b


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of one source file in a folder of its own."""
    one = [os.path.join(b.CSRC, "geglu.cu")]
    monkeypatch.setattr(b, "_sources", lambda: one)
    for name, file in (("BUILD", "objects"), ("LIB", "libcompfp32.so"), ("BINDING", "_attn_binding.so")):
        monkeypatch.setattr(b, name, str(tmp_path / file))
    return tmp_path


@pytest.mark.parametrize("torch", ["none", "without CUDA"])
def test_without_torch(elsewhere, monkeypatch, torch):
    there = elsewhere / "torch"
    (there / "lib").mkdir(parents=True)
    spec = None if torch == "none" else type("Spec", (), {"submodule_search_locations": [str(there)]})
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: spec)
    assert not b.up_to_date()
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.BINDING)
    assert b.up_to_date()


def test_a_binding_that_fails_leaves_the_library(elsewhere, monkeypatch):
    monkeypatch.setenv("CXX", "false")
    monkeypatch.setattr(b, "_torch_dir", lambda: str(elsewhere))
    with pytest.raises(RuntimeError, match="attn_binding"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)
    assert not b.up_to_date()


def test_another_torch_is_seen(elsewhere, monkeypatch):
    """The binding's ABI is its torch's: another version is built for again."""
    made = []
    monkeypatch.setattr(b, "_torch_dir", lambda: str(elsewhere))
    monkeypatch.setattr(b, "_compile_binding", lambda torch: made.append(torch) or "obj")
    monkeypatch.setattr(b.subprocess, "run", lambda cmd, **kw: open(cmd[cmd.index("-o") + 1], "w").close() or type(
        "P", (), {"returncode": 0, "stdout": "", "stderr": ""}))
    (elsewhere / "version.py").write_text("__version__ = '2.9.1+cu130'\n")
    b.build()
    assert b.up_to_date() and len(made) == 1
    (elsewhere / "version.py").write_text("__version__ = '2.11.0+cu130'\n")
    assert not b.up_to_date()
    b.build()
    assert b.up_to_date() and len(made) == 2
