"""What a build needs: the library nothing but hipcc; the binding's compiled step also torch's headers and a host
compiler, without which the library is there all the same.  The compilers are stand-ins that write empty files."""
import importlib.util
import os
import subprocess

import pytest

from tensor_transformer_mlp_02_amd import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build into an empty folder; returns the compilers' command lines and what g++ is to do."""
    ran, gxx = [], {"fails": False}

    def run(cmd, **kw):
        ran.append(cmd)
        host = "marshal.cpp" in " ".join(cmd)
        if host and gxx["fails"]:
            raise subprocess.CalledProcessError(1, cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b, "HERE", str(tmp_path))
    monkeypatch.setattr(b, "OUT", str(tmp_path / "libtpmlp.so"))
    if hasattr(b, "MARSHAL"):
        monkeypatch.setattr(b, "MARSHAL", str(tmp_path / os.path.basename(b.MARSHAL)))
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(b.subprocess, "run", run)
    return tmp_path, ran, gxx


def marshals(path):
    return sorted(p.name for p in path.iterdir() if p.name.startswith("_marshal"))


def test_both_are_built(tree):
    path, ran, _ = tree
    assert b.build() == str(path / "libtpmlp.so") and os.path.exists(path / "libtpmlp.so")
    assert len(marshals(path)) == 1
    assert sum("marshal.cpp" in " ".join(c) for c in ran) == 1


def test_without_torch(tree, monkeypatch, capfd):
    path, _, _ = tree
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else found(name, *a))
    b.build()
    assert os.path.exists(path / "libtpmlp.so") and marshals(path) == []
    assert "torch is not installed" in capfd.readouterr().err


def test_without_a_host_compiler(tree, capfd):
    path, _, gxx = tree
    b.build()
    assert len(marshals(path)) == 1
    gxx["fails"] = True
    b.build()                       # and the one that an earlier build left is taken away
    assert os.path.exists(path / "libtpmlp.so") and marshals(path) == []
    assert "marshal" in capfd.readouterr().err


def test_a_library_that_does_not_compile_is_an_error(tree, monkeypatch):
    def fails(*a):
        raise RuntimeError("hipcc failed")
    monkeypatch.setattr(b, "_compile", fails)
    with pytest.raises(RuntimeError, match="hipcc failed"):
        b.build()


def test_the_compiled_step_is_for_this_python(tree):
    import sysconfig
    path, _, _ = tree
    (path / "_marshal.so").write_text("of an earlier build")
    b.build()
    assert marshals(path) == ["_marshal" + sysconfig.get_config_var("EXT_SUFFIX")]


def test_a_compiled_step_for_another_torch_is_not_used(monkeypatch):
    import types
    torch = pytest.importorskip("torch")
    import tensor_transformer_mlp_02_amd as tp
    ran = []
    fake = types.SimpleNamespace(torch_version="1.0.0", setup=lambda *a: ran.append(a))
    monkeypatch.setattr(tp, "_marshal", fake, raising=False)
    monkeypatch.setattr(tp, "_compiled", None)
    assert tp._marshaller() is False and not ran
    fake.torch_version = torch.__version__.split("+")[0]
    monkeypatch.setattr(tp, "_compiled", None)
    assert tp._marshaller() is fake and ran
