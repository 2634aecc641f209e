"""The build on the CPU: the library is built whatever becomes of the paged
helpers' extension.  (In a folder of its own, with a source of one line.)"""
import ctypes
import os

import pytest

from transformer_scaled_dot_02_gb300 import build as sd_build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    (tmp_path / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (tmp_path / "bind.cpp").write_text("int two() { return 2; }\n")
    for name, value in (("SOURCES", ["one.cu"]), ("HEADERS", []), ("CSRC", str(tmp_path)),
                        ("BUILD_DIR", str(tmp_path / "_build")), ("LIB", str(tmp_path / "libone.so")),
                        ("BIND", str(tmp_path / os.path.basename(sd_build.BIND))),
                        ("BIND_SOURCE", str(tmp_path / "bind.cpp"))):
        monkeypatch.setattr(sd_build, name, value)
    return tmp_path


@pytest.fixture
def torch_dir():
    torch = sd_build._torch_dir()
    if torch is None:
        pytest.skip("no torch for CUDA")
    return torch


@pytest.mark.parametrize("why", ["source", "compiler", "version"])
def test_the_library_is_built_where_the_extension_is_not(tree, torch_dir, why, monkeypatch, capfd):
    if why == "source":
        (tree / "bind.cpp").write_text("#error no\n")
    elif why == "compiler":
        monkeypatch.setenv("CXX", str(tree / "no_such_compiler"))
    else:
        real = open
        monkeypatch.setattr("builtins.open", lambda path, *a, **k: real(
            str(tree / "one.cu") if str(path) == os.path.join(torch_dir, "version.py") else path, *a, **k))
    open(sd_build.BIND, "w").write("an older one")
    os.utime(sd_build.BIND, (1, 1))
    sd_build.build()
    assert ctypes.CDLL(sd_build.LIB).one() == 1
    assert not os.path.exists(sd_build.BIND)
    assert "extension was not built" in capfd.readouterr().err


def test_without_a_torch_the_library_alone_is_built(tree, monkeypatch):
    monkeypatch.setattr(sd_build, "_torch_dir", lambda: None)
    sd_build.build()
    assert ctypes.CDLL(sd_build.LIB).one() == 1 and not os.path.exists(sd_build.BIND)


def test_a_torch_without_cuda_counts_as_none(tmp_path, monkeypatch):
    (tmp_path / "torch").mkdir()
    (tmp_path / "torch" / "__init__.py").write_text("")
    spec = type("spec", (), {"origin": str(tmp_path / "torch" / "__init__.py")})
    monkeypatch.setattr(sd_build.importlib.util, "find_spec", lambda name: spec)
    assert sd_build._torch_dir() is None


def test_the_extension_follows_the_interpreter_and_the_torch(tree, torch_dir, monkeypatch):
    import sysconfig
    assert sd_build.BIND.endswith(sysconfig.get_config_var("EXT_SUFFIX"))

    def rebuilt():
        before = os.stat(sd_build.BIND).st_ino if os.path.exists(sd_build.BIND) else None
        sd_build.build()
        return os.stat(sd_build.BIND).st_ino != before

    assert rebuilt() and not rebuilt()
    monkeypatch.setattr(sd_build, "_torch_version", lambda torch: "0.0.1")
    assert rebuilt() and not rebuilt()          # another torch, though its files are the older ones
    os.remove(sd_build._bind_stamp())
    assert rebuilt() and not rebuilt()


def test_an_extension_of_another_torch_is_not_used(torch_dir, monkeypatch):
    import torch
    import transformer_scaled_dot_02_gb300 as sd
    sd_build.build()
    monkeypatch.setattr(sd, "_bind_module", None)
    assert sd._paged().torch_version == str(torch.__version__)
    monkeypatch.setattr(sd, "_bind_module", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(ImportError, match="built against torch"):
        sd._paged()
