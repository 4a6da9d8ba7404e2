"""What build() makes: the library whether or not the part of the binding that needs torch can be made, and that part for
the interpreter and the torch that load it."""
import importlib.util
import os
import stat
import sysconfig

import pytest

torch = pytest.importorskip("torch")

COMPILER = """#!/bin/sh
# stands for a compiler: makes the file behind -o, or fails
[ -e "%s" ] && { echo no >&2; exit 1; }
while [ $# -gt 0 ]; do
  if [ "$1" = -o ]; then echo x > "$2"; fi
  shift
done
"""


@pytest.fixture
def b(tmp_path, monkeypatch):
    """build.py with a folder of its own and compilers that take no time; fail(name) makes one fail."""
    from causal_gqa_attention_flashattention_gb300 import build
    spec = importlib.util.spec_from_file_location("build_of_its_own", build.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.BUILD = str(tmp_path / "_build")
    m.LIB = os.path.join(m.BUILD, "libneattn.so")
    for name in ("nvcc", "g++"):
        f = tmp_path / name
        f.write_text(COMPILER % (tmp_path / (name + ".fails")))
        f.chmod(f.stat().st_mode | stat.S_IXUSR)
    m.NVCC = str(tmp_path / "nvcc")
    monkeypatch.setenv("PATH", str(tmp_path) + os.pathsep + os.environ["PATH"])
    m.fail = lambda name, on=True: (tmp_path / (name + ".fails")).write_text("") if on else (tmp_path / (name + ".fails")).unlink()
    return m


def made(b):
    return sorted(f for f in os.listdir(b.BUILD) if f.endswith(".so"))


def test_both(b):
    assert b.build() == b.LIB
    assert made(b) == sorted(["libneattn.so", os.path.basename(b.bind_path())])
    b.fail("nvcc"), b.fail("g++")
    b.build()  # all is new: nothing is compiled
    with pytest.raises(RuntimeError):
        b.build(force=True)


def test_library_without_torch(b, monkeypatch, capfd):
    monkeypatch.setitem(__import__("sys").modules, "torch", None)
    assert b.build() == b.LIB and made(b) == ["libneattn.so"]
    assert "torch" in capfd.readouterr().err


def test_library_where_the_binding_does_not_compile(b):
    b.fail("g++")
    with pytest.raises(RuntimeError, match="bind.cpp"):
        b.build()
    assert made(b) == ["libneattn.so"]
    b.fail("g++", False), b.fail("nvcc")
    b.build()  # only what is missing
    assert len(made(b)) == 2


def test_binding_of_another_torch_or_python(b, monkeypatch):
    b.build()
    first = b.bind_path()
    monkeypatch.setattr(torch, "__version__", "0.1+other")
    second = b.bind_path()
    assert second != first and not os.path.exists(second)
    b.fail("nvcc")  # the library stays
    b.build()
    assert os.path.exists(second)
    get = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: ".other.so" if name == "EXT_SUFFIX" else get(name))
    b.build()
    assert len({first, second, b.bind_path()}) == 3 and os.path.exists(b.bind_path())


def test_the_binding_loads_what_is_built():
    from causal_gqa_attention_flashattention_gb300 import binding, build
    assert binding.BIND_PATH == build.bind_path() and torch.__version__ in binding.BIND_PATH
