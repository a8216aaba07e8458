"""The build's two parts (no GPU): the C library, which needs nvcc alone, and the native part of the Python binding. What
the second lacks does not keep the first from being made, and it is made again for another torch or interpreter."""
import importlib.util
import os
import shutil

import pytest

import fp8_block_scaled_quant_gb300 as fb

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build module with one small source, making its files in a folder of its own."""
    if not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")):
        pytest.skip("nvcc not available")
    spec = importlib.util.spec_from_file_location("own_build", os.path.join(os.path.dirname(fb.lib_path()), "_build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(m, "sources", lambda: [str(src)])
    for name, path in (("LIB", "lib.so"), ("BIND", "bind.so"), ("BUILD", "build"), ("BIND_FOR", "build/bind.for")):
        monkeypatch.setattr(m, name, str(tmp_path / path))
    return m


@pytest.mark.parametrize("compiler", [["false"], ["/nonexistent/g++"]])
def test_the_library_is_there_where_the_binding_fails(build, monkeypatch, compiler):
    monkeypatch.setattr(build, "bind_command", lambda out: compiler)
    with pytest.raises(RuntimeError) as e:
        build.build()
    assert type(e.value).__name__ == "BindError"
    assert os.path.exists(build.LIB) and not os.path.exists(build.BIND)


def test_the_library_without_torch(build, monkeypatch):
    def gone(*a):
        raise ImportError("No module named torch")

    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(build, "bind_command", gone)
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BIND)


def test_the_binding_follows_torch_and_python(build, monkeypatch):
    made = []
    monkeypatch.setattr(build, "bind_command", lambda out: made.append(out) or ["touch", out])
    build.build()
    build.build()
    assert len(made) == 1 and os.path.exists(build.BIND)
    monkeypatch.setattr(build, "bind_for", lambda: "another torch")
    build.build()
    build.build()
    assert len(made) == 2


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    from fp8_block_scaled_quant_gb300 import _build
    _build.build()
    monkeypatch.setattr(fb, "_bind", None)
    monkeypatch.setattr(_build, "bind_for", lambda: "another torch")
    with pytest.raises(fb.Fp8BlkError, match="another torch"):
        fb._native()
