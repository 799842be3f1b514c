"""What is built when, with compilers that only record their command: the library
by itself where there is no torch, the binding again for another torch."""
import os
import sys

import pytest

from dense_gemm_07_gb300 import _build


@pytest.fixture()
def commands(tmp_path, monkeypatch):
    """An empty tree; the commands run since the list was last cleared."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return type("Result", (), dict(returncode=0, stderr=""))()

    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build, "_nvcc", lambda: os.path.join("cuda", "bin", "nvcc"))
    for name, value in (("BUILD_DIR", "b"), ("LIB_DIR", "l"), ("LIB_PATH", "l/libgemm07.so"),
                        ("BINDING_PATH", "l/layer_binding.so"),
                        ("BINDING_STAMP", "b/layer_binding.txt")):
        monkeypatch.setattr(_build, name, str(tmp_path / value))
    return ran


def _compilers(ran):
    return {os.path.basename(c[0]) for c in ran}


def test_the_library_builds_without_torch(commands, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it fails
    assert _build.build() == _build.LIB_PATH
    assert _compilers(commands) == {"nvcc"}
    assert len(commands) == len(_build.sources()) + 1
    assert os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.BINDING_PATH)
    commands.clear()
    _build.build()
    assert not commands
    with pytest.raises(RuntimeError, match="torch"):
        _build.build_binding()


def test_the_binding_is_built_with_the_library_and_again_for_another_torch(commands, monkeypatch):
    pytest.importorskip("torch")
    if _build._torch_dir() is None:
        pytest.skip("torch without CUDA")
    _build.build()
    assert _compilers(commands) == {"nvcc", "g++"}
    assert os.path.exists(_build.LIB_PATH) and os.path.exists(_build.BINDING_PATH)
    commands.clear()
    _build.build()
    _build.build_binding()
    assert not commands
    for change in (("_torch_version", lambda d: "another"), ("_torch_dir", lambda: str(os.sep))):
        monkeypatch.setattr(_build, *change)
        _build.build()
        assert _compilers(commands) == {"g++"} and len(commands) == 2  # compiled and linked
        commands.clear()
        _build.build_binding()
        assert not commands


def test_the_ctypes_layer_asks_for_the_library_alone(commands):
    from dense_gemm_07_gb300 import _abi
    loaded, _abi._lib = _abi._lib, None
    try:
        with pytest.raises(RuntimeError, match="could not be loaded"):  # an empty file
            _abi.lib()
    finally:
        _abi._lib = loaded
    assert _compilers(commands) == {"nvcc"} and os.path.exists(_build.LIB_PATH)
