"""The build of the library and of the native call beside it: neither waits for what only the other one needs.
Compilers are stood in for."""
import os

import pytest
import torch

from block_eigenbasis_preconditioning_gb300 import binding, build


@pytest.fixture
def folder(tmp_path, monkeypatch):
    """An empty build folder, and the commands that would run in it."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    for name, file in (("LIB", "libdobb.so"), ("CALL", "_lm_call.so"), ("CALL_FOR", "_lm_call.for")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    ran = []

    def run(cmd, what):
        ran.append(what)
        open(cmd[cmd.index("-o") + 1], "w").close()

    def compile_one(nvcc, src, extra):
        ran.append(os.path.basename(src))
        return src
    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "_compile", compile_one)
    return ran


CALL = ["g++ lm_call.cpp", "link of _lm_call.so"]


def test_both_are_built_once(folder):
    assert build.build() == build.LIB and os.path.exists(build.LIB) and os.path.exists(build.CALL)
    assert sorted(folder) == sorted([os.path.basename(s) for s in build.sources()] + ["link"] + CALL)
    assert folder.index("link") < folder.index(CALL[1])
    folder.clear()
    assert build.build() == build.build_library() == build.LIB and build.build_call() == build.CALL and folder == []


def test_the_library_alone_needs_no_headers(folder, monkeypatch, tmp_path, capsys):
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "nowhere")})
    assert build.build_library() == build.LIB and not set(folder) & set(CALL)
    assert build.build(force=True) == build.LIB and not set(folder) & set(CALL) and "left out" in capsys.readouterr().out
    with pytest.raises(build.NoHeaders, match="Python.h"):
        build.build_call()
    # a module that was built before the headers went away does not make the library stale
    folder.clear()
    assert build.build() == build.LIB and folder == []


def test_calls_without_the_native_module(monkeypatch):
    def none(*args):
        raise build.NoHeaders("Python.h does not exist")
    monkeypatch.setattr(build, "build_call", none)
    monkeypatch.setattr(binding, "_CALL", None)
    with pytest.warns(RuntimeWarning, match="Python.h"):
        call = binding.load_call()
    x = torch.zeros(3, 4)
    assert call.layer_norm(x, None, None, 1e-5, None) is None and call.sample() is None and binding.load_call() is call
    with pytest.raises(ValueError, match="CUDA device"):  # (the interpreter's way speaks)
        from block_eigenbasis_preconditioning_gb300 import layer_norm
        layer_norm(x)


def test_another_pytorch_or_python_compiles_the_call_again(folder, monkeypatch):
    build.build()
    folder.clear()
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert build.build_library() == build.LIB and folder == []
    assert build.build_call() == build.CALL and folder == CALL
    folder.clear()
    assert build.build_call() == build.CALL and folder == []
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399")
    assert build.build() == build.LIB and folder == CALL
    folder.clear()
    os.remove(build.CALL_FOR)  # built by whoever kept no note of it
    assert build.build() == build.LIB and folder == CALL


def test_newer_sources(folder):
    build.build()
    folder.clear()
    now = os.path.getmtime(build.LIB)
    stale = lambda *files: [os.utime(f, (now - 10 ** 9, now - 10 ** 9)) for f in files]  # noqa: E731
    stale(build.CALL)
    assert build.build() == build.LIB and folder == CALL
    folder.clear()
    stale(build.LIB)
    assert build.build() == build.LIB and "link" in folder and not set(folder) & set(CALL)
    folder.clear()
    assert build.build(force=True) == build.LIB and set(CALL) < set(folder)


def test_a_compiler_that_fails_is_an_error(folder, monkeypatch):
    def run(cmd, what):
        if what == CALL[0]:
            raise RuntimeError("g++ lm_call.cpp failed")
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(build, "_run", run)
    with pytest.raises(RuntimeError, match="lm_call"):
        build.build()
    assert os.path.exists(build.LIB)  # (the library is there)


def test_a_pytorch_without_cuda(folder, monkeypatch, capsys):
    monkeypatch.setattr(torch.version, "cuda", None)
    assert build.build() == build.LIB and not set(folder) & set(CALL) and "without CUDA" in capsys.readouterr().out
