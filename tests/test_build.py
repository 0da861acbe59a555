"""The build on the CPU: the library does not hang on its Python extension, and an
extension of another PyTorch or Python is neither kept nor loaded."""
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

from paged_kv_cache_276_gb300 import build, native


@pytest.fixture
def scratch(tmp_path, monkeypatch):
    """A build folder of its own, in which every source compiles to an empty object."""
    def empty_object(src):
        obj = str(tmp_path / (src + ".o"))
        subprocess.run(["g++", "-c", "-x", "c++", "-fPIC", "/dev/null", "-o", obj], check=True)
        return obj

    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libpkv.so"))
    monkeypatch.setattr(build, "_compile", empty_object)
    return tmp_path


@pytest.mark.parametrize("error", [subprocess.CalledProcessError(1, "g++"), FileNotFoundError("g++"), RuntimeError("nvcc")])
def test_the_library_is_built_where_the_extension_cannot_be(scratch, monkeypatch, error):
    calls = []

    def no_headers():
        calls.append(1)
        raise error

    monkeypatch.setattr(build, "_compile_bind", no_headers)
    monkeypatch.setattr(native, "bind_path", lambda: str(scratch / "_bind.so"))
    monkeypatch.setattr(build, "_bind_failed", False)
    with pytest.warns(UserWarning, match="Python extension"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(native.bind_path())
    assert build.build() == build.LIB and len(calls) == 1  # one try in a process
    monkeypatch.setattr(native, "_bind_module", None)
    with pytest.raises(RuntimeError, match="is missing"):
        native._bind()


def test_an_extension_of_another_torch_or_python_does_not_count(monkeypatch):
    build.build()
    assert build.up_to_date()
    monkeypatch.setattr(native, "_bind_module", None)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1+other")
        assert not build.up_to_date()
        with pytest.raises(RuntimeError, match="is missing"):
            native._bind()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: ".cpython-300-other.so")
        assert not build.up_to_date()
    assert build.up_to_date() and native._bind() is not None


@pytest.mark.parametrize("torch_there", [True, False])
def test_the_build_runs_as_a_script_and_without_torch(tmp_path, torch_there):
    build.build()
    if not torch_there:
        (tmp_path / "torch.py").write_text("raise ImportError('no torch here')\n")
    done = subprocess.run([sys.executable, build.__file__], cwd=tmp_path, capture_output=True, text=True,
                          env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert done.returncode == 0, done.stderr
    assert done.stdout.strip() == build.LIB
    assert ("Python extension" in done.stderr) is not torch_there
