"""The torch-tensor forms beside torch itself."""
import subprocess

import pytest

torch = pytest.importorskip("torch")


# ------------------------------------------------------------------ a torch without the host module

def test_build_without_torch_s_hip_libraries(tmp_path, monkeypatch):
    from importlib.machinery import ModuleSpec

    from tile_hierarchy_linear_amd import build

    lib = tmp_path / "torch" / "lib"
    lib.mkdir(parents=True)
    (lib / "libc10.so").write_bytes(b"")
    spec = ModuleSpec("torch", None, is_package=True)
    spec.submodule_search_locations = [str(tmp_path / "torch")]
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: spec)
    monkeypatch.setattr(build, "TORCH_OPS", str(tmp_path / "_torch_ops.so"))
    started = []

    def check_call(cmd, **kw):
        started.append(cmd)
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(build.subprocess, "check_call", check_call)
    build.build_torch_ops()  # a CPU-only torch: nothing to build, no error
    assert not started
    (lib / "libc10_hip.so").write_bytes(b"")
    with pytest.raises(subprocess.CalledProcessError):
        build.build_torch_ops()  # with them it is built, and a failure is one
    assert len(started) == 1
