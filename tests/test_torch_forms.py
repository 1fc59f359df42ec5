"""The torch-tensor forms beside torch itself."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import tile_hierarchy_linear_amd as thl

PKG = os.path.dirname(os.path.abspath(thl.__file__))


# ------------------------------------------------------------------ out of memory

@pytest.mark.gpu
def test_a_workspace_that_does_not_fit_raises_torch_s_error():
    m = 1 << 24
    s, dy, dx = (torch.zeros(8, m, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    w, dw = torch.ones(m, device="cuda"), torch.zeros(m, device="cuda")
    assert thl.thl_rmsnorm_backward_workspace(m, 8) == 8 * m * 4
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (64 << 20)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            thl.rmsnorm_backward(s, dy, w, dx, dw)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    thl.rmsnorm_backward(s, dy, w, dx, dw)  # and goes on
    torch.cuda.synchronize()
    assert not bool(dw.any())


# ------------------------------------------------------------------ a torch without the host module

def _package_without_the_module(tmp_path):
    """A copy of the package (its library linked) that has no _torch_ops.so."""
    pkg = tmp_path / "tile_hierarchy_linear_amd"
    pkg.mkdir()
    for name in os.listdir(PKG):
        if name.endswith(".py") or name == "libthl.so":
            os.symlink(os.path.join(PKG, name), pkg / name)
    return pkg


_USE = """
import tile_hierarchy_linear_amd as thl
assert thl.__file__.startswith({root!r}), thl.__file__
assert thl.thl_status_string(0) and thl.thl_variant_count() > 0
assert thl.thl_rmsnorm(0, 0, None, 1, None, 1, None, 1, None, 1e-6, 1.0, None, 1, None, 1,
                       thl.thl_norm_types(0, 0, 0, 0)) == 0
try:
    thl.rmsnorm(None, None, None)
except ImportError as e:
    assert "_torch_ops" in str(e), e
else:
    raise AssertionError("rmsnorm took its arguments")
print("done")
"""


@pytest.mark.parametrize("broken", ["absent", "another"])
def test_the_library_loads_without_the_torch_forms(tmp_path, broken):
    pkg = _package_without_the_module(tmp_path)
    if broken == "another":  # one that this torch cannot load
        (pkg / "_torch_ops.so").write_bytes(b"no library")
    # run from a path-loaded copy: the C binding works, a torch form says what it misses
    code = f"import sys; sys.path.insert(0, {str(tmp_path)!r})\n" + _USE.format(root=str(tmp_path))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=tmp_path, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), r.stderr


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


@pytest.mark.parametrize("symbol", ["PyModule_Create2", "thl_not_a_symbol_of_torch"])
def test_build_fails_where_the_module_would_not_load(tmp_path, monkeypatch, symbol):
    from tile_hierarchy_linear_amd import build

    (tmp_path / "torch_ops.cpp").write_text(f'extern "C" void {symbol}(); extern "C" void use() {{ {symbol}(); }}\n')
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build, "TORCH_OPS", str(tmp_path / "_torch_ops.so"))
    if symbol.startswith("thl"):
        with pytest.raises(subprocess.CalledProcessError):
            build.build_torch_ops()
    else:
        build.build_torch_ops()
    assert os.path.exists(tmp_path / "_torch_ops.so") == (not symbol.startswith("thl"))


def test_a_module_for_another_torch_goes(tmp_path, monkeypatch):
    from importlib.machinery import ModuleSpec

    from tile_hierarchy_linear_amd import build

    spec = ModuleSpec("torch", None, is_package=True)
    spec.submodule_search_locations = [str(tmp_path / "torch")]
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: spec)
    monkeypatch.setattr(build, "TORCH_OPS", str(tmp_path / "_torch_ops.so"))
    (tmp_path / "_torch_ops.so").write_bytes(b"built with a HIP torch")
    build.build_torch_ops()
    assert not os.path.exists(tmp_path / "_torch_ops.so")
