"""The torch-tensor forms beside torch itself."""
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import tile_hierarchy_linear_amd as thl

PKG = os.path.dirname(os.path.abspath(thl.__file__))


def _calls(device):
    """One call of every form: its function, its tensors by name, its other arguments, and the names it writes."""
    f, i, u = torch.float32, torch.int32, torch.uint8

    def t(*shape, dtype=f):
        return torch.zeros(*shape, dtype=dtype, device=device)

    places = torch.arange(8, dtype=i, device=device).reshape(4, 2)
    return {
        "rmsnorm": (thl.rmsnorm, dict(x=t(4, 64), w=t(64), y=t(4, 64), residual=t(4, 64), residual_out=t(4, 64)), {},
                    ("y", "residual_out")),
        "rmsnorm_mx": (thl.rmsnorm, dict(x=t(4, 64), w=t(64), y=t(4, 64, dtype=torch.float8_e4m3fn),
                                         sf=t(4, 16, dtype=u)), {}, ("y", "sf")),
        "rmsnorm_backward": (thl.rmsnorm_backward, dict(s=t(4, 64), dy=t(4, 64), w=t(64), dx=t(4, 64), dw=t(64),
                                                        dres=t(4, 64)), {}, ("dx", "dw")),
        "moe_sort": (thl.moe_sort, dict(ids=t(4, 2, dtype=i), rows=t(4, 2, dtype=i), offsets=t(6, dtype=i),
                                        order=t(8, dtype=i)), dict(experts=5), ("rows", "offsets", "order")),
        "moe_gather": (thl.moe_gather, dict(x=t(4, 64), rows=places, y=t(8, 64)), {}, ("y",)),
        "moe_gather_mx": (thl.moe_gather, dict(x=t(4, 64, dtype=u), rows=places, y=t(8, 64, dtype=u),
                                               sf=t(4, 16, dtype=u), sf_y=t(8, 16, dtype=u)), {}, ("y", "sf_y")),
        "moe_combine": (thl.moe_combine, dict(x=t(8, 64), rows=places, y=t(4, 64), weights=t(4, 2)), {},
                        ("y",)),
        "moe_combine_backward": (thl.moe_combine_backward,
                                 dict(dy=t(4, 64), x=t(8, 64), rows=places, weights=t(4, 2), dx=t(8, 64),
                                      dweights=t(4, 2)), {}, ("dx", "dweights")),
        "gemm_w4": (thl.gemm_w4, dict(w=t(32, 64, dtype=u), x=t(3, 128, dtype=torch.float16), d=t(3, 32),
                                      scales=t(32, 1, dtype=torch.float16), zeros=t(32, 1, dtype=u), c=t(3, 32),
                                      bias=t(32)), dict(group=128, beta=1.0), ("d",)),
    }


FORMS = ["rmsnorm", "rmsnorm_mx", "rmsnorm_backward", "moe_sort", "moe_gather", "moe_gather_mx", "moe_combine",
         "moe_combine_backward", "gemm_w4"]


# ------------------------------------------------------------------ autograd

def _floats(form, device):
    return [k for k, v in _calls(device)[form][1].items() if v.dtype in (torch.float32, torch.float16)]


def _refused_where_recorded(form, device, names):
    for name in names:
        call, tensors, rest, _ = _calls(device)[form]
        tensors[name].requires_grad_()
        with pytest.raises(ValueError, match=f"{name}: requires a gradient"):
            call(**tensors, **rest)
        call, tensors, rest, _ = _calls(device)[form]
        with torch.autograd.forward_ad.dual_level():
            tensors[name] = torch.autograd.forward_ad.make_dual(tensors[name], torch.ones_like(tensors[name]))
            with pytest.raises(ValueError, match=f"{name}: requires a gradient"):
                call(**tensors, **rest)


@pytest.mark.parametrize("form,first", [
    ("rmsnorm", "x"), ("rmsnorm", "w"), ("rmsnorm", "y"), ("rmsnorm_backward", "s"), ("rmsnorm_backward", "dy"),
    ("moe_gather", "x"), ("moe_combine", "x"), ("moe_combine_backward", "dy"), ("gemm_w4", "x"), ("gemm_w4", "scales")])
def test_a_tensor_that_requires_a_gradient_is_refused(form, first):
    # (seen before the device, so that it shows without a GPU)
    _refused_where_recorded(form, "cpu", [first])


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
def test_every_tensor_that_requires_a_gradient_is_refused(form):
    _refused_where_recorded(form, "cuda", _floats(form, "cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
def test_such_tensors_are_taken_where_nothing_is_recorded(form):
    call, tensors, rest, written = _calls("cuda")[form]
    for name in _floats(form, "cuda"):
        tensors[name].requires_grad_()
    with torch.no_grad():
        call(**tensors, **rest)
    with torch.inference_mode():
        call(**tensors, **rest)
    torch.cuda.synchronize()


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w):
        y = torch.empty_like(x)
        thl.rmsnorm(x, w, y, eps=1e-5)
        ctx.save_for_backward(x, w)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, w = ctx.saved_tensors
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        thl.rmsnorm_backward(x, dy, w, dx, dw, eps=1e-5)
        return dx, dw


@pytest.mark.gpu
def test_inside_an_autograd_function():
    # fp32 sums of 200 terms: each side within 1e-5 of the gradient's norm
    g = torch.Generator().manual_seed(0)
    x, w, up = torch.randn(30, 200, generator=g), 1 + 0.2 * torch.randn(200, generator=g), torch.randn(30, 200, generator=g)
    X, W = x.double().requires_grad_(), w.double().requires_grad_()
    ((X * torch.rsqrt(X.square().mean(dim=1, keepdim=True) + 1e-5) * W) * up.double()).sum().backward()
    xd, wd = x.cuda().requires_grad_(), w.cuda().requires_grad_()
    (_Norm.apply(xd, wd) * up.cuda()).sum().backward()
    for got, want in ((xd.grad, X.grad), (wd.grad, W.grad)):
        assert float((got.cpu().double() - want).norm()) <= 1e-5 * float(want.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("form", FORMS)
def test_outputs_count_as_written(form):
    call, tensors, rest, written = _calls("cuda")[form]
    before = {k: v._version for k, v in tensors.items()}
    call(**tensors, **rest)
    torch.cuda.synchronize()
    for k, v in tensors.items():
        assert (v._version > before[k]) == (k in written), k


@pytest.mark.gpu
def test_a_saved_tensor_that_is_overwritten_is_noticed():
    p = torch.ones(4, 64, device="cuda", requires_grad=True)
    h, x, w = torch.ones(4, 64, device="cuda"), torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    loss = (p * h).sum()  # keeps h
    thl.rmsnorm(x, w, torch.empty_like(x), residual=h, residual_out=h)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


@pytest.mark.gpu
def test_inference_tensors():
    with torch.inference_mode():
        x, w, y = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda"), torch.empty(4, 64, device="cuda")
        thl.rmsnorm(x, w, y, eps=0.0)
    assert bool((y == 1).all())
    y2 = y.clone()
    thl.rmsnorm(x, w, y, eps=0.0)  # and outside
    torch.cuda.synchronize()
    assert torch.equal(y, y2)


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
