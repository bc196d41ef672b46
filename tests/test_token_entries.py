"""The token operators' Python entry points: what they do around a call, without a GPU."""
import os
import re

import pytest
import torch

import routed_expert_ffn_route_gb300 as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "routed_expert_ffn_route_gb300")


@pytest.fixture(scope="module")
def native():
    moe.build()
    moe.lib()
    from routed_expert_ffn_route_gb300 import _tokens_native
    return _tokens_native


class Stream:
    def __init__(self, handle, device):
        self.cuda_stream, self.device_index = handle, device


# -------------------------------------------------------------------- device and stream
@pytest.mark.parametrize("dev", [0, 1, 7])
def test_a_call_runs_with_its_operands_device_current(native, dev):
    """A default stream's handle is 0 on every device: the device has to be current."""
    assert native.trace(dev, None) == [f"current stream of {dev}", f"set {dev}", "call on 0",
                                       "restore"]
    assert native.trace(dev, Stream(0, dev)) == [f"set {dev}", "call on 0", "restore"]
    assert native.trace(dev, Stream(4096, dev)) == [f"set {dev}", "call on 4096", "restore"]


def test_a_stream_of_another_device_is_refused(native):
    for on, dev in [(0, 1), (1, 0)]:
        with pytest.raises(ValueError, match="device"):
            native.trace(dev, Stream(0, on))
    with pytest.raises(ValueError, match="CUDA device"):
        native.trace(-1, None)
    with pytest.raises(AttributeError):
        native.trace(0, object())


def test_every_entry_point_calls_through_the_device_guard():
    """Each C call of the extension module stands in the one function that sets the device."""
    with open(os.path.join(PKG, "csrc", "tokens_py.cpp")) as f:
        src = f.read()
    calls = re.findall(r"return (moe_\w+)\(", src)
    launched = re.findall(r"c\.launch\(a\[\d+\], \[&\]\(void \*st\) \{\s*return (moe_\w+)\(", src)
    assert sorted(calls) == sorted(launched) and len(calls) == 7
    assert "on_device<Cuda>" in src and "c10::cuda::OptionalCUDAGuard g;" in src


def test_a_torch_stream_says_its_device():
    """handle() reads these two attributes of torch.cuda.Stream."""
    assert hasattr(torch.cuda.Stream, "device_index") and hasattr(torch.cuda.Stream, "cuda_stream")


# ---------------------------------------------------------- the extension module's versions
@pytest.fixture
def build_dir(tmp_path, monkeypatch):
    """The build module on an empty folder, its compiler calls recorded (each makes its output)."""
    from routed_expert_ffn_route_gb300 import _build
    ran = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("x")
        return Done

    monkeypatch.setattr(_build.subprocess, "run", run)
    monkeypatch.setattr(_build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(_build, "HERE", str(tmp_path))
    monkeypatch.setattr(_build, "PY_EXT", str(tmp_path / os.path.basename(_build.PY_EXT)))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libmoe_gb300.so"))
    (tmp_path / "libmoe_gb300.so").write_text("x")
    monkeypatch.setattr(_build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    return _build, ran, tmp_path


def test_the_object_is_made_again_for_another_torch_or_python(build_dir, monkeypatch):
    """Also when the other torch's files are older than the object."""
    build, ran, _ = build_dir
    obj = build._entries_obj(False)
    assert len(ran) == 1 and build._entries_obj(False) == obj and len(ran) == 1
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "2.0.0+other")
        assert build._entries_obj(False) == obj and len(ran) == 2
        assert build._entries_obj(False) == obj and len(ran) == 2
    assert build._entries_obj(False) == obj and len(ran) == 3
    with monkeypatch.context() as m:
        m.setattr(build.sys, "version", "3.99.0 (another)")
        assert build._entries_obj(False) == obj and len(ran) == 4


def test_the_module_carries_the_interpreters_abi(build_dir):
    build, ran, folder = build_dir
    import importlib.machinery
    import sysconfig
    assert build.PY_EXT.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert importlib.machinery.EXTENSION_SUFFIXES[0] == sysconfig.get_config_var("EXT_SUFFIX")
    old = folder / "_tokens_native.so"  # a module without a tag, which any interpreter loads
    old.write_text("x")
    build._link_entries(build._entries_obj(False), False)
    assert not old.exists() and os.path.exists(build.PY_EXT)


def test_a_module_of_another_torch_is_refused(native):
    from routed_expert_ffn_route_gb300 import tokens
    assert native.torch_version == str(torch.__version__)
    assert tokens._made_for_this_torch(native) is native

    class Other:
        torch_version = "2.0.0+other"

    with pytest.raises(ImportError, match="2.0.0"):
        tokens._made_for_this_torch(Other)


def test_the_library_builds_where_the_module_cannot(build_dir, monkeypatch):
    """A torch without CUDA, or a Python without headers, is no reason to fail: the C library needs
    neither."""
    build, ran, folder = build_dir
    with monkeypatch.context() as m:
        m.setattr(torch.version, "cuda", None)
        assert build._entries_obj(False) is None
    with monkeypatch.context() as m:
        m.setattr(build.sysconfig, "get_paths", lambda: {"include": str(folder)})
        assert build._entries_obj(False) is None
    assert not ran
    build._link_entries(None, False)
    assert not ran


def test_a_call_without_the_module_says_so(native, monkeypatch):
    import sys

    from routed_expert_ffn_route_gb300 import tokens
    monkeypatch.setattr(tokens, "_native", tokens._Late())
    monkeypatch.delattr(moe, "_tokens_native", raising=False)
    monkeypatch.setitem(sys.modules, "routed_expert_ffn_route_gb300._tokens_native", None)
    x = torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ImportError, match="have not been built"):
        moe.moe_sort_tokens(x, 1, x, x, x)


@pytest.mark.parametrize("torch_there", [True, False])
def test_star_import_does_not_need_torch(torch_there):
    """The binding of the packed layer imports without torch; the token operators need it."""
    import subprocess
    import sys
    code = ("import sys\n" + ("" if torch_there else "sys.modules['torch'] = None\n")
            + "from routed_expert_ffn_route_gb300 import *\n"
              "assert callable(moe_layer_forward) and callable(make_config)\n"
              f"assert ('moe_linear' in globals()) == {torch_there}\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


# ------------------------------------------------------------------------------ autograd
def zeros(*shape, dtype=torch.bfloat16, grad=False):
    return torch.zeros(*shape, dtype=dtype, requires_grad=grad)


OUTPUTS = ["q_scale", "resid", "xs", "scale_s", "combined", "dy", "dw", "dx", "product"]


def write(which):
    """A call whose output `which` requires a gradient (on the host: other checks come later)."""
    g = {n: n == which for n in OUTPUTS}
    T, k, H, f32 = 4, 2, 64, torch.float32
    x, pos = zeros(T, H), torch.zeros(T, k, dtype=torch.int32)
    off, xs = torch.zeros(9, dtype=torch.int32), zeros(T * k, H)
    w = zeros(T, k, dtype=f32)
    if which in ("q_scale", "resid"):
        moe.moe_rmsnorm_e4m3(x, torch.zeros(T, H, dtype=torch.float8_e4m3fn),
                             zeros(T, 1, dtype=f32, grad=g["q_scale"]),
                             resid=zeros(T, H, grad=g["resid"]))
    elif which in ("xs", "scale_s"):
        moe.moe_dispatch_rows(x, pos, off, zeros(T * k, H, grad=g["xs"]),
                              scale=zeros(T, 1, dtype=f32),
                              scale_s=zeros(T * k, 1, dtype=f32, grad=g["scale_s"]))
    elif which == "combined":
        moe.moe_combine_rows(xs, pos, zeros(T, H, grad=True), w=w)
    elif which in ("dy", "dw"):
        moe.moe_combine_rows_grad(x, xs, pos, off, w, zeros(T * k, H, grad=g["dy"]),
                                  zeros(T, k, dtype=f32, grad=g["dw"]))
    elif which == "dx":
        moe.moe_dispatch_rows_grad(xs, pos, zeros(T, H, grad=True))
    else:
        moe.moe_linear(x, zeros(32, H), zeros(T, 32, grad=True))


@pytest.mark.parametrize("which", OUTPUTS)
def test_an_output_in_a_recorded_graph_is_refused(native, which):
    with pytest.raises(ValueError, match="requires a gradient"):
        write(which)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):
        write(which)  # passes that check


def test_inputs_that_require_gradients_are_taken(native):
    x, pos = zeros(8, 64, grad=True), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        moe.moe_combine_rows(x, pos, zeros(4, 64), w=zeros(4, 2, dtype=torch.float32, grad=True))


# ------------------------------------------------------------------------ 32-bit numbers
@pytest.mark.parametrize("group", [-2 ** 32, 2 ** 32, -2 ** 31 - 1, 2 ** 31, -2 ** 40 + 128])
def test_numbers_beyond_32_bits_are_refused(native, group):
    """A group of -2^32 is not one of 0."""
    x, q = zeros(4, 256), torch.zeros(4, 256, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="group is out of range"):
        moe.moe_rmsnorm_e4m3(x, q, zeros(4, 1, dtype=torch.float32), group=group)
