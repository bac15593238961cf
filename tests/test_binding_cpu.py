"""The native part of the Python binding on a host without a GPU: what is reachable
without it, and, against a stand-in for the library, what it does around a call."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "w4a8_rotated_quantized_amd")
NATIVE = os.path.join(PKG, "_native" + sysconfig.get_config_var("EXT_SUFFIX"))
pytestmark = pytest.mark.skipif(not os.path.exists(os.path.join(PKG, "libconvrot.so")), reason="libconvrot.so not built")


def _python(code, cwd, *args):
    env = {k: v for k, v in os.environ.items() if k != "PYTHONPATH"}
    r = subprocess.run([sys.executable, "-c", code, *map(str, args)], cwd=cwd, env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    return r.stdout


WITHOUT = """
import torch
import w4a8_rotated_quantized_amd as cr
assert cr.status_string(0) and cr._native is not None and isinstance(cr.device_check(), int)
assert cr.convrot_layer_norm_backward_workspace_size(5, 64, 1) > 0
z = torch.zeros((4, 256), dtype=torch.bfloat16)
try:
    cr.convrot_act_checkpoint(z, cr.ACT.GELU)
except ValueError:                             # a tensor that is not on a GPU: refused as ever
    pass
else:
    raise SystemExit("a host tensor was taken")
try:
    cr.mxfp4_quantize(z)
except ImportError as e:
    assert "_native" in str(e) and "build()" in str(e), e
else:
    raise SystemExit("mxfp4_quantize ran without the native module")
print("ok")
"""


@pytest.mark.parametrize("kind", ["absent", "another file", "another torch"])
def test_package_without_its_native_module(tmp_path, kind):
    """Everything that goes through ctypes needs libconvrot.so alone; the rest says what is missing when it is called."""
    pkg = tmp_path / os.path.basename(PKG)
    pkg.mkdir()
    shutil.copy(os.path.join(PKG, "__init__.py"), pkg)
    os.symlink(os.path.join(PKG, "libconvrot.so"), pkg / "libconvrot.so")
    code = WITHOUT
    if kind == "another file":
        (pkg / os.path.basename(NATIVE)).write_bytes(b"no shared object")
    elif kind == "another torch":
        os.symlink(NATIVE, pkg / os.path.basename(NATIVE))
        code = "import torch\ntorch.__version__ = '0.0.1'\n" + code
    assert "ok" in _python(code, tmp_path)


def test_native_module_is_named_for_its_python():
    """No other Python takes the file for its own: the interface that it uses is not the stable one."""
    import w4a8_rotated_quantized_amd as cr
    assert cr._native.__file__ == NATIVE


# ---------------------------------------------------------------------------
# Around a call: the native module linked to a stand-in for the library
# (binding_stub.cpp), on tensors that are said to be on a GPU and have no memory.
# ---------------------------------------------------------------------------
def _stub_missing():
    if not shutil.which("g++"):
        return "g++ not available"
    if not os.path.isdir("/opt/rocm/include/hip"):
        return "HIP headers not available"
    if not os.path.exists(NATIVE):
        return "the native module is not built"
    return None


@pytest.fixture(scope="module")
def stub(tmp_path_factory):
    if _stub_missing():
        pytest.skip(_stub_missing())
    to = tmp_path_factory.mktemp("stub") / "libconvrot.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-pthread", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    f"-I{os.path.join(ROOT, 'include')}", "-Wl,-soname,libconvrot.so", os.path.join(ROOT, "tests", "binding_stub.cpp"),
                    "-o", str(to)], check=True)
    return to


HARNESS = """
import ctypes, importlib.util, sys, threading, time, weakref
import torch
stub = ctypes.CDLL(sys.argv[1], ctypes.RTLD_GLOBAL)
spec = importlib.util.spec_from_file_location("_native", sys.argv[2])
n = importlib.util.module_from_spec(spec)
spec.loader.exec_module(n)

class OnGpu(torch.Tensor):
    @staticmethod
    def __new__(cls, dtype, *shape):
        return torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cuda:0")
    @classmethod
    def __torch_dispatch__(cls, f, types, args=(), kwargs=None):
        raise AssertionError(str(f))

T = OnGpu
bf, f32, u8, i8 = torch.bfloat16, torch.float32, torch.uint8, torch.int8
M, C, N = 4, 64, 8
moments = lambda: ([T(i8, 300), T(i8, 5)], [T(u8, 300), T(u8, 5)], [T(f32, 2), T(f32, 1)], [T(f32, 2), T(f32, 1)])
two = lambda dtype: [T(dtype, 300), T(dtype, 5)]

def calls():
    # function, arguments, places of the tensors that it writes for others than itself (in lists: all of a list)
    m, v, ms, vs = moments()
    yield "mxfp4_quantize", [T(bf, M, C), 0, T(u8, 1, M, 64), T(u8, 1, M, 4), 0], [2, 3]
    yield "mxfp4_dequantize", [T(u8, 1, M, 64), T(u8, 1, M, 4), C, 0, 0, T(bf, M, C), 0], [5]
    yield "mxfp4_gemm", [T(u8, 1, M, 64), T(u8, 1, M, 4), T(u8, 1, N, 64), T(u8, 1, N, 4), None, 1, T(f32, M, N), 0], [6]
    yield "layer_norm_forward", [T(bf, M, C), T(bf, C), T(bf, C), None, 1e-6, False, 0, T(bf, M, C), T(f32, M), T(f32, M), 0], [7, 8, 9]
    yield "layer_norm_backward", [T(bf, M, C), T(bf, M, C), T(f32, M), T(f32, M), T(bf, C), None, False, None, 0, T(bf, M, C), T(f32, C),
                                  T(f32, C), True, True, True, T(u8, 64), 0], [9, 10, 11, 15]
    yield "adamw_step", [two(f32), two(f32), two(f32), two(f32), None, None, None, None, 1, .1, .9, .99, 1e-8, 0., 0, 0], [0]
    yield "adamw_step", [two(f32), two(bf), m, v, two(bf), ms, vs, T(f32, 1), 1, .1, .9, .99, 1e-8, 0., 0, 0], [0, 4]
    m, v, ms, vs = moments()
    yield "adamw_moments", [m, v, ms, vs, T(f32, 305), T(f32, 305), 0], [4, 5]

def flat(args):
    return [t for a in args for t in (a if type(a) is list else [a]) if isinstance(t, torch.Tensor)]
"""

OTHERS = HARNESS + """
for i, (name, args, _) in enumerate(calls()):
    held, alive = [weakref.ref(t) for t in flat(args)], []
    lists = [a for a in args if type(a) is list]
    def other():
        while stub.stub_calls() <= i:
            time.sleep(0.001)
        for l in lists:                        # the caller's lists change under the call
            l.clear()
        alive.append(all(r() is not None for r in held))
        stub.stub_word()
    t = threading.Thread(target=other)
    t.start()
    result = getattr(n, name)(*args)
    t.join()
    assert type(result) is not int or result == 0, f"{name}: no other thread ran during the call"
    assert alive == [True], name
print("ok")
"""


def test_other_threads_run_during_a_call(stub):
    """A call may wait, for memory or for a place in the queue, for what another Python thread has yet to do."""
    assert "ok" in _python(OTHERS, ROOT, stub, NATIVE)


VERSIONS = HARNESS + """
stub.stub_wait(0)
for name, args, written in calls():
    places = [flat([args[k]]) for k in written]
    ours = [t for p in places for t in p]
    result = getattr(n, name)(*args)
    assert type(result) is not int or result == 0, name
    for t in flat(args):
        assert t._version == any(t is o for o in ours), (name, tuple(t.shape), t.dtype, t._version)
with torch.inference_mode():
    inner = T(f32, M, C)
assert inner.is_inference()
for mode in (torch.inference_mode, torch.no_grad):     # tensors without a version are left alone
    with mode():
        assert type(n.mxfp4_gemm(T(u8, 1, M, 64), T(u8, 1, M, 4), T(u8, 1, 64, 64), T(u8, 1, 64, 4), None, 1, inner, 0)) is not int
print("ok")
"""


def test_written_tensors_change_their_version(stub):
    """Autograd then refuses a backward pass that needs what was there before."""
    assert "ok" in _python(VERSIONS, ROOT, stub, NATIVE)


LEFT = HARNESS + """
name, args, _ = [c for c in calls() if c[0] == sys.argv[3]][-1]
stub.stub_linger()
threading.Thread(target=lambda: getattr(n, name)(*args), daemon=True).start()
while stub.stub_calls() == 0:
    time.sleep(0.001)
print("ok", flush=True)
"""


@pytest.mark.parametrize("name", ["mxfp4_gemm", "layer_norm_backward", "adamw_step"])
def test_a_call_that_outlives_the_interpreter(stub, name):
    """A daemon thread whose call ends when the interpreter is gone ends quietly, and the process as it would have."""
    assert "ok" in _python(LEFT, ROOT, stub, NATIVE, name)
