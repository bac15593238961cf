"""The C ABI of the batched adapters and activation checkpoints rejects bad
arguments with the documented status before touching a device, and the Python
binding rejects bad tensors. No compute call runs here."""
import ctypes
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "w4a8_rotated_quantized_amd")
pytestmark = pytest.mark.skipif(not os.path.exists(os.path.join(PKG, "libconvrot.so")), reason="libconvrot.so not built")

A = 0x10000      # aligned, never dereferenced
MIS = A + 4


@pytest.fixture(scope="module")
def cr():
    import w4a8_rotated_quantized_amd as m
    if m.device_check() == 0:
        pytest.skip("a device is visible: fake addresses are for hosts without one")
    return m


def _fwd(cr, x=A, ldx=64, down=A, up=A, R=16, n=2, off=A, ids=A, S=3, scale=None, base=None, ldb=128, out=A, ot=0,
         ldo=128, la=A, M=5, N=128, K=64):
    return cr.lib.convrot_lora_forward(x, ldx, down, up, R, n, off, ids, S, scale, base, ldb, out, ot, ldo, la, M, N, K,
                                       None)


def test_forward_validation(cr):
    assert _fwd(cr) == 4                                     # valid: no device here
    assert _fwd(cr, scale=A, base=A, ot=1) == 4              # in place
    assert _fwd(cr, base=A + 4096, ldb=136) == 4
    for k in ("x", "down", "up", "off", "ids", "out", "la"):
        assert _fwd(cr, **{k: None}) == 1, k
        assert _fwd(cr, **{k: MIS}) == 1, k
    assert _fwd(cr, scale=MIS) == 1 and _fwd(cr, base=MIS) == 1
    assert _fwd(cr, base=A, ldb=136) == 1                    # in place with another leading dimension
    assert _fwd(cr, ot=-1) == 1 and _fwd(cr, ot=3) == 1
    assert _fwd(cr, ot=2) == 3                               # no integer output
    for R in (0, -8, 4, 12, 136):
        assert _fwd(cr, R=R) == 3, R
    for R in (8, 24, 128):
        assert _fwd(cr, R=R) == 4, R
    for M in (0, -1, 1 << 26):
        assert _fwd(cr, M=M) == 2, M
    assert _fwd(cr, M=(1 << 26) - 1) == 4
    assert _fwd(cr, N=0) == 2 and _fwd(cr, N=132, ldo=136) == 2 and _fwd(cr, N=32776, ldo=32776) == 2
    assert _fwd(cr, K=60) == 2 and _fwd(cr, K=72) == 2 and _fwd(cr, K=32776, ldx=32776) == 2   # ldx < K
    assert _fwd(cr, ldx=68) == 2 and _fwd(cr, ldx=1 << 31) == 2
    assert _fwd(cr, ldo=120) == 2 and _fwd(cr, ldo=132) == 2 and _fwd(cr, base=A + 16, ldb=120) == 2
    assert _fwd(cr, ldb=1) == 4                              # no base: its leading dimension is not read
    for n in (0, -1, 4097):
        assert _fwd(cr, n=n) == 2, n
    for S in (0, -1, 65537):
        assert _fwd(cr, S=S) == 2, S


def _bwd(cr, dy=A, lddy=128, la=A, x=A, ldx=256, xs=None, xg=1, rot=256, down=A, up=A, R=16, n=2, off=A, ids=A, S=3,
         scale=None, base=None, ldb=256, dx=A, dt=0, lddx=256, dd=A, du=A, acc=0, M=5, N=128, K=256, ws=A, wsb=1 << 30):
    return cr.lib.convrot_lora_backward(dy, lddy, la, x, ldx, xs, xg, rot, down, up, R, n, off, ids, S, scale, base, ldb,
                                        dx, dt, lddx, dd, du, acc, M, N, K, ws, wsb, None)


def test_backward_validation(cr):
    assert _bwd(cr) == 4
    assert _bwd(cr, dx=None) == 4 and _bwd(cr, dd=None, x=None) == 4 and _bwd(cr, du=None, la=None) == 4
    assert _bwd(cr, dx=None, dd=None, du=None) == 1          # nothing wanted
    assert _bwd(cr, x=None) == 1 and _bwd(cr, la=None) == 1
    for k in ("dy", "down", "up", "off", "ids", "ws"):
        assert _bwd(cr, **{k: None}) == 1, k
        assert _bwd(cr, **{k: MIS}) == 1, k
    for k in ("x", "la", "xs", "scale", "base", "dx", "dd", "du"):
        assert _bwd(cr, **{k: MIS}) == 1, k
    need = cr.convrot_lora_backward_workspace_size(5, 128, 256, 16, 2)
    assert need > 0 and _bwd(cr, wsb=need) == 4 and _bwd(cr, wsb=need - 1) == 6
    for rot in (16, 64, 256):
        assert _bwd(cr, xs=A, rot=rot) == 4
    assert _bwd(cr, xs=A, rot=1024) == 2                     # K % rot_group
    assert _bwd(cr, xs=A, rot=0) == 3 and _bwd(cr, xs=A, rot=128) == 3
    assert _bwd(cr, rot=0) == 4                              # not read for bf16 inputs
    assert _bwd(cr, xs=A, xg=0) == 4 and _bwd(cr, xs=A, xg=2) == 3 and _bwd(cr, xs=A, xg=5) == 1
    assert _bwd(cr, xs=A, K=264, ldx=264, ldb=264, lddx=264) == 2     # codes come in groups of 256
    assert _bwd(cr, K=264, ldx=264, ldb=264, lddx=264) == 4
    assert _bwd(cr, xs=A, ldx=264) == 2 and _bwd(cr, ldx=264) == 4
    assert _bwd(cr, lddy=120) == 2 and _bwd(cr, lddx=248) == 2 and _bwd(cr, dt=2) == 3 and _bwd(cr, dt=7) == 1
    assert _bwd(cr, R=12) == 3 and _bwd(cr, M=0) == 2 and _bwd(cr, S=0) == 2 and _bwd(cr, n=0) == 2
    assert _bwd(cr, n=4096, R=128, N=8192, lddy=8192) == 2   # weights beyond 2^31 elements
    assert cr.convrot_lora_backward_workspace_size(5, 8192, 256, 128, 4096) == 0
    assert cr.convrot_lora_backward_workspace_size(0, 128, 256, 16, 2) == 0
    assert cr.convrot_lora_backward_workspace_size(5, 128, 256, 12, 2) == 0


def test_act_validation(cr):
    L = cr.lib
    def f(z=A, ldz=256, rows=3, C=128, act=0, y=A, ldy=128, c=A, s=A):
        return L.convrot_act_checkpoint(z, ldz, rows, C, act, y, ldy, c, s, None)
    def b(dy=A, lddy=128, c=A, s=A, rows=3, C=128, act=0, dz=A, lddz=256):
        return L.convrot_act_backward(dy, lddy, c, s, rows, C, act, dz, lddz, None)
    for act in (0, 1, 2):
        assert f(act=act) == 4 and b(act=act) == 4
    assert f(act=0, ldz=128) == 4 and f(act=2, ldz=248) == 2 and b(act=2, lddz=248) == 2
    assert f(act=3) == 1 and b(act=-1) == 1
    for k in ("z", "y", "c", "s"):
        assert f(**{k: None}) == 1 and f(**{k: MIS}) == 1
    for k in ("dy", "dz", "c", "s"):
        assert b(**{k: None}) == 1 and b(**{k: MIS}) == 1
    for k in ({"rows": 0}, {"rows": 1 << 31}, {"C": 32}, {"C": 96}, {"C": 0}, {"C": 32832}, {"rows": 1 << 29, "C": 64}):
        assert f(**k) == 2 and b(**k) == 2, k
    assert f(ldy=120) == 2 and f(ldz=132) == 2 and b(lddy=64) == 2


def test_binding_refuses_tensors(cr):
    bf = torch.bfloat16
    x, down, up = torch.zeros((4, 64), dtype=bf), torch.zeros((2, 8, 64), dtype=bf), torch.zeros((2, 128, 8), dtype=bf)
    off, ids = torch.tensor([0, 4], dtype=torch.int32), torch.tensor([0], dtype=torch.int32)
    for args in ((x, down, up, off, ids),                                    # not on the GPU
                 (x.float(), down, up, off, ids), (x, down[:, :, :32], up, off, ids), (x, down, up[:, :, :4], off, ids),
                 (x, down, up, off.long(), ids), (x, down, up, off[:1], ids), (x[0], down, up, off, ids),
                 (x, down[0], up, off, ids), (x, down, up, off, ids[0])):
        with pytest.raises(ValueError):
            cr.convrot_lora_forward(*args)
    dy, la = torch.zeros((4, 128), dtype=bf), torch.zeros((4, 8))
    for k in ({}, {"want_dx": False, "want_weights": False}, {"accumulate": True}, {"dx_type": 2},
              {"x_scales": torch.zeros(3)}):
        with pytest.raises(ValueError):
            cr.convrot_lora_backward(dy, la, x, down, up, off, ids, **k)
    with pytest.raises(ValueError):
        cr.convrot_act_checkpoint(x, 0)
    with pytest.raises(ValueError):
        cr.convrot_act_checkpoint(x, 7)
    with pytest.raises(ValueError):
        cr.convrot_act_backward(x, torch.zeros((4, 64), dtype=torch.int8), torch.zeros((4, 1)), 0)


BUILD = os.path.join(PKG, "_build")
OBJS = [f + ".o" for f in ("rq", "pack", "merge", "gemm_w4a4", "gemm_int", "gemm_w4a8", "gemm_f6", "lora", "act")]
ROCM = "/opt/rocm"


def _missing():
    if not shutil.which("g++"):
        return "g++ not available"
    if not os.path.isdir(os.path.join(ROCM, "include", "hip")):
        return "HIP headers not available"
    if not all(os.path.exists(os.path.join(BUILD, o)) for o in OBJS):
        return "kernel objects not built (run the build first)"
    return None


@pytest.mark.skipif(_missing() is not None, reason=str(_missing()))
def test_host_layer_under_sanitizers(tmp_path):
    """adapter_abi.cpp with AddressSanitizer and UndefinedBehaviorSanitizer over
    seeded random arguments (tests/adapter_host_check.cpp)."""
    flags = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
             "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
             f"-I{os.path.join(ROOT, 'include')}"]
    objs = []
    for src in (os.path.join(PKG, "csrc", "abi.cpp"), os.path.join(PKG, "csrc", "adapter_abi.cpp"),
                os.path.join(ROOT, "tests", "adapter_host_check.cpp")):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        subprocess.run(["g++", *flags, "-c", src, "-o", objs[-1]], check=True)
    exe = str(tmp_path / "check")
    subprocess.run(["g++", "-fsanitize=address,undefined", *objs, *[os.path.join(BUILD, o) for o in OBJS],
                    f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib", "-o", exe], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "all ok" in r.stdout or "skipped" in r.stdout
