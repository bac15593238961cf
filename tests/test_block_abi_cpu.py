"""The C ABI of the microscaled 4-bit linear, of layer norm and of the optimizer
step rejects bad arguments with the documented status before touching a device,
and the Python binding rejects bad tensors. No compute call runs here."""
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


def test_mx_validation(cr):
    def q(x=A, ldx=1024, rows=3, K=1024, rot=0, c=A, s=A):
        return cr.lib.mxfp4_quantize(x, ldx, rows, K, rot, c, s, None)

    def d(c=A, s=A, rows=3, K=1024, rot=0, out=A, ot=0, ldo=1024):
        return cr.lib.mxfp4_dequantize(c, s, rows, K, rot, out, ot, ldo, None)

    def g(ac=A, asc=A, wc=A, ws=A, bias=None, out=A, ot=0, ldc=64, M=3, N=64, K=1024):
        return cr.lib.mxfp4_gemm(ac, asc, wc, ws, bias, out, ot, ldc, M, N, K, None)

    assert q() == 4 and d() == 4 and g() == 4 and g(bias=A, ot=1) == 4
    for k in ("x", "c", "s"):
        assert q(**{k: None}) == 1 and q(**{k: MIS}) == 1
    for k in ("c", "s", "out"):
        assert d(**{k: None}) == 1 and d(**{k: MIS}) == 1
    for k in ("ac", "asc", "wc", "ws", "out"):
        assert g(**{k: None}) == 1 and g(**{k: MIS}) == 1
    assert g(bias=MIS) == 1
    for rot in (16, 64, 256, 1024):
        assert q(rot=rot) == 4 and d(rot=rot) == 4
    for rot in (-1, 4, 32, 128, 512, 4096):
        assert q(rot=rot) == 3 and d(rot=rot) == 3
    assert q(K=1056, ldx=1056) == 4 and q(K=1056, ldx=1056, rot=16) == 4 and q(K=1056, ldx=1056, rot=64) == 2
    for k in ({"rows": 0}, {"rows": 1 << 26}, {"K": 0}, {"K": 16}, {"K": 1000}, {"K": 32800}):
        assert q(ldx=32800, **k) == 2 and d(ldo=32800, **k) == 2, k
    for ld in (1016, 1028, 1 << 31):
        assert q(ldx=ld) == 2 and d(ldo=ld) == 2
    assert d(ot=2) == 3 and d(ot=3) == 1 and d(ot=-1) == 1 and g(ot=2) == 3 and g(ot=7) == 1
    for k in ({"M": 0}, {"M": 1 << 26}, {"N": 0}, {"N": 60}, {"N": 1 << 26, "ldc": 1 << 26}, {"K": 48}, {"ldc": 56}, {"ldc": 68},
              {"M": (1 << 26) - 1, "N": (1 << 26) - 8, "ldc": 1 << 26}):
        assert g(**k) == 2, k


def test_norm_validation(cr):
    def f(x=A, xt=0, ldx=64, w=A, ldw=16392, b=A, ldbias=16392, at=0, plus=0, off=None, S=1, eps=1e-6, y=A, yt=0, ldy=64, m=A, r=A, rows=5, C=64):
        return cr.lib.convrot_layer_norm_forward(x, xt, ldx, w, ldw, b, ldbias, at, plus, off, S, eps, y, yt, ldy, m, r, rows, C, None)

    def b(dy=A, dyt=0, lddy=64, x=A, xt=0, ldx=64, m=A, r=A, w=A, ldw=16392, at=0, plus=0, off=None, S=1, base=None, ldb=64, dx=A, dxt=0,
          lddx=64, dw=A, db=A, acc=0, rows=5, C=64, ws=A, wsb=1 << 30):
        return cr.lib.convrot_layer_norm_backward(dy, dyt, lddy, x, xt, ldx, m, r, w, ldw, at, plus, off, S, base, ldb, dx, dxt, lddx, dw,
                                                  db, acc, rows, C, ws, wsb, None)

    assert f() == 4 and f(w=None, b=None) == 4 and f(off=A, S=7, plus=1) == 4
    assert b() == 4 and b(w=None) == 4 and b(off=A, S=7, plus=1) == 4 and b(base=A, dx=A) == 4
    assert b(dx=None) == 4 and b(dw=None, db=None, ws=None, wsb=0) == 4 and b(dw=None) == 4
    assert b(dx=None, dw=None, db=None) == 1 and b(ws=None) == 1 and b(base=A, ldb=72) == 1
    for k in ("x", "y", "m", "r"):
        assert f(**{k: None}) == 1 and f(**{k: MIS}) == 1, k
    for k in ("dy", "x", "m", "r"):
        assert b(**{k: None}) == 1 and b(**{k: MIS}) == 1, k
    for k in ("w", "b", "off"):
        assert f(**{k: MIS}) == 1
    for k in ("w", "off", "base", "dx", "dw", "db", "ws"):
        assert b(**{k: MIS}) == 1
    for t in ("xt", "at", "yt"):
        assert f(**{t: 2}) == 3 and f(**{t: 3}) == 1 and f(**{t: 1}) == 4
    for t in ("dyt", "xt", "at", "dxt"):
        assert b(**{t: 2}) == 3 and b(**{t: -1}) == 1 and b(**{t: 1}) == 4
    assert f(plus=2) == 1 and b(plus=-1) == 1 and f(eps=-1e-6) == 1 and f(eps=float("nan")) == 1 and f(eps=0.0) == 4
    assert f(S=2) == 1 and b(S=2) == 1                       # sequences without offsets
    for k in ({"rows": 0}, {"rows": 1 << 26}, {"C": 0}, {"C": 12}, {"C": 16392}, {"off": A, "S": 0}, {"off": A, "S": 4097}):
        wide = {n: 16392 for n in ("ldx", "ldy")}
        assert f(**wide, **k) == 2, k
        assert b(lddy=16392, ldx=16392, lddx=16392, **k) == 2, k
    assert f(ldx=56) == 2 and f(ldy=68) == 2 and b(lddy=56) == 2 and b(lddx=1 << 31) == 2 and b(base=A + 64, ldb=56) == 2
    for ld in (0, 56, 68, 1 << 31):
        assert f(off=A, S=2, ldw=ld) == 2 and f(off=A, S=2, ldbias=ld) == 2 and b(off=A, S=2, ldw=ld) == 2
        assert f(ldw=ld, ldbias=ld) == 4 and b(ldw=ld) == 4                # one row: not read
        assert f(off=A, S=2, w=None, ldw=ld) == 4 and f(off=A, S=2, b=None, ldbias=ld) == 4
    need = cr.convrot_layer_norm_backward_workspace_size(5, 64, 1)
    assert need > 0 and b(wsb=need) == 4 and b(wsb=need - 1) == 6
    for k in ((0, 64, 1), (5, 12, 1), (5, 64, 0), (5, 64, 4097)):
        assert cr.convrot_layer_norm_backward_workspace_size(*k) == 0


class _Entry(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "avg", "sq", "avg_scales", "sq_scales", "copy")] + [("n", ctypes.c_int64)]


def test_adamw_validation(cr):
    def one(**k):
        e = dict(param=A, grad=A, avg=A, sq=A, avg_scales=A, sq_scales=A, copy=None, n=100)
        e.update(k)
        return _Entry(**e)

    def s(*entries, count=None, gt=1, bits=32, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.01, step=1, gs=None, seed=1):
        arr = (_Entry * max(1, len(entries)))(*entries)
        return cr.lib.convrot_adamw_step(ctypes.addressof(arr), len(entries) if count is None else count, gt, bits, lr, b1, b2, eps, wd,
                                         step, gs, seed, None)

    assert s(one()) == 4 and s(one(), one(n=0, param=None, grad=None), one(copy=A)) == 4 and s(one(), bits=8) == 4
    assert s(one(avg_scales=None, sq_scales=None)) == 4 and s(one(avg_scales=MIS)) == 4
    assert s(one(avg_scales=MIS, sq_scales=MIS), bits=8) == 4              # scales need 4 bytes
    for k in ("param", "grad", "avg", "sq"):
        assert s(one(**{k: None})) == 1 and s(one(), one(**{k: MIS})) == 1, k
    assert s(one(copy=MIS)) == 1
    for k in ("avg_scales", "sq_scales"):
        assert s(one(**{k: None}), bits=8) == 1 and s(one(**{k: A + 2}), bits=8) == 1
    assert s(one(n=-1)) == 2 and s(one(n=1 << 31)) == 2 and s(one(n=(1 << 31) - 1)) == 4
    assert s(count=0) == 2 and s(one(), count=-3) == 2 and s(one(), count=65537) == 2
    assert cr.lib.convrot_adamw_step(None, 1, 1, 32, 1e-3, 0.9, 0.999, 1e-8, 0.0, 1, None, 0, None) == 1
    assert s(one(), gt=0) == 4 and s(one(), gt=2) == 3 and s(one(), gt=5) == 1
    for bits in (0, 4, 16, 64):
        assert s(one(), bits=bits) == 3
    nan = float("nan")
    for k in ({"lr": -1.0}, {"lr": nan}, {"b1": 1.0}, {"b1": -0.1}, {"b2": 1.0}, {"b2": nan}, {"eps": -1e-9}, {"wd": -0.1}, {"step": 0},
              {"step": -4}, {"gs": A + 2}):
        assert s(one(), **k) == 1, k
    assert s(one(), gs=MIS) == 4 and s(one(), lr=0.0, eps=0.0, wd=0.0, b1=0.0, b2=0.0) == 4

    def m(*entries, av=A, sq=A):
        arr = (_Entry * len(entries))(*entries)
        return cr.lib.convrot_adamw_moments(ctypes.addressof(arr), len(entries), av, sq, None)

    assert m(one(param=None, grad=None)) == 4 and m(one(), av=None) == 1 and m(one(), sq=MIS) == 1
    assert m(one(avg_scales=None)) == 1 and m(one(avg=MIS)) == 1


def test_binding_refuses_tensors(cr):
    """No tensor here is on the GPU; what is wrong is named before that where it can be."""
    bf = torch.bfloat16
    x = torch.zeros((4, 64), dtype=bf)
    codes, scales = torch.zeros((1, 4, 64), dtype=torch.uint8), torch.zeros((1, 4, 4), dtype=torch.uint8)
    for call in (lambda: cr.mxfp4_quantize(x, 64), lambda: cr.mxfp4_dequantize(codes, scales, 64),
                 lambda: cr.mxfp4_gemm(codes, scales, codes, scales), lambda: cr.convrot_layer_norm_forward(x),
                 lambda: cr.convrot_layer_norm_backward(x, x, x[0], x[0]),
                 lambda: cr.convrot_adamw_step([x], [x], [x], [x], step=1, lr=1e-3),
                 lambda: cr.convrot_adamw_step([], [], [], [], step=1, lr=1e-3),
                 lambda: cr.convrot_adamw_moments([x], [x], [x], [x]), lambda: cr.convrot_adamw_moments([], [], [], [])):
        with pytest.raises(ValueError):
            call()
    # the native module by itself: sizes, types and what is no tensor
    n = cr._native
    for call in (lambda: n.mxfp4_quantize(x, 64, None, None, 0), lambda: n.mxfp4_quantize(3, 64, None, None, 0),
                 lambda: n.mxfp4_gemm(codes, scales, codes, None, None, 0, None, 0),
                 lambda: n.layer_norm_forward(x, None, None, None, 1e-6, False, 0, None, None, None, 0),
                 lambda: n.adamw_step([x, 3], [x, x], [x], [x], None, None, None, None, 1, .1, .9, .9, .1, 0., 0, 0)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        n.mxfp4_quantize(x)


def test_documented_where_it_cannot_be_checked(cr):
    with open(os.path.join(ROOT, "include", "convrot.h")) as f:
        header = " ".join(f.read().replace("\n *", " ").split())
    assert "a captured graph replays those of the capture" in header
    assert "One below an earlier one counts as that earlier one." in header
    assert "their places in y, mean, rstd and dx are left as they are" in header
    for call in (cr.mxfp4_gemm, cr.convrot_layer_norm_forward):
        assert "Not recorded by autograd" in " ".join(call.__doc__.split())


BUILD = os.path.join(PKG, "_build")
OBJS = [f + ".o" for f in ("rq", "pack", "merge", "gemm_w4a4", "gemm_int", "gemm_w4a8", "gemm_f6", "mx", "gemm_mx", "norm", "adamw")]
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
    """block_abi.cpp with AddressSanitizer and UndefinedBehaviorSanitizer over
    seeded random arguments (tests/block_host_check.cpp)."""
    flags = ["-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
             "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include",
             f"-I{os.path.join(ROOT, 'include')}"]
    objs = []
    for src in (os.path.join(PKG, "csrc", "abi.cpp"), os.path.join(PKG, "csrc", "block_abi.cpp"),
                os.path.join(ROOT, "tests", "block_host_check.cpp")):
        objs.append(str(tmp_path / (os.path.basename(src) + ".o")))
        subprocess.run(["g++", *flags, "-c", src, "-o", objs[-1]], check=True)
    exe = str(tmp_path / "check")
    subprocess.run(["g++", "-fsanitize=address,undefined", *objs, *[os.path.join(BUILD, o) for o in OBJS],
                    f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib", "-o", exe], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert "all ok" in r.stdout or "skipped" in r.stdout


def test_adamw_refuses_an_eps_whose_reciprocal_is_infinite(cr):
    """Below 2^-126 a float32 eps is subnormal (or zero): without a gradient the update would be 0 times infinity, not 0."""
    e = (_Entry * 1)(_Entry(param=A, grad=A, avg=A, sq=A, n=100))

    def s(eps):
        return cr.lib.convrot_adamw_step(ctypes.addressof(e), 1, 1, 32, 1e-3, 0.9, 0.999, eps, 0.0, 1, None, 0, None)

    assert [s(eps) for eps in (0.0, 2.0 ** -126, 1e-30, 1e-8, 1.0)] == [4] * 5
    assert [s(eps) for eps in (2.0 ** -126 * (1 - 2.0 ** -23), 2.0 ** -127, 1e-40, 1e-50, 5e-324)] == [1] * 5


def test_norm_refuses_an_eps_that_rounds_to_zero(cr):
    """As a float32 it would be 0: a row without variance then has no rstd, where the formula's is finite and xh 0."""
    def f(eps):
        return cr.lib.convrot_layer_norm_forward(A, 0, 64, None, 64, None, 64, 0, 0, None, 1, eps, A, 0, 64, A, A, 5, 64, None)

    assert [f(eps) for eps in (0.0, 2.0 ** -149, 1e-40, 1e-6, 1.0)] == [4] * 5
    assert [f(eps) for eps in (2.0 ** -151, 1e-50, 5e-324)] == [1] * 3
