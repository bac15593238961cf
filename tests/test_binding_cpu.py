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
    assert cr._native.__file__ == NATIVE and not os.path.exists(os.path.join(PKG, "_native.so"))
