"""The package without a usable native half of the binding: W4A16 imports and runs, MXFP4 says what is missing."""
import os
import shutil
import subprocess
import sys

import pytest

fp4 = pytest.importorskip("block_scaled_fp4_w4a16_amd")

SCRIPT = """
import torch, block_scaled_fp4_w4a16_amd as fp4
assert fp4.__file__.startswith({root!r})
assert fp4.fp4_layout_bytes("nvfp4", 2048, 2048) == (2048 * 2048 // 2, 2048 * 2048 // 16)
x, t = torch.zeros(4, 64), torch.zeros(4, 32, dtype=torch.uint8)
for call in (lambda: fp4.MXTensor.quantize(x), lambda: fp4.MXTensor.from_canonical(t, t[:, :2]),
             lambda: fp4.mx_linear(x, x), lambda: fp4.fp4_quantize_mxfp4(4, 64, x, t, t[:, :2])):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e) and "_fp4bind" in str(e) and e.__cause__ is not None
    else:
        raise AssertionError("no error")
print("done")
"""


@pytest.mark.parametrize("native", ["absent", "broken"])
def test_w4a16_without_the_native_half(native, tmp_path):
    package = tmp_path / "block_scaled_fp4_w4a16_amd"
    package.mkdir()
    here = os.path.dirname(fp4.__file__)
    for name in ("__init__.py", "libfp4w4a16.so"):
        shutil.copy(os.path.join(here, name), package / name)
    if native == "broken":
        (package / "_fp4bind.so").write_bytes(b"not a library")
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(root=str(tmp_path))], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)}, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("done\n"), r.stderr
