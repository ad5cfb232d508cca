"""Layer norm where libtaco_rms was not built: it is a library of its own, and what needs
it says so when it is called."""
import os
import shutil
import subprocess
import sys

import pytest

from conftest import ROOT

pytest.importorskip("torch")
PACKAGE = os.path.join(ROOT, "gradients_taco_compress_amd")
LIBRARIES = ["libtaco.so", "libtaco_norm.so", "_norm_torch.so"]
if not all(os.path.exists(os.path.join(PACKAGE, f)) for f in LIBRARIES):
    pytest.skip("libtaco_norm is not built", allow_module_level=True)

PROGRAM = """
import torch
from gradients_taco_compress_amd import norm
assert norm.checkpoint_scale(64) > 0
x = torch.zeros(4, 64)

def error(call):
    try:
        call()
    except Exception as e:
        return f"{type(e).__name__}: {e}"

for call in (lambda: norm.layer_norm(x), lambda: norm.norm(x), lambda: norm.layer_norm_backward(x, x, x, x)):
    assert error(call).startswith("TypeError") and "CUDA/HIP" in error(call), error(call)
norm._even = lambda t: t             # (which would ask for a device tensor first)
for call in (lambda: norm.rms_norm(x), lambda: norm.rms_norm_mx(x),
             lambda: norm.rms_norm_backward(x, x, x[:, 0]), lambda: norm.rms(x),
             lambda: norm.rms(x, residual=x), lambda: norm.taco_rms_backward_workspace(4, 64)):
    assert error(call).startswith("ImportError: ") and "build.py" in error(call), error(call)
    assert "{missing}" in error(call), error(call)
print("ok")
"""


@pytest.mark.parametrize("also", [[], ["libtaco_rms.so"]])
def test_layer_norm_does_not_need_the_other_norm(tmp_path, also):
    package = tmp_path / "gradients_taco_compress_amd"
    package.mkdir()
    for f in os.listdir(PACKAGE):
        if f.endswith(".py") or f in LIBRARIES + also:
            shutil.copy(os.path.join(PACKAGE, f), package / f)
    program = PROGRAM.replace("{missing}", "torch module" if also else "libtaco_rms.so")
    done = subprocess.run([sys.executable, "-c", program], cwd=tmp_path, capture_output=True, text=True,
                          timeout=300, env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert done.returncode == 0 and done.stdout.strip() == "ok", done.stderr
