"""Every tile of the 4-bit product's kernel: the 4-bit tests of test_gpu_mx.py
with the tile forced (GEMM_GB300_MX_TILE, read once per process): 0 and 1 block
pairs of 256 x 256 and 256 x 128, 2 and 3 single blocks of 128 x 128 and 128 x
64."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("tile", range(4))
def test_forced_tile(lib_path, gpu, tile):
    env = dict(os.environ, GEMM_GB300_MX_TILE=str(tile))
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(HERE, "test_gpu_mx.py"), "-q",
                        "-x", "-m", "gpu", "-k", "mx4"], env=env, capture_output=True, text=True,
                       timeout=600, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]


@pytest.mark.parametrize("form", [0, 1, 2, 5])
def test_forced_converted_form(lib_path, gpu, form):
    """Products with a 16-bit operand (GEMM_GB300_MX_MIXED): 0 the stored operand
    always expanded, otherwise always converted where there is such a kernel,
    with K in that many slices."""
    env = dict(os.environ, GEMM_GB300_MX_MIXED=str(form))
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(HERE, "test_gpu_mx.py"), "-q",
                        "-x", "-m", "gpu", "-k", "converted or hard_scales"], env=env,
                       capture_output=True, text=True, timeout=600, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
