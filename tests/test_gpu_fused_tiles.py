"""Every tile of the fused products' kernel: the 16-bit tests of test_gpu_fused.py with
the tile forced (GEMM_GB300_FUSED_TILE, read once per process): 0 block pairs of 256 x
256, 1 and 2 single blocks of 128 x 128 and 128 x 64."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("tile", range(3))
def test_forced_tile(lib_path, gpu, tile):
    env = dict(os.environ, GEMM_GB300_FUSED_TILE=str(tile))
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(HERE, "test_gpu_fused.py"), "-q",
                        "-x", "-m", "gpu", "-k", "not f32"], env=env, capture_output=True, text=True,
                       timeout=600, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
