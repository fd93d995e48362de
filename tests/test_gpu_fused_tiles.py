"""Every tile of the fused products' kernel: the 16-bit tests of test_gpu_fused.py with
the tile forced (GEMM_GB300_FUSED_TILE, read once per process): 0 block pairs of 256 x
256, 1 to 3 single blocks of 128 x 192, 128 x 128 and 128 x 64; and K in slices wherever it is
long enough (GEMM_GB300_FUSED_SPLITS)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("tile,splits", [(0, 1), (1, 1), (2, 1), (3, 1), (0, 2), (1, 2),
                                         (2, 3), (3, 4)])
def test_forced_tile(lib_path, gpu, tile, splits):
    env = dict(os.environ, GEMM_GB300_FUSED_TILE=str(tile), GEMM_GB300_FUSED_SPLITS=str(splits))
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(HERE, "test_gpu_fused.py"), "-q",
                        "-x", "-m", "gpu", "-k",
                        "not f32 and not few_rows" if splits == 1 else "test_fused and not f32"], env=env, capture_output=True, text=True,
                       timeout=600, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
