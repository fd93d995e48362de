"""Fused and grouped products whose rows begin on 16 bytes and end anywhere: nothing past a
row's last column is written, in a wider matrix or behind a single row."""
import os
import subprocess
import sys

import pytest
import torch

import fused_ref as ref
from fused_ref import DT

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture
def g(lib_path, gpu):
    from dense_gemm_tiled_gb300 import binding
    yield binding
    torch.cuda.synchronize()
    assert binding.check_device_status() == binding.OK


def new(dtype, *shape, seed=0, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * std).to(DT[dtype]).cuda()


class Inside:
    """A matrix (or several) of aligned rows inside a buffer of sevens."""

    def __init__(self, dtype, *shape):
        *outer, n = shape
        ld = (n + 7) // 8 * 8 + 8
        self.buf = torch.full((4096 + ld * torch.Size(outer).numel(),), 7.0, dtype=DT[dtype], device="cuda")
        strides = (ld, 1) if len(outer) == 1 else (ld * outer[1], ld, 1)
        self.t = self.buf.as_strided(shape, strides, 2048)
        self.t.fill_(float("nan"))
        self.out = torch.ones_like(self.buf, dtype=torch.bool)
        self.out.as_strided(shape, strides, 2048).fill_(False)

    def check(self, what=""):
        changed = (self.out & (self.buf != 7)).nonzero().flatten() - 2048
        assert changed.numel() == 0, (what, changed[:8].tolist())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M", [1, 2, 20, 40, 300])
@pytest.mark.parametrize("K", [16, 600])
def test_row_ends(g, dtype, M, K):
    for N in (1, 2, 3, 5, 7, 8, 9, 31, 33, 65, 127, 130, 257, 420):
        A, B = new(dtype, M, K, seed=1), new(dtype, K, N, seed=2, std=0.2)
        Y, U = Inside(dtype, M, N), Inside(dtype, M, N)
        R = new(dtype, M, N, seed=3)
        g.gemm_fused(A, B, Y.t, act="gelu", residual=R, preact=U.t)
        u, eu, y, ey = ref.forward(A.double(), B.double(), dtype, name="gelu", residual=R.double())
        ref.check(Y.t, y, ey, N)
        ref.check(U.t, u, eu, N)
        Y.check(N)
        U.check(N)
        dX, db = Inside(dtype, M, N), torch.empty(N, device="cuda")
        g.gemm_fused_backward(A, B, dX.t, U.t, dbias=db)
        d, ed, s, es = ref.backward(A.double(), B.double(), dtype, U.t.double())
        ref.check(dX.t, d, ed, N)
        ref.check(db, s, es, N)
        dX.check(N)
        U.check(N)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("sizes", [[1], [64, 0, 32, 96], [100, 1, 31]])
def test_row_ends_of_groups(g, dtype, sizes):
    """Whole boxes and boxes that a group's end cuts; weights' gradients with and without
    what was there."""
    at = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
    offs = torch.tensor(at, dtype=torch.int32, device="cuda")
    rows, E, K = at[-1], len(sizes), 40
    for N in (1, 5, 8, 33, 65, 130, 257):
        A, B = new(dtype, rows, K, seed=1), new(dtype, E, N, K, seed=2, std=0.2)
        Y = Inside(dtype, rows, N)
        g.gemm_grouped(A, B, Y.t, offs, transB=True, act="relu")
        Y.check(N)
        C = Inside(dtype, E, K, N)
        g.gemm_grouped_wgrad(A, Y.t, C.t, offs)
        C.check(N)
        C.t.fill_(1.0)
        C2 = Inside(dtype, E, K, N)
        C2.t.copy_(C.t)
        g.gemm_grouped_wgrad(A, Y.t, C2.t, offs, beta=0.5)
        C2.check(N)
        g.gemm_grouped_wgrad(A, Y.t, C.t, offs)
        for e, (lo, hi) in enumerate(zip(at, at[1:])):
            _, _, y, ey = ref.forward(A[lo:hi].double(), B[e].double().t(), dtype, name="relu")
            ref.check(Y.t[lo:hi], y, ey, (N, e))
            a, b = A[lo:hi].double().t(), Y.t[lo:hi].double()
            _, _, y, ey = ref.forward(a, b, dtype)
            ref.check(C.t[e], y, ey, (N, e))
            _, _, y, ey = ref.forward(a, b, dtype, residual=torch.ones_like(y), beta=0.5)
            ref.check(C2.t[e], y, ey, (N, e))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_operands_end_where_they_end(g, dtype):
    """What lies behind the last column of an operand's aligned row does not matter."""
    for M, N, K in ((1, 24, 5), (20, 72, 63), (40, 24, 65), (300, 130, 127), (17, 40, 1001), (3, 257, 70)):
        for ta in (False, True):
            for tb in (False, True):
                A, B = Inside(dtype, *((K, M) if ta else (M, K))), Inside(dtype, *((N, K) if tb else (K, N)))
                for x, seed in ((A, 1), (B, 2)):
                    x.buf.fill_(float("nan"))
                    x.t.copy_(new(dtype, *x.t.shape, seed=seed))
                Y = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda")
                g.gemm_fused(A.t, B.t, Y, transA=ta, transB=tb)
                a, b = A.t.double(), B.t.double()
                _, _, y, ey = ref.forward(a.t() if ta else a, b.t() if tb else b, dtype)
                ref.check(Y, y, ey, (M, N, K, ta, tb))


@pytest.mark.parametrize("tile", [0, 1, 2, 3])
def test_row_ends_of_every_tile(lib_path, gpu, tile):
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-q", "-x", "-m", "gpu",
                        "-k", "not f32 and not every_tile"],
                       env=dict(os.environ, GEMM_GB300_FUSED_TILE=str(tile), GEMM_GB300_FUSED_SPLITS="1"),
                       capture_output=True, text=True, timeout=600, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
