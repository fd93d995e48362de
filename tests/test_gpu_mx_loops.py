"""The loops of persistent kernels past their first turn: several tiles a worker
in the 4-bit product (every tile shape), several row tiles a block in the
elementwise kernels, with the column sums carried across them."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import mx_ref
from helpers import to_np
from oracle import compare

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(autouse=True)
def _lib(lib_path, gpu):
    yield


@pytest.fixture
def g():
    from dense_gemm_tiled_gb300 import binding
    return binding


def f64(t):
    return t.detach().double().cpu().numpy()


def stored(g, x64, fmt):
    codes, st, v = mx_ref.store(x64, fmt)
    return g.Mx(torch.from_numpy(codes).cuda(), torch.from_numpy(st).cuda(), fmt, *x64.shape), v


# tiles of 256 x 256 (76 pairs at most), 256 x 128, 128 x 128 and 128 x 64 (152 blocks)
SHAPE = {0: (256, 256, 76), 1: (256, 128, 76), 2: (128, 128, 152), 3: (128, 64, 152)}
# tile -> (M, N): at least three tiles for some workers, edges ragged both ways
SIZES = {0: (3900, 2700), 1: (3900, 1400), 2: (3700, 2100), 3: (3700, 1090)}


@pytest.mark.parametrize("fmt", ["fp4", "fp4_e4m3"])
@pytest.mark.parametrize("dtype", list(DT))
def test_many_tiles(g, fmt, dtype):
    """Run by test_forced_tile_loops with the tile forced; by itself on the rule's
    choice.  K of several ring fills, so that phases carry over between tiles."""
    tile = int(os.environ.get("GEMM_GB300_MX_TILE", "0"))
    (M, N), (bm, bn, slots) = SIZES[tile], SHAPE[tile]
    assert -(-M // bm) * -(-N // bn) > 2 * slots
    K = 1100
    r = np.random.default_rng(tile)
    A, a = stored(g, r.standard_normal((M, K)).astype(np.float32), fmt)
    B, b = stored(g, (r.standard_normal((N, K)) * 0.05).astype(np.float32), fmt)
    at, bt = torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda()
    ref, mag = (at @ bt.T).cpu().numpy(), (at.abs() @ bt.abs().T).cpu().numpy()
    # stored by TMA; then read back with beta, and rows off alignment
    C = torch.full((M, -(-N // 8) * 8), float("nan"), dtype=DT[dtype], device="cuda")[:, :N]
    g.gemm_mx(A, B, C)
    assert g.last_path() == "mx_tc"
    res = compare.check(to_np(C), ref, mag, dtype)
    assert res["ok"], res
    first = C.clone()
    g.gemm_mx(A, B, C)
    assert torch.equal(C, first)
    for base in (torch.randn((M, -(-N // 8) * 8), device="cuda").to(DT[dtype])[:, :N],
                 torch.randn((M, N + 3), device="cuda").to(DT[dtype])[:, 1: N + 1]):
        c0 = f64(base)
        g.gemm_mx(A, B, base, alpha=0.5, beta=-1.0)
        res = compare.check(to_np(base), 0.5 * ref - c0, 0.5 * mag + np.abs(c0), dtype)
        assert res["ok"], res
    assert g.check_device_status() == g.OK


@pytest.mark.parametrize("tile", range(4))
def test_forced_tile_loops(tile):
    env = dict(os.environ, GEMM_GB300_MX_TILE=str(tile))
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-q", "-x", "-m",
                        "gpu", "-k", "many_tiles"], env=env, capture_output=True, text=True,
                       timeout=600, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]


ROWS = [(16384, 640), (9000, 5632), (40000, 70), (33000, 129)]


@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_many_row_tiles(g, rows, cols, dtype):
    """More row tiles than a strip's blocks: stored bytes as the reference's (on
    rows spread over the whole), the read back, the transposed form, and the
    activation's backward pass with its sums."""
    gen = torch.Generator(device="cuda").manual_seed(rows)
    X = torch.randn((rows, cols), generator=gen, device="cuda").to(DT[dtype])
    dY = torch.randn((rows, cols), generator=gen, device="cuda").to(DT[dtype])
    some = np.unique(np.concatenate([np.arange(0, rows, 97), np.arange(rows - 130, rows)]))
    for fmt in mx_ref.BLOCK:
        Q, Y = g.mx_empty(rows, cols, fmt), torch.empty_like(X)
        Q.codes.fill_(0xA5)
        Q.scales.fill_(0xFF)
        g.mx_quantize(X, Q, act="relu", Y=Y)
        assert g.last_grid() < -(-rows // 64) * -(-cols // 128)
        assert torch.equal(Y, X.clamp(min=0))
        codes, _, v = mx_ref.store(f64(X[some]), fmt)
        assert np.array_equal(Q.codes.cpu().numpy()[some], codes)
        g.mx_dequantize(Q, Y)
        assert torch.equal(Y[some].cpu(), torch.from_numpy(v).float().to(DT[dtype]))
        T = g.mx_empty(rows, cols, fmt)
        g.mx_quantize(X.t().contiguous(), T, transX=True)
        assert torch.equal(T.codes, Q.codes) and torch.equal(T.scales, Q.scales)
    dX, db = torch.empty_like(dY), torch.full((cols,), float("nan"), device="cuda")
    g.mx_act_backward(dY, Q, dX, act="relu", dbias=db)  # (Q: the last format, int8)
    x = g.mx_dequantize(Q, torch.empty((rows, cols), device="cuda"))
    want = dY.double() * (x > 0)
    assert torch.equal(dX.double(), want)
    # sums of exact terms in fp32: at most `rows` additions of half an ulp of what
    # has been summed
    tol = rows * 2.0 ** -24 * want.abs().sum(0)
    assert torch.all((db.double() - want.sum(0)).abs() <= tol)
    again = torch.empty_like(db)
    g.mx_act_backward(dY, Q, dY, act="relu", dbias=again)
    assert torch.equal(db, again) and torch.equal(dY, dX)
