"""Grouped products of many ragged groups, more tiles than workers, whose residual or
pre-activation is asked for ahead: boxes that a group's end cuts give their staging buffer
back to the next tile's load."""
import os
import re
import subprocess
import sys

import pytest
import torch

import fused_ref as ref
from fused_ref import DT

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "dense_gemm_tiled_gb300", "csrc")


def test_every_way_out_of_a_staging_buffer_is_fenced():
    """Stores to a staging buffer are ordered before what the tensor-memory-access unit
    does with it next, whichever way the box leaves it."""
    text = open(os.path.join(CSRC, "fused_tcgen05.cuh")).read()
    end = text[text.index("// a box that the group's end cuts"):]
    end = end[: end.index("\n    if (lane == 0) {\n      bulk_wait_all();")]
    ways = end.split("} else {")
    assert len(ways) == 2 and "fu_rows_out" in ways[0] and "tma_store_3d" in ways[1]
    for way in ways:
        way = re.sub(r"//[^\n]*", "", way)
        assert "fence_proxy_async_smem();" in way
        assert way.index("fence_proxy_async_smem();") < way.index("__syncwarp();")


def case(dtype, N, K, off=0, seed=0):
    """Some 700 groups of 0 to 45 rows: operands, 64-bit products by row, offsets."""
    gen = torch.Generator().manual_seed(seed)
    sizes = torch.randint(0, 46, (700,), generator=gen)
    at = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)])
    rows = int(at[-1])

    def new(*shape, std=1.0):
        return (torch.randn(shape, generator=gen) * std).to(DT[dtype]).cuda()
    A, B = new(rows, K), new(700, K, N, std=0.2)
    return A, B, at, rows, new


def products(A, B, at, alpha, bias=None):
    """U and its bound (fused_ref.py), group by group."""
    got = [ref.product(A[lo:hi].double(), B[g].double(), alpha, None if bias is None else bias[g].double())
           for g, (lo, hi) in enumerate(zip(at.tolist(), at[1:].tolist()))]
    return torch.cat([u for u, _ in got]), torch.cat([e for _, e in got])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("N,K", [(520, 16), (264, 72)])
def test_cut_boxes(lib_path, gpu, dtype, N, K):
    from dense_gemm_tiled_gb300 import binding as g
    A, B, at, rows, new = case(dtype, N, K)
    offs = at.to(torch.int32).cuda()
    bias, R = new(700, N), new(rows, N)
    u, eu = products(A, B, at, 1.25, bias)
    y, ey = ref.act(u, "gelu") + 0.5 * R.double(), 1.13 * eu + 2.0 ** -22 * (2 * u.abs() + R.double().abs())
    ey = ey + ref.rounding(y.abs() + ey, dtype)
    first = None
    for i in range(12):
        Y = R.clone() if i % 3 == 1 else torch.full_like(R, float("nan"))
        if i % 3 == 2:  # (results off 16-byte alignment: every box leaves row by row)
            Y = torch.empty(rows * N + 1, dtype=R.dtype, device="cuda")[1:].view(rows, N)
        g.gemm_grouped(A, B, Y, offs, alpha=1.25, bias=bias, act="gelu",
                       residual=Y if i % 3 == 1 else R, beta=0.5)
        assert g.last_path() == "fused_tc"
        if first is None:
            ref.check(Y, y, ey)
            first = Y
        assert torch.equal(Y, first), i
    # the slope of a kept U, in place and apart, and its column sums
    U = new(rows, N, std=2.0)
    p, ep = products(A, B, at, 0.75)
    d = p * ref.slope(U.double(), "gelu")
    ed = 1.13 * ep + 2.0 ** -20 * p.abs()
    first = None
    for i in range(8):
        dX = U.clone() if i % 2 else torch.full_like(U, float("nan"))
        db = torch.full((700, N), float("nan"), device="cuda")
        g.gemm_grouped_backward(A, B, dX, offs, dX if i % 2 else U, alpha=0.75, dbias=db)
        if first is None:
            ref.check(dX, d, ed + ref.rounding(d.abs() + ed, dtype))
            for e, (lo, hi) in enumerate(zip(at.tolist(), at[1:].tolist())):
                bound = ed[lo:hi].sum(0) + (hi - lo + 8) * 2.0 ** -23 * d[lo:hi].abs().sum(0)
                ref.check(db[e], d[lo:hi].sum(0), bound, e)
            first = dX, db
        assert torch.equal(dX, first[0]) and torch.equal(db, first[1]), i
    torch.cuda.synchronize()
    assert g.check_device_status() == g.OK


@pytest.mark.gpu
@pytest.mark.parametrize("tile", [0, 1, 2, 3])
def test_cut_boxes_of_every_tile(lib_path, gpu, tile):
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-q", "-x", "-m", "gpu",
                        "-k", "test_cut_boxes and not every_tile"],
                       env=dict(os.environ, GEMM_GB300_FUSED_TILE=str(tile)), capture_output=True,
                       text=True, timeout=600, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
