"""Results whose rows begin on 16 bytes and end anywhere, inside a wider buffer: every path
writes all of a row and nothing behind it."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
COLS = (1, 2, 3, 4, 5, 7, 8, 9, 31, 33, 65, 66, 127, 130, 257, 420)
ROWS = (1, 2, 20, 40, 129, 300)
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# What is stored of a one: a fp4_e4m3 block's scale is 1 / 6 rounded to e4m3, whose steps
# there are 1 / 64: 11 / 64, and the code 6 reads as 66 / 64 = 1.03125.
ONE = {"fp4": 1.0, "int8": 1.0, "fp4_e4m3": 1.03125}


@pytest.fixture
def g(lib_path, gpu):
    from dense_gemm_tiled_gb300 import binding
    yield binding
    torch.cuda.synchronize()
    assert binding.check_device_status() == binding.OK


class Inside:
    """[rows, n] (or [b, rows, n]) of aligned rows inside a buffer of sevens."""

    def __init__(self, dt, *shape, off=0):
        *outer, n = shape
        ld = (n + 7) // 8 * 8 + 8
        at = 2048 + off
        self.buf = torch.full((4096 + ld * torch.Size(outer).numel(),), 7.0, dtype=dt, device="cuda")
        strides = (ld, 1) if len(outer) == 1 else (ld * outer[1], ld, 1)
        self.t = self.buf.as_strided(shape, strides, at)
        self.t.fill_(2.0)
        self.out = torch.ones_like(self.buf, dtype=torch.bool)
        self.out.as_strided(shape, strides, at).fill_(False)

    def check(self, value, what):
        assert (self.t == value).all(), (what, self.t.flatten()[:4].tolist())
        assert (self.buf[self.out] == 7).all(), (what, (self.out & (self.buf != 7)).nonzero().flatten()[:8].tolist())


def ones(dt, *shape):
    return torch.ones(shape, dtype=dt, device="cuda")


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("dtype,opt", [("f16", {}), ("bf16", {}), ("f32", {}), ("f32", dict(tf32=True)),
                                       ("f32", dict(tf32x3=True))])
def test_gemm(g, dtype, opt, M):
    dt = DT[dtype]
    for N in COLS:
        for K in (16, 240):
            for ta, tb in ((False, False), (False, True), (True, False)):
                A, B = ones(dt, *((K, M) if ta else (M, K))), ones(dt, *((N, K) if tb else (K, N)))
                for beta, bias in ((0.0, None), (0.5, None), (0.0, ones(dt, N))):
                    if bias is not None and opt:
                        continue
                    C = Inside(dt, M, N)
                    g.gemm(A, B, C.t, ta, tb, beta=beta, bias=bias, **opt)
                    C.check(K + 2 * beta + (bias is not None), (M, N, K, ta, tb, beta, g.last_path()))


@pytest.mark.parametrize("dtype,opt", [("f16", {}), ("bf16", {}), ("f32", dict(tf32=True))])
@pytest.mark.parametrize("off", [0, 1])
def test_large(g, dtype, opt, off):
    """Many tiles a worker, shared tiles, block pairs; rows off alignment through an aligned copy."""
    dt = DT[dtype]
    for M, N, K in ((1500, 1501, 64), (1037, 2050, 240), (130, 2049, 2000), (3000, 705, 200)):
        A, B = ones(dt, M, K), ones(dt, N, K)
        for beta in (0.0, 0.5):
            C = Inside(dt, M, N, off=off)
            g.gemm(A, B, C.t, False, True, alpha=0.125, beta=beta, **opt)
            C.check(K / 8 + 2 * beta, (M, N, K, beta, g.last_path()))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
def test_batched(g, dtype):
    dt = DT[dtype]
    for M, N, K in ((40, 33, 64), (1, 5, 16), (130, 130, 64), (257, 65, 240)):
        A, B, C = ones(dt, 5, M, K), ones(dt, 5, N, K), Inside(dt, 5, M, N)
        g.gemm_strided_batched(A, B, C.t, False, True)
        C.check(K, (M, N, K, g.last_path()))


@pytest.mark.parametrize("fmt", ["fp4", "fp4_e4m3", "int8"])
@pytest.mark.parametrize("M", ROWS)
def test_stored_operands(g, fmt, M):
    paths = set()
    for N in COLS:
        for K in (64, 240):
            W = g.mx_empty(N, K, fmt)
            g.mx_quantize(ones(torch.float16, N, K), W)
            V = g.mx_empty(K, N, fmt)
            g.mx_quantize(ones(torch.float16, K, N), V)
            X = g.mx_empty(M, K, fmt)
            g.mx_quantize(ones(torch.float16, M, K), X)
            for dtype in ("f16", "bf16", "f32"):
                dt = DT[dtype]
                calls = [(ones(dt, M, K), W, dict(transB=True)), (ones(dt, M, K), V, {}),
                         (ones(dt, K, M), V, dict(transA=True))]
                if fmt != "int8":
                    calls.append((X, W, {}))
                for A, B, opt in calls:
                    for beta in (0.0, 0.5):
                        C = Inside(dt, M, N)
                        g.gemm_mx(A, B, C.t, beta=beta, **opt)
                        paths.add(g.last_path())
                        # (sums of so few bits are exact in fp32, and rounded once)
                        one = ONE[fmt] ** (2 if A is X else 1)
                        C.check(torch.tensor(K * one + 2 * beta, dtype=torch.float64).to(dt).cuda(), (fmt, dtype, M, N, K, opt, beta, g.last_path()))
    assert len(paths) >= 2, paths


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M", ROWS)
def test_elementwise(g, dtype, M):
    dt = DT[dtype]
    for N in COLS:
        for fmt in ("int8", "fp4", "fp4_e4m3"):
            Q, Y = g.mx_empty(M, N, fmt), Inside(dt, M, N)
            g.mx_quantize(ones(dt, M, N), Q, act="relu", Y=Y.t)
            Y.check(1, (fmt, "Y", M, N))
            D = Inside(dt, M, N)
            g.mx_dequantize(Q, D.t)
            D.check(ONE[fmt], (fmt, "dequantize", M, N))
            if fmt == "int8":
                X = Inside(dt, M, N)
                g.mx_act_backward(ones(dt, M, N), Q, X.t, act="relu")
                X.check(1, (fmt, "backward", M, N))


@pytest.mark.parametrize("ctma", ["0", "2"])
def test_stores_of_either_kind(lib_path, gpu, ctma):
    """(the switch is read once per process)"""
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.abspath(__file__), "-q", "-x", "-m", "gpu",
                        "-k", "test_large or test_gemm and 300 or test_batched"],
                       env=dict(os.environ, GEMM_GB300_HG_CTMA=ctma), capture_output=True, text=True,
                       timeout=600, cwd=os.path.dirname(HERE))
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-2000:]
