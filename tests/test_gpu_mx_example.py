"""The LoRA block of examples/lora_mlp_block.py: its step against the formulas in
64 bits on the values that its stored operands stand for, and gelu's backward
pass against differences of the forward pass."""
import os
import sys

import numpy as np
import pytest
import torch

import mx_ref
from helpers import to_np
from oracle import compare

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def f64(t):
    return t.detach().double().cpu().numpy()


def values(Q):
    return mx_ref.load(Q.codes.cpu().numpy(), Q.scales.cpu().numpy(), Q.rows, Q.cols, Q.fmt)


def near(got, a, b, dtype, extra=None):
    """got against a @ b within the GEMM's bound, plus `extra`."""
    ref, mag = a @ b, np.abs(a) @ np.abs(b)
    if extra is not None:
        ref, mag = ref + extra, mag + np.abs(extra)
    res = compare.check(to_np(got), ref, mag, dtype)
    assert res["ok"], res


@pytest.mark.parametrize("T", [1, 40, 130])
def test_block_step(lib_path, gpu, T):
    from lora_mlp_block import Block
    blk = Block(d=192, F=330, r=8)
    gen = torch.Generator().manual_seed(T)
    x, dout = (torch.randn((T, 192), generator=gen).half().cuda() for _ in range(2))
    out, saved = blk.forward(x)
    dx, dA, dB, dbias = blk.backward(dout, saved)
    torch.cuda.synchronize()
    x8, h8, xa = saved
    W1, W2, A, B = values(blk.W1), values(blk.W2), f64(blk.A), f64(blk.B)
    # each stage from what the one before it wrote (16-bit tensors round between)
    near(xa, f64(x), A.T, "f16")
    h = f64(x) @ W1.T + f64(xa) @ B.T + f64(blk.bias)
    step = np.repeat(2.0 ** np.floor(np.log2(np.maximum(np.abs(h), 1e-9))).max(1, keepdims=True), 330, 1)
    # the checkpoint: half a step of its block (at most 2^-6 of the row's largest
    # power of two) and the two fp16 roundings of h on its way
    assert np.all(np.abs(values(h8) - h) <= step * 2.0 ** -6 + 2.0 ** -9 * (np.abs(h) + 1))
    dy = f64(dout) @ W2
    dh = dy * mx_ref.slope(values(h8), "gelu")
    # dbias: fp16 dy (2^-11, and 1e-4 of its terms' sum) times a slope of at most 1.13
    err = 1.13 * (2.0 ** -10 * np.abs(dy) + 1e-4 * (np.abs(f64(dout)) @ np.abs(W2)) + 2.0 ** -20)
    assert np.all(np.abs(f64(dbias) - dh.sum(0)) <= err.sum(0))
    # the adapter's gradients from the tensors that the step itself used
    dh16 = dh.astype(np.float16).astype(np.float64)
    rel = lambda got, want: np.linalg.norm(f64(got) - want) / np.linalg.norm(want)  # noqa: E731
    # (fp16 roundings of dy, dh, dh B and the result, each 2^-11 of a term)
    assert rel(dB, dh16.T @ f64(xa)) < 4 * 2.0 ** -10
    assert rel(dA, (dh16 @ B).T @ values(x8)) < 6 * 2.0 ** -10
    assert rel(dx, dh16 @ W1 + (dh16 @ B) @ A) < 6 * 2.0 ** -10


def test_gelu_gradient_against_differences(lib_path, gpu):
    """At values that the checkpoint holds exactly, dX for dY = 1 against central
    differences of the forward pass, fp32: h^2 / 6 max|f'''| (below 1.2 * h^2 / 6)
    and two evaluations' errors (2^-20 (|x| + |y|) each) over 2 h."""
    from dense_gemm_tiled_gb300 import binding as g
    # every block's largest magnitude is 4: steps of 1/16
    x = (torch.arange(-64, 64, dtype=torch.float32) / 16).view(4, 32)
    x[:, 0] = 4.0
    Q, dX = g.mx_empty(4, 32, "int8"), torch.empty((4, 32), device="cuda")
    g.mx_quantize(x.cuda(), Q)
    assert torch.equal(g.mx_dequantize(Q, torch.empty((4, 32), device="cuda")).cpu(), x)
    g.mx_act_backward(torch.ones((4, 32), device="cuda"), Q, dX)
    h = 2.0 ** -6
    y = []
    for s in (h, -h):
        Y = torch.empty((4, 32), device="cuda")
        g.mx_quantize((x + s).cuda(), g.mx_empty(4, 32, "int8"), act="gelu", Y=Y)
        y.append(f64(Y))
    diff = (y[0] - y[1]) / (2 * h)
    tol = 1.2 * h * h / 6 + 2 * 2.0 ** -20 * 2 * (np.abs(f64(x)) + h) / (2 * h)
    assert np.all(np.abs(f64(dX) - diff) <= tol)
