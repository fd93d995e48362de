"""gelu and its slope in mx_quantize and mx_act_backward against 64 bits, within
what the arithmetic of each type can lose (u = 2^-24, half an ulp of fp32).

fp32: x Phi(x) = max(x, 0) - |x| Phi(-|x|) with CUDA's normcdff (within 5 ulp: 10
u) and one FMA; the slope, h = Phi(-|x|) - |x| phi(x) below 0 and 1 - h above,
with expf (2 ulp: 4 u; its argument x^2 / 2 rounded once: x^2 / 2 u of the result),
three more roundings on phi's term and one on each sum.

16-bit types: the rational form 7.1.26 of Abramowitz and Stegun.  Its own error is
evaluated here in 64 bits at every point; of its evaluation in fp32,
  t = 1 / (1 + p z)   constants 3 u, sum u, reciprocal 2 u: 6 u, which the
                      polynomial carries on at most 3.5-fold (its condition at
                      t = 1): 21 u
  polynomial          five FMAs over terms that sum to at most 4.5 times the
                      result: 49 u
  exp(-x^2 / 2)       argument 1.5 x^2 u, exponential 4 u, two products 2 u
in all (76 + 1.5 x^2) u of Phi(-|x|); then the rounding to the type.
"""
import math

import numpy as np
import pytest
import torch

import mx_ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = 2.0 ** -24
HALF_ULP = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
HALF_SUB = {"f32": 2.0 ** -140, "f16": 2.0 ** -25 * 1.001, "bf16": 2.0 ** -120}


@pytest.fixture(autouse=True)
def _lib(lib_path, gpu):
    yield


@pytest.fixture
def g():
    from dense_gemm_tiled_gb300 import binding
    return binding


def f64(t):
    return t.detach().double().cpu().numpy()


def tail(a):
    """Phi(-a) in 64 bits."""
    return 0.5 * np.vectorize(math.erfc, otypes=[np.float64])(a / math.sqrt(2.0))


def method_error(a):
    """|7.1.26 - erfc| / 2 at a / sqrt 2, in 64 bits."""
    z = a / math.sqrt(2.0)
    t = 1 / (1 + 0.3275911 * z)
    p = t * (0.254829592 + t * (-0.284496736 + t * (1.421413741 + t * (-1.453152027 +
                                                                       t * 1.061405429))))
    return np.abs(0.5 * p * np.exp(-z * z) - tail(a))


def rounded(bound, want, dtype):
    """The bound before rounding to the type, and that rounding."""
    if dtype == "f32":
        return bound + HALF_SUB[dtype]
    return bound + HALF_ULP[dtype] * (np.abs(want) + bound) + HALF_SUB[dtype]


def points(dtype):
    """Both signs, dense where the tail's terms nearly cancel, out to where the
    tail leaves fp32."""
    x = torch.cat([torch.linspace(-14, 14, 20001), torch.linspace(-1.2, -0.3, 4001),
                   torch.linspace(-5.5, -3.5, 4001), torch.randn(3012, generator=torch.Generator().manual_seed(1))])
    return x.to(DT[dtype])[: x.numel() // 32 * 32].view(-1, 32).contiguous()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("extra", [0, 1])
def test_gelu(g, dtype, extra):
    X = points(dtype).cuda()
    if extra:  # rows off 16-byte alignment
        base = torch.empty((X.shape[0], 33), dtype=X.dtype, device="cuda")
        base[:, :32] = X
        X = base[:, :32]
    Y = torch.empty_like(X) if not extra else torch.empty_like(base)[:, :32]
    g.mx_quantize(X, g.mx_empty(*X.shape, "int8"), act="gelu", Y=Y)
    x, y = f64(X), f64(Y)
    a = np.abs(x)
    want = np.where(x > 0, x, 0.0) - a * tail(a)
    if dtype == "f32":
        bound = 10 * U * a * tail(a) + U * np.abs(want)
    else:
        bound = a * (method_error(a) + (76 + 1.5 * a * a) * U * tail(a)) + U * np.abs(want)
    bad = np.abs(y - want) > rounded(bound, want, dtype)
    assert not bad.any(), (x[bad][:5], y[bad][:5], want[bad][:5])


@pytest.mark.parametrize("dtype", list(DT))
def test_gelu_slope(g, dtype):
    """At the values of the checkpoint, for gradients of many sizes."""
    X = points(dtype).cuda()
    gen = torch.Generator().manual_seed(2)
    dY = torch.randn(X.shape, generator=gen).to(DT[dtype]).cuda()
    Q, dX = g.mx_empty(*X.shape, "int8"), torch.empty_like(X)
    g.mx_quantize(X, Q)
    g.mx_act_backward(dY, Q, dX)
    x = mx_ref.load(Q.codes.cpu().numpy(), Q.scales.cpu().numpy(), *X.shape, "int8")
    dy, a = f64(dY), np.abs(x)
    phi = np.exp(-a * a / 2) / math.sqrt(2 * math.pi)
    h = tail(a) - a * phi
    s = np.where(x < 0, h, 1 - h)
    if dtype == "f32":
        e = 10 * U * tail(a) + (8 + a * a / 2) * U * a * phi
    else:
        e = method_error(a) + (76 + 1.5 * a * a) * U * tail(a) + (10 + 1.5 * a * a) * U * a * phi
    e = e + U * np.abs(h) + np.where(x < 0, 0.0, U)
    want = dy * s
    bound = np.abs(dy) * e + U * np.abs(want)
    bad = np.abs(f64(dX) - want) > rounded(bound, want, dtype)
    assert not bad.any(), (x[bad][:5], f64(dX)[bad][:5], want[bad][:5])


def test_fp32_gelu_beside_the_epilogues(g):
    """A GEMM's fused gelu and mx_quantize's on the same fp32 values: the former
    is v / 2 (1 + erff(v / sqrt 2)), where erff is within 2 ulp (4 u), its argument
    2 u off (at most 0.97 of which reach Phi's twice the value) and the sum rounded
    to u: 8 u of |v| / 2 (1 + erf) at most |v|, besides the latter's own bound."""
    X = points("f32").cuda()
    n, Y = X.shape[1], torch.empty_like(X)
    g.mx_quantize(X, g.mx_empty(*X.shape, "int8"), act="gelu", Y=Y)
    C = torch.empty_like(X)
    g.gemm(X, torch.eye(n, device="cuda"), C, act="gelu")
    x, a = f64(X), np.abs(f64(X))
    assert np.all(np.abs(f64(C) - f64(Y)) <= 8 * U * a + 10 * U * a * tail(a) + 2.0 ** -140)


def test_relu_of_a_bad_block(g):
    """relu is v > 0 ? v : 0 and its slope 1 where x > 0, 0 elsewhere, as in the
    GEMM epilogue: a NaN becomes 0 forward, and a block that holds one (its
    checkpoint is NaN) passes no gradient; gelu passes NaN on."""
    x = torch.ones((2, 64))
    x[0, 3], x[0, 40], x[1, 33] = float("nan"), -1.0, float("inf")
    for dtype in DT.values():
        X, dY = x.to(dtype).cuda(), torch.full((2, 64), 2.0, dtype=dtype, device="cuda")
        Q, Y, dX = g.mx_empty(2, 64, "int8"), torch.empty_like(X), torch.empty_like(X)
        g.mx_quantize(X, Q, act="relu", Y=Y)
        assert Y[0, 3] == 0 and Y[0, 40] == 0 and torch.isinf(Y[1, 33])
        g.mx_act_backward(dY, Q, dX, act="relu")
        want = torch.full((2, 64), 2.0)
        want[0, :32], want[0, 40], want[1, 32:] = 0.0, 0.0, 0.0
        assert torch.equal(dX.float().cpu(), want)
        g.mx_act_backward(dY, Q, dX, act="gelu")
        assert torch.isnan(dX[0, :32]).all() and torch.isnan(dX[1, 32:]).all()
        assert torch.isfinite(dX[0, 32:]).all() and torch.isfinite(dX[1, :32]).all()
