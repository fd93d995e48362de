"""Fused and grouped products: every finite 16-bit value through gelu, relu and their slopes;
columns of a wider result that are written as well as those that are not; forward passes of
offsets that do not ascend, with guards around every result."""
import pytest
import torch

import fused_ref as ref
from fused_ref import DT

pytestmark = pytest.mark.gpu


@pytest.fixture
def g(lib_path, gpu):
    from dense_gemm_tiled_gb300 import binding
    yield binding
    torch.cuda.synchronize()
    assert binding.check_device_status() == binding.OK


def matrix(shape, dtype, seed, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * std).to(DT[dtype]).cuda()


def finite(dtype):
    v = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(DT[dtype])
    v = v[v.isfinite()].contiguous()
    assert v.numel() == 65536 - {"f16": 2048, "bf16": 256}[dtype]
    assert v.max() == torch.finfo(DT[dtype]).max and v.min() == torch.finfo(DT[dtype]).min
    return v


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [20, 3])  # (either kernel)
def test_activations_of_every_16_bit_value(g, dtype, rows):
    v = finite(dtype)
    x, n = v.double(), v.numel()
    zero = torch.zeros((rows, 16), dtype=DT[dtype], device="cuda")
    W = torch.ones((n, 16), dtype=DT[dtype], device="cuda")
    Y, U = (torch.empty((rows, n), dtype=DT[dtype], device="cuda") for _ in range(2))
    g.gemm_fused(zero, W, Y, transB=True, bias=v, act="gelu", preact=U)
    assert torch.equal(U, v.expand(rows, n))
    # Phi within 1.5e-7 of itself, times |x|: 2^-22 |x|; beyond 20 it is 0 or 1
    y, e = ref.act(x, "gelu"), torch.where(x.abs() > 20, 0.0, 2.0 ** -22 * x.abs())
    ref.check(Y, y.expand(rows, n), (e + ref.rounding(y.abs() + e, dtype)).expand(rows, n), "gelu")
    assert (Y[:, x > 20] == v[x > 20]).all() and (Y[:, x < -20] == 0).all()
    g.gemm_fused(zero, W, Y, transB=True, bias=v, act="relu")
    assert torch.equal(Y, torch.relu(v).expand(rows, n))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_slopes_of_every_16_bit_value(g, dtype):
    v = finite(dtype)
    x, n = v.double(), v.numel()
    one = torch.zeros((20, 16), dtype=DT[dtype], device="cuda")
    one[:, 0] = 1
    W = torch.ones((n, 16), dtype=DT[dtype], device="cuda")
    U, dX = v.expand(20, n).contiguous(), torch.empty((20, n), dtype=DT[dtype], device="cuda")
    g.gemm_fused_backward(one, W, dX, U, transB=True)
    d = ref.slope(x.clamp(-40, 40), "gelu")  # (whose x * x is finite; it is 0 or 1 there)
    e = torch.where(x.abs() > 20, 0.0, 2.0 ** -20)
    ref.check(dX, d.expand(20, n), (e + ref.rounding(d.abs() + e, dtype)).expand(20, n), "slope")
    g.gemm_fused_backward(one, W, dX, U, transB=True, act="relu")
    assert torch.equal(dX, (v > 0).to(DT[dtype]).expand(20, n))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [70, 5])
@pytest.mark.parametrize("width,lo,hi", [(100, 3, 92), (160, 16, 104)])
def test_written_columns(g, dtype, rows, width, lo, hi):
    N = hi - lo
    A, B = matrix((rows, 24), dtype, 1), matrix((N, 24), dtype, 2)
    bufs = [torch.full((rows, width), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    Y, U = (b[:, lo:hi] for b in bufs)
    g.gemm_fused(A, B, Y, transB=True, act="relu", preact=U)
    u, eu, y, ey = ref.forward(A.double(), B.double().t(), dtype, name="relu")
    ref.check(Y, y, ey)
    ref.check(U, u, eu)
    for b in bufs:
        assert (b[:, :lo] == 7).all() and (b[:, hi:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows", [300, 16, 12, 5])
@pytest.mark.parametrize("transB", [False, True])
def test_offsets_that_do_not_ascend_forward(g, dtype, rows, transB):
    """Nothing outside the results is written, whichever kernel takes the call (the rows
    that wrong groups share hold unspecified values), and the status says so."""
    E, N, K = 40, 72, 40
    r, far = rows, 2 ** 31 - 1
    bads = [[0, r] * 20 + [0], [r] + [0] * 39 + [r], [-5, 2, 2, r] + [r + 1] * 37,
            [0, far, -far] + list(range(38)), [-far] * 20 + [far] * 21, [1, 0] * 20 + [r]]
    A, B = matrix((rows, K), dtype, 1), matrix((E, N, K) if transB else (E, K, N), dtype, 2)
    b, R = matrix((E, N), dtype, 3), matrix((rows, N), dtype, 4)
    for bad in bads:
        offs = torch.tensor(bad, dtype=torch.int64).to(torch.int32).cuda()
        guards = [torch.full((rows + 64, N), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
        Y, U = (t[32:-32] for t in guards)
        g.gemm_grouped(A, B, Y, offs, transB=transB, bias=b, act="gelu", residual=R, preact=U)
        assert g.check_device_status() == g.ERR_INVALID_ARG, bad
        for t in guards:
            assert (t[:32] == 7).all() and (t[-32:] == 7).all()
    # the next call is right
    at = [0, rows // 2] + [rows] * (E - 1)
    offs = torch.tensor(at, dtype=torch.int32, device="cuda")
    Y = torch.empty_like(R)
    g.gemm_grouped(A, B, Y, offs, transB=transB)
    for e in (0, 1):
        lo, hi = at[e], at[e + 1]
        _, _, y, ey = ref.forward(A[lo:hi].double(), B[e].double().t() if transB else B[e].double(), dtype)
        ref.check(Y[lo:hi], y, ey, e)
