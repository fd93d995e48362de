"""Stored operands at the ends of their ranges: signs of zeros, padding after a
negative factor, scales far from 1 whose products are ordinary numbers, 16-bit
values that would overflow before their scale is applied, and scales that are no
fp16 numbers."""
import numpy as np
import pytest
import torch

import mx_ref
from helpers import to_np
from oracle import compare

pytestmark = pytest.mark.gpu

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


def check(C, a, bT, dtype):
    res = compare.check(to_np(C), a @ bT, np.abs(a) @ np.abs(bT), dtype)
    assert res["ok"], res


@pytest.mark.parametrize("fmt", ["fp4", "fp4_e4m3"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("trans", [False, True])
def test_zeros_keep_their_sign(g, fmt, dtype, trans):
    """In blocks of zeros alone and beside other values; a value too small for a
    code is a zero of its sign as well."""
    gen = torch.Generator().manual_seed(4)
    x = torch.randn((40, 200), generator=gen)
    x[:, ::3], x[:, ::6], x[:, 1::7], x[7, :70] = 0.0, -0.0, -2.0 ** -9, -0.0
    x = x.to(DT[dtype])
    Q = g.mx_empty(40, 200, fmt)
    g.mx_quantize((x.t() if trans else x).contiguous().cuda(), Q, transX=trans)
    codes, st, _ = mx_ref.store(x.double().numpy(), fmt)
    assert np.array_equal(Q.scales.cpu().numpy(), st)
    assert np.array_equal(Q.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("fmt", list(mx_ref.BLOCK))
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("trans", [False, True])
def test_padding_after_a_negative_factor(g, fmt, dtype, trans):
    """Codes past a row's last column are zero bytes whatever mult's sign; zeros
    inside it keep theirs (-1 * 0 is -0)."""
    for rows, cols in [(1, 1), (3, 17), (130, 77), (33, 259), (70, 129)]:
        gen = torch.Generator().manual_seed(cols)
        x = torch.randn((rows, cols), generator=gen).to(DT[dtype])
        x[:, ::5] = 0.0
        x[:, ::10] = -0.0
        Q = g.mx_empty(rows, cols, fmt)
        Q.codes.fill_(0xA5)
        X = (x.t() if trans else x).contiguous().cuda()
        g.mx_quantize(X, Q, transX=trans, mult=-1.0)
        codes, st, _ = mx_ref.store(x.double().numpy(), fmt, -1.0)
        assert np.array_equal(Q.scales.cpu().numpy(), st)
        assert np.array_equal(Q.codes.cpu().numpy(), codes), (rows, cols)


@pytest.mark.parametrize("shift", [124, -124, 125, -125])
def test_opposite_scales_of_two_stored_operands(g, shift):
    """Values about 2^124 and 2^-124 (2^125 and its inverse: scaled codes below 2^-126): every product of a
    block is an ordinary number, in whatever order the scales are applied."""
    for M, N, K in [(1, 40, 64), (7, 130, 700), (32, 200, 300)]:
        r = np.random.default_rng(M)
        A, a = stored(g, (r.standard_normal((M, K)) * 2.0 ** shift).astype(np.float32), "fp4")
        B, b = stored(g, (r.standard_normal((N, K)) * 2.0 ** -shift).astype(np.float32), "fp4")
        C = torch.empty((M, N), device="cuda")
        g.gemm_mx(A, B, C)
        assert g.last_path() == "mx_stream"
        check(C, a, b.T, "f32")


@pytest.mark.parametrize("shift", [124, -124, 125, -125])
def test_opposite_scales_on_the_tensor_core(g, shift):
    """The same past the streaming kernel's rows: the block-scaled MMA takes both
    scales at once."""
    for M, N, K in [(40, 50, 300), (200, 300, 600)]:
        r = np.random.default_rng(M)
        A, a = stored(g, (r.standard_normal((M, K)) * 2.0 ** shift).astype(np.float32), "fp4")
        B, b = stored(g, (r.standard_normal((N, K)) * 2.0 ** -shift).astype(np.float32), "fp4")
        C = torch.empty((M, N), device="cuda")
        g.gemm_mx(A, B, C)
        assert g.last_path() == "mx_tc"
        check(C, a, b.T, "f32")


def test_opposite_scales_keep_nan(g):
    r = np.random.default_rng(1)
    x = (r.standard_normal((5, 96)) * 2.0 ** 124).astype(np.float32)
    w = (r.standard_normal((40, 96)) * 2.0 ** -124).astype(np.float32)
    x[1, 40], w[3, 0], w[7] = np.nan, np.inf, 0.0
    (A, a), (B, b) = stored(g, x, "fp4"), stored(g, w, "fp4")
    C = torch.empty((5, 40), device="cuda")
    g.gemm_mx(A, B, C)
    want = np.zeros((5, 40), dtype=bool)
    want[1], want[:, 3] = True, True
    assert np.array_equal(torch.isnan(C).cpu().numpy(), want)
    assert torch.equal(C[[0, 2, 3, 4], 7].cpu(), torch.zeros(4))


@pytest.mark.parametrize("fmt", ["fp4", "fp4_e4m3"])
def test_large_bf16_rows_times_small_weights(g, fmt):
    """bf16 rows of 2^126: a sum of unscaled codes would leave fp32 while the
    products with the weights do not; the same for every number of rows."""
    r = np.random.default_rng(2)
    B, b = stored(g, (r.standard_normal((70, 320)) * 2.0 ** -5).astype(np.float32), fmt)
    for M in (1, 9, 32, 40):
        x = torch.from_numpy(r.uniform(0.5, 1.0, (M, 320)) * 2.0 ** 122).to(torch.bfloat16).cuda()
        x[:, ::7] *= 16.0
        C = torch.empty((M, 70), dtype=torch.bfloat16, device="cuda")
        g.gemm_mx(x, B, C, transB=True)
        check(C, f64(x), b.T, "bf16")


def test_fp16_rows_times_scales_past_fp16(g):
    """A power-of-two scale that is no fp16 number: up to 32 rows of A, with B
    stored [N, K], it stays in fp32; in every other product of 16-bit rows the
    values are rounded to fp16 first."""
    r = np.random.default_rng(3)
    w = r.standard_normal((96, 256)).astype(np.float32)
    w[0] *= 2.0 ** -20   # values of fp16's subnormal range
    w[1] *= 2.0 ** -40   # below it
    w[2] *= 2.0 ** 13    # scales up to 2^13, values within range
    w[3] *= 2.0 ** 30    # beyond it
    B, b = stored(g, w, "fp4")
    with np.errstate(over="ignore"):
        half = b.astype(np.float16).astype(np.float64)
    for M in (1, 32, 33, 100):
        gen = torch.Generator().manual_seed(M)
        A = torch.randn((M, 256), generator=gen).half().cuda() / 16
        C = torch.empty((M, 96), dtype=torch.float16, device="cuda")
        g.gemm_mx(A, B, C, transB=True)
        assert (g.last_path() == "mx_stream") == (M <= 32)
        v = b if M <= 32 else half
        keep = [j for j in range(96) if j != 3]
        check(C[:, keep].contiguous(), f64(A), v[keep].T, "f16")
        if M <= 32:  # finite products of about 2^30, past fp16 only in C
            want = (f64(A) @ b[3]).astype(np.float32)
            assert np.all(np.abs(want) > 65520) and np.array_equal(f64(C[:, 3]), np.sign(want) * np.inf)
        else:
            assert not torch.isfinite(C[:, 3]).any()
    # stored [K, N]: always rounded
    At = torch.randn((4, 96), generator=torch.Generator().manual_seed(5)).half().cuda() / 16
    At[:, 3] = 0.25
    C = torch.empty((4, 256), dtype=torch.float16, device="cuda")
    g.gemm_mx(At, B, C)
    big = np.abs(b[3]) > 65520
    keep = np.flatnonzero(~big)
    check(C[:, keep].contiguous(), f64(At), half[:, keep], "f16")
    assert not torch.isfinite(C[:, np.flatnonzero(big)]).any()
