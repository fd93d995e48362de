"""Microscaled operands without a GPU: the reference's own pins (hand-worked
values, the gradient against differences), the storage sizes, and every refusal
of the entry points before anything is launched."""
import ctypes
import math

import numpy as np
import pytest

import mx_ref


# ---------------------------------------------------------------- the reference
def test_reference_blocks_by_hand():
    x = np.zeros((1, 32))
    # amax 7: 2^(2 - 2) = 1; 7 saturates to 6, 5 is a tie (4 and 6: 4 is even),
    # 2.5 a tie (2 and 3: 2), 0.25 a tie (0 and .5: 0), 1.75 a tie (1.5, 2: 2)
    x[0, :7] = [7, 5, 2.5, 0.25, -1.75, -0.75, 3.4]
    codes, st, v = mx_ref.store(x, "fp4")
    assert st[0] == 127 and list(v[0, :7]) == [6, 4, 2, 0, -2, -1, 3]
    assert codes[0, 0] == (7 | 6 << 4) and codes[0, 2] == (0xC | 0xA << 4)
    # int8: amax 3 -> 2^(1 - 6) = 1/32; 3 * 32 = 96; 0.015625 * 32 = .5 -> 0
    x = np.zeros((1, 32)); x[0, :3] = [3, 0.015625, -0.046875]
    codes, st, v = mx_ref.store(x, "int8")
    assert st[0] == 122 and codes[0, 0] == 96 and codes[0, 1] == 0 and codes[0, 2] == 254
    # just under a power of two rounds past the largest code and stays there
    x = np.zeros((1, 32)); x[0, 0] = 1.9999
    assert mx_ref.store(x, "int8")[2][0, 0] == 127 / 64
    # e4m3: amax 3 -> scale 0.5; 0.125 / .5 = .25 is a tie
    x = np.zeros((1, 16)); x[0, :3] = [3, 0.125, 0.2]
    codes, st, v = mx_ref.store(x, "fp4_e4m3")
    assert st[0] == 0x30 and list(v[0, :3]) == [3, 0, 0.25]


@pytest.mark.parametrize("fmt", list(mx_ref.BLOCK))
def test_reference_store_and_load_agree(fmt):
    r = np.random.default_rng(1)
    for rows, cols in [(1, 1), (3, 17), (130, 77), (5, 129), (2, 300)]:
        x = r.standard_normal((rows, cols)).astype(np.float32)
        codes, st, v = mx_ref.store(x, fmt)
        assert np.array_equal(mx_ref.load(codes, st, rows, cols, fmt), v)
        # the step at a block's largest value bounds the error of each element
        b = mx_ref.BLOCK[fmt]
        amax = np.array([[np.abs(x[i, j // b * b:(j // b + 1) * b]).max() for j in range(cols)]
                         for i in range(rows)])
        worst = {"fp4": 1 / 4, "fp4_e4m3": 1 / 6 + 1 / 16, "int8": 1 / 64}[fmt]
        assert np.all(np.abs(v - x) <= worst * amax)


@pytest.mark.parametrize("act", ["gelu", "none"])
def test_reference_slope_against_differences(act):
    x = np.linspace(-6, 6, 241)
    f = mx_ref.gelu if act == "gelu" else (lambda t: t)
    h = 1e-5
    # central difference: h^2/6 max|f'''| (below 2) plus 64-bit rounding over h
    assert np.all(np.abs((f(x + h) - f(x - h)) / (2 * h) - mx_ref.slope(x, act)) < 1e-9)


# ---------------------------------------------------------------- the library
@pytest.fixture(scope="module")
def b(lib_path):
    from dense_gemm_tiled_gb300 import binding
    return binding


@pytest.mark.parametrize("fmt", list(mx_ref.BLOCK))
def test_sizes(b, fmt):
    for rows, cols in [(0, 0), (1, 1), (1, 33), (128, 128), (129, 513), (7, 2**31 - 1)]:
        assert b.mx_row_bytes(fmt, cols) == mx_ref.row_bytes(fmt, cols)
        nb = -(-cols // mx_ref.BLOCK[fmt])
        assert b.mx_scale_bytes(fmt, rows, cols) == -(-rows // 128) * -(-nb // 4) * 512
    assert b._lib.gemm_mx_row_bytes(3, 4) == -1 and b._lib.gemm_mx_row_bytes(0, -1) == -1
    assert b._lib.gemm_mx_scale_bytes(0, 1 << 31, 4) == -1


# fake, aligned, disjoint device addresses (never dereferenced: the call fails)
X, Y, Q, S, D, BQ, BS = (0x100000000 * i for i in range(1, 8))
OK, INV, UNS, ALIAS = 0, 1, 2, 3


def quant(**k):
    a = dict(format=0, transX=0, rows=4, cols=64, dtype=0, mult=1.0, X=X, ldx=64, act=0, Y=None,
             ldy=0, q=Q, ldq=32, s=S)
    a.update(k)
    return list(a.values()) + [None]


@pytest.mark.parametrize("k,code", [
    (dict(format=3), INV), (dict(format=-1), INV), (dict(transX=2), INV), (dict(dtype=3), INV),
    (dict(act=3), INV), (dict(act=2), INV), (dict(mult=math.inf), INV), (dict(mult=math.nan), INV),
    (dict(rows=-1), INV), (dict(cols=-1), INV), (dict(rows=1 << 31), UNS), (dict(ldx=63), INV),
    (dict(X=None), INV), (dict(X=X + 2), INV), (dict(ldq=16), INV), (dict(ldq=40), INV),
    (dict(q=Q + 8), INV), (dict(q=None), INV), (dict(s=None), INV), (dict(s=S + 4), INV),
    (dict(transX=1, ldx=3), INV), (dict(Y=Y, ldy=63), INV), (dict(Y=Y, ldy=64, transX=1, ldx=4), UNS),
    (dict(q=X + 64), ALIAS), (dict(s=X), ALIAS), (dict(q=S + 256), ALIAS),
    (dict(Y=X + 4, ldy=64), ALIAS), (dict(Y=X, ldy=65), ALIAS), (dict(Y=Q, ldy=64), ALIAS),
    (dict(rows=0, X=None), OK), (dict(cols=0, X=None), OK),
])
def test_quantize_refusals(b, k, code):
    assert b._lib.gemm_mx_quantize(*quant(**k)) == code
    assert b.last_path() == "none"


def dequant(**k):
    a = dict(format=0, rows=4, cols=64, q=Q, ldq=32, s=S, dtype=0, Y=Y, ldy=64)
    a.update(k)
    return list(a.values()) + [None]


@pytest.mark.parametrize("k,code", [
    (dict(format=7), INV), (dict(dtype=4), INV), (dict(rows=-1), INV), (dict(cols=1 << 31), UNS),
    (dict(ldy=63), INV), (dict(Y=Y + 1), INV), (dict(ldq=24), INV), (dict(q=Q + 1), INV),
    (dict(Y=Q + 4), ALIAS), (dict(Y=S), ALIAS), (dict(rows=0, q=None), OK),
])
def test_dequantize_refusals(b, k, code):
    assert b._lib.gemm_mx_dequantize(*dequant(**k)) == code


def act_bwd(**k):
    a = dict(rows=4, cols=64, dtype=1, act=2, dY=Y, lddy=64, q=Q, ldq=64, s=S, dX=X, lddx=64,
             dbias=D)
    a.update(k)
    return list(a.values()) + [None]


@pytest.mark.parametrize("k,code", [
    (dict(dtype=3), INV), (dict(act=4), INV), (dict(rows=-1), INV), (dict(cols=1 << 31), UNS),
    (dict(lddy=63), INV), (dict(dX=None), INV), (dict(dX=X + 1), INV), (dict(ldq=48), INV),
    (dict(dbias=D + 2), INV), (dict(dX=Y + 2), ALIAS), (dict(dX=Y, lddx=65), ALIAS),
    (dict(dX=Q), ALIAS), (dict(dbias=Y + 4), ALIAS), (dict(dbias=X), ALIAS),
    (dict(cols=0), OK), (dict(rows=0, dbias=None), OK),
])
def test_act_backward_refusals(b, k, code):
    assert b._lib.gemm_mx_act_backward(*act_bwd(**k)) == code


def mx4(**k):
    a = dict(format=0, M=4, N=8, K=64, dtype=1, alpha=1.0, beta=0.0, A=X, lda=32, As=S, B=BQ,
             ldb=32, Bs=BS, C=D, ldc=8, bias=None, act=0)
    a.update(k)
    return list(a.values()) + [None]


@pytest.mark.parametrize("k,code", [
    (dict(format=2), UNS), (dict(format=5), INV), (dict(dtype=3), INV), (dict(act=9), INV),
    (dict(M=-1), INV), (dict(N=1 << 31), UNS), (dict(ldc=7), INV), (dict(C=D + 1), INV),
    (dict(lda=16), INV), (dict(ldb=33), INV), (dict(A=X + 8), INV), (dict(Bs=None), INV),
    (dict(As=S + 2), INV), (dict(C=X), ALIAS), (dict(C=BS + 16), ALIAS), (dict(bias=D + 1), INV),
    (dict(bias=D + 4), ALIAS), (dict(M=0, A=None), OK), (dict(N=0), OK),
])
def test_mx4_refusals(b, k, code):
    assert b._lib.gemm_mx4(*mx4(**k)) == code


def mixed(**k):
    a = dict(format=0, tA=0, tB=1, M=4, N=8, K=64, dtype=1, alpha=1.0, beta=0.0, A=X, lda=64, B=BQ,
             ldb=32, Bs=BS, C=D, ldc=8, bias=None, act=0)
    a.update(k)
    return list(a.values()) + [None]


@pytest.mark.parametrize("k,code", [
    (dict(format=3), INV), (dict(tA=2), INV), (dict(tB=-1), INV), (dict(dtype=4), INV),
    (dict(K=-1), INV), (dict(K=1 << 31), UNS), (dict(lda=63), INV), (dict(tA=1, lda=3), INV),
    (dict(ldb=16), INV), (dict(tB=0, ldb=16), OK + 4), (dict(format=2, ldb=32), INV),
    (dict(C=X + 2), ALIAS), (dict(C=BQ), ALIAS), (dict(C=BS), ALIAS), (dict(M=0), OK),
])
def test_mixed_refusals(b, k, code):
    # (code 4: the arguments are valid; without a device the call ends there)
    if code == 4:
        import torch
        if torch.cuda.is_available():
            pytest.skip("valid arguments with made-up addresses: not launched on a GPU")
        assert b._lib.gemm_mx(*mixed(**k)) == code
        return
    assert b._lib.gemm_mx(*mixed(**k)) == code


def test_binding_refuses(b):
    import torch
    q, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    with pytest.raises(ValueError):
        b.Mx(q, s, "fp4", 4, 64)  # host tensors
    with pytest.raises(ValueError):
        b.Mx(q, s, "fp5", 4, 64)
    with pytest.raises(ValueError):
        b.mx_empty(4, 64, "mx")
    with pytest.raises(ValueError):
        b.gemm_mx(torch.zeros(4, 64), None, torch.zeros(4, 8))
