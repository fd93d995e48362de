"""Fused and grouped products: what they refuse, before anything reaches a GPU."""
import pytest
import torch

# fake, aligned device addresses: argument checks never read them
PA, PB, PY, PR, PU, PO, PD, PV = (0x10000000 * i for i in range(1, 9))
INVALID, UNSUPPORTED, ALIAS = 1, 2, 3


@pytest.fixture(scope="module")
def b(lib_path):
    from dense_gemm_tiled_gb300 import binding
    return binding


def fused(b, **k):
    a = dict(tA=0, tB=1, M=16, N=24, K=8, dt=1, alpha=1.0, A=PA, lda=8, B=PB, ldb=8, bias=None, act=0,
             beta=1.0, R=None, ldr=0, U=None, ldu=0, Y=PY, ldy=24)
    a.update(k)
    return b._lib.gemm_fused(*(a[n] for n in ("tA", "tB", "M", "N", "K", "dt", "alpha", "A", "lda", "B",
                                              "ldb", "bias", "act", "beta", "R", "ldr", "U", "ldu", "Y",
                                              "ldy")), None)


def fused_bwd(b, **k):
    a = dict(tA=0, tB=0, M=16, N=24, K=8, dt=1, alpha=1.0, A=PA, lda=8, B=PB, ldb=24, act=2, U=PU,
             ldu=24, Y=PY, ldy=24, db=None)
    a.update(k)
    return b._lib.gemm_fused_backward(*(a[n] for n in ("tA", "tB", "M", "N", "K", "dt", "alpha", "A",
                                                       "lda", "B", "ldb", "act", "U", "ldu", "Y", "ldy",
                                                       "db")), None)


def grouped(b, **k):
    a = dict(tB=1, T=16, N=24, K=8, E=3, o=PO, dt=2, alpha=1.0, A=PA, lda=8, B=PB, ldb=8, sb=192,
             bias=None, act=0, beta=1.0, R=None, ldr=0, U=None, ldu=0, Y=PY, ldy=24)
    a.update(k)
    return b._lib.gemm_grouped(*(a[n] for n in ("tB", "T", "N", "K", "E", "o", "dt", "alpha", "A", "lda",
                                                "B", "ldb", "sb", "bias", "act", "beta", "R", "ldr", "U",
                                                "ldu", "Y", "ldy")), None)


def grouped_bwd(b, **k):
    a = dict(tB=0, T=16, N=24, K=8, E=3, o=PO, dt=2, alpha=1.0, A=PA, lda=8, B=PB, ldb=24, sb=192,
             act=2, U=PU, ldu=24, Y=PY, ldy=24, db=None)
    a.update(k)
    return b._lib.gemm_grouped_backward(*(a[n] for n in ("tB", "T", "N", "K", "E", "o", "dt", "alpha",
                                                         "A", "lda", "B", "ldb", "sb", "act", "U", "ldu",
                                                         "Y", "ldy", "db")), None)


def wgrad(b, **k):
    a = dict(T=16, M=8, N=24, E=3, o=PO, dt=2, alpha=1.0, beta=0.0, A=PA, lda=8, B=PB, ldb=24, C=PY,
             ldc=24, sc=192)
    a.update(k)
    return b._lib.gemm_grouped_wgrad(*(a[n] for n in ("T", "M", "N", "E", "o", "dt", "alpha", "beta", "A",
                                                      "lda", "B", "ldb", "C", "ldc", "sc")), None)


BIG = 2 ** 31 - 2 ** 18 + 1
FORWARD = [
    (dict(dt=3), INVALID), (dict(dt=7), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID),
    (dict(tB=2), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(lda=7), INVALID),
    (dict(ldb=7), INVALID), (dict(ldy=23), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID),
    (dict(Y=None), INVALID), (dict(A=PA + 1), INVALID), (dict(Y=PY + 1), INVALID),
    (dict(bias=PD + 1), INVALID), (dict(R=PR, ldr=23), INVALID), (dict(R=PR + 1, ldr=24), INVALID),
    (dict(U=PU, ldu=23), INVALID), (dict(U=PU + 1, ldu=24), INVALID),
    (dict(N=BIG, ldy=BIG, bias=None), UNSUPPORTED), (dict(K=BIG, lda=BIG, ldb=BIG), UNSUPPORTED),
    (dict(lda=2 ** 60), UNSUPPORTED),
    (dict(Y=PA + 16), ALIAS), (dict(Y=PB + 16), ALIAS), (dict(bias=PY), ALIAS),
    (dict(R=PY + 2, ldr=24), ALIAS), (dict(R=PY, ldr=25), ALIAS), (dict(U=PY, ldu=24), ALIAS),
    (dict(U=PA, ldu=24), ALIAS), (dict(U=PB, ldu=24), ALIAS), (dict(U=PR, ldu=24, R=PR, ldr=24), ALIAS),
    (dict(U=PU, ldu=24, bias=PU), ALIAS),
]


@pytest.mark.parametrize("args,code", FORWARD + [(dict(tA=2), INVALID), (dict(M=-1), INVALID),
                                                 (dict(M=BIG), UNSUPPORTED)])
def test_fused_refuses(b, args, code):
    assert fused(b, **args) == code
    assert b.last_path() == "none" and b.last_launches() == 0


@pytest.mark.parametrize("args,code", FORWARD + [
    (dict(T=-1), INVALID), (dict(E=-1), INVALID), (dict(o=None), INVALID), (dict(o=PO + 2), INVALID),
    (dict(sb=-8), INVALID), (dict(E=65536), UNSUPPORTED), (dict(T=BIG), UNSUPPORTED),
    (dict(sb=2 ** 60), UNSUPPORTED), (dict(o=PY), ALIAS), (dict(U=PO, ldu=24), ALIAS)])
def test_grouped_refuses(b, args, code):
    assert grouped(b, **args) == code
    assert b.last_path() == "none" and b.last_launches() == 0


BACKWARD = [
    (dict(dt=4), INVALID), (dict(act=5), INVALID), (dict(U=None), INVALID), (dict(ldu=23), INVALID),
    (dict(U=PU + 1), INVALID), (dict(db=PD + 2), INVALID), (dict(Y=None), INVALID),
    (dict(ldy=23), INVALID), (dict(U=PY + 2), ALIAS), (dict(U=PY, ldu=25), ALIAS), (dict(Y=PA), ALIAS),
    (dict(db=PY), ALIAS), (dict(db=PA), ALIAS), (dict(db=PB), ALIAS), (dict(db=PU), ALIAS),
]


@pytest.mark.parametrize("args,code", BACKWARD)
def test_fused_backward_refuses(b, args, code):
    assert fused_bwd(b, **args) == code


@pytest.mark.parametrize("args,code", BACKWARD + [(dict(o=None), INVALID), (dict(db=PO), ALIAS),
                                                  (dict(E=65536), UNSUPPORTED)])
def test_grouped_backward_refuses(b, args, code):
    assert grouped_bwd(b, **args) == code


@pytest.mark.parametrize("args,code", [
    (dict(dt=3), INVALID), (dict(T=-1), INVALID), (dict(M=-1), INVALID), (dict(E=-1), INVALID),
    (dict(lda=7), INVALID), (dict(ldb=23), INVALID), (dict(ldc=23), INVALID), (dict(o=None), INVALID),
    (dict(C=None), INVALID), (dict(sc=-192), INVALID), (dict(sc=191), ALIAS), (dict(sc=0), ALIAS),
    (dict(C=PA), ALIAS), (dict(C=PB), ALIAS), (dict(o=PY), ALIAS), (dict(T=BIG), UNSUPPORTED),
    (dict(M=BIG, lda=BIG, sc=2 ** 40), UNSUPPORTED), (dict(E=65536), UNSUPPORTED)])
def test_wgrad_refuses(b, args, code):
    assert wgrad(b, **args) == code


def test_nothing_to_do(b):
    assert fused(b, M=0) == 0 and fused(b, N=0, ldb=8) == 0
    assert grouped(b, T=0) == 0 and grouped(b, E=0, o=None) == 0 and grouped(b, N=0) == 0
    assert fused_bwd(b, M=0) == 0 and grouped_bwd(b, T=0) == 0 and grouped_bwd(b, E=0) == 0
    assert wgrad(b, M=0) == 0 and wgrad(b, E=0) == 0
    assert b.last_path() == "none"


def test_binding_refuses(b):
    f = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt)  # noqa: E731
    o = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(TypeError):
        b.gemm_fused(f(4, 8), f(8, 6, dt=torch.float32), f(4, 6))
    with pytest.raises(TypeError):
        b.gemm_fused(f(4, 8, dt=torch.int8), f(8, 6, dt=torch.int8), f(4, 6, dt=torch.int8))
    with pytest.raises(ValueError):
        b.gemm_fused(f(4, 8), f(8, 6), f(4, 6))  # host tensors
    with pytest.raises(ValueError):
        b.gemm_grouped(f(4, 8), f(2, 8, 6), f(4, 6), o)
    with pytest.raises(ValueError):
        b.gemm_grouped_wgrad(f(4, 8), f(4, 6), f(2, 8, 6), o)


def test_path_names(b):
    assert b.PATHS[13] == "fused_tc" and b.PATHS[14] == "fused_ffma"
