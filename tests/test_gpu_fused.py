"""Products with a full epilogue and products grouped by expert, on the GPU, against
their definition in 64 bits (fused_ref.py)."""
import pytest
import torch

import fused_ref as ref
from fused_ref import DT

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(autouse=True)
def _lib(lib_path, gpu):
    yield


@pytest.fixture
def g():
    from dense_gemm_tiled_gb300 import binding
    yield binding
    torch.cuda.synchronize()
    assert binding.check_device_status() == binding.OK


def matrix(shape, dtype, seed, std=1.0, off=0, pad=0):
    """A CUDA tensor (2-D or 3-D), optionally `off` elements into a buffer whose rows
    are `pad` elements wider, the rest of it NaN."""
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(shape, generator=gen) * std).to(DT[dtype]).cuda()
    if not off and not pad:
        return x
    buf = torch.full((x[..., 0].numel() * (shape[-1] + pad) + off,), NAN, dtype=DT[dtype],
                     device="cuda")
    out = buf[off:].view(*shape[:-1], shape[-1] + pad)[..., : shape[-1]]
    out.copy_(x)
    return out


def offsets_of(sizes, first=0):
    at = [first]
    for n in sizes:
        at.append(at[-1] + n)
    return at, torch.tensor(at, dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().double()


SHAPES = [
    # M, N, K
    (1, 1, 1), (1, 5632, 2048), (3, 40, 8), (17, 33, 65), (32, 64, 64), (33, 65, 63),
    (128, 128, 128), (129, 257, 192), (200, 304, 136), (255, 64, 1024), (300, 513, 70),
    (512, 520, 333), (1000, 200, 48),
    (17, 72, 4104), (130, 264, 4100), (300, 1030, 2056), (512, 2048, 1030),
    (4200, 72, 40),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_fused(g, M, N, K, dtype):
    seed = M + 7 * N + K
    for i, (ta, tb, act, bias, res, pre) in enumerate([
            (False, True, "gelu", True, True, True), (False, False, "relu", True, False, False),
            (True, False, "none", False, True, False), (True, True, "gelu", False, False, True)]):
        A = matrix((K, M) if ta else (M, K), dtype, seed + i)
        B = matrix((N, K) if tb else (K, N), dtype, seed + 10 + i, 0.2)
        b = matrix((N,), dtype, seed + 20) if bias else None
        R = matrix((M, N), dtype, seed + 30) if res else None
        Y = torch.full((M, N), NAN, dtype=DT[dtype], device="cuda")
        U = torch.full_like(Y, NAN) if pre else None
        out = g.gemm_fused(A, B, Y, transA=ta, transB=tb, alpha=1.25, bias=b, act=act, residual=R,
                           beta=-0.5, preact=U)
        assert out is Y
        a64, b64 = f64(A.t() if ta else A), f64(B.t() if tb else B)
        u, eu, y, ey = ref.forward(a64, b64, dtype, 1.25, None if b is None else f64(b), act,
                                   None if R is None else f64(R), -0.5)
        ref.check(Y, y, ey, (ta, tb, act))
        if pre:
            ref.check(U, u, eu, "U")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_fused_backward(g, M, N, K, dtype):
    seed = M + 7 * N + K
    for i, (ta, tb, act, sums) in enumerate([(False, False, "gelu", True), (False, True, "relu", True),
                                             (True, False, "none", True),
                                             (True, True, "gelu", False)]):
        A = matrix((K, M) if ta else (M, K), dtype, seed + i)
        B = matrix((N, K) if tb else (K, N), dtype, seed + 10 + i, 0.2)
        U = matrix((M, N), dtype, seed + 30, 2.0) if act != "none" else None
        dX = torch.full((M, N), NAN, dtype=DT[dtype], device="cuda")
        db = torch.full((N,), NAN, device="cuda") if sums else None
        g.gemm_fused_backward(A, B, dX, U, transA=ta, transB=tb, alpha=0.75, act=act, dbias=db)
        u = f64(U) if U is not None else torch.zeros((M, N), dtype=torch.float64, device="cuda")
        d, ed, s, es = ref.backward(f64(A.t() if ta else A), f64(B.t() if tb else B), dtype, u, 0.75,
                                    act)
        ref.check(dX, d, ed, (ta, tb, act))
        if sums:
            ref.check(db, s, es, "dbias")


# (sizes, rows ahead of the first group, rows behind the last)
GROUPS = [
    ([5], 0, 0), ([0], 0, 3), ([1], 2, 0), ([1, 0, 1], 0, 0), ([0, 0, 70, 0], 3, 5),
    ([128, 128], 0, 0), ([127, 129, 1, 300], 1, 33), ([32, 31, 33, 0, 64, 65], 0, 0),
    ([3] * 70 + [0] * 10 + [200], 0, 1), ([0] * 40 + [7], 0, 0), ([520, 17, 256], 5, 100),
]


def grouped_call(g, sizes, ahead, behind, N, K, dtype, tb, act, bias, res, pre, seed=0, pad=0, off=0):
    at, offs = offsets_of(sizes, ahead)
    rows, E = at[-1] + behind, len(sizes)
    A = matrix((rows, K), dtype, seed, off=off, pad=pad)
    B = matrix((E, N, K) if tb else (E, K, N), dtype, seed + 1, 0.2, off=off, pad=pad)
    b = matrix((E, N), dtype, seed + 2) if bias else None
    R = matrix((rows, N), dtype, seed + 3, off=off, pad=pad) if res else None
    Y = matrix((rows, N), dtype, seed + 4, off=off, pad=pad)
    U = matrix((rows, N), dtype, seed + 5, off=off, pad=pad) if pre else None
    y0, u0 = Y.clone(), None if U is None else U.clone()
    # what is not a group's row must not matter
    for t in (A, R):
        if t is not None:
            t[:ahead] = NAN
            t[at[-1]:] = float("inf")
    g.gemm_grouped(A, B, Y, offs, transB=tb, alpha=1.5, bias=b, act=act, residual=R, beta=0.5,
                   preact=U)
    for e, (lo, hi) in enumerate(zip(at, at[1:])):
        w = f64(B[e].t() if tb else B[e])
        u, eu, y, ey = ref.forward(f64(A[lo:hi]), w, dtype, 1.5, None if b is None else f64(b[e]),
                                   act, None if R is None else f64(R[lo:hi]), 0.5)
        ref.check(Y[lo:hi], y, ey, e)
        if pre:
            ref.check(U[lo:hi], u, eu, ("U", e))
    for t, t0 in ((Y, y0), (U, u0)):
        if t is not None:
            assert torch.equal(t[:ahead], t0[:ahead]) and torch.equal(t[at[-1]:], t0[at[-1]:])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("sizes,ahead,behind", GROUPS)
def test_grouped(g, sizes, ahead, behind, dtype):
    grouped_call(g, sizes, ahead, behind, 72, 40, dtype, True, "gelu", True, True, True)
    grouped_call(g, sizes, ahead, behind, 136, 200, dtype, False, "relu", True, False, False, 50)
    grouped_call(g, sizes, ahead, behind, 264, 64, dtype, True, "none", False, True, False, 60)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("sizes,ahead,behind", GROUPS)
def test_grouped_backward(g, sizes, ahead, behind, dtype):
    at, offs = offsets_of(sizes, ahead)
    rows, E = at[-1] + behind, len(sizes)
    for i, (N, K, tb, act) in enumerate([(72, 40, False, "gelu"), (200, 136, True, "relu"),
                                         (264, 72, False, "none")]):
        A = matrix((rows, K), dtype, 3 + i)
        B = matrix((E, N, K) if tb else (E, K, N), dtype, 13 + i, 0.2)
        U = matrix((rows, N), dtype, 23 + i, 2.0) if act != "none" else None
        for t in (A, U):
            if t is not None:
                t[:ahead] = NAN
                t[at[-1]:] = float("inf")
        dX = matrix((rows, N), dtype, 33 + i)
        d0 = dX.clone()
        db = torch.full((E, N), NAN, device="cuda")
        g.gemm_grouped_backward(A, B, dX, offs, U, transB=tb, alpha=0.5, act=act, dbias=db)
        for e, (lo, hi) in enumerate(zip(at, at[1:])):
            u = f64(U[lo:hi]) if U is not None else torch.zeros((hi - lo, N), dtype=torch.float64,
                                                                device="cuda")
            d, ed, s, es = ref.backward(f64(A[lo:hi]), f64(B[e].t() if tb else B[e]), dtype, u, 0.5,
                                        act)
            ref.check(dX[lo:hi], d, ed, e)
            ref.check(db[e], s, es, ("dbias", e))
        assert torch.equal(dX[:ahead], d0[:ahead]) and torch.equal(dX[at[-1]:], d0[at[-1]:])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("sizes,ahead,behind", GROUPS)
def test_grouped_wgrad(g, sizes, ahead, behind, dtype):
    at, offs = offsets_of(sizes, ahead)
    rows, E = at[-1] + behind, len(sizes)
    for i, (M, N, beta) in enumerate([(40, 72, 0.0), (136, 264, 1.0), (300, 64, -0.5), (1, 1, 0.0),
                                      (1, 65, 1.0)]):
        A, B = matrix((rows, M), dtype, 3 + i), matrix((rows, N), dtype, 13 + i)
        for t in (A, B):
            t[:ahead] = NAN
            t[at[-1]:] = float("inf")
        C = matrix((E, M, N), dtype, 23 + i) if beta else torch.full((E, M, N), NAN, dtype=DT[dtype],
                                                                    device="cuda")
        c0 = C.clone()
        g.gemm_grouped_wgrad(A, B, C, offs, alpha=0.5, beta=beta)
        for e, (lo, hi) in enumerate(zip(at, at[1:])):
            c = f64(c0[e]) if beta else None
            _, _, y, ey = ref.forward(f64(A[lo:hi].t()), f64(B[lo:hi]), dtype, 0.5, residual=c,
                                      beta=beta)
            ref.check(C[e], y, ey, e)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sizes,N,K", [([455], 130, 1332), ([3, 0, 2], 72, 3000), ([40] * 9, 30, 257)])
def test_long_inner_dimension(g, sizes, N, K, dtype):
    """Few tiles and a long inner dimension: slices of it (fp32), for weights too."""
    grouped_call(g, sizes, 1, 4, N, K, dtype, True, "gelu", True, True, True, 7)
    grouped_call(g, sizes, 0, 0, N, K, dtype, False, "none", False, True, False, 8, 3, 1)
    at, offs = offsets_of([K, 0, K // 3, 1], 2)
    A, B = matrix((at[-1], 49), dtype, 1), matrix((at[-1], N), dtype, 2)
    for pad in (0, 5):
        C = matrix((4, 49, N), dtype, 3, pad=pad)
        c0 = f64(C)
        g.gemm_grouped_wgrad(A, B, C, offs, alpha=0.5, beta=-1.0)
        for e, (lo, hi) in enumerate(zip(at, at[1:])):
            _, _, y, ey = ref.forward(f64(A[lo:hi].t()), f64(B[lo:hi]), dtype, 0.5, residual=c0[e],
                                      beta=-1.0)
            ref.check(C[e], y, ey, e)
    C = torch.zeros((8, 49, N), dtype=DT[dtype], device="cuda")[::2]  # (apart from one another)
    g.gemm_grouped_wgrad(A, B, C, offs)
    for e, (lo, hi) in enumerate(zip(at, at[1:])):
        _, _, y, ey = ref.forward(f64(A[lo:hi].t()), f64(B[lo:hi]), dtype)
        ref.check(C[e], y, ey, e)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("off,pad", [(0, 8), (1, 0), (0, 1), (3, 5)])
def test_pitches_and_alignment(g, off, pad, dtype):
    """Matrices inside wider ones, on and off 16-byte alignment."""
    for K in (64, 65):
        grouped_call(g, [100, 0, 31], 2, 9, 130, K, dtype, True, "gelu", True, True, True, 5, pad, off)
        grouped_call(g, [40, 97], 0, 0, 77, K, dtype, False, "none", True, False, False, 6, pad, off)
    _, offs = offsets_of([50, 0, 81], 1)
    A, B = matrix((140, 77), dtype, 1, off=off, pad=pad), matrix((140, 130), dtype, 2, off=off, pad=pad)
    C = matrix((3, 77, 130), dtype, 3, off=off, pad=pad)
    c0 = f64(C)
    g.gemm_grouped_wgrad(A, B, C, offs, beta=1.0)
    for e, (lo, hi) in enumerate([(1, 51), (51, 51), (51, 132)]):
        _, _, y, ey = ref.forward(f64(A[lo:hi].t()), f64(B[lo:hi]), dtype, residual=c0[e])
        ref.check(C[e], y, ey, e)
    M, N, K = 100, 130, 65
    A, B = matrix((M, K), dtype, 1, off=off, pad=pad), matrix((K, N), dtype, 2, 0.2, off=off, pad=pad)
    U = matrix((M, N), dtype, 3, off=off, pad=pad)
    dX, db = matrix((M, N), dtype, 4, off=off, pad=pad), torch.empty(N, device="cuda")
    g.gemm_fused_backward(A, B, dX, U, dbias=db)
    d, ed, s, es = ref.backward(f64(A), f64(B), dtype, f64(U))
    ref.check(dX, d, ed)
    ref.check(db, s, es)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_written_columns_alone(g, dtype):
    """What lies between the rows of a wider result stays."""
    buf = torch.full((70, 100), 7.0, dtype=DT[dtype], device="cuda")
    Y = buf[:, 3:92]
    A, B = matrix((70, 24), dtype, 1), matrix((89, 24), dtype, 2)
    g.gemm_fused(A, B, Y, transB=True)
    assert (buf[:, :3] == 7).all() and (buf[:, 92:] == 7).all()
    buf = torch.full((70, 160), 7.0, dtype=DT[dtype], device="cuda")
    Y = buf[:, 16:104]
    g.gemm_fused(A, B[:88], Y, transB=True)
    assert (buf[:, :16] == 7).all() and (buf[:, 104:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_nonfinite_stays_in_its_group(g, dtype):
    """A NaN or an infinity of one group's rows or matrix reaches that group alone."""
    at, offs = offsets_of([50, 30, 60, 20])
    A, B = matrix((160, 64), dtype, 1), matrix((4, 64, 72), dtype, 2)
    U = matrix((160, 72), dtype, 3)
    A[60] = NAN
    A[75] = float("inf")
    U[55] = NAN
    B[3] = NAN
    dX, db = torch.zeros((160, 72), dtype=DT[dtype], device="cuda"), torch.zeros((4, 72), device="cuda")
    g.gemm_grouped_backward(A, B, dX, offs, U, dbias=db)
    assert dX[:50].isfinite().all() and dX[80:140].isfinite().all()
    assert db[0].isfinite().all() and db[2].isfinite().all()
    assert dX[60].isnan().all() and dX[55].isnan().all() and dX[140:].isnan().all()
    assert dX[50:55].isfinite().all() and db[1].isnan().all() and db[3].isnan().all()
    Y = torch.zeros_like(dX)
    g.gemm_grouped(A, B, Y, offs, act="gelu")
    assert Y[:60].isfinite().all() and Y[61:75].isfinite().all() and Y[76:140].isfinite().all()
    assert Y[60].isnan().all()
    C = torch.zeros((4, 64, 72), dtype=DT[dtype], device="cuda")
    g.gemm_grouped_wgrad(A, Y.nan_to_num(0.0, 0.0, 0.0), C, offs)
    assert C[0].isfinite().all() and C[2].isfinite().all() and C[3].isfinite().all()
    assert C[1].isnan().all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_relu_gradient_of_nonfinite(g, dtype):
    """relu's gradient is zero where U is not above zero, whatever comes in."""
    A = matrix((40, 32), dtype, 1)
    A[3] = float("inf")
    A[4] = NAN
    U = matrix((40, 48), dtype, 2)
    U[5] = NAN
    dX = torch.empty((40, 48), dtype=DT[dtype], device="cuda")
    g.gemm_fused_backward(A, matrix((32, 48), dtype, 3), dX, U, act="relu")
    assert (dX[~(U > 0)] == 0).all()


@pytest.mark.parametrize("act", ["relu", "gelu"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_infinite_preactivations(g, dtype, act):
    """act(+inf) = inf, act(-inf) = 0; their slopes 1 and 0."""
    one = torch.ones((8, 8), dtype=DT[dtype], device="cuda")
    b = torch.tensor([float("inf"), float("-inf"), NAN, 0, 1, -1, 3, -3], dtype=DT[dtype], device="cuda")
    Y, U = torch.empty_like(one), torch.empty_like(one)
    g.gemm_fused(0 * one, one, Y, bias=b, act=act, preact=U)
    assert (Y[:, 0] == float("inf")).all() and (Y[:, 1] == 0).all()
    if act == "gelu":
        assert Y[:, 2].isnan().all()
    dX = torch.empty_like(one)
    g.gemm_fused_backward(one, one, dX, U, act=act)
    assert (dX[:, 0] == 8).all() and (dX[:, 1] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_results_over_inputs(g, dtype):
    """The residual, and the pre-activation of a backward pass, may be the result."""
    for M, N, K, off in ((150, 140, 72, 0), (30, 65, 33, 1)):
        A, B = matrix((M, K), dtype, 1), matrix((N, K), dtype, 2, 0.2)
        Y = matrix((M, N), dtype, 3, off=off)
        r = f64(Y)
        g.gemm_fused(A, B, Y, transB=True, act="gelu", residual=Y)
        _, _, y, ey = ref.forward(f64(A), f64(B.t()), dtype, name="gelu", residual=r)
        ref.check(Y, y, ey)
        U = matrix((M, N), dtype, 4, off=off)
        d, ed, s, es = ref.backward(f64(A), f64(B.t()), dtype, f64(U))
        db = torch.empty(N, device="cuda")
        g.gemm_fused_backward(A, B, U, U, transB=True, dbias=db)
        ref.check(U, d, ed)
        ref.check(db, s, es)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [9, 70])
def test_offsets_past_32_bits(g, rows, dtype):
    """Rows and matrices whose offsets (in elements) pass 2^31."""
    dt, ld, far = DT[dtype], (1 << 31) // rows + 16 - (1 << 31) // rows % 16 + (1 << 25), 1_200_000_000
    N, K = 72, 40
    bufs = [torch.empty(ld * rows, dtype=dt, device="cuda") for _ in range(2)]
    wide = torch.empty(2 * far + N * K, dtype=dt, device="cuda")
    A = bufs[0].as_strided((rows, K), (ld, 1))
    Y = bufs[1].as_strided((rows, N), (ld, 1))
    B = wide.as_strided((3, N, K), (far, K, 1))
    A.copy_(matrix((rows, K), dtype, 1))
    B.copy_(matrix((3, N, K), dtype, 2))
    at, offs = offsets_of([3, 0, rows - 3])
    g.gemm_grouped(A, B, Y, offs, transB=True, act="gelu")
    for e, (lo, hi) in enumerate(zip(at, at[1:])):
        _, _, y, ey = ref.forward(f64(A[lo:hi]), f64(B[e].t()), dtype, name="gelu")
        ref.check(Y[lo:hi], y, ey, e)
    U, db = matrix((rows, K), dtype, 4), torch.empty((3, K), device="cuda")
    dX = bufs[0].as_strided((rows, K), (ld, 1), K)
    g.gemm_grouped_backward(Y, B, dX, offs, U, dbias=db)
    for e, (lo, hi) in enumerate(zip(at, at[1:])):
        d, ed, s, es = ref.backward(f64(Y[lo:hi]), f64(B[e]), dtype, f64(U[lo:hi]))
        ref.check(dX[lo:hi], d, ed, e)
        ref.check(db[e], s, es, e)
    C = wide.as_strided((3, K, N), (far, N, 1))
    g.gemm_grouped_wgrad(A, Y, C, offs)
    for e, (lo, hi) in enumerate(zip(at, at[1:])):
        _, _, y, ey = ref.forward(f64(A[lo:hi].t()), f64(Y[lo:hi]), dtype)
        ref.check(C[e], y, ey, e)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_shared_matrix(g, dtype):
    """One matrix for every group (a stride of 0)."""
    at, offs = offsets_of([20, 0, 45])
    A = matrix((65, 48), dtype, 1)
    for w in (matrix((40, 48), dtype, 2), matrix((40, 48), dtype, 2, off=1, pad=1)):
        Y = torch.empty((65, 40), dtype=DT[dtype], device="cuda")
        g.gemm_grouped(A, w.expand(3, 40, 48), Y, offs, transB=True)
        _, _, y, ey = ref.forward(f64(A), f64(w.t()), dtype)
        ref.check(Y, y, ey)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", [[3, 0, 7], [40, 0, 61]])
def test_interleaved_matrices(g, sizes, dtype):
    """Matrices of B whose rows lie between one another's."""
    at, offs = offsets_of(sizes)
    A = matrix((at[-1], 48), dtype, 1)
    for tb, w in ((False, matrix((48, 3, 72), dtype, 2).permute(1, 0, 2)),
                  (True, matrix((72, 3, 48), dtype, 3).permute(1, 0, 2)),
                  (True, matrix((72, 3, 48), dtype, 3, pad=8).permute(1, 0, 2)),
                  (False, matrix((48, 3, 77), dtype, 4).permute(1, 0, 2))):
        N = w.shape[1] if tb else w.shape[2]
        Y = torch.empty((at[-1], N), dtype=DT[dtype], device="cuda")
        g.gemm_grouped(A, w, Y, offs, transB=tb)
        for e, (lo, hi) in enumerate(zip(at, at[1:])):
            _, _, y, ey = ref.forward(f64(A[lo:hi]), f64(w[e].t() if tb else w[e]), dtype)
            ref.check(Y[lo:hi], y, ey, e)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_16_bit_value(g, dtype):
    """gelu and its slope of every finite 16-bit value, the product being 0 or 1."""
    v = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(DT[dtype])
    v = v[v.isfinite()][: 65536 // 64 * 64 - 4096].contiguous()
    x, n = v.double(), v.numel()
    zero, one = torch.zeros((20, 16), dtype=DT[dtype], device="cuda"), torch.zeros((20, 16), dtype=DT[dtype], device="cuda")
    one[:, 0] = 1
    W = torch.ones((n, 16), dtype=DT[dtype], device="cuda")
    for rows in (20, 3):  # (either kernel)
        Y = torch.empty((rows, n), dtype=DT[dtype], device="cuda")
        g.gemm_fused(zero[:rows], W, Y, transB=True, bias=v, act="gelu")
        y = ref.act(x, "gelu").expand(rows, n)
        e = 2.0 ** -22 * x.abs().expand(rows, n)
        ref.check(Y, y, e + ref.rounding(y.abs() + e, dtype), "gelu")
    dX = torch.empty((20, n), dtype=DT[dtype], device="cuda")
    g.gemm_fused_backward(one, W, dX, v.expand(20, n).contiguous(), transB=True)
    d = ref.slope(x, "gelu").expand(20, n)
    ref.check(dX, d, 2.0 ** -20 + ref.rounding(d.abs() + 2.0 ** -20, dtype), "slope")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_single_rows(g, dtype):
    """The pitch of a single row does not matter, however far."""
    far = 1 << 42
    A, W = matrix((1, 77), dtype, 1), matrix((1, 77), dtype, 2)
    B, R = matrix((30, 77), dtype, 3, 0.2), matrix((1, 30), dtype, 4)
    Y, U = torch.empty((1, 30), dtype=DT[dtype], device="cuda"), torch.empty((1, 30), dtype=DT[dtype], device="cuda")
    one = lambda t: t.as_strided((1, t.shape[1]), (far, 1))  # noqa: E731
    g.gemm_fused(one(A), B, one(Y), transB=True, residual=one(R), preact=one(U), act="gelu")
    u, eu, y, ey = ref.forward(f64(A), f64(B.t()), dtype, name="gelu", residual=f64(R))
    ref.check(Y, y, ey)
    ref.check(U, u, eu)
    d, ed, _, _ = ref.backward(f64(A), f64(B.t()), dtype, f64(U))
    g.gemm_fused_backward(one(A), B, one(Y), one(U), transB=True)
    ref.check(Y, d, ed)
    X = matrix((40, 77), dtype, 5)
    Z = torch.empty((40, 1), dtype=DT[dtype], device="cuda")
    g.gemm_fused(X, one(W), Z, transB=True)  # one row of B
    _, _, y, ey = ref.forward(f64(X), f64(W.t()), dtype)
    ref.check(Z, y, ey)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty_sizes(g, dtype):
    dt = DT[dtype]

    def new(*shape):
        return torch.full(shape, NAN, dtype=dt, device="cuda")
    # no inner dimension: the product is zero
    Y, b = new(20, 24), matrix((24,), dtype, 1)
    g.gemm_fused(new(20, 0), new(24, 0), Y, transB=True, bias=b, act="relu")
    assert torch.equal(Y, torch.relu(b).expand(20, 24))
    _, offs = offsets_of([15, 0, 5])
    g.gemm_grouped(new(20, 0), new(3, 24, 0), Y, offs, transB=True)
    assert (Y == 0).all()
    Y = g.gemm_fused(new(3, 0), new(24, 0), new(3, 24), transB=True, bias=b, act="relu")
    assert torch.equal(Y, torch.relu(b).expand(3, 24))  # (few rows)
    # no rows: nothing is written but sums and gradients, which are zero
    db = torch.full((24,), NAN, device="cuda")
    g.gemm_fused_backward(new(0, 8), new(8, 24), new(0, 24), new(0, 24), dbias=db)
    assert (db == 0).all()
    _, none = offsets_of([0, 0])
    db = torch.full((2, 24), NAN, device="cuda")
    g.gemm_grouped_backward(new(0, 8), new(2, 8, 24), new(0, 24), none, new(0, 24), dbias=db)
    assert (db == 0).all()
    C = new(2, 8, 24)
    g.gemm_grouped_wgrad(new(0, 8), new(0, 24), C, none)
    assert (C == 0).all()
    C = torch.ones((2, 8, 24), dtype=dt, device="cuda")
    g.gemm_grouped_wgrad(new(0, 8), new(0, 24), C, none, beta=0.5)
    assert (C == 0.5).all()
    # no columns, no groups
    g.gemm_fused(new(4, 8), new(0, 8), new(4, 0), transB=True)
    g.gemm_grouped(new(4, 8), new(0, 8, 8), new(4, 8), offs[:1])
    # beta 0 reads no residual
    Y = g.gemm_fused(matrix((20, 8), dtype, 1), matrix((8, 24), dtype, 2), new(20, 24),
                     residual=new(20, 24), beta=0.0)
    assert Y.isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_results_every_time(g, dtype):
    _, offs = offsets_of([700, 0, 1000, 348])
    A, B = matrix((2048, 512), dtype, 1), matrix((4, 512, 320), dtype, 2)
    U = matrix((2048, 320), dtype, 3)

    def once():
        dX, db = torch.empty_like(U), torch.empty((4, 320), device="cuda")
        C = torch.empty((4, 512, 320), dtype=DT[dtype], device="cuda")
        g.gemm_grouped_backward(A, B, dX, offs, U, dbias=db)
        g.gemm_grouped_wgrad(A, dX, C, offs)
        return dX, db, C
    first = once()
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(first, once()))


def test_streams_and_graphs(g):
    """On a stream of the caller's, two streams at once, and in two captured graphs
    replayed in turn and together, with offsets that change between replays."""
    dtype = "bf16"
    E, N, K, rows = 5, 200, 136, 400
    A, W = matrix((rows, K), dtype, 1), matrix((E, N, K), dtype, 2, 0.2)
    U = matrix((rows, K), dtype, 3)

    def call(offs, Y, dX, db, stream=None):
        g.gemm_grouped(A, W, Y, offs, transB=True, act="gelu", stream=stream)
        g.gemm_grouped_backward(Y, W, dX, offs, U, dbias=db, stream=stream)

    def outs():
        return (torch.zeros((rows, N), dtype=DT[dtype], device="cuda"),
                torch.zeros((rows, K), dtype=DT[dtype], device="cuda"),
                torch.zeros((E, K), device="cuda"))
    sizes = [[100, 0, 50, 200, 50], [0, 0, 399, 1, 0], [80, 80, 80, 80, 80]]
    want = []
    for s in sizes:
        o = outs()
        call(offsets_of(s)[1], *o)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [outs() for _ in range(2)]
    offs = [offsets_of(s)[1] for s in sizes]
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            call(offs[i], *got[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(got[i], want[i]))
    graphs, held = [], []
    for i in range(2):
        o, live = outs(), offs[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[i]):
            call(live, *o)
        graphs.append(graph)
        held.append((o, live))
    for i, s in [(0, 0), (1, 1), (0, 2), (1, 0), (0, 1)]:
        o, live = held[i]
        for t in o:
            t.zero_()
        live.copy_(offs[s])
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(o, want[s]))
    for i in range(2):
        held[i][1].copy_(offs[i])
    torch.cuda.synchronize()
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for x, y in zip(held[i][0], want[i]))


def test_capture_with_cached_operands(g):
    """A captured call that copies operands (rows off alignment) keeps its own scratch."""
    A, W = matrix((60, 33), "f16", 1), matrix((3, 33, 70), "f16", 2)
    _, offs = offsets_of([20, 10, 30])
    want = torch.empty((60, 70), dtype=torch.float16, device="cuda")
    g.gemm_grouped(A, W, want, offs)
    torch.cuda.synchronize()
    Y = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gemm_grouped(A, W, Y, offs)
    big = torch.empty_like(want)
    for _ in range(3):
        Y.zero_()
        g.gemm_grouped(A * 2, W, big, offs)  # (scratch of the same size in between)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)


def test_offsets_that_do_not_ascend(g):
    """Bad offsets: nothing outside the matrices is touched, the status says so."""
    rows, E, N, K = 300, 6, 72, 40
    for dtype in ("bf16", "f32"):
        for bad in ([0, 50, 20, 100, 90, 200, 300], [-5, 10, 10, 20, 30, 40, 50],
                    [0, 10, 400, 500, 2 ** 31 - 1, 100, 300], [300, 0, 0, 0, 0, 0, -2 ** 31]):
            offs = torch.tensor(bad, dtype=torch.int32, device="cuda")
            A, B = matrix((rows, K), dtype, 1), matrix((E, K, N), dtype, 2)
            guard = torch.full((rows + 64, N), 7.0, dtype=DT[dtype], device="cuda")
            db = torch.zeros((E + 2, N), device="cuda")
            U = matrix((rows, N), dtype, 3)
            g.gemm_grouped_backward(A, B, guard[32:-32], offs, U, dbias=db[1:-1])
            assert g.check_device_status() == g.ERR_INVALID_ARG
            C = torch.zeros((E, K, N), dtype=DT[dtype], device="cuda")
            g.gemm_grouped_wgrad(A, U, C, offs)
            assert g.check_device_status() == g.ERR_INVALID_ARG
            assert (guard[:32] == 7).all() and (guard[-32:] == 7).all()
            assert (db[0] == 0).all() and (db[-1] == 0).all()
    assert g.check_device_status() == g.OK


@pytest.mark.parametrize("sizes", [[130, 170], [3, 8]])
def test_wait_that_runs_out(g, sizes):
    """A load that never comes: the waits end, the status says so, the next call is right."""
    at, offs = offsets_of(sizes)
    A, W = matrix((at[-1], 256), "bf16", 1), matrix((2, 512, 256), "bf16", 2)
    Y = torch.empty((at[-1], 512), dtype=torch.bfloat16, device="cuda")
    g.set_wait_timeout_ns(50_000_000)
    try:
        g.set_fault_injection(1)
        g.gemm_grouped(A, W, Y, offs, transB=True)
        g.set_fault_injection(0)
        assert g.check_device_status() == g.ERR_TIMEOUT
    finally:
        g.set_fault_injection(0)
        g.set_wait_timeout_ns(0)
    g.gemm_grouped(A, W, Y, offs, transB=True)
    for e, (lo, hi) in enumerate(zip(at, at[1:])):
        _, _, y, ey = ref.forward(f64(A[lo:hi]), f64(W[e].t()), "bf16")
        ref.check(Y[lo:hi], y, ey)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sizes,ahead,behind", [
    ([1], 0, 0), ([8], 0, 0), ([9], 0, 0), ([16], 0, 0), ([0, 1, 0], 0, 0), ([2, 0, 0, 7, 1], 1, 2),
    ([1] * 16, 0, 0), ([0] * 33 + [5] + [0] * 40 + [9], 2, 0), ([0, 0], 0, 4),
    ([9] + [1] * 7 + [0] * 40, 0, 0)])
@pytest.mark.parametrize("N,K", [(1, 1), (7, 8), (40, 65), (72, 512), (130, 520), (64, 1000),
                                 (1408, 2048), (24, 5000)])
def test_few_rows(g, sizes, ahead, behind, N, K, dtype):
    """Up to 16 rows in all: the streaming kernel, every depth of its copies."""
    for act, bias, res, pre in (("gelu", True, True, True), ("none", False, False, False)):
        grouped_call(g, sizes, ahead, behind, N, K, dtype, True, act, bias, res, pre, N + K)
        assert g.last_path() == "fused_stream"
    grouped_call(g, sizes, ahead, behind, N, K, dtype, True, "relu", True, True, False, 3, 8, 8)
    grouped_call(g, sizes, ahead, behind, N, K, dtype, True, "relu", True, True, False, 3, 3, 1)


# ------------------------------------------------------------------ an expert's MLP
def experts(g, x, offs, W1, b1, W2, dout):
    """y = gelu(x W1^T + b1) W2^T + x and every gradient, by groups."""
    rows, d = x.shape
    E, F, _ = W1.shape
    new = lambda *s: torch.zeros(s, dtype=x.dtype, device="cuda")  # noqa: E731
    h, u, y, dh, dx = new(rows, F), new(rows, F), new(rows, d), new(rows, F), new(rows, d)
    db, dW1, dW2 = torch.zeros((E, F), device="cuda"), new(E, F, d), new(E, d, F)
    g.gemm_grouped(x, W1, h, offs, transB=True, bias=b1, act="gelu", preact=u)
    g.gemm_grouped(h, W2, y, offs, transB=True, residual=x)
    g.gemm_grouped_backward(dout, W2, dh, offs, u, dbias=db)
    g.gemm_grouped_wgrad(dout, h, dW2, offs)
    g.gemm_grouped_wgrad(dh, x, dW1, offs)
    g.gemm_grouped(dh, W1, dx, offs, residual=dout)
    return y, dx, dW1, db, dW2


def test_experts_gradients(g):
    """The whole run together in fp32: against the formula by autograd in 64 bits, and
    against differences."""
    sizes = [37, 0, 90, 5]
    at, offs = offsets_of(sizes)
    d, F, rows = 24, 40, at[-1]
    x, dout = matrix((rows, d), "f32", 1), matrix((rows, d), "f32", 2)
    W1, W2 = matrix((4, F, d), "f32", 3, 0.3), matrix((4, d, F), "f32", 4, 0.3)
    b1 = matrix((4, F), "f32", 5, 0.3)
    y, dx, dW1, db, dW2 = experts(g, x, offs, W1, b1, W2, dout)
    p = [t.double().requires_grad_() for t in (x, W1, b1, W2)]

    def loss(x, W1, b1, W2):
        ys = []
        for e, (lo, hi) in enumerate(zip(at, at[1:])):
            u = x[lo:hi] @ W1[e].t() + b1[e]
            ys.append(ref.act(u, "gelu") @ W2[e].t() + x[lo:hi])
        y = torch.cat(ys)
        return y, (y * dout.double()).sum()
    y64, total = loss(*p)
    total.backward()
    # fp32 all along, terms of order 1: 2^-23 per operation, a few hundred of them
    for got, want in ((y, y64.detach()), (dx, p[0].grad), (dW1, p[1].grad), (db, p[2].grad),
                      (dW2, p[3].grad)):
        assert (got.double() - want).abs().max() <= 2.0 ** -23 * 400 * want.abs().max()
    # central differences of the library's own forward pass along random directions:
    # error O(h^2) of the step and 2 * 2^-24 * |total|'s terms / h of the roundings
    h = 2.0 ** -6
    for i, (w, grad) in enumerate(((x, dx), (W1, dW1), (b1, db), (W2, dW2))):
        v = matrix(tuple(w.shape), "f32", 50 + i)
        v /= v.norm()
        vals = []
        for s in (h, -h):
            args = [x, W1, b1, W2]
            args[i] = w + s * v
            ys = experts(g, args[0], offs, args[1], args[2], args[3], dout)[0]
            vals.append((ys.double() * dout.double()).sum())
        diff = (vals[0] - vals[1]) / (2 * h)
        want = (grad.double() * v.double()).sum()
        assert abs(diff - want) <= 0.01 * grad.double().norm(), i


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_experts_16bit(g, dtype):
    """The same in 16 bits, each step against 64 bits on the step's own inputs."""
    at, offs = offsets_of([130, 0, 257, 1])
    d, F, rows = 96, 200, at[-1]
    x, dout = matrix((rows, d), dtype, 1), matrix((rows, d), dtype, 2)
    W1, W2 = matrix((4, F, d), dtype, 3, 0.1), matrix((4, d, F), dtype, 4, 0.1)
    b1 = matrix((4, F), dtype, 5, 0.3)
    y, dx, dW1, db, dW2 = experts(g, x, offs, W1, b1, W2, dout)
    for e, (lo, hi) in enumerate(zip(at, at[1:])):
        u, _, h, _ = ref.forward(f64(x[lo:hi]), f64(W1[e].t()), dtype, bias=f64(b1[e]), name="gelu")
        u, h = u.to(DT[dtype]).double(), h.to(DT[dtype]).double()
        # (h and u differ from the library's by roundings of one step at most, which
        # the sums below average over: 4 steps of their magnitude)
        eps = 4 * torch.finfo(DT[dtype]).eps
        want = h @ f64(W2[e].t()) + f64(x[lo:hi])
        mag = h.abs() @ f64(W2[e].t()).abs() + f64(x[lo:hi]).abs()
        assert ((y[lo:hi].double() - want).abs() <= eps * mag).all()
        dh = f64(dout[lo:hi]) @ f64(W2[e]) * ref.slope(u, "gelu")
        mh = f64(dout[lo:hi]).abs() @ f64(W2[e]).abs() * 1.13
        assert ((db[e].double() - dh.sum(0)).abs() <= eps * mh.sum(0)).all()
        assert ((dW1[e].double() - dh.t() @ f64(x[lo:hi])).abs() <=
                eps * (mh.t() @ f64(x[lo:hi]).abs())).all()
        assert ((dW2[e].double() - f64(dout[lo:hi]).t() @ h).abs() <=
                eps * (f64(dout[lo:hi]).abs().t() @ (h.abs() + 0.2))).all()
        assert ((dx[lo:hi].double() - dh @ f64(W1[e]) - f64(dout[lo:hi])).abs() <=
                eps * (mh @ f64(W1[e]).abs() + f64(dout[lo:hi]).abs())).all()
