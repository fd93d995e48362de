"""Microscaled operands on the GPU against their definition in 64 bits
(mx_ref.py): stored bytes bit for bit, products within the GEMM's own bounds
(oracle/compare.py), the activation's backward pass within fp32 evaluation."""
import numpy as np
import pytest
import torch

import mx_ref
from helpers import to_np
from oracle import bf16_to_double, compare

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FMTS = list(mx_ref.BLOCK)


@pytest.fixture(autouse=True)
def _lib(lib_path, gpu):
    yield


@pytest.fixture
def g():
    from dense_gemm_tiled_gb300 import binding
    yield binding
    torch.cuda.synchronize()
    assert binding.check_device_status() == binding.OK


def f64(t):
    return t.detach().double().cpu().numpy()


def matrix(rows, cols, dtype, seed, std=1.0, offset=0, pitch=None):
    """A CUDA matrix [rows, cols], optionally inside a wider one and off
    alignment (the rest filled with NaN)."""
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn((rows, cols), generator=gen) * std).to(DT[dtype])
    if offset == 0 and pitch is None:
        return x.cuda()
    pitch = pitch or cols
    base = torch.full((rows * pitch + offset + 64,), float("nan"), dtype=DT[dtype], device="cuda")
    v = base[offset: offset + rows * pitch].view(rows, pitch)[:, :cols]
    v.copy_(x)
    return v


def filled(g, rows, cols, fmt):
    """An Mx whose buffers hold noise: everything that is read must be written."""
    Q = g.mx_empty(rows, cols, fmt)
    Q.codes.fill_(0xA5)
    Q.scales.fill_(0xFF)
    return Q


def stored(g, x64, fmt):
    """An Mx made from the reference's bytes, and its values."""
    codes, st, v = mx_ref.store(x64, fmt)
    rows, cols = x64.shape
    return g.Mx(torch.from_numpy(codes).cuda(), torch.from_numpy(st).cuda(), fmt, rows, cols), v


SIZES = [(1, 1), (1, 32), (3, 17), (128, 128), (130, 77), (33, 259), (257, 1000), (5, 4096)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("trans", [False, True])
def test_quantize_bytes(g, fmt, dtype, trans):
    for i, (rows, cols) in enumerate(SIZES):
        for off, extra in ((0, 0), (1, 3), (0, 8)):
            sr, sc = (cols, rows) if trans else (rows, cols)
            X = matrix(sr, sc, dtype, 10 + i, offset=off, pitch=sc + extra)
            Q = filled(g, rows, cols, fmt)
            g.mx_quantize(X, Q, transX=trans, mult=1.0 if i % 2 else 0.75)
            x = f64(X).T if trans else f64(X)
            codes, st, v = mx_ref.store(np.ascontiguousarray(x), fmt, 1.0 if i % 2 else 0.75)
            assert np.array_equal(Q.codes.cpu().numpy(), codes), (rows, cols, off, extra)
            assert np.array_equal(Q.scales.cpu().numpy(), st), (rows, cols, off, extra)
            for out in DT:
                Y = matrix(rows, cols, out, 0, offset=off, pitch=cols + extra)
                g.mx_dequantize(Q, Y)
                want = torch.from_numpy(v).float().to(DT[out])
                assert torch.equal(Y.cpu(), want), (rows, cols, out)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_hard_values(g, fmt):
    """Zeros, subnormals, the ends of the types' range, every tie, and blocks
    with a NaN or an infinity (alone in becoming NaN)."""
    big = torch.finfo(torch.float32).max
    tiny = 2.0 ** -149
    x = torch.zeros((12, 70))
    x[1, :] = tiny
    x[2, :40] = torch.linspace(-big, big, 40)
    x[3, 0] = 2.0 ** -126
    x[4, :] = torch.arange(70) / 8.0
    x[5, :] = -torch.arange(70) / 16.0
    x[6, 5] = float("nan"); x[6, 40] = 3.0
    x[7, 69] = float("inf"); x[7, 1] = 1.0
    x[8, 33] = float("-inf")
    x[9, :] = -0.0
    x[10, :] = torch.tensor([2.0 ** (i - 60) for i in range(70)])
    x[11, :] = 448.0 * 6.0 * 3.0
    Q = filled(g, 12, 70, fmt)
    g.mx_quantize(x.cuda(), Q)
    codes, st, v = mx_ref.store(x.numpy().astype(np.float64), fmt)
    got = Q.codes.cpu().numpy()
    assert np.array_equal(Q.scales.cpu().numpy(), st)
    assert np.array_equal(got, codes)
    Y = torch.empty((12, 70), device="cuda")
    g.mx_dequantize(Q, Y)
    assert np.array_equal(f64(Y), v.astype(np.float32).astype(np.float64), equal_nan=True)
    b = mx_ref.BLOCK[fmt]
    assert torch.isnan(Y[6, :b]).all() and torch.isfinite(Y[6, 2 * b:]).all()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
def test_activation_forward_and_backward(g, dtype, act):
    for i, (rows, cols) in enumerate([(1, 1), (2, 45), (129, 131), (300, 512), (1000, 64)]):
        for off, extra in ((0, 0), (1, 1)):
            X = matrix(rows, cols, dtype, 40 + i, std=2.0, offset=off, pitch=cols + extra)
            dY = matrix(rows, cols, dtype, 50 + i, offset=off, pitch=cols + extra)
            Y, dX = torch.empty_like(X), torch.empty_like(dY)
            db = torch.full((cols,), float("nan"), device="cuda")
            Q = filled(g, rows, cols, "int8")
            g.mx_quantize(X, Q, act=act, Y=Y)
            codes, st, xq = mx_ref.store(f64(X), "int8")
            assert np.array_equal(Q.codes.cpu().numpy(), codes)
            x = f64(X)
            y = {"none": x, "relu": np.maximum(x, 0), "gelu": mx_ref.gelu(x)}[act]
            # fp32 evaluation as the GEMM epilogue's, then one rounding to the type
            rnd = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
            sub = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}[dtype]
            ev = 0.0 if act != "gelu" else 2.0 ** -20
            assert np.all(np.abs(f64(Y) - y) <= ev * (np.abs(x) + np.abs(y)) + rnd * np.abs(y) * 1.001 + sub)
            g.mx_act_backward(dY, Q, dX, act=act, dbias=db)
            dy = f64(dY)
            dx = dy * mx_ref.slope(xq, act)
            # the slope (at most 1.13) within 2^-20, the product one fp32 rounding
            err = (0.0 if act != "gelu" else 2.0 ** -20) * np.abs(dy) + 2.0 ** -23 * np.abs(dx)
            assert np.all(np.abs(f64(dX) - dx) <= err + rnd * np.abs(dx) * 1.001 + sub)
            # column sums: each term's error and one fp32 rounding of the sum of
            # magnitudes for each of the ceil(log)-free additions (rows of them)
            tol = err.sum(0) + rows * 2.0 ** -24 * np.abs(dx).sum(0) + 1e-38
            assert np.all(np.abs(f64(db) - dx.sum(0)) <= tol)
            # the same into the gradient's own buffer, without the sums
            g.mx_act_backward(dY, Q, dY, act=act)
            assert torch.equal(dY, dX)
            # and the forward pass into its own input
            g.mx_quantize(X, Q, act=act, Y=X)
            assert torch.equal(X, Y) and np.array_equal(Q.codes.cpu().numpy(), codes)


def test_act_backward_no_rows_and_stability(g):
    db = torch.full((33,), float("nan"), device="cuda")
    Q = g.mx_empty(0, 33, "int8")
    E = torch.empty((0, 33), device="cuda")
    g.mx_act_backward(E, Q, E.clone(), dbias=db)
    assert torch.equal(db.cpu(), torch.zeros(33))
    X, dY = matrix(3000, 200, "f16", 1), matrix(3000, 200, "f16", 2)
    Q = g.mx_empty(3000, 200, "int8")
    g.mx_quantize(X, Q)
    outs = []
    for _ in range(3):
        db = torch.empty(200, device="cuda")
        g.mx_act_backward(dY, Q, torch.empty_like(dY), dbias=db)
        outs.append(db)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def check_product(C, a, bT, dtype, alpha=1.0, beta=0.0, C0=None, bias=None, act="none"):
    """C against alpha * a @ bT + beta * C0 (+ bias, act), all in 64 bits."""
    ref = alpha * (a @ bT)
    mag = abs(alpha) * (np.abs(a) @ np.abs(bT))
    if beta != 0.0:
        ref = ref + beta * C0
        mag = mag + np.abs(beta * C0)
    res = compare.check_epilogue(to_np(C), ref, mag, dtype, bias, act)
    assert res["ok"], res


FP4 = ["fp4", "fp4_e4m3"]
MX4_SIZES = [(1, 1, 1), (1, 8, 32), (2, 130, 64), (128, 128, 256), (129, 257, 300), (77, 301, 777),
             (300, 520, 1031), (16, 4096, 512), (520, 136, 4096)]


@pytest.mark.parametrize("fmt", FP4)
@pytest.mark.parametrize("dtype", list(DT))
def test_mx4_product(g, fmt, dtype):
    for i, (M, N, K) in enumerate(MX4_SIZES):
        r = np.random.default_rng(100 + i)
        A, a = stored(g, r.standard_normal((M, K)).astype(np.float32), fmt)
        B, b = stored(g, (r.standard_normal((N, K)) * 0.05).astype(np.float32), fmt)
        C = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda")
        g.gemm_mx(A, B, C)
        check_product(C, a, b.T, dtype)
        # an odd pitch off alignment, everything in the epilogue
        bias = matrix(1, N, dtype, 7)[0]
        C0 = matrix(M, N, dtype, 8, offset=1, pitch=N + 5)
        c0 = f64(C0)
        g.gemm_mx(A, B, C0, alpha=-0.5, beta=2.0, bias=bias, act="gelu" if i % 2 else "relu")
        check_product(C0, a, b.T, dtype, -0.5, 2.0, c0, f64(bias), "gelu" if i % 2 else "relu")


@pytest.mark.parametrize("fmt", FP4)
def test_mx4_exact_on_integers(g, fmt):
    """Codes 0, 1, 2 and scales 1 and 2: every partial sum is a small integer."""
    r = np.random.default_rng(3)
    M, N, K = 260, 390, 700
    a, b = (r.integers(-2, 3, (n, K)).astype(np.float64) for n in (M, N))
    for v in (a, b):
        v[:, ::mx_ref.BLOCK[fmt]] = 6.0  # every block's scale is exact
    b[:, : mx_ref.BLOCK[fmt]] *= 2
    (A, av), (B, bv) = stored(g, a, fmt), stored(g, b, fmt)
    assert np.array_equal(av, a) and np.array_equal(bv, b)
    C = torch.empty((M, N), device="cuda")
    g.gemm_mx(A, B, C)
    assert np.array_equal(f64(C), a @ b.T)


@pytest.mark.parametrize("fmt", FP4)
def test_mx4_nan_scale_reaches_its_row_only(g, fmt):
    r = np.random.default_rng(4)
    x = r.standard_normal((200, 300)).astype(np.float32)
    x[130, 299] = np.nan
    w = r.standard_normal((150, 300)).astype(np.float32)
    w[7, 0] = np.inf
    (A, a), (B, b) = stored(g, x, fmt), stored(g, w, fmt)
    C = torch.empty((200, 150), device="cuda")
    g.gemm_mx(A, B, C)
    got = torch.isnan(C).cpu().numpy()
    want = np.zeros_like(got)
    want[130] = True
    want[:, 7] = True
    assert np.array_equal(got, want)


MIXED_SIZES = [(1, 1, 1), (1, 130, 64), (3, 77, 33), (8, 512, 512), (17, 300, 1031), (33, 64, 2048),
               (130, 257, 259), (300, 520, 700), (32, 640, 1500), (2, 4096, 4096), (31, 96, 96)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("variant", ["nt", "nn", "tn", "tt"])
def test_mixed_product(g, fmt, dtype, variant):
    tA, tB = variant[0] == "t", variant[1] == "t"
    for i, (M, N, K) in enumerate(MIXED_SIZES):
        r = np.random.default_rng(200 + i)
        A = matrix(K if tA else M, M if tA else K, dtype, 60 + i)
        B, b = stored(g, (r.standard_normal((N, K) if tB else (K, N)) * 0.05).astype(np.float32), fmt)
        a, b = f64(A), b
        a, b = (a.T if tA else a), (b.T if tB else b)
        C = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda")
        g.gemm_mx(A, B, C, transA=tA, transB=tB)
        check_product(C, a, b, dtype)
        A = matrix(*A.shape, dtype, 60 + i, offset=1, pitch=A.shape[1] + 3)
        bias = matrix(1, N, dtype, 7)[0]
        C0 = matrix(M, N, dtype, 8, offset=1, pitch=N + 5)
        c0 = f64(C0)
        g.gemm_mx(A, B, C0, transA=tA, transB=tB, alpha=-0.5, beta=2.0, bias=bias, act="relu")
        check_product(C0, a, b, dtype, -0.5, 2.0, c0, f64(bias), "relu")


@pytest.mark.parametrize("fmt", FMTS)
def test_mixed_hard_scales(g, fmt):
    """A stored operand with the scales of very small and large values, a NaN
    block, and K of 0."""
    r = np.random.default_rng(5)
    w = r.standard_normal((64, 256)).astype(np.float32)
    w[0] *= 2.0 ** -60
    w[1] *= 2.0 ** 60
    w[2, 40] = np.nan
    B, b = stored(g, w, fmt)
    for M in (1, 9, 40):
        A = matrix(M, 256, "bf16", 3)
        C = torch.empty((M, 64), dtype=torch.bfloat16, device="cuda")
        g.gemm_mx(A, B, C, transB=True)
        got = f64(C)
        assert np.isnan(got[:, 2]).all()
        keep = [j for j in range(64) if j != 2]
        res = compare.check(to_np(C[:, keep]), f64(A) @ b[keep].T,
                            np.abs(f64(A)) @ np.abs(b[keep]).T, "bf16")
        assert res["ok"], res
    E = g.mx_empty(64, 0, fmt)
    C = torch.ones((3, 64), device="cuda")
    g.gemm_mx(torch.empty((3, 0), device="cuda"), E, C, transB=True, beta=0.5)
    assert torch.equal(C.cpu(), torch.full((3, 64), 0.5))


def test_other_stream_and_graph(g):
    """The calls on a stream of their own, captured once and replayed."""
    X, W = matrix(100, 512, "f16", 1), matrix(300, 512, "f16", 2, std=0.05)
    dY = matrix(100, 512, "f16", 3)
    A, B, Q = (g.mx_empty(*s) for s in ((100, 512, "fp4"), (300, 512, "fp4"), (100, 512, "int8")))
    C, C1 = (torch.empty((100, 300), dtype=torch.float16, device="cuda") for _ in range(2))
    Y, dX = torch.empty_like(X), torch.empty_like(X)
    db = torch.empty(512, device="cuda")
    dW = torch.empty((300, 512), dtype=torch.float16, device="cuda")
    s = torch.cuda.Stream()

    def step():
        g.mx_quantize(X, A, stream=s)
        g.mx_quantize(W, B, stream=s)
        g.gemm_mx(A, B, C, stream=s)
        g.gemm_mx(X[:1], B, C1[:1], transB=True, stream=s)
        g.mx_quantize(X, Q, act="gelu", Y=Y, stream=s)
        g.mx_act_backward(dY, Q, dX, dbias=db, stream=s)
        g.gemm_mx(C, Q, dW, transA=True, stream=s)

    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    outs = [C, C1[:1], Y, dX, db, dW]
    eager = [t.clone() for t in outs]
    for t in outs:
        t.fill_(float("nan"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    graph.replay()
    torch.cuda.synchronize()
    for t, e in zip(outs, eager):
        assert torch.equal(t, e)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fmt,variant,M,N,K", [
    ("fp4", "nt", 1, 300, 20000), ("fp4", "nt", 13, 200, 20001), ("fp4_e4m3", "nt", 32, 130, 17000),
    ("fp4_e4m3", "nt", 5, 20000, 300), ("int8", "tn", 32, 200, 20000), ("int8", "tn", 7, 130, 20001),
    ("int8", "tn", 31, 9000, 300), ("int8", "tn", 16, 70, 9000)])
def test_few_rows_long_sums(g, dtype, fmt, variant, M, N, K):
    """The streaming kernels past one fill of their rings and one cluster."""
    tA, tB = variant[0] == "t", variant[1] == "t"
    r = np.random.default_rng(300 + M)
    A = matrix(K if tA else M, M if tA else K, dtype, 61)
    B, b = stored(g, (r.standard_normal((N, K) if tB else (K, N)) * 0.05).astype(np.float32), fmt)
    a = f64(A)
    a, b = (a.T if tA else a), (b.T if tB else b)
    C = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda")
    g.gemm_mx(A, B, C, transA=tA, transB=tB)
    assert g.last_path() == "mx_stream"
    check_product(C, a, b, dtype)
    first = C.clone()
    g.gemm_mx(A, B, C, transA=tA, transB=tB)
    assert torch.equal(C, first)


@pytest.mark.parametrize("fmt", FP4)
def test_few_rows_of_two_stored_operands(g, fmt):
    for M, N, K in [(1, 5000, 700), (9, 300, 9001), (32, 200, 12000), (17, 129, 31)]:
        r = np.random.default_rng(400 + M)
        A, a = stored(g, r.standard_normal((M, K)).astype(np.float32), fmt)
        B, b = stored(g, (r.standard_normal((N, K)) * 0.05).astype(np.float32), fmt)
        C = torch.full((M, N), float("nan"), device="cuda")
        g.gemm_mx(A, B, C)
        assert g.last_path() == "mx_stream"
        check_product(C, a, b.T, "f32")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_wgrad_scales_past_fp16(g, dtype):
    """Checkpoint rows whose power of two is no normal fp16 number, beside
    ordinary ones; their products are far below or within fp32's range."""
    r = np.random.default_rng(9)
    x = r.standard_normal((200, 140)).astype(np.float32)
    x[3] *= 2.0 ** -17
    x[70] *= 2.0 ** -12
    x[71, :32] = 0.0
    if dtype == "bf16":
        x[5] *= 2.0 ** 40
        x[6] *= 2.0 ** -40
    B, b = stored(g, x, "int8")
    A = matrix(200, 24, dtype, 3)
    C = torch.empty((24, 140), dtype=DT[dtype], device="cuda")
    g.gemm_mx(A, B, C, transA=True)
    assert g.last_path() == "mx_stream"
    check_product(C, f64(A).T, b, dtype)


@pytest.mark.parametrize("case", ["mx4", "stream", "wgrad", "convert"])
def test_bounded_waits(lib_path, gpu, case):
    """A load that never comes ends as a status, not as a hang (the library's own
    test hook: the producer leaves out its first load)."""
    from dense_gemm_tiled_gb300 import binding as g
    r = np.random.default_rng(1)
    B, _ = stored(g, r.standard_normal((256, 512)).astype(np.float32), "int8" if case == "wgrad" else "fp4")
    M = 200 if case == "mx4" else 8
    A = stored(g, r.standard_normal((M, 512)).astype(np.float32), "fp4")[0] if case == "mx4" else \
        matrix(*{"wgrad": (256, 8), "convert": (8, 256), "stream": (8, 512)}[case], "f16", 1)
    C = torch.empty((M, 512 if case in ("wgrad", "convert") else 256), dtype=torch.float16,
                    device="cuda")
    call = lambda: g.gemm_mx(A, B, C, transA=case == "wgrad", transB=case == "stream")  # noqa: E731
    call()
    torch.cuda.synchronize()
    assert g.last_path() == {"mx4": "mx_tc", "convert": "mx_convert"}.get(case, "mx_stream")
    want = C.clone()
    g.set_wait_timeout_ns(20_000_000)
    g.set_fault_injection(1)
    try:
        call()
        assert g.check_device_status() == g.ERR_TIMEOUT
    finally:
        g.set_fault_injection(0)
        g.set_wait_timeout_ns(0)
    call()
    assert g.check_device_status() == g.OK
    assert torch.equal(C, want)


@pytest.mark.parametrize("dtype", list(DT))
def test_activation_at_the_ends(g, dtype):
    """gelu far out on both sides, at the type's ends and at infinities; a NaN
    stays one; an infinite gradient stays infinite where the slope is not 0."""
    top = torch.finfo(DT[dtype]).max
    x = torch.tensor([[-top, -100.0, -64.0, -20.0, -8.0, -5.0, -0.0, 0.0, 5.0, 8.0, 20.0, 64.0, 100.0,
                       top, float("inf"), float("-inf"), float("nan")]]).to(DT[dtype])
    X = x.cuda()
    Y, Q = torch.empty_like(X), filled(g, 1, 17, "int8")
    g.mx_quantize(X, Q, act="gelu", Y=Y)
    y, want = f64(Y)[0], mx_ref.gelu(f64(x)[0][:14])
    assert np.all(np.abs(y[:14] - want) <= 2.0 ** -20 * (np.abs(f64(x)[0][:14]) + np.abs(want)) +
                  2.0 ** -8 * np.abs(want))
    assert y[14] == np.inf and y[15] == 0.0 and np.isnan(y[16])
    X = torch.tensor([[-4.0, -1.0, 0.0, 1.0, 4.0, 0.5]], dtype=DT[dtype], device="cuda")
    dY = torch.tensor([[1.0, 1.0, float("inf"), float("-inf"), float("nan"), 2.0]],
                      dtype=DT[dtype], device="cuda")
    Q, dX = filled(g, 1, 6, "int8"), torch.empty_like(dY)
    g.mx_quantize(X, Q)
    g.mx_act_backward(dY, Q, dX)
    d = f64(dX)[0]
    assert d[2] == np.inf and d[3] == -np.inf and np.isnan(d[4]) and np.isfinite(d[[0, 1, 5]]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("fmt,variant,M,N,K", [
    ("fp4", "nt", 700, 600, 2100), ("fp4_e4m3", "nt", 513, 1000, 777), ("fp4", "nn", 300, 900, 1300),
    ("fp4_e4m3", "nn", 130, 515, 2050), ("int8", "tn", 900, 700, 1000), ("int8", "tn", 66, 4000, 130),
    ("fp4_e4m3", "nn", 1, 3000, 500), ("fp4", "nt", 33, 8000, 96)])
def test_converted_product(g, dtype, fmt, variant, M, N, K):
    """The kernel that converts the stored operand: several tiles both ways,
    ragged, more stages than its ring; the same twice."""
    tA, tB = variant[0] == "t", variant[1] == "t"
    r = np.random.default_rng(500 + M)
    A = matrix(K if tA else M, M if tA else K, dtype, 71)
    B, b = stored(g, (r.standard_normal((N, K) if tB else (K, N)) * 0.05).astype(np.float32), fmt)
    a = f64(A)
    a, b = (a.T if tA else a), (b.T if tB else b)
    C = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda")
    g.gemm_mx(A, B, C, transA=tA, transB=tB)
    check_product(C, a, b, dtype)
    C1 = torch.full_like(C, float("nan"))
    g.gemm_mx(A, B, C1, transA=tA, transB=tB)
    assert torch.equal(C, C1)
    bias, C0 = matrix(1, N, dtype, 7)[0], matrix(M, N, dtype, 8, offset=1, pitch=N + 3)
    c0 = f64(C0)
    g.gemm_mx(A, B, C0, transA=tA, transB=tB, alpha=0.5, beta=-1.0, bias=bias, act="gelu")
    check_product(C0, a, b, dtype, 0.5, -1.0, c0, f64(bias), "gelu")


def far_rows(rows, cols, pitch, dtype, seed):
    """A matrix whose rows lie `pitch` elements apart in one large allocation."""
    base = torch.empty((rows - 1) * pitch + cols, dtype=DT[dtype], device="cuda")
    v = base.as_strided((rows, cols), (pitch, 1))
    if seed is not None:
        v.copy_(matrix(rows, cols, dtype, seed))
    return v


def test_offsets_past_32_bits(g):
    """Rows 2^31 elements (or bytes of codes) apart, and 130 rows 2^25 apart:
    every byte and element offset passes 32 bits (allocations of 4 to 9 GB)."""
    P = 1 << 31
    X = far_rows(3, 100, P, "f16", 1)
    codes = torch.empty(2 * P + 112, dtype=torch.uint8, device="cuda").as_strided((3, 112), (P, 1))
    Q = g.Mx(codes, torch.empty(g.mx_scale_bytes("int8", 3, 100), dtype=torch.uint8, device="cuda"),
             "int8", 3, 100)
    Y = far_rows(3, 100, P, "f16", None)
    g.mx_quantize(X, Q, act="gelu", Y=Y)
    want, st, xq = mx_ref.store(f64(X), "int8")
    assert np.array_equal(codes.cpu().numpy(), want) and np.array_equal(Q.scales.cpu().numpy(), st)
    y = mx_ref.gelu(f64(X))
    assert np.all(np.abs(f64(Y) - y) <= 2.0 ** -20 * (np.abs(f64(X)) + np.abs(y)) + 2.0 ** -10 * np.abs(y) + 2.0 ** -24)
    g.mx_dequantize(Q, Y)
    assert torch.equal(Y.cpu(), torch.from_numpy(xq).to(torch.float16))
    g.mx_act_backward(X, Q, Y, act="relu")
    assert torch.equal(Y.cpu(), (torch.from_numpy(xq) > 0).half() * X.cpu())
    del X, Y, codes, Q
    torch.cuda.empty_cache()
    P = 1 << 25
    r = np.random.default_rng(6)
    (A, a), (B, b) = (stored(g, r.standard_normal((n, 96)).astype(np.float32), "fp4") for n in (130, 104))
    C = far_rows(130, 104, P, "f16", None)
    g.gemm_mx(A, B, C)
    check_product(C, a, b.T, "f16")
    c0 = f64(C)
    g.gemm_mx(A, B, C, alpha=0.5, beta=1.0)
    check_product(C, a, b.T, "f16", 0.5, 1.0, c0)
    X = far_rows(130, 96, P, "f16", 7)
    for M in (130, 5):  # expanded or converted, and streamed
        g.gemm_mx(X[:M], B, C[:M], transB=True)
        check_product(C[:M].contiguous(), f64(X[:M]), b.T, "f16")
    Q, q = stored(g, r.standard_normal((130, 200)).astype(np.float32), "int8")
    W = torch.empty((96, 200), dtype=torch.float16, device="cuda")
    g.gemm_mx(X, Q, W, transA=True)
    check_product(W, f64(X).T, q, "f16")
    g.gemm_mx(X[:, :24], Q, W[:24], transA=True)
    check_product(W[:24], f64(X[:, :24]).T, q, "f16")
