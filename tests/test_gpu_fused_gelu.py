"""gelu of fused fp32 products: one function whether or not the pre-activation is kept."""
import pytest
import torch

import fused_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture
def g(lib_path, gpu):
    from dense_gemm_tiled_gb300 import binding
    yield binding
    torch.cuda.synchronize()
    assert binding.check_device_status() == binding.OK


def new(*shape, seed=0, std=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=gen) * std).cuda()


@pytest.mark.parametrize("M,N,K", [(1, 40, 64), (17, 72, 4104), (33, 65, 63), (130, 264, 100), (64, 32, 2000),
                                   (300, 1030, 2056), (1024, 1024, 1024), (700, 512, 0), (2100, 1300, 300)])
def test_kept_or_not(g, M, N, K):
    """The same values, bit for bit, in inference and in training (every path of the fp32
    products: whole tiles, slices of K, shared tiles, no inner dimension)."""
    A, B, b = new(M, K, seed=1), new(N, K, seed=2, std=0.2), new(N, seed=3)
    Y, Y2, U = (torch.full((M, N), float("nan"), device="cuda") for _ in range(3))
    g.gemm_fused(A, B, Y, transB=True, bias=b, act="gelu")
    g.gemm_fused(A, B, Y2, transB=True, bias=b, act="gelu", preact=U)
    assert torch.equal(Y, Y2)
    _, _, y, ey = ref.forward(A.double(), B.double().t(), "f32", bias=b.double(), name="gelu")
    ref.check(Y, y, ey)


@pytest.mark.parametrize("rows,K", [(3, 0), (3, 8), (200, 40), (20, 4000)])
@pytest.mark.parametrize("keep", [False, True])
def test_tails(g, rows, K, keep):
    """The negative tail keeps its relative accuracy: CUDA gives 5 ulp for normcdff, the
    product with |u| and the sum with max(u, 0) half an ulp each: 6 ulp, 2^-23 each."""
    v = torch.linspace(-12, 12, 4 * 1201, device="cuda")
    A, B = torch.zeros((rows, K), device="cuda"), torch.ones((v.numel(), K), device="cuda")
    Y = torch.full((rows, v.numel()), float("nan"), device="cuda")
    g.gemm_fused(A, B, Y, transB=True, bias=v, act="gelu", preact=torch.empty_like(Y) if keep else None)
    y = ref.act(v.double(), "gelu").expand_as(Y)
    ref.check(Y, y, 6 * 2.0 ** -23 * y.abs())
