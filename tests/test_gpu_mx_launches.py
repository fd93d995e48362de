"""What a product with a stored operand launches where rows of A are off 16-byte
alignment: one copy of A, whichever kernel takes the product."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("fmt,variant,M,N,K", [
    ("fp4", "nt", 4000, 1024, 520), ("fp4_e4m3", "nn", 4000, 1024, 520),
    ("int8", "tn", 4000, 1024, 520), ("fp4", "tn", 40, 512, 520), ("int8", "nt", 40, 512, 520),
    ("int8", "nn", 4, 512, 520), ("fp4", "nt", 100, 512, 520), ("fp4", "nt", 8, 512, 520),
    ("int8", "tn", 8, 512, 520)])
def test_one_copy_of_an_unaligned_operand(lib_path, gpu, dtype, fmt, variant, M, N, K):
    from dense_gemm_tiled_gb300 import binding as g
    tA, tB = variant[0] == "t", variant[1] == "t"
    shape = (K, M) if tA else (M, K)
    gen = torch.Generator(device="cuda").manual_seed(M)
    A = torch.randn(shape, generator=gen, device="cuda").to(dtype)
    off = torch.empty((shape[0], shape[1] + 3), dtype=dtype, device="cuda")[:, 1: shape[1] + 1]
    off.copy_(A)
    W = torch.randn((N, K) if tB else (K, N), generator=gen, device="cuda") * 0.05
    B = g.mx_quantize(W, g.mx_empty(*W.shape, fmt))
    C, D = (torch.empty((M, N), dtype=dtype, device="cuda") for _ in range(2))
    g.gemm_mx(A, B, C, transA=tA, transB=tB)
    aligned, path = g.last_launches(), g.last_path()
    torch.cuda.synchronize()
    g.scratch_high_water(reset=True)
    g.gemm_mx(off, B, D, transA=tA, transB=tB)
    assert g.last_path() == path and g.last_launches() == aligned + 1
    torch.cuda.synchronize()
    # the copy, at most the expanded B and the 16-bit kernel's own scratch: not two
    # copies
    copy = 2 * shape[0] * (-(-shape[1] // 8) * 8)
    if copy > 2 * N * K + (1 << 21):
        assert g.scratch_high_water() < 2 * copy
    assert torch.equal(C, D)
