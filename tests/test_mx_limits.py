"""The products with stored operands at the largest sizes that their kernels'
32-bit counts hold (no GPU: made-up addresses, refused or stopped before a launch)."""
import pytest

D, X, S, BQ, BS = (0x10000000000 * i for i in range(1, 6))
TOP = (1 << 31) - (1 << 18)
UNSUPPORTED, NO_DEVICE = 2, 4


@pytest.fixture(scope="module")
def b(lib_path):
    from dense_gemm_tiled_gb300 import binding
    return binding


def call(b, which, M, N, K):
    pad = lambda n: -(-n // 16) * 16  # noqa: E731
    if which == "mx4":
        ld = pad(-(-K // 2))
        return b._lib.gemm_mx4(0, M, N, K, 1, 1.0, 0.0, X, ld, S, BQ, ld, BS, D, N, None, 0, None)
    fmt, tA, tB = which
    row = K if tB else N
    return b._lib.gemm_mx(fmt, tA, tB, M, N, K, 1, 1.0, 0.0, X, M if tA else K, BQ,
                          pad(row if fmt == 2 else -(-row // 2)), BS, D, N, None, 0, None)


WHICH = ["mx4", (0, 0, 1), (1, 0, 0), (2, 1, 0), (2, 0, 1)]


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("place", range(3))
def test_sizes_past_the_end(b, which, place):
    for n in (TOP + 1, 2**31 - 256, 2**31 - 255, 2**31 - 1, 2**31):
        size = [1, 1, 1]
        size[place] = n
        assert call(b, which, *size) == UNSUPPORTED, n
        assert b.last_path() == "none"


@pytest.mark.parametrize("which", WHICH)
@pytest.mark.parametrize("place", range(3))
def test_largest_size_is_taken(b, which, place):
    import torch
    if torch.cuda.is_available():
        pytest.skip("valid arguments with made-up addresses: not launched on a GPU")
    size = [1, 1, 1]
    size[place] = TOP
    assert call(b, which, *size) == NO_DEVICE
