"""Stored operands whose tensors get other storage after the Mx was made."""
import numpy as np
import pytest
import torch

import mx_ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["data", "set_", "module", "tensor"])
def test_replaced_storage(lib_path, gpu, how):
    from dense_gemm_tiled_gb300 import binding as g
    r = np.random.default_rng(1)
    w = [r.standard_normal((64, 96)).astype(np.float32) for _ in range(2)]
    (c0, s0, v0), (c1, s1, v1) = (mx_ref.store(x, "fp4") for x in w)
    codes, scales = (torch.nn.Parameter(torch.from_numpy(t).cuda(), requires_grad=False)
                     for t in (c0, s0))
    Q = g.Mx(codes, scales, "fp4", 64, 96)
    Y = torch.empty((64, 96), device="cuda")
    assert np.array_equal(g.mx_dequantize(Q, Y).cpu().numpy(), v0)
    n0, n1 = torch.from_numpy(c1).cuda(), torch.from_numpy(s1).cuda()
    if how == "data":
        codes.data, scales.data = n0, n1
    elif how == "set_":
        codes.set_(n0), scales.set_(n1)
    elif how == "tensor":
        Q.codes, Q.scales = n0, n1
    else:  # a module that goes to the host, is loaded there, and comes back
        m = torch.nn.Module()
        m.codes, m.scales = codes, scales
        m.to("cpu")
        with pytest.raises(ValueError):
            g.mx_dequantize(Q, Y)
        m.codes.copy_(n0), m.scales.copy_(n1)
        m.to("cuda")
    Y.fill_(float("nan"))
    assert np.array_equal(g.mx_dequantize(Q, Y).cpu().numpy(), v1)
    A = torch.eye(96, device="cuda")
    C = torch.empty((96, 64), device="cuda")
    assert np.array_equal(g.gemm_mx(A, Q, C, transB=True).cpu().numpy(), v1.T)
