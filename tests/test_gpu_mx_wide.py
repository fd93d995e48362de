"""The activation's backward pass at the most columns that a row may have (2^31 -
1; about 30 GB on the device)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_column_sums_of_the_widest_row(lib_path, gpu):
    from dense_gemm_tiled_gb300 import binding as g
    cols = (1 << 31) - 1
    Q = g.mx_empty(1, cols, "int8")
    Q.codes.zero_()
    Q.scales.fill_(121)  # 2^-6
    lit = [0, 1, 63, 64, (1 << 30) + 5] + list(range(cols - 70, cols))
    at = torch.tensor(lit, device="cuda")
    Q.codes[0, at] = 64  # x = 1; 0 elsewhere
    dY = torch.full((1, cols), 0.5, dtype=torch.float16, device="cuda")
    dY[0, at] = torch.arange(1, len(lit) + 1, device="cuda").half()
    want = dY[0, at].float()
    db = torch.full((cols,), float("nan"), device="cuda")
    g.mx_act_backward(dY, Q, dY, act="relu", dbias=db)
    assert torch.equal(db[at], want) and torch.equal(dY[0, at].float(), want)
    for t in (db, dY[0]):  # and 0 in every other column
        assert sum(int(torch.count_nonzero(p)) for p in t.split(1 << 28)) == len(lit)
    assert g.check_device_status() == g.OK
