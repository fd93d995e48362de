"""Grouped products whose offsets do not ascend: what is guarded, and that the work stays
bounded; and the tile count that bounds it, on the host."""
import os
import random

import pytest
import torch

from fused_ref import DT

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "dense_gemm_tiled_gb300", "csrc")


def test_ascending_offsets_stay_within_the_bound():
    """ceil(rows / tile) + min(groups, rows) row tiles are enough for any ascending
    offsets, and the kernel's walk ends there."""
    rng = random.Random(1)
    for _ in range(2000):
        rows, groups, tile = rng.choice([0, 1, 5, 300, 5000]), rng.choice([1, 2, 9, 400]), rng.choice([128, 256])
        at = sorted(rng.randint(0, rows) for _ in range(groups + 1))
        used = sum(-(-(b - a) // tile) for a, b in zip(at, at[1:]))
        assert used <= -(-rows // tile) + min(groups, rows)
    # (alternating ones would ask for half the groups times all rows)
    text = open(os.path.join(CSRC, "fused_tcgen05.cuh")).read()
    walk = text[text.index("bool find(const FuParams& p"):]
    assert walk.index("if (t >= p.tiles) return false;") < walk.index("rows.find(")


@pytest.mark.gpu
def test_work_is_bounded(lib_path, gpu):
    """Offsets 0, rows, 0, rows ...: no more tiles than a group for each row has, where
    every second group's would be 128 times as many."""
    from dense_gemm_tiled_gb300 import binding as g
    rows, E, N, K = 4096, 65535, 512, 64
    A = torch.ones((rows, K), dtype=torch.bfloat16, device="cuda")
    B = torch.ones((K, N), dtype=torch.bfloat16, device="cuda").expand(E, K, N)
    Y = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    each = torch.arange(E + 1, device="cuda").clamp(max=rows).to(torch.int32)
    bad = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    bad[1::2] = rows
    ms = {}
    for name, offs in (("each", each), ("bad", bad)):
        for _ in range(3):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            g.gemm_grouped(A, B, Y, offs)
            end.record()
            torch.cuda.synchronize()
            ms[name] = start.elapsed_time(end)
        assert g.check_device_status() == (g.OK if name == "each" else g.ERR_INVALID_ARG)
        if name == "each":
            assert (Y == K).all()
    assert ms["bad"] <= 16 * ms["each"], ms
