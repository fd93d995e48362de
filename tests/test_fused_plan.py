"""The choice of a fused product's tile and slices of K (csrc/fused_plan.h), on the host:
every size that a call may have, none of them trapping, and what the kernel asks of it."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_gemm_tiled_gb300", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include "fused_plan.h"
using namespace gb300;
int main() {
  // (none, one, those about the tiles and the largest)
  const int sizes[] = {0, 1, 2, 15, 16, 17, 63, 64, 65, 128, 255, 257, 1000, 4096, 30001, 2147221504};
  int n = 0;
  for (int kind = FUSED_DENSE; kind <= FUSED_INNER; ++kind)
    for (int M : sizes) for (int N : sizes) for (int K : sizes)
      for (int groups : {1, 2, 7, 300, 65535}) {
        if (N == 0 || (kind == FUSED_DENSE && groups > 1)) continue;
        // (C without rows is no call, and one past any memory is not either)
        if (kind == FUSED_INNER && (M == 0 || (double)M * N * groups > 1e12)) continue;
        FusedArgs a = {};
        a.kind = kind;
        a.dtype = 1;
        a.transA = kind == FUSED_INNER;
        a.transB = M & 1;
        a.M = M; a.N = N; a.K = K;
        a.groups = groups;
        a.num_sms = 152;
        fused_plan(a);
        const int steps = (K + 63) / 64, each = (steps + a.splits - 1) / a.splits;
        if (a.tile < 0 || a.tile >= FUSED_TILES || a.splits < 1 || a.splits > FUSED_MAX_SPLITS ||
            (a.splits > 1 && (kind != FUSED_DENSE || (a.splits - 1) * each >= steps))) {
          printf("kind %d %d x %d x %d, %d groups: tile %d, %d slices\n", kind, M, N, K, groups, a.tile,
                 a.splits);
          return 1;
        }
        ++n;
      }
  printf("ok %d\n", n);
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    from dense_gemm_tiled_gb300 import build
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "t.cpp", d / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all",
                    "-I" + CSRC, "-I" + cuda, str(src), "-o", str(exe)], check=True)
    return str(exe)


@pytest.mark.parametrize("env", [{}] + [{"GEMM_GB300_FUSED_TILE": t, "GEMM_GB300_FUSED_SPLITS": s}
                                        for t, s in (("0", "4"), ("1", "2"), ("3", "1"), ("9", "9"))])
def test_every_size_has_a_plan(program, env):
    """Without rows too: a rank whose experts got no tokens asks for zero column sums."""
    r = subprocess.run([program], env=dict(os.environ, **env), capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout + r.stderr


def test_no_plan_without_rows():
    """A call without rows has no product to plan."""
    text = open(os.path.join(CSRC, "fused_api.cu")).read()
    assert "if (!few && !none) fused_plan(a);" in text
