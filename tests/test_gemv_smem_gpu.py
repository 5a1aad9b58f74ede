"""CUDA-core decode kernels whose staged x takes a little less than the 48 KB of shared memory
that a kernel has without asking: its static arrays count towards them."""

import pytest

import moe_expert_routed_b200 as M
from tests.gpu_util import check_full, run
from workloads.gen import (DT_BF16, DT_F32, FMT_AFFINE, FMT_CODEBOOK, FMT_NVFP4, make_problem)

pytestmark = pytest.mark.gpu


# bytes of 8 rows of staged x: units of 32 codes (16 of 8 bits) take 33 (17) floats
@pytest.mark.parametrize("fmt,bits,gs,k", [(FMT_CODEBOOK, 4, 16, 1472),   # 48,576
                                           (FMT_AFFINE, 8, 16, 1440),     # 48,960
                                           (FMT_AFFINE, 4, 16, 1472),     # 48,576
                                           (FMT_NVFP4, 4, 16, 1488),      # 49,104 with the last half unit
                                           (FMT_AFFINE, 8, 16, 1424),     # 48,416
                                           (FMT_AFFINE, 8, 16, 1456)])    # 49,504: above 48 KB
@pytest.mark.parametrize("m,E", [(27, 1), (40, 2), (130, 40)])
def test_staged_x_near_48_kb(fmt, bits, gs, k, m, E):
    P = make_problem("near", fmt=fmt, bits=bits, group_size=gs, m=m, k=k, n=72, n_expert_used=1 + (E > 1),
                     num_experts=E, x_dtype=DT_BF16, out_dtype=DT_F32, seed=k)
    ws = M.new_workspace(P.m, P.n_expert_used, P.num_experts)
    out = run(P, "decode", workspace=ws)
    assert M.poll_error(ws) == 0
    nviol, ratio, _ = check_full(P, out)
    assert nviol == 0, f"worst err / bound {ratio:.3g}"


@pytest.mark.parametrize("fmt,bits,gs,k", [(FMT_CODEBOOK, 4, 64, 7936), (FMT_AFFINE, 4, 16, 7936),
                                           (FMT_AFFINE, 4, 64, 7936), (FMT_NVFP4, 4, 16, 8192)])
@pytest.mark.parametrize("m", [3, 5, 6, 7, 8])
def test_long_rows_for_five_to_seven_tokens(fmt, bits, gs, k, m):
    """Rows of which fewer than eight fit in shared memory: kernels have room for 1, 2, 4 or 8 pairs,
    so five to seven count as eight."""
    P = make_problem("long", fmt=fmt, bits=bits, group_size=gs, m=m, k=k, n=40, n_expert_used=1, num_experts=1,
                     x_dtype=DT_F32, out_dtype=DT_F32, seed=m)
    ws = M.new_workspace(P.m, 1, 1)
    out = run(P, "decode", workspace=ws)
    assert M.poll_error(ws) == 0
    nviol, ratio, _ = check_full(P, out)
    assert nviol == 0, f"worst err / bound {ratio:.3g}"
