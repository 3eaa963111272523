"""GPU test of a fused product at the most columns the library takes."""
import pytest

import microscaled_block_scaled_amd as mxg
from gpu_util import log

pytestmark = pytest.mark.gpu


def test_most_columns():
    """2^30 columns: ones times ones, K of them, plus a bias that tells the
    columns apart; exact in BF16."""
    import torch
    M, N, K = 2, 1 << 30, 128
    log("fused product of %d columns" % N)
    a = torch.full((M, K // 2), 0x22, dtype=torch.uint8, device="cuda")       # E2M1 ones
    b = torch.full((N, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    sa = torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda")
    sb = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    bias = torch.arange(N, device="cuda", dtype=torch.int32).remainder(127).to(torch.bfloat16)
    p = mxg.plan_fused(mxg.FMT_E2M1, M, N, K)
    assert p["workgroups"] * p["threads"] < 1 << 32
    c = mxg.mx_gemm_fused(a, sa, b, sb, mxg.FMT_E2M1, bias=bias)
    del b, sb
    step = 1 << 27
    for at in range(0, N, step):
        assert (c[:, at:at + step] == bias[at:at + step] + K).all(), at
