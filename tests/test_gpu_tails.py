"""GPU tests of the arithmetic's far ends.

Tolerances: rstd with an exact mean and eps 0 has only its own rounding, half
a unit in the last place; the correction's own error is below 2^-20 of one."""
import numpy as np
import pytest

import block_ref as ref
import microscaled_block_scaled_amd as mxg
import oracle
from gpu_util import log

pytestmark = pytest.mark.gpu

U = ref.U32


def _dev(a, dtype="float32"):
    import torch
    return torch.from_numpy(np.asarray(a, np.float32)).to(getattr(torch, dtype)).cuda()


def _h64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype,top", [("float32", 64), ("bfloat16", 16)])
@pytest.mark.parametrize("width", [32, 1024, 8192, 32768])
def test_rstd_is_rounded_once(width, dtype, top):
    """Integers whose squares' sum is exact in any order: rstd is 1 / sqrt of
    an exact mean."""
    log("rstd of exact means, width %d %s" % (width, dtype))
    rng = np.random.default_rng(width + top)
    most = min(top, int((2.0 ** 24 / width) ** 0.5))
    x = rng.integers(-most, most + 1, (400, width)).astype(np.float64)
    x *= 2.0 ** rng.integers(-50, 50, (400, 1))            # exact too
    x[:3] = [[2.0 ** -70], [2.0 ** 55], [1.0]]
    o = mxg.mx_rmsnorm_quantize(_dev(x, dtype), _dev(np.ones(width)), mxg.FMT_E4M3, eps=0.0,
                                need_rstd=True)
    got = o.rstd.cpu().numpy()
    want = 1.0 / np.sqrt((x * x).mean(1))
    assert (abs(got - want) <= 0.501 * np.spacing(got).astype(np.float64)).all(), \
        float((abs(got - want) / np.spacing(got)).max())


@pytest.mark.parametrize("fmt", [mxg.FMT_E4M3, mxg.FMT_E5M2, mxg.FMT_E2M1])
def test_y_overflows_bf16_beside_saturating_elements(fmt):
    """y beyond BF16's range becomes an infinity in the same call that
    saturates 8-bit elements to their largest value."""
    import torch
    log("overflowing y beside fmt %d" % fmt)
    width = 2048
    x = torch.ones((5, width), dtype=torch.bfloat16, device="cuda")
    w = torch.full((width,), 3.4e38, device="cuda")   # past BF16's largest, in FP32
    w[1::2] = 1.9 * 2.0 ** 127                              # in range for both
    w[::64] = -3.4e38
    o = mxg.mx_rmsnorm_quantize(x, w, fmt, eps=0.0, need_y=True)
    y = w.expand(5, width)
    assert torch.equal(o.y, y.to(torch.bfloat16)) and torch.isinf(o.y).any()
    rq, rs = oracle.quantize(fmt, _h64(y))
    assert (o.q.cpu().numpy() == rq).all() and (o.q_scale.cpu().numpy() == rs).all()
