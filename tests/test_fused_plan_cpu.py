"""The fused products' plans over the sizes that the library takes (host logic
only)."""
import pytest

import microscaled_block_scaled_amd as mxg

TOP = 1 << 30                           # MX_MAX_DIM
FORMATS = [(mxg.FMT_E2M1, None), (mxg.FMT_E4M3, None), (mxg.FMT_E4M3, mxg.FMT_E2M1), (None, None)]


@pytest.mark.parametrize("fmt,fmt_b", FORMATS)
def test_grids_can_be_launched(fmt, fmt_b):
    """A launch has less than 2^32 threads, as mx_gemm's plans for the same
    sizes have: small tiles must not go beyond."""
    for M, N in ((8, TOP), (64, TOP), (33, TOP - 63), (64, TOP - 64), (TOP, 8), (TOP, 64),
                 (TOP - 1, 33), (100, TOP // 2), (TOP // 2, 129), (1, TOP)):
        for K in (128, 512, 16384):
            p = mxg.plan_fused(fmt, M, N, K, fmt_b=fmt_b)
            assert p["tile_m"] > 0 and 0 < p["workgroups"] * p["threads"] < 1 << 32, (M, N, K, p)


@pytest.mark.parametrize("fmt,fmt_b", FORMATS)
def test_grids_that_cannot_be_numbered_are_refused(fmt, fmt_b):
    with pytest.raises(ValueError):
        mxg.plan_fused(fmt, TOP, TOP, 128, fmt_b=fmt_b)
