"""The CPU models and the register checks of the GEMM kernels, for those with
the fused epilogue (no GPU): their tiles' copies stay inside the operands, they
have the ring that the copy model checks, and neither they nor the row kernels
of ordinary widths spill registers."""
import os
import re

import pytest

import test_copy_bounds_cpu as cb
import test_kernel_resources_cpu as res
from microscaled_block_scaled_amd import build as B

PAIRS = [(cb.FP4, cb.FP4), (cb.FP8, cb.FP8), (cb.FP8, cb.FP4), (cb.B16, cb.B16)]


def fused_tiles():
    """(BM, BN, waves along M, waves along N) of the fused products' table."""
    src = open(os.path.join(B.CSRC, "mxfused.hip")).read()
    body = src[src.index("kFusedTiles[] = {"):]
    rows = re.findall(r"\{(\d+), (\d+), (\d+), (\d+), [\d.]+\}", body[:body.index("};")])
    return [tuple(int(v) for v in r) for r in rows]


def test_the_table_is_read_whole():
    tiles = fused_tiles()
    assert len(tiles) == 6 and {(128, 128, 4, 2), (128, 64, 2, 2), (64, 64, 2, 2)} <= set(tiles)


@pytest.mark.parametrize("tile", fused_tiles(), ids=["%dx%d" % t[:2] for t in fused_tiles()])
def test_fused_copies_stay_inside_their_operands(tile):
    BM, BN, WGM, WGN = tile
    shapes = [(8, 8192, 4096), (1, 1, 512), (300, 200, 1536), (BM, BN, 2048), (BM, 3 * BN, 384),
              (BM + 5, 2 * BN - 3, 640), (2 * BM - 1, BN + 1, 1664), (40, 203, 2560), (70, 512, 8192)]
    bad = []
    for fa, fb in PAIRS:
        for M, N, K in shapes:
            for kchunk in sorted({K, max(512, -(-K // 3) // 512 * 512)}):
                for prob in cb.check(fa, fb, BM, BN, WGM, WGN, M, N, K, kchunk):
                    bad.append(((fa, fb), (M, N, K), kchunk, prob))
    assert not bad, bad[:5]


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if not os.path.exists(res.LIB):
        pytest.skip("libmxgemm.so is not built")
    for tool in ("llvm-objcopy", "clang-offload-bundler", "llvm-readelf"):
        if not os.path.exists(os.path.join(res.LLVM, tool)):
            pytest.skip("ROCm LLVM tools not available")
    return res._kernels(tmp_path_factory.mktemp("kernels"))


def test_fused_decode_kernels_have_the_model_s_ring(kernels):
    seen = 0
    for name, v in kernels.items():
        m = re.search(r"fused_decodeILi(\d)ELi(\d)ELi(\d)ELi(\d+)E", name)
        if not m:
            continue
        fa, fb, wide = int(m.group(1)), int(m.group(2)), int(m.group(4))
        kv, RA, RB, MA, ncopy, S, R = cb.decode_geo(fa, fb, wide)
        want = (cb.DECODE_WAVES * (S * (MA * RA + cb.DECODE_ROWS * RB) + R * 1024)
                + cb.DECODE_OFFS)
        assert v.get("group_segment_fixed_size") == want, (name, v, want)
        assert v.get("vgpr_spill_count", 0) == 0, (name, v)
        seen += 1
    assert seen == 10


def test_row_kernels_of_ordinary_widths_do_not_spill(kernels):
    """Rows of up to 8192 values, and everything that does not hold a row."""
    names = ["norm_quantizeILi%dELi%dELi512ELi2E" % (i, f) for i in (1, 2) for f in (1, 2, 3, 5, 6)]
    names += ["norm_gradILi%dELi1024ELi1E" % i for i in (1, 2)]
    names += ["norm_grad_fewILi%dELi1024ELi1E" % i for i in (1, 2)]
    names += ["column_sum", "swiglu_quantize", "swiglu_grad", "moe_sort", "moe_count", "moe_gather",
              "moe_combine", "moe_combine_grad", "splitk_fused"]
    for name in names:
        found = {k: v for k, v in kernels.items() if name in k}
        assert found, name
        assert not [(k, v) for k, v in found.items() if v.get("vgpr_spill_count", 0)], name
