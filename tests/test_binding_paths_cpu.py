"""What block.py hands to the compiled half of the binding (no GPU: a stand-in
takes the calls)."""
import pytest

import microscaled_block_scaled_amd as mxg
from microscaled_block_scaled_amd import block


class _Handed(Exception):
    pass


def test_no_format_differs_from_every_format_code(monkeypatch):
    """fmt None, no quantized output, reaches the compiled call as what no
    integer can be."""
    handed = []

    def fast(name, stream, like, *args):
        handed.append(args)
        raise _Handed

    monkeypatch.setattr(block, "_fast", fast)
    for fmt in (None, 0, -1, mxg.FMT_E4M3):
        with pytest.raises(_Handed):
            mxg.mx_rmsnorm_quantize("x", "weight", fmt, eps=1e-5, need_y=True)
    assert [a[3] for a in handed] == [None, 0, -1, mxg.FMT_E4M3]


def test_an_activation_beyond_32_bits_does_not_wrap():
    for act in (-1, 5, 1 << 32, (1 << 32) + 1, None, "relu", 1.5):
        with pytest.raises(ValueError):
            block._act(act)
    assert [block._act(a) for a in (0, 1, 2, 3, 4)] == [0, 1, 2, 3, 4]
