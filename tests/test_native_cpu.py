"""The compiled half of the binding without a GPU: it loads, is bound to the
library, and answers None -- no crash, no exception -- to whatever is not
plain tensors on the device."""
import pytest

import microscaled_block_scaled_amd as mxg
from microscaled_block_scaled_amd import block

# arguments of each entry, without device and stream
COUNTS = {"rmsnorm_quantize": 7, "rmsnorm_backward": 6, "swiglu_quantize": 2, "swiglu_backward": 2,
          "moe_sort": 2, "moe_gather": 3, "moe_combine": 4, "moe_combine_backward": 4,
          "gemm_fused": 11, "gemm_bf16_fused": 7}


def test_every_entry_is_there():
    n = block.native()
    assert {k for k in dir(n) if not k.startswith("__")} == set(COUNTS) | {"bind"}


@pytest.mark.parametrize("name", sorted(COUNTS))
def test_anything_else_is_none(name):
    import torch
    f = getattr(block.native(), name)
    cpu = torch.zeros((4, 64))
    for value in (None, 3, -1, 1 << 70, 2.5, "x", [cpu], cpu, cpu[0], cpu.t(), torch.zeros(()),
                  torch.zeros((2, 2, 2)), torch.nn.Parameter(cpu), cpu.to_sparse(), object()):
        assert f(*([value] * COUNTS[name]), 0, 0) is None
        assert f(*([cpu] + [value] * (COUNTS[name] - 1)), 0, 0) is None
    assert f() is None
    assert f(*([cpu] * (COUNTS[name] + 1)), 0, 0) is None
    assert f(*([cpu] * COUNTS[name]), None, None) is None
    assert f(*([cpu] * COUNTS[name]), 0, 1 << 70) is None


def test_bind_takes_all_addresses_or_none():
    n = block.native()
    with pytest.raises(ValueError):
        n.bind((1, 2))
    with pytest.raises(ValueError):
        n.bind([1] * len(block._NATIVE_ORDER))
    with pytest.raises((TypeError, OverflowError)):
        n.bind(("x",) * len(block._NATIVE_ORDER))


def test_order_is_the_structs():
    """block.py hands the addresses over in the order of struct Library."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(block.__file__), "csrc", "binding.cpp")).read()
    body = src[src.index("struct Library {"):src.index("} lib;")]
    assert tuple(re.findall(r"decltype\(&(mx_\w+)\)", body)) == block._NATIVE_ORDER


def test_wrong_arguments_raise_as_in_python():
    import torch
    cpu = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(cpu, cpu[0], mxg.FMT_E4M3)
    with pytest.raises(TypeError):
        mxg.mx_swiglu_quantize([1.0], mxg.FMT_E4M3)
    with pytest.raises(ValueError):
        mxg.mx_gemm_bf16_fused(cpu.bfloat16(), cpu.bfloat16())
