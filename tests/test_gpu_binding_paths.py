"""The two ways into the operators between the products -- the compiled one on
the current stream, the Python one on a named stream -- refuse the same calls,
and a named stream is the one that a call's allocations belong to."""
import pytest

import microscaled_block_scaled_amd as mxg
from gpu_util import log

pytestmark = pytest.mark.gpu


def _here():
    import torch
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("path", ["compiled", "python"])
@pytest.mark.parametrize("fmt", [0, -1, 6, 9, 1 << 32, (1 << 32) + 1])
def test_what_is_no_format_is_refused(fmt, path):
    import torch
    log("format %d, %s path" % (fmt, path))
    s = None if path == "compiled" else _here()
    x, w = torch.ones((4, 64), device="cuda"), torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x, w, fmt, need_y=True, stream=s)
    with pytest.raises(ValueError):
        mxg.mx_swiglu_quantize(x, fmt, stream=s)
    q, qs = mxg.mx_quantize(torch.ones((4, 128), device="cuda"), mxg.FMT_E4M3)
    with pytest.raises(ValueError):
        mxg.mx_gemm_fused(q, qs, q, qs, fmt, stream=s)
    with pytest.raises(ValueError):
        mxg.mx_gemm_fused(q, qs, q, qs, mxg.FMT_E4M3, fmt_b=fmt, stream=s)


@pytest.mark.parametrize("path", ["compiled", "python"])
@pytest.mark.parametrize("act", [-1, 5, 1 << 32, (1 << 32) + 1, -(1 << 32)])
def test_what_is_no_activation_is_refused(act, path):
    import torch
    log("activation %d, %s path" % (act, path))
    s = None if path == "compiled" else _here()
    q, qs = mxg.mx_quantize(torch.ones((4, 128), device="cuda"), mxg.FMT_E4M3)
    a = torch.ones((4, 128), device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mxg.mx_gemm_fused(q, qs, q, qs, mxg.FMT_E4M3, act=act, stream=s)
    with pytest.raises(ValueError):
        mxg.mx_gemm_bf16_fused(a, a, act=act, stream=s)


class _NoTruth:
    def __bool__(self):
        raise LookupError("neither true nor false")


@pytest.mark.parametrize("path", ["compiled", "python"])
def test_a_flag_without_truth_raises_its_own_error(path):
    import torch
    log("flags without truth, %s path" % path)
    s = None if path == "compiled" else _here()
    x, w = torch.ones((4, 64), device="cuda"), torch.ones(64, device="cuda")
    for kw in (dict(need_y=_NoTruth()), dict(need_y=True, need_rstd=_NoTruth())):
        with pytest.raises(LookupError):
            mxg.mx_rmsnorm_quantize(x, w, mxg.FMT_E4M3, stream=s, **kw)
    with pytest.raises(LookupError):
        mxg.mx_rmsnorm_backward(x, x, torch.ones(4, device="cuda"), w, need_dw=_NoTruth(), stream=s)


def test_the_default_stream_by_its_handle(monkeypatch):
    """stream=0 from inside another stream: outputs are allocated for the
    default stream, on which the call runs, and not for some third one."""
    import torch
    log("the default stream by its handle")
    x, w = torch.randn((4, 64), device="cuda"), torch.ones(64, device="cuda")
    want = mxg.mx_rmsnorm_quantize(x, w, mxg.FMT_E4M3)
    torch.cuda.synchronize()
    entered = []
    enter = torch.cuda.stream

    def spy(s):
        entered.append(s.cuda_stream)
        return enter(s)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        monkeypatch.setattr(torch.cuda, "stream", spy)
        got = mxg.mx_rmsnorm_quantize(x, w, mxg.FMT_E4M3, stream=0)
        monkeypatch.undo()
        assert torch.cuda.current_stream() == side
    torch.cuda.synchronize()
    assert entered == [0]
    assert torch.equal(got.q, want.q) and torch.equal(got.q_scale, want.q_scale)
