"""The compiled half of the binding and the Python one give the same results:
naming the current stream takes the Python path."""
import pytest

import microscaled_block_scaled_amd as mxg
from microscaled_block_scaled_amd import block
from gpu_util import log

pytestmark = pytest.mark.gpu


def _same(a, b):
    import torch
    if a is None or b is None:
        return a is b
    if isinstance(a, (tuple, list)):
        return len(a) == len(b) and all(_same(x, y) for x, y in zip(a, b))
    return a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride() and torch.equal(a, b)


def _cases():
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, device="cuda", generator=g).to(dtype)

    x, r, big = rand(6, 128), rand(6, 128), rand(6, 400)
    gub = rand(72, 256)
    w = rand(128, dtype=torch.float32)
    rstd = mxg.mx_rmsnorm_quantize(x, w, None, need_y=True, need_rstd=True).rstd
    gu = rand(6, 256)
    ids = torch.randint(-1, 4, (6, 2), device="cuda", generator=g)
    plan = mxg.mx_moe_sort(ids, 4)
    y, wt = rand(12, 128), rand(6, 2, dtype=torch.float32)
    qa, sa = mxg.mx_quantize(rand(6, 512), mxg.FMT_E4M3)
    qb, sb = mxg.mx_quantize(rand(72, 512), mxg.FMT_E2M1)
    q8, s8 = mxg.mx_quantize(rand(72, 512), mxg.FMT_E4M3)
    xq, xs = mxg.mx_quantize(x, mxg.FMT_E2M3)
    bias, res = rand(72), rand(6, 72)
    for fmt in (None, 1, 2, 3, 4, 5):
        for kw in (dict(), dict(residual=r), dict(residual=big[:, 136:264]),
                   dict(need_rstd=True, residual=r)):
            yield "rmsnorm_quantize", lambda s, fmt=fmt, kw=kw: mxg.mx_rmsnorm_quantize(
                x, w, fmt, need_y=True, eps=1e-5, stream=s, **kw)
    yield "rmsnorm_backward", lambda s: mxg.mx_rmsnorm_backward(r, x, rstd, w, dh=r, stream=s)
    yield "rmsnorm_backward", lambda s: mxg.mx_rmsnorm_backward(r, x, rstd, w, need_dw=False, stream=s)
    for fmt in (1, 2, 3, 4, 5):
        yield "swiglu_quantize", lambda s, fmt=fmt: mxg.mx_swiglu_quantize(gu, fmt, stream=s)
        yield "swiglu_quantize", lambda s, fmt=fmt: mxg.mx_swiglu_quantize(big[:, 8:264], fmt, stream=s)
    yield "swiglu_backward", lambda s: mxg.mx_swiglu_backward(x, gu, stream=s)
    for dt in (torch.int32, torch.int64):
        yield "moe_sort", lambda s, dt=dt: mxg.mx_moe_sort(ids.to(dt), 4, stream=s)
    yield "moe_gather", lambda s: mxg.mx_moe_gather(plan, x, stream=s)
    yield "moe_gather", lambda s: mxg.mx_moe_gather(plan, xq, xs, stream=s)
    for kw in (dict(), dict(weights=wt), dict(weights=wt, residual=x)):
        yield "moe_combine", lambda s, kw=kw: mxg.mx_moe_combine(plan, y, stream=s, **kw)
    yield "moe_combine_backward", lambda s: mxg.mx_moe_combine_backward(plan, x, y, wt, stream=s)
    for kw in (dict(), dict(bias=bias, act=mxg.ACT_SILU), dict(residual=res, out_dtype=torch.bfloat16),
               dict(out_dtype=torch.float32, bias=bias.float())):
        yield "gemm_fused", lambda s, kw=kw: mxg.mx_gemm_fused(qa, sa, qb, sb, 2, fmt_b=1, stream=s, **kw)
        yield "gemm_fused", lambda s, kw=kw: mxg.mx_gemm_fused(qa, sa, q8, s8, 2, stream=s, **kw)
        yield "gemm_bf16_fused", lambda s, kw=kw: mxg.mx_gemm_bf16_fused(gu, gub, stream=s, **kw)
    out = torch.empty((6, 72), dtype=torch.bfloat16, device="cuda")
    yield "gemm_fused", lambda s: mxg.mx_gemm_fused(qa, sa, q8, s8, 2, residual=res, out=out, stream=s).clone()


def test_both_paths_agree(monkeypatch):
    import torch
    here = torch.cuda.current_stream().cuda_stream
    taken = []
    fast = block._fast

    def spy(name, stream, *args):
        r = fast(name, stream, *args)
        taken.append((name, stream is None, r is not None))
        return r

    monkeypatch.setattr(block, "_fast", spy)
    cases = list(_cases())
    assert {n for n, _ in cases} == {"rmsnorm_quantize", "rmsnorm_backward", "swiglu_quantize",
                                     "swiglu_backward", "moe_sort", "moe_gather", "moe_combine",
                                     "moe_combine_backward", "gemm_fused", "gemm_bf16_fused"}
    for i, (name, call) in enumerate(cases):
        log("native %d: %s" % (i, name))
        taken.clear()
        a = call(None)
        b = call(here)
        assert taken == [(name, True, True), (name, False, False)]
        assert _same(a, b), name


def test_refusals_of_the_library_raise():
    import torch
    x = torch.zeros((4, 48), device="cuda")              # not whole scale blocks
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x, x[0], mxg.FMT_E4M3)
    with pytest.raises(ValueError):
        mxg.mx_moe_sort(torch.zeros((4, 2), dtype=torch.int64, device="cuda"), 300)
