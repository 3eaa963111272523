"""GPU tests of the arithmetic's far ends: the norm's reciprocal root, and the
sigmoid where it is below FP32's normal range while its products are not.

Tolerances in u = 2^-24.
* rstd: with an exact mean and eps 0 its only error is its own rounding, half
  a unit in the last place; the correction's own error is below 2^-20 of one.
* sigmoid's tail: exp2 2 u, its argument 2 u, three products 1 u each: 7 u;
  the gradient's two products more 9 u, and 1 + gate 1 u: 10 u.  The tests
  take 10 u and 12 u.
* a fused epilogue's SiLU the same, 16 u like its other tests, and half the
  spacing 2^-149 of the subnormals.
* GELU's tanh form: its argument w has a relative error of at most 6 u
  (constants and products), which is 6 u |w| of the result."""
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


def _tail():
    """Gates from where the sigmoid leaves FP32's normal range, one per block
    of 32, with ups that bring the product back into it."""
    rng = np.random.default_rng(1)
    g = np.concatenate([np.arange(-80.0, -104.5, -0.5), np.arange(-105.0, -171.0, -3.0),
                        [-87.0, -87.25, -87.3125, -87.375, -88.0, -88.75]])
    up = 2.0 ** np.minimum(np.round(-g / np.log(2) - 20), 126)
    g, up = np.repeat(g, 32), np.repeat(up, 32) * (1 + rng.random(32 * len(g)))
    up *= np.where(rng.random(len(up)) < 0.5, -1, 1)
    return g, up


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_gated_activation_in_the_tail(dtype):
    g, up = _tail()
    gu = _dev(np.concatenate([g, up])[None].repeat(3, 0), dtype)
    gu[1, 5::7] = 0.5                                       # ordinary gates among them
    y = ref.swiglu(_h64(gu))
    assert (abs(y) > 2.0 ** -120).all()
    for fmt in (mxg.FMT_E4M3, mxg.FMT_E5M2, mxg.FMT_E2M1, mxg.FMT_E2M3, mxg.FMT_E3M2):
        log("gated activation's tail %s fmt %d" % (dtype, fmt))
        q, s = (t.cpu().numpy() for t in mxg.mx_swiglu_quantize(gu, fmt))
        (ql, sl), (qh, sh) = (oracle.quantize(fmt, y * (1 + d)) for d in (-10 * U, 10 * U))
        assert ((s == sl) | (s == sh)).all()
        # blocks on which both ends agree leave no choice
        n = s.shape[1]
        sure = (sl == sh) & (ql.reshape(3, n, -1) == qh.reshape(3, n, -1)).all(-1)
        assert sure.mean() > 0.9
        assert (q.reshape(3, n, -1) == ql.reshape(3, n, -1))[sure].all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_gated_activation_gradient_in_the_tail(dtype):
    log("gated activation's gradient in the tail, %s" % dtype)
    g, up = _tail()
    gu = _dev(np.concatenate([g, up])[None].repeat(2, 0), dtype)
    dy = _dev(1 + np.random.default_rng(2).random((2, len(g))), dtype)
    got = _h64(mxg.mx_swiglu_backward(dy, gu))
    want = ref.swiglu_grad(_h64(dy), _h64(gu))
    half = ref.UBF if dtype == "bfloat16" else U
    spacing = 2.0 ** -133 if dtype == "bfloat16" else 2.0 ** -149
    assert (abs(got - want) <= (12 * U + half) * abs(want) + spacing).all()
    assert (abs(got[:, :len(g)]) > 2.0 ** -120).all()       # d_gate is far from underflow


def test_gated_activation_gradient_in_place():
    """dGU may be GU itself, also where a wave writes its values twice."""
    import torch
    log("gated activation's gradient in place")
    g, up = _tail()
    gu = _dev(np.concatenate([g, up])[None].repeat(3, 0))
    gu[1:, 3::5] = 0.25
    dy = _dev(np.random.default_rng(3).random((3, len(g))))
    want = mxg.mx_swiglu_backward(dy, gu)
    rc = mxg.lib().mx_swiglu_backward(mxg.IN_FP32, 3, len(g), dy.data_ptr(), len(g), gu.data_ptr(),
                                      2 * len(g), gu.data_ptr(),
                                      torch.cuda.current_stream().cuda_stream or None)
    torch.cuda.synchronize()
    assert rc == mxg.MX_OK and torch.equal(gu, want)


@pytest.mark.parametrize("M", [3, 70])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_epilogue_in_the_tail(act, M):
    """Products of zeros, so the epilogue's argument is the bias: single
    values, whole tiles and split sums."""
    import torch
    v = np.arange(-80.0, -103.0, -0.125) if act == "silu" else np.arange(-9.5, -10.7, -0.01)
    v = np.float64(np.float32(v))
    want = ref.act(v, act) if act == "silu" else None
    if act == "gelu_tanh":
        w = 2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)
        want = v * ref.sigmoid(w)
        tol = (16 + 6 * abs(w)) * U * abs(want)
    else:
        tol = 16 * U * abs(want)
    code = {"silu": mxg.ACT_SILU, "gelu_tanh": mxg.ACT_GELU_TANH}[act]
    for K, N in ((128, len(v)), (1024, len(v)), (8192, len(v))):
        log("fused %s tail %dx%dx%d" % (act, M, N, K))
        bias = _dev(v)
        a = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
        b = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
        qa, sa = mxg.mx_quantize(a.float(), mxg.FMT_E4M3)
        qb, sb = mxg.mx_quantize(b.float(), mxg.FMT_E4M3)
        for got in (mxg.mx_gemm_bf16_fused(a, b, bias=bias, act=code, out_dtype=torch.float32),
                    mxg.mx_gemm_fused(qa, sa, qb, sb, mxg.FMT_E4M3, bias=bias, act=code,
                                      out_dtype=torch.float32)):
            assert (abs(_h64(got) - want) <= tol + 2.0 ** -149).all(), (K, N)


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
