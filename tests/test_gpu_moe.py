"""GPU tests of expert routing: the sort and the gather exactly, the
combination and its gradients against 64-bit references (tests/block_ref.py).

Tolerances in u = 2^-24: the combination adds top products and a residual one
after the other, (top + 2) u of the terms' magnitudes; the weight gradient's
products and sums are width / 512 + 8 + 6 additions deep per lane and over
lanes; BF16 outputs half a unit in the last place more."""
import numpy as np
import pytest

import block_ref as ref
import microscaled_block_scaled_amd as mxg
from gpu_util import log

pytestmark = pytest.mark.gpu

U, UBF = ref.U32, ref.UBF
DTYPES = ["float32", "bfloat16"]


def _torch():
    import torch
    return torch


def _dev(a, dtype="float32"):
    torch = _torch()
    return torch.from_numpy(np.asarray(a, np.float32)).to(getattr(torch, dtype)).cuda()


def _h64(t):
    return t.double().cpu().numpy()


def _ids(tokens, top, experts, seed, drop=0.1):
    rng = np.random.default_rng(seed)
    ids = np.minimum(rng.integers(0, experts, (tokens, top)),
                     rng.integers(0, experts, (tokens, top)))        # uneven experts
    ids[rng.random((tokens, top)) < drop] = -1
    return ids


def _plan(ids, experts, dtype="int64"):
    torch = _torch()
    return mxg.mx_moe_sort(torch.from_numpy(ids).to(getattr(torch, dtype)).cuda(), experts)


def _check_sort(ids, experts, dtype="int64"):
    plan = _plan(ids, experts, dtype)
    rows, row_of = ref.sort(ids, experts)
    assert plan.group_rows.tolist() == rows.tolist()
    assert (plan.row_of.cpu().numpy() == row_of).all()


@pytest.mark.parametrize("dtype", ["int32", "int64"])
@pytest.mark.parametrize("tokens,top,experts", [
    (1, 1, 1), (1, 8, 256), (5, 3, 4), (64, 2, 8), (63, 1, 2), (1000, 8, 255), (1024, 8, 256),
    (4096, 1, 7), (4097, 1, 7), (8193, 1, 7), (4099, 3, 64), (20001, 6, 128), (70000, 8, 256)])
def test_sort(tokens, top, experts, dtype):
    log("sort %dx%d over %d experts, %s" % (tokens, top, experts, dtype))
    _check_sort(_ids(tokens, top, experts, tokens + experts), experts, dtype)


@pytest.mark.parametrize("tokens", [300, 9000])
def test_sort_one_expert_none_and_outside_ids(tokens):
    log("sort of degenerate ids, %d tokens" % tokens)
    _check_sort(np.full((tokens, 2), 3), 5)
    _check_sort(np.full((tokens, 2), -1), 5)
    ids = _ids(tokens, 2, 5, 1)
    ids[::7, 0] = 5
    ids[1::7, 1] = 2 ** 40 + 1
    ids[2::7, 0] = -2 ** 40
    ids[3::7, 0] = 2 ** 32
    _check_sort(ids, 5)
    _check_sort(np.clip(ids, -2 ** 31, 2 ** 31 - 1), 5, "int32")


def test_sort_no_tokens():
    torch = _torch()
    plan = mxg.mx_moe_sort(torch.empty((0, 4), dtype=torch.int64, device="cuda"), 9)
    assert plan.group_rows.tolist() == [0] * 9 and plan.row_of.shape == (0, 4)
    xs, ss = mxg.mx_moe_gather(plan, torch.empty((0, 64), device="cuda"))
    assert xs.shape == (0, 64) and ss is None
    out = mxg.mx_moe_combine(plan, torch.empty((0, 64), device="cuda"))
    assert out.shape == (0, 64)


@pytest.mark.parametrize("tokens,top,width", [(1, 1, 4096), (7, 8, 4096), (64, 2, 4100),
                                              (33, 3, 1), (100, 4, 33), (257, 6, 1040)])
def test_gather_bytes(tokens, top, width):
    torch = _torch()
    log("gather %dx%d rows of %d bytes" % (tokens, top, width))
    ids = _ids(tokens, top, 16, tokens)
    _, row_of = ref.sort(ids, 16)
    plan = _plan(ids, 16)
    rng = np.random.default_rng(width)
    x = rng.integers(0, 256, (tokens, width)).astype(np.uint8)
    sc = rng.integers(0, 256, (tokens, (width + 31) // 32)).astype(np.uint8)
    xd, sd = torch.from_numpy(x).cuda(), torch.from_numpy(sc).cuda()
    xs, ss = mxg.mx_moe_gather(plan, xd, sd)
    assert (xs.cpu().numpy() == ref.gather(row_of, x)).all()
    assert (ss.cpu().numpy() == ref.gather(row_of, sc)).all()
    alone, none = mxg.mx_moe_gather(plan, xd)
    assert none is None and torch.equal(alone, xs)
    wide = torch.zeros((tokens, width + 5), dtype=torch.uint8, device="cuda")
    wide[:, 3:3 + width] = xd                      # another pitch, another alignment
    xs2, ss2 = mxg.mx_moe_gather(plan, wide[:, 3:3 + width], sd)
    assert torch.equal(xs2, xs) and torch.equal(ss2, ss)


def test_gather_keeps_value_types():
    torch = _torch()
    ids = _ids(40, 2, 4, 3)
    _, row_of = ref.sort(ids, 4)
    for dt in (torch.bfloat16, torch.float32, torch.float8_e4m3fn):
        log("gather of %s" % dt)
        x = torch.randn((40, 64), device="cuda").to(dt)
        xs, _ = mxg.mx_moe_gather(_plan(ids, 4), x)
        assert xs.dtype == dt and xs.shape == (80, 64)
        want = ref.gather(row_of, x.float().cpu().numpy())
        assert (xs.float().cpu().numpy() == want).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,top,width", [(1, 1, 8), (3, 2, 4096), (70, 8, 520), (129, 3, 1544),
                                              (500, 64, 64)])
def test_combine(tokens, top, width, dtype):
    torch = _torch()
    log("combine %dx%d width %d %s" % (tokens, top, width, dtype))
    ids = _ids(tokens, top, 8, tokens, drop=0.2)
    ids[-1] = -1                                   # a token without any expert
    rows, row_of = ref.sort(ids, 8)
    plan = _plan(ids, 8)
    rng = np.random.default_rng(width)
    y = _dev(rng.standard_normal((tokens * top, width)), dtype)
    y[int(rows.sum()):] = float("nan")             # rows that nobody may read
    w = rng.standard_normal((tokens, top))
    w[ids < 0] = np.nan
    w, res = _dev(w), _dev(rng.standard_normal((tokens, width)), dtype)
    half = UBF if dtype == "bfloat16" else U
    for weights, residual in ((w, res), (w, None), (None, res), (None, None)):
        want, mag = ref.combine(row_of, _h64(y), None if weights is None else _h64(w),
                                None if residual is None else _h64(res))
        for yy in (y, y[:int(rows.sum())]):        # with and without the rows of no expert
            out = mxg.mx_moe_combine(plan, yy, weights, residual=residual)
            assert (abs(_h64(out) - want) <= (top + 2) * U * mag + half * abs(want)).all()


def test_combine_pitches_and_side_stream():
    torch = _torch()
    log("combine pitches")
    ids = _ids(50, 2, 4, 5)
    plan = _plan(ids, 4)
    big = torch.randn((100, 3 * 64), device="cuda").to(torch.bfloat16)
    y, res = big[:, :64], big[:50, 128:]
    w = torch.rand((50, 2), device="cuda")
    want = mxg.mx_moe_combine(plan, y.contiguous(), w, residual=res.contiguous())
    assert torch.equal(mxg.mx_moe_combine(plan, y, w, residual=res), want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    ids_d = torch.from_numpy(ids).cuda()
    st.wait_stream(torch.cuda.current_stream())
    p2 = mxg.mx_moe_sort(ids_d, 4, stream=st.cuda_stream)
    out = mxg.mx_moe_combine(p2, y, w, residual=res, stream=st.cuda_stream)
    st.synchronize()
    assert torch.equal(p2.row_of, plan.row_of) and torch.equal(out, want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,top,width", [(1, 1, 8), (3, 2, 4096), (70, 8, 520), (129, 3, 1544)])
def test_combine_gradient(tokens, top, width, dtype):
    torch = _torch()
    log("combine gradient %dx%d width %d %s" % (tokens, top, width, dtype))
    ids = _ids(tokens, top, 8, tokens + 1, drop=0.2)
    rows, row_of = ref.sort(ids, 8)
    plan = _plan(ids, 8)
    rng = np.random.default_rng(width + 1)
    y = _dev(rng.standard_normal((tokens * top, width)), dtype)
    y[int(rows.sum()):] = float("nan")
    w = rng.standard_normal((tokens, top))
    w[ids < 0] = np.nan
    w, dout = _dev(w), _dev(rng.standard_normal((tokens, width)), dtype)
    want_dy, want_dw, mag = ref.combine_grad(row_of, _h64(dout), _h64(y), _h64(w))
    half = UBF if dtype == "bfloat16" else U
    for yy in (y, y[:int(rows.sum())]):
        dy, dw = mxg.mx_moe_combine_backward(plan, dout, yy, w)
        assert dy.shape == yy.shape
        assert (abs(_h64(dy) - want_dy[:len(yy)]) <= (U + half) * abs(want_dy[:len(yy)])).all()
        assert (abs(_h64(dw) - want_dw) <= (width / 512 + 8 + 8) * U * mag).all()


def test_combine_gradient_matches_differences():
    """Steps of y and of the weights change the loss by the gradients."""
    log("combine gradient differences")
    ids = _ids(20, 4, 6, 7)
    _, row_of = ref.sort(ids, 6)
    rng = np.random.default_rng(7)
    y, vy = rng.standard_normal((80, 64)), rng.standard_normal((80, 64))
    w, vw = rng.random((20, 4)), rng.standard_normal((20, 4))
    dout = rng.standard_normal((20, 64))
    y, w, dout = (np.float64(np.float32(a)) for a in (y, w, dout))
    dy, dw = mxg.mx_moe_combine_backward(_plan(ids, 6), _dev(dout), _dev(y), _dev(w))
    e = 1e-3
    loss = [(ref.combine(row_of, y + t * vy, w + t * vw)[0] * dout).sum() for t in (e, -e)]
    got = (_h64(dy) * vy).sum() + (_h64(dw) * vw).sum()
    mag = abs(_h64(dy) * vy).sum() + (ref.combine_grad(row_of, dout, y, w)[2] * abs(vw)).sum()
    assert abs(got - (loss[0] - loss[1]) / (2 * e)) <= 16 * U * mag + 1e-9


def test_gather_past_32_bit_offsets():
    torch = _torch()
    tokens, top, width = 36000, 8, 16384
    log("gather into %d rows of %d bytes" % (tokens * top, width))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ids = torch.randint(0, 32, (tokens, top), device="cuda", generator=g)
    x = torch.randint(0, 256, (tokens, width), dtype=torch.uint8, device="cuda", generator=g)
    plan = mxg.mx_moe_sort(ids, 32)
    xs, _ = mxg.mx_moe_gather(plan, x)
    for t in (0, 1, tokens // 2, tokens - 1):
        for j in range(top):
            assert torch.equal(xs[int(plan.row_of[t, j])], x[t])
    rows = plan.row_of.long().view(-1)
    assert torch.equal(xs[rows, 5], x[:, 5].repeat_interleave(top))
    # and the rows past 2^31 elements come back
    out = mxg.mx_moe_combine(plan, xs.view(torch.bfloat16)[:, :64].contiguous())
    assert out.shape == (tokens, 64)
    y = xs.view(torch.bfloat16).view(torch.int16) & 0x3fff        # finite, small values
    y = y.view(torch.bfloat16)
    out = mxg.mx_moe_combine(plan, y)
    at = [0, tokens - 1]
    want = sum(y[rows.view(tokens, top)[at, j]].double() for j in range(top))
    mag = sum(y[rows.view(tokens, top)[at, j]].double().abs() for j in range(top))
    assert ((out[at].double() - want).abs() <= (top + 2) * U * mag + UBF * want.abs()).all()


def test_refusals():
    torch = _torch()
    log("routing refusals")
    ids = torch.zeros((4, 2), dtype=torch.int64, device="cuda")
    plan = mxg.mx_moe_sort(ids, 3)
    x = torch.zeros((4, 64), device="cuda")
    for bad in (lambda: mxg.mx_moe_sort(ids.float(), 3), lambda: mxg.mx_moe_sort(ids, 0),
                lambda: mxg.mx_moe_sort(ids, 257), lambda: mxg.mx_moe_sort(ids[:, :1], 3),
                lambda: mxg.mx_moe_sort(ids.cpu(), 3), lambda: mxg.mx_moe_sort(ids[0], 3),
                lambda: mxg.mx_moe_sort(torch.zeros((2, 65), dtype=torch.int64, device="cuda"), 3),
                lambda: mxg.mx_moe_gather(plan, x[:3]), lambda: mxg.mx_moe_gather(plan, x, x[:3]),
                lambda: mxg.mx_moe_gather(plan, x.t()),
                lambda: mxg.mx_moe_combine(plan, x.half()),
                lambda: mxg.mx_moe_combine(plan, x[:, :12].contiguous()),
                lambda: mxg.mx_moe_combine(plan, x, torch.ones((4, 3), device="cuda")),
                lambda: mxg.mx_moe_combine(plan, x, residual=x[:, :32]),
                lambda: mxg.mx_moe_combine_backward(plan, x, torch.zeros((9, 64), device="cuda"),
                                                    torch.ones((4, 2), device="cuda"))):
        with pytest.raises(ValueError):
            bad()
