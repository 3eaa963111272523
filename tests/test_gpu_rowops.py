"""GPU tests of the row operators: RMS norm with residual and MX output, its
gradient, the gated activation with MX output, and its gradient, against
64-bit references (tests/block_ref.py) and the oracle's quantizer.

Tolerances, in units u = 2^-24 of FP32 rounding:
* norm: a row's sum of squares is at most 64 + 6 + 16 additions of positive
  terms deep (87 u relative with the squares' own rounding), half of that in
  rstd, plus mean, eps, square root and quotient (4 u) and two products: 50 u.
* norm gradient: 90 u of the row sum's terms, plus the outer arithmetic: 100 u
  of the sum of the terms' magnitudes; dw adds its rows one by one per
  workgroup (rows / 256), then by 128 threads over 256 partial rows; for few
  rows one thread in eight of the row's workgroup walks them.
* sigmoid: exp2 and reciprocal of 2 u each, their arguments 2 u, the sum and
  the products 1 u each: 10 u; the gradient's products 16 u of the magnitudes.
* BF16 outputs: half a unit in the last place more."""
import numpy as np
import pytest

import block_ref as ref
import microscaled_block_scaled_amd as mxg
import mxinputs
import oracle
from gpu_util import log

pytestmark = pytest.mark.gpu

U, UBF = ref.U32, ref.UBF
FMTS = [mxg.FMT_E2M1, mxg.FMT_E4M3, mxg.FMT_E5M2, mxg.FMT_E2M3, mxg.FMT_E3M2]
FMT_IDS = ["e2m1", "e4m3", "e5m2", "e2m3", "e3m2"]
DTYPES = ["float32", "bfloat16"]


def _torch():
    import torch
    return torch


def _dev(a, dtype="float32"):
    torch = _torch()
    return torch.from_numpy(np.asarray(a, np.float32)).to(getattr(torch, dtype)).cuda()


def _h64(t):
    return t.double().cpu().numpy()


def _decode(fmt, q, s):
    """MX bytes -> float64 values (finite scales)."""
    q = q.cpu().numpy()
    if fmt == mxg.FMT_E2M1:
        codes = np.stack([q & 15, q >> 4], -1).reshape(len(q), -1)
        v = np.concatenate([oracle.tables()[0][:8], -oracle.tables()[0][:8]])[codes]
    elif fmt in (mxg.FMT_E2M3, mxg.FMT_E3M2):
        bits = np.unpackbits(q, axis=1, bitorder="little").reshape(len(q), -1, 6)
        codes = (bits << np.arange(6, dtype=np.uint8)).sum(-1)
        m = np.asarray(mxinputs._fp6_magnitudes(fmt), np.float64)
        v = np.concatenate([m, -m])[codes]
    else:
        torch = _torch()
        dt = torch.float8_e4m3fn if fmt == mxg.FMT_E4M3 else torch.float8_e5m2
        v = torch.from_numpy(q).view(dt).double().numpy()
    return v * np.repeat(2.0 ** (s.cpu().numpy().astype(np.float64) - 127), 32, 1)


# widths of every workgroup shape, its smallest and its largest row
SHAPES = [(1, 32), (3, 96), (5, 512), (4, 544), (2, 2048), (3, 2080), (7, 4096), (2, 5120),
          (3, 8192), (2, 8224), (1, 16384), (2, 16416), (1, 32768), (1, 32800), (2, 65536),
          (600, 32), (520, 1056), (514, 8192)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("rows,width", SHAPES)
def test_norm_f32(rows, width, residual):
    torch = _torch()
    log("norm f32 %dx%d residual=%s" % (rows, width, residual))
    rng = np.random.default_rng(rows * 7 + width)
    x = _dev(rng.standard_normal((rows, width)) * np.exp2(rng.integers(-20, 20, (rows, 1))))
    r = _dev(rng.standard_normal((rows, width))) if residual else None
    w = _dev(rng.standard_normal(width))
    fmt = FMTS[(rows + width // 32) % 5]
    o = mxg.mx_rmsnorm_quantize(x, w, fmt, residual=r, eps=1e-5, need_y=True, need_rstd=True)
    torch.cuda.synchronize()
    h = x if r is None else x + r
    assert torch.equal(o.h, h)
    y, rstd = ref.norm(_h64(h), _h64(w), np.float64(np.float32(1e-5)))
    assert (abs(_h64(o.rstd) - rstd) <= 50 * U * rstd).all()
    assert (abs(_h64(o.y) - y) <= 50 * U * abs(y) + 2.0 ** -149).all()
    for f in FMTS:                       # every format quantizes the very y that was returned
        p = mxg.mx_rmsnorm_quantize(x, w, f, residual=r, eps=1e-5)
        rq, rs = oracle.quantize(f, _h64(o.y))
        assert (p.q.cpu().numpy() == rq).all() and (p.q_scale.cpu().numpy() == rs).all(), f
    assert torch.equal(o.q, mxg.mx_rmsnorm_quantize(x, w, fmt, residual=r, eps=1e-5).q)


@pytest.mark.parametrize("fmt", FMTS, ids=FMT_IDS)
@pytest.mark.parametrize("rows,width", [(1, 8192), (33, 5120), (5, 16416), (130, 288)])
def test_norm_bf16_is_the_f32_norm_of_the_same_values(rows, width, fmt):
    torch = _torch()
    log("norm bf16 %dx%d fmt %d" % (rows, width, fmt))
    rng = np.random.default_rng(width + fmt)
    x = _dev(rng.standard_normal((rows, width)), "bfloat16")
    r = _dev(rng.standard_normal((rows, width)) * 3, "bfloat16")
    for wt in DTYPES:
        w = _dev(rng.standard_normal(width), wt)
        o = mxg.mx_rmsnorm_quantize(x, w, fmt, residual=r, need_y=True, need_rstd=True)
        h = (x.float() + r.float()).to(torch.bfloat16)
        p = mxg.mx_rmsnorm_quantize(h.float(), w.float(), fmt, need_y=True, need_rstd=True)
        torch.cuda.synchronize()
        assert torch.equal(o.h, h)
        assert torch.equal(o.rstd, p.rstd)
        assert torch.equal(o.y, p.y.to(torch.bfloat16))
        assert torch.equal(o.q, p.q) and torch.equal(o.q_scale, p.q_scale)


@pytest.mark.parametrize("fmt", FMTS, ids=FMT_IDS)
def test_norm_quantizes_edge_values(fmt):
    """Rows of ones with eps 0 have rstd 1, so y is the weights exactly: every
    element value, midpoint and value next to overflow, at block scales from
    the smallest subnormals to the largest finite values, both signs, zeros;
    and overflowing residual sums round to infinities."""
    torch = _torch()
    log("norm edge values fmt %d" % fmt)
    top = {mxg.FMT_E2M1: 6.0, mxg.FMT_E4M3: 448.0, mxg.FMT_E5M2: 57344.0, mxg.FMT_E2M3: 7.5,
           mxg.FMT_E3M2: 28.0}[fmt]
    # every code of the format, in whole rows of bytes
    codes = torch.arange(768, dtype=torch.int64).remainder(256).to(torch.uint8)
    values = {mxg.FMT_E2M1: 64, mxg.FMT_E4M3: 32, mxg.FMT_E5M2: 32}.get(fmt, 128)
    row = {mxg.FMT_E2M1: 32, mxg.FMT_E4M3: 32, mxg.FMT_E5M2: 32}.get(fmt, 96)
    grid = _decode(fmt, codes.view(-1, row), torch.full((768 // row, values // 32), 127,
                                                        dtype=torch.uint8))
    g = np.unique(np.abs(grid[np.isfinite(grid)]))
    mids = (g[1:] + g[:-1]) / 2
    over = top * (1 + np.arange(1, 9) / 32.0)
    vals = np.concatenate([g, mids, mids * (1 + 2.0 ** -22), mids * (1 - 2.0 ** -22), over, [0.0]])
    vals = np.concatenate([vals, -vals])
    vals = np.concatenate([vals, np.zeros(-len(vals) % 31)]).reshape(-1, 31)
    rows = []
    for e in (0, -3, 40, 100, -60, -100, -118, -126, -132, -140, -149):
        block = np.concatenate([np.full((len(vals), 1), top), vals], 1) / top * 2.0 ** e
        rows.append(block.reshape(-1))
    w = np.concatenate(rows + [np.zeros(32), np.full(32, 3.0e38), np.full(32, -1e-45)])
    w = w.astype(np.float32)
    for at in range(0, len(w), 65536):
        part = w[at:at + 65536]
        o = mxg.mx_rmsnorm_quantize(torch.ones((2, len(part)), device="cuda"), _dev(part), fmt,
                                    eps=0.0, need_y=True)
        assert (_h64(o.y) == part.astype(np.float64)).all()
        rq, rs = oracle.quantize(fmt, np.stack([part, part]).astype(np.float64))
        assert (o.q_scale.cpu().numpy() == rs).all() and (o.q.cpu().numpy() == rq).all()
    big = torch.tensor([[3.3895313892515355e38] * 32], device="cuda").to(torch.bfloat16)
    more = torch.full_like(big, 6.7e35)
    o = mxg.mx_rmsnorm_quantize(big, torch.ones(32, device="cuda"), fmt, residual=more)
    want = (big.float() + more.float()).to(torch.bfloat16)
    assert torch.isinf(want).all() and torch.equal(o.h, want)


def test_norm_pitches_streams_and_single_outputs():
    torch = _torch()
    log("norm pitches")
    rng = np.random.default_rng(5)
    big = _dev(rng.standard_normal((9, 1024)), "bfloat16")
    w = _dev(rng.standard_normal(512))
    x, r = big[:, :512], big[::3, 512:][:3]
    want = mxg.mx_rmsnorm_quantize(x[:3].contiguous(), w, mxg.FMT_E4M3, residual=r.contiguous())
    got = mxg.mx_rmsnorm_quantize(x[:3], w, mxg.FMT_E4M3, residual=r)
    only_y = mxg.mx_rmsnorm_quantize(x[:3], w, None, residual=r, need_y=True)
    assert only_y.q is None and only_y.q_scale is None
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    on = mxg.mx_rmsnorm_quantize(x[:3], w, mxg.FMT_E4M3, residual=r, stream=st.cuda_stream)
    st.synchronize()
    for o in (got, on):
        assert torch.equal(o.q, want.q) and torch.equal(o.h, want.h)
        assert torch.equal(o.q_scale, want.q_scale)
    assert torch.equal(only_y.h, want.h)
    empty = mxg.mx_rmsnorm_quantize(x[:0], w, mxg.FMT_E4M3, need_y=True, need_rstd=True)
    assert empty.q.shape == (0, 512) and empty.q_scale.shape == (0, 16) and empty.y.shape == (0, 512)


def test_norm_non_finite_and_zero_rows():
    """Rows are alone: a NaN or an infinity marks its own row's blocks (scale
    255, zero codes), a zero row with eps is zeros, without eps not a number."""
    torch = _torch()
    log("norm non-finite rows")
    x = np.ones((5, 128))
    x[1, 3], x[2, 70], x[3] = np.nan, np.inf, 0.0
    for dt in DTYPES:
        o = mxg.mx_rmsnorm_quantize(_dev(x, dt), _dev(np.ones(128)), mxg.FMT_E4M3, eps=1e-6,
                                    need_y=True)
        z = mxg.mx_rmsnorm_quantize(_dev(x, dt), _dev(np.ones(128)), mxg.FMT_E4M3, eps=0.0)
        s = o.q_scale.cpu().numpy()
        # an infinity makes rstd 0: only its own value is 0 * inf
        assert (s[1] == 255).all() and list(s[2]) == [0, 0, 255, 0] and (s[3] == 0).all()
        assert (s[0] == s[4]).all() and (s[0] < 255).all()
        assert (o.q.cpu().numpy()[[1, 2, 3]] == 0).all()
        assert torch.isnan(o.y[1]).all() and torch.isnan(o.y[2, 70]) and (o.y[3] == 0).all()
        assert (z.q_scale.cpu().numpy()[3] == 255).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,width", [(1, 32), (3, 96), (512, 32), (513, 32), (1500, 64),
                                        (600, 2080), (33, 5120), (5, 8192), (511, 8192), (9, 8224),
                                        (3, 16416), (2, 65536)])
def test_norm_gradient(rows, width, dtype):
    torch = _torch()
    log("norm gradient %dx%d %s" % (rows, width, dtype))
    rng = np.random.default_rng(rows + width)
    h, dy, dh = (_dev(rng.standard_normal((rows, width)), dtype) for _ in range(3))
    w = _dev(rng.standard_normal(width), DTYPES[(rows + width) % 2])
    eps = 1e-5
    rstd = mxg.mx_rmsnorm_quantize(h, w, mxg.FMT_E4M3, eps=eps, need_rstd=True).rstd
    dx, dw = mxg.mx_rmsnorm_backward(dy, h, rstd, w, dh=dh)
    dx0, none = mxg.mx_rmsnorm_backward(dy, h, rstd, w, need_dw=False)
    again = mxg.mx_rmsnorm_backward(dy, h, rstd, w, dh=dh)
    torch.cuda.synchronize()
    assert none is None and torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    half = UBF if dtype == "bfloat16" else U
    for got, extra in ((dx, _h64(dh)), (dx0, None)):
        want, want_dw, mag, mag_dw = ref.norm_grad(_h64(dy), _h64(h), _h64(w), eps, extra)
        # rstd is itself 50 u off, and appears up to three times in a term
        assert (abs(_h64(got) - want) <= 250 * U * mag + half * abs(want)).all()
    if rows <= 512 and width <= 8192:              # one launch: threads / 8 down the rows
        depth = rows / (-(-width // 512) * 8) + 8 + 55
    else:
        depth = rows / 256 + 1 + 16 + 32 + 55
    assert (abs(_h64(dw) - want_dw) <= depth * U * mag_dw).all()


def test_norm_gradient_matches_differences():
    """A step of the rows along a direction changes the loss by the gradient."""
    log("norm gradient differences")
    rng = np.random.default_rng(8)
    h, dy, v = (rng.standard_normal((4, 256)) for _ in range(3))
    w = rng.standard_normal(256)
    h, dy, w = (np.float64(np.float32(a)) for a in (h, dy, w))
    hd = _dev(h)
    rstd = mxg.mx_rmsnorm_quantize(hd, _dev(w), mxg.FMT_E4M3, eps=1e-5, need_rstd=True).rstd
    dx, _ = mxg.mx_rmsnorm_backward(_dev(dy), hd, rstd, _dev(w))
    e = 1e-5
    f = [(ref.norm(h + t * v, w, 1e-5)[0] * dy).sum() for t in (e, -e)]
    _, _, mag, _ = ref.norm_grad(dy, h, w, 1e-5)
    assert abs((_h64(dx) * v).sum() - (f[0] - f[1]) / (2 * e)) <= 250 * U * (mag * abs(v)).sum() + 1e-7


def test_norm_gradient_zero_rows_and_pitches():
    torch = _torch()
    log("norm gradient zero rows, pitches")
    rng = np.random.default_rng(9)
    big = _dev(rng.standard_normal((6, 3 * 96)))
    dy, h, dh = big[:, :96], big[:, 96:192], big[:, 192:]
    w = _dev(rng.standard_normal(96))
    rstd = _dev(rng.random(6) + 0.5)
    got = mxg.mx_rmsnorm_backward(dy, h, rstd, w, dh=dh)
    want = mxg.mx_rmsnorm_backward(dy.contiguous(), h.contiguous(), rstd, w, dh=dh.contiguous())
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dx, dw = mxg.mx_rmsnorm_backward(dy[:0], h[:0], rstd[:0], w)
    assert dx.shape == (0, 96) and (dw == 0).all()


GLU_SHAPES = [(1, 32), (3, 96), (2, 2048), (5, 2080), (3, 14336), (2, 28672), (70, 1056)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,width", GLU_SHAPES)
def test_swiglu(rows, width, dtype):
    """The bytes lie between those of the exact result times 1 -+ 10 u."""
    torch = _torch()
    rng = np.random.default_rng(rows * 3 + width)
    gu = _dev(rng.standard_normal((rows, 2 * width)) * np.exp2(rng.integers(-6, 6, (rows, 1))), dtype)
    y = ref.swiglu(_h64(gu))
    for fmt in FMTS:
        log("swiglu %dx%d %s fmt %d" % (rows, width, dtype, fmt))
        q, s = mxg.mx_swiglu_quantize(gu, fmt)
        torch.cuda.synchronize()
        (ql, sl), (qh, sh) = (oracle.quantize(fmt, y * (1 + d)) for d in (-10 * U, 10 * U))
        s_np = s.cpu().numpy()
        assert ((s_np == sl) | (s_np == sh)).all()
        same = np.repeat((sl == sh), 32, 1)
        got = abs(_decode(fmt, q, s))
        lo, hi = (abs(_decode(fmt, torch.from_numpy(a), torch.from_numpy(b)))
                  for a, b in ((ql, sl), (qh, sh)))
        assert (((got >= lo) & (got <= hi)) | ~same).all()
        assert (np.sign(_decode(fmt, q, s)) * np.sign(y) >= 0).all()


def test_swiglu_extremes():
    """Gates far out: sigmoid 0 and 1; NaN and infinities mark their block."""
    torch = _torch()
    log("swiglu extremes")
    g = np.zeros((1, 256))
    u = np.ones((1, 256))
    g[0, :32], u[0, :32] = -200.0, 3e30
    g[0, 32:64] = 3e4
    g[0, 64], g[0, 96], g[0, 128] = np.nan, np.inf, -np.inf
    u[0, 160], u[0, 192] = np.nan, -np.inf
    g[0, 193], g[0, 160:192] = 1.0, 1.0
    gu = _dev(np.concatenate([g, u], 1))
    q, s = mxg.mx_swiglu_quantize(gu, mxg.FMT_E4M3)
    s = s.cpu().numpy()[0]
    assert s[0] == 0 and (q[0, :32] & 0x7f == 0).all()
    assert s[1] == 127 + 14 - 8
    assert (s[2:7] == 255).all() and (q[0, 64:224] == 0).all() and s[7] == 0
    dgu = mxg.mx_swiglu_backward(torch.ones_like(gu[:, :256]), gu)
    d = dgu.cpu().numpy()[0]
    assert (d[:32] == 0).all() and (d[256:288] == 0).all()            # sigmoid 0
    assert (d[32:64] == 1).all() and (d[288:320] == 3e4).all()        # sigmoid 1
    assert np.isnan(d[64]) and np.isnan(d[256 + 64])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,width", GLU_SHAPES)
def test_swiglu_gradient(rows, width, dtype):
    torch = _torch()
    log("swiglu gradient %dx%d %s" % (rows, width, dtype))
    rng = np.random.default_rng(rows + 5 * width)
    gu = _dev(rng.standard_normal((rows, 2 * width)) * 3, dtype)
    dy = _dev(rng.standard_normal((rows, width)), dtype)
    dgu = mxg.mx_swiglu_backward(dy, gu)
    torch.cuda.synchronize()
    d, (g, up) = _h64(dy), np.split(_h64(gu), 2, 1)
    sig = ref.sigmoid(g)
    want = ref.swiglu_grad(d, _h64(gu))
    mag = np.concatenate([abs(d * up) * sig * (1 + abs(g)), abs(d * g) * sig], 1)
    half = UBF if dtype == "bfloat16" else U
    assert (abs(_h64(dgu) - want) <= 16 * U * mag + half * abs(want)).all()


def test_swiglu_pitches_and_zero_rows():
    torch = _torch()
    log("swiglu pitches")
    rng = np.random.default_rng(11)
    big = _dev(rng.standard_normal((7, 400)), "bfloat16")
    gu, dy = big[:, :192], big[:, 200:296]
    q, s = mxg.mx_swiglu_quantize(gu, mxg.FMT_E5M2)
    q1, s1 = mxg.mx_swiglu_quantize(gu.contiguous(), mxg.FMT_E5M2)
    assert torch.equal(q, q1) and torch.equal(s, s1)
    assert torch.equal(mxg.mx_swiglu_backward(dy, gu),
                       mxg.mx_swiglu_backward(dy.contiguous(), gu.contiguous()))
    q, s = mxg.mx_swiglu_quantize(gu[:0], mxg.FMT_E2M1)
    assert q.shape == (0, 48) and s.shape == (0, 3)
    assert mxg.mx_swiglu_backward(dy[:0], gu[:0]).shape == (0, 192)


def test_row_operators_past_32_bit_offsets():
    """Rows whose elements lie past 2^31 (and bytes past 2^32) give what they
    give alone."""
    torch = _torch()
    rows, width = 66000, 32768
    log("row operators past 2^31 elements (%dx%d bf16)" % (rows, width))
    x = torch.empty((rows, width), dtype=torch.bfloat16, device="cuda")
    block = torch.randn((600, width), device="cuda").to(torch.bfloat16)
    for at in range(0, rows, 600):
        x[at:at + 600] = block[:min(600, rows - at)]
    w = torch.ones(width, device="cuda")
    o = mxg.mx_rmsnorm_quantize(x, w, mxg.FMT_E4M3)
    p = mxg.mx_rmsnorm_quantize(block, w, mxg.FMT_E4M3)
    for at in (0, 32400, 65400):
        assert torch.equal(o.q[at:at + 600], p.q) and torch.equal(o.q_scale[at:at + 600], p.q_scale)
    del o
    q, s = mxg.mx_swiglu_quantize(x, mxg.FMT_E2M1)
    q1, s1 = mxg.mx_swiglu_quantize(block, mxg.FMT_E2M1)
    for at in (0, 32400, 65400):
        assert torch.equal(q[at:at + 600], q1) and torch.equal(s[at:at + 600], s1)


def test_refusals():
    torch = _torch()
    log("row operator refusals")
    x = torch.zeros((4, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x, w, 9)
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x.half(), w, mxg.FMT_E4M3)
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x, w[:32], mxg.FMT_E4M3)
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x, w, mxg.FMT_E4M3, residual=x[:2])
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x, w, mxg.FMT_E4M3, residual=x.to(torch.bfloat16))
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x.t(), torch.ones(4, device="cuda"), mxg.FMT_E4M3)
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x[:, :48], torch.ones(48, device="cuda"), mxg.FMT_E4M3)
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x[:, 1:33], torch.ones(32, device="cuda"), mxg.FMT_E4M3)
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x, w, None)
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x, w, mxg.FMT_E4M3, eps=-1.0)
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_quantize(x.cpu(), w, mxg.FMT_E4M3)
    with pytest.raises(TypeError):
        mxg.mx_swiglu_quantize([1.0], mxg.FMT_E4M3)
    with pytest.raises(ValueError):
        mxg.mx_swiglu_quantize(x[:, :32], mxg.FMT_E4M3)           # width 16
    with pytest.raises(ValueError):
        mxg.mx_swiglu_backward(x, x)
    with pytest.raises(ValueError):
        mxg.mx_rmsnorm_backward(x, x, w[:4].double(), w)
