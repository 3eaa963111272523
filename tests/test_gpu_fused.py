"""GPU tests of the products with a fused epilogue, C = residual +
act(A * B^T + bias), on every kernel a plan can choose (decode, tiles, split-K).

With nothing to fuse and no K split the result is mx_gemm's, bit for bit, on
the same kernel or another tile.  Otherwise it is held to the 64-bit result within: the product's own bound (1e-5 T, and the
oracle's term E for 8-bit operands), which an activation's slope (below 1.13)
carries on; 16 units u = 2^-24 of the activation's value and argument; two
units for the sums with bias and residual; half a unit in the last place of
BF16 output."""
import numpy as np
import pytest

import block_ref as ref
import microscaled_block_scaled_amd as mxg
import mxinputs
import oracle
from gpu_util import log

pytestmark = pytest.mark.gpu

U, UBF = ref.U32, ref.UBF
ACT = {"none": mxg.ACT_NONE, "relu": mxg.ACT_RELU, "silu": mxg.ACT_SILU, "gelu": mxg.ACT_GELU,
       "gelu_tanh": mxg.ACT_GELU_TANH}
PAIRS = [(mxg.FMT_E4M3, mxg.FMT_E4M3), (mxg.FMT_E2M1, mxg.FMT_E2M1), (mxg.FMT_E4M3, mxg.FMT_E2M1),
         None]                          # None: BF16
PAIR_IDS = ["e4m3", "e2m1", "w4a8", "bf16"]
# decode (M <= 32, K >= 512), its edges, short tiles, every 256-row tile, and
# split-K: few tiles and a long K
SHAPES = [(1, 64, 512), (8, 1000, 1024), (9, 33, 512), (16, 40, 640), (32, 257, 512),
          (1, 7, 128), (33, 520, 256), (64, 257, 384), (100, 130, 256), (130, 264, 384),
          (300, 1000, 256), (256, 2048, 128), (70, 512, 8192), (200, 130, 4096),
          (520, 2052, 384), (700, 4102, 256), (1030, 4097, 128), (2000, 6144, 128),
          (1500, 7000, 128), (2040, 8100, 128)]


def _torch():
    import torch
    return torch


def _case(pair, M, N, K, seed):
    """Operands on the device and the oracle's (C, T, E)."""
    torch = _torch()
    if pair is None:
        a, b = mxinputs.make_bf16(M, K, seed=seed, tensor=0), mxinputs.make_bf16(N, K, seed=seed, tensor=1)
        C, T = oracle.gemm_bf16(a, b)
        dev = [torch.from_numpy(v.view(np.int16)).cuda().view(torch.bfloat16) for v in (a, b)]
        return dev, C, T, 0.0
    rng = np.random.default_rng(seed)
    qa, sa = oracle.quantize(pair[0], np.float64(np.float32(rng.standard_normal((M, K)))))
    qb, sb = oracle.quantize(pair[1], np.float64(np.float32(rng.standard_normal((N, K)) / np.sqrt(K))))
    eight = mxg.FMT_E4M3 in pair
    if pair[0] == pair[1]:
        out = oracle.gemm(pair[0], qa, sa, qb, sb, K, group_bound=eight)
    else:
        out = oracle.gemm(pair[0], qa, sa, qb, sb, K, group_bound=True, fmt_b=pair[1])
    return ([torch.from_numpy(v).cuda() for v in (qa, sa, qb, sb)], out[0], out[1],
            out[2] if eight else 0.0)


def _fused(pair, dev, **kw):
    if pair is None:
        return mxg.mx_gemm_bf16_fused(dev[0], dev[1], **kw)
    return mxg.mx_gemm_fused(*dev, pair[0], fmt_b=pair[1], **kw)


def _plain(pair, dev, **kw):
    if pair is None:
        return mxg.mx_gemm_bf16(dev[0], dev[1], **kw)
    return mxg.mx_gemm(*dev, pair[0], fmt_b=pair[1], **kw)


def _bound(C, T, E, bias, act, res, bf16):
    pre = C + (0 if bias is None else bias)
    v = ref.act(pre, act)
    out = v + (0 if res is None else res)
    tol = 1.13 * (1e-5 * T + E + 2 * U * (abs(C) + abs(pre))) + 2 * U * (abs(v) + abs(out))
    if act != "none":
        tol = tol + 16 * U * abs(pre)
    return out, tol + (UBF * (abs(out) + tol) if bf16 else 0) + 2.0 ** -126


@pytest.mark.parametrize("pair", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_against_the_oracle(pair, M, N, K):
    torch = _torch()
    dev, C, T, E = _case(pair, M, N, K, seed=M + N)
    rng = np.random.default_rng(K + N)
    bias32 = np.float64(np.float32(rng.standard_normal(N)))
    for out_dtype in (torch.float32, torch.bfloat16):
        bf16 = out_dtype == torch.bfloat16
        res = torch.from_numpy(rng.standard_normal((M, N))).to(out_dtype).cuda()
        resw = torch.zeros((M, N + 3), dtype=out_dtype, device="cuda")     # an odd pitch
        resw[:, :N] = res
        bias = torch.from_numpy(bias32).float().cuda()
        log("fused %s %dx%dx%d %s" % (pair, M, N, K, out_dtype))
        plan = mxg.plan_fused(None if pair is None else pair[0], M, N, K,
                              fmt_b=None if pair is None else pair[1])
        if plan["split_k"] == 1:
            dec = plan["variant"] == mxg.VARIANT_DECODE
            plain = _plain(pair, dev, out_dtype=out_dtype,
                           tile=(32, 32) if dec else (256, 128), split_k=1)
            assert torch.equal(_fused(pair, dev, out_dtype=out_dtype), plain)
        for i, act in enumerate(ref.ACTS):
            b = None if i == 1 else bias.to(torch.bfloat16) if i == 2 else bias
            r = None if i == 3 else resw[:, :N] if i == 4 else res
            got = _fused(pair, dev, bias=b, act=ACT[act], residual=r, out_dtype=out_dtype)
            want, tol = _bound(C, T, E, None if b is None else b.double().cpu().numpy(), act,
                               None if r is None else res.double().cpu().numpy(), bf16)
            err = abs(got.double().cpu().numpy() - want)
            assert (err <= tol).all(), (act, float((err / tol).max()))


@pytest.mark.parametrize("pair", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("M,N,K", [(8, 1000, 1024), (130, 264, 384), (70, 512, 8192), (5, 33, 128)])
def test_residual_in_place(pair, M, N, K):
    """C may be the residual itself."""
    torch = _torch()
    dev, _, _, _ = _case(pair, M, N, K, seed=3)
    for dt in (torch.float32, torch.bfloat16):
        log("fused in place %s %dx%dx%d %s" % (pair, M, N, K, dt))
        h = torch.randn((M, N), device="cuda").to(dt)
        want = _fused(pair, dev, act=mxg.ACT_SILU, residual=h, out_dtype=dt)
        got = _fused(pair, dev, act=mxg.ACT_SILU, residual=h, out=h, out_dtype=dt)
        assert got is h and torch.equal(got, want)


def test_every_kernel_is_reached():
    """The shapes above take every tile, the decode kernel and a split."""
    seen, split = set(), 0
    for pair in PAIRS:
        for M, N, K in SHAPES:
            p = mxg.plan_fused(None if pair is None else pair[0], M, N, K,
                               fmt_b=None if pair is None else pair[1])
            seen.add((p["tile_m"], p["tile_n"]))
            split += p["split_k"] > 1
    log("fused tiles %s, %d split" % (sorted(seen), split))
    assert seen == {(256, 256), (256, 192), (256, 128), (128, 128), (128, 64), (64, 64), (32, 32)}
    assert split


@pytest.mark.parametrize("pair", PAIRS, ids=PAIR_IDS)
def test_without_a_workspace_k_is_not_split(pair):
    """The same call through the C ABI with too small a workspace: unsplit, so
    mx_gemm's unsplit result bit for bit, and nothing written beside C."""
    torch = _torch()
    M, N, K = 70, 512, 8192
    dev, _, _, _ = _case(pair, M, N, K, seed=9)
    plan = mxg.plan_fused(None if pair is None else pair[0], M, N, K,
                          fmt_b=None if pair is None else pair[1])
    assert plan["split_k"] > 1
    want = _plain(pair, dev, out_dtype=torch.float32, tile=(256, 128), split_k=1)
    ws = torch.full((plan["workspace_bytes"],), 7, dtype=torch.uint8, device="cuda")
    for w, nbytes in ((None, 0), (None, 1 << 40), (ws, plan["workspace_bytes"] - 1)):
        log("fused without workspace %s %s" % (pair, nbytes))
        out = torch.zeros((M, N), device="cuda")
        p = [t.data_ptr() for t in dev]
        tail = [None, 0, mxg.ACT_NONE, None, 0, out.data_ptr(), mxg.OUT_FP32,
                None if w is None else w.data_ptr(), nbytes,
                torch.cuda.current_stream().cuda_stream or None]
        rc = mxg.lib().mx_gemm_bf16_fused(M, N, K, *p, *tail) if pair is None else \
            mxg.lib().mx_gemm_fused(pair[0], pair[1], M, N, K, *p, *tail)
        torch.cuda.synchronize()
        assert rc == mxg.MX_OK and torch.equal(out, want) and (ws == 7).all()


def test_activation_edges():
    """Signed zeros, far tails, NaN and infinities through each activation: a
    product of exact values, so the sums are known."""
    torch = _torch()
    M, N, K = 3, 40, 128
    vals = [0.0, -0.0, 1.0, -1.0, 30.0, -30.0, 200.0, -200.0, 3e38, -3e38, np.inf, -np.inf, np.nan]
    bias = torch.zeros(N, device="cuda")
    bias[:len(vals)] = torch.tensor(vals)
    a = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    b = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    v = np.array(vals)
    for name in ref.ACTS:
        log("fused activation edges %s" % name)
        got = mxg.mx_gemm_bf16_fused(a, b, bias=bias, act=ACT[name], out_dtype=torch.float32)
        got = got.cpu().numpy().astype(np.float64)[:, :len(vals)]
        assert (np.isnan(got[:, -1])).all()
        with np.errstate(all="ignore"):
            want = ref.act(v[:-1].copy(), name)
        if name not in ("none", "relu"):           # -inf * 0: not a number
            assert np.isnan(got[:, 11]).all()
            want, got = np.delete(want, 11), np.delete(got, 11, axis=1)
        ok = (got[:, :len(want)] == want) | (abs(got[:, :len(want)] - want) <= 16 * U * abs(want) + 1e-9)
        assert ok.all(), (name, got[0], want)


def test_full_size_rows():
    """The 70B down projection over 2048 tokens: sampled rows."""
    torch = _torch()
    M, N, K = 2048, 8192, 28672
    log("fused full size %dx%dx%d" % (M, N, K))
    rows = [0, 1, 255, 256, 1000, 2046, 2047]
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    qa, sa = mxg.mx_quantize(torch.randn((M, K), device="cuda", generator=g), mxg.FMT_E2M1)
    qb, sb = mxg.mx_quantize(torch.randn((N, K), device="cuda", generator=g) / K ** 0.5, mxg.FMT_E2M1)
    bias = torch.randn(N, device="cuda", generator=g)
    res = torch.randn((M, N), device="cuda", generator=g).to(torch.bfloat16)
    got = mxg.mx_gemm_fused(qa, sa, qb, sb, mxg.FMT_E2M1, bias=bias, act=mxg.ACT_GELU, residual=res)
    C, T = oracle.gemm(mxg.FMT_E2M1, qa.cpu().numpy(), sa.cpu().numpy(), qb.cpu().numpy(),
                       sb.cpu().numpy(), K, rows=rows)[:2]
    want, tol = _bound(C, T, 0.0, bias.double().cpu().numpy(), "gelu",
                       res[rows].double().cpu().numpy(), True)
    assert (abs(got[rows].double().cpu().numpy() - want) <= tol).all()


def test_graph_replays():
    """A block captured in a graph: norm, decode product, routing, gated
    activation; every replay equals the eager result on the same inputs."""
    torch = _torch()
    log("graph of the block operators")
    x = torch.randn((8, 1024), device="cuda").to(torch.bfloat16)
    r = torch.randn((8, 1024), device="cuda").to(torch.bfloat16)
    w = torch.ones(1024, device="cuda")
    qb, sb = mxg.mx_quantize(torch.randn((2048, 1024), device="cuda"), mxg.FMT_E4M3)
    qk, sk = mxg.mx_quantize(torch.randn((512, 8192), device="cuda"), mxg.FMT_E4M3)
    long, ls = mxg.mx_quantize(torch.randn((70, 8192), device="cuda"), mxg.FMT_E4M3)
    assert mxg.plan_fused(mxg.FMT_E4M3, 70, 512, 8192)["split_k"] > 1
    ids = torch.randint(-1, 4, (8, 2), device="cuda")
    wt = torch.rand((8, 2), device="cuda")

    def block():
        o = mxg.mx_rmsnorm_quantize(x, w, mxg.FMT_E4M3, residual=r)
        plan = mxg.mx_moe_sort(ids, 4)
        xs, ss = mxg.mx_moe_gather(plan, o.q, o.q_scale)
        gu = mxg.mx_gemm_fused(xs, ss, qb, sb, mxg.FMT_E4M3, act=mxg.ACT_NONE)
        q, s = mxg.mx_swiglu_quantize(gu, mxg.FMT_E4M3)
        y = mxg.mx_gemm_fused(q, s, qb[:1024], sb[:1024], mxg.FMT_E4M3)
        split = mxg.mx_gemm_fused(long, ls, qk, sk, mxg.FMT_E4M3, act=mxg.ACT_GELU)
        return mxg.mx_moe_combine(plan, y, wt, residual=o.h), q, s, plan.row_of, split

    block()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = block()
    for i in range(4):
        x.copy_(torch.randn((8, 1024), device="cuda").to(torch.bfloat16))
        long.copy_(mxg.mx_quantize(torch.randn((70, 8192), device="cuda"), mxg.FMT_E4M3)[0])
        ids.copy_(torch.randint(-1, 4, (8, 2), device="cuda"))
        want = [t.clone() for t in block()]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        live = want[3].view(-1) >= 0
        n = int(live.sum())
        for got, ref_t in zip(out, want):
            if got.shape[0] == 16 and got.dim() == 2 and got.dtype == torch.uint8:
                got, ref_t = got[:n], ref_t[:n]
            assert torch.equal(got, ref_t), i


def test_refusals():
    torch = _torch()
    log("fused refusals")
    q, s = mxg.mx_quantize(torch.randn((32, 128), device="cuda"), mxg.FMT_E4M3)
    a = torch.zeros((32, 128), dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: mxg.mx_gemm_fused(q, s, q, s, mxg.FMT_E5M2),
                lambda: mxg.mx_gemm_fused(q, s, q, s, mxg.FMT_E4M3, fmt_b=mxg.FMT_E5M2),
                lambda: mxg.mx_gemm_fused(q, s, q, s, mxg.FMT_E4M3, act=7),
                lambda: mxg.mx_gemm_fused(q, s, q, s, mxg.FMT_E4M3, act=-1),
                lambda: mxg.mx_gemm_fused(q, s, q, s, mxg.FMT_E4M3, bias=a[0, :31]),
                lambda: mxg.mx_gemm_fused(q, s, q, s, mxg.FMT_E4M3, bias=a[0, :32].half()),
                lambda: mxg.mx_gemm_fused(q, s, q, s, mxg.FMT_E4M3, residual=a[:, :31]),
                lambda: mxg.mx_gemm_fused(q, s, q, s, mxg.FMT_E4M3, residual=a[:, :32].float()),
                lambda: mxg.mx_gemm_fused(q, s, q, s, mxg.FMT_E4M3, residual=a[:, 1:33]),
                lambda: mxg.mx_gemm_fused(q, s[:, :2], q, s, mxg.FMT_E4M3),
                lambda: mxg.mx_gemm_bf16_fused(a, a[:, :64].contiguous()),
                lambda: mxg.mx_gemm_bf16_fused(a, a, out_dtype=torch.float16),
                lambda: mxg.mx_gemm_bf16_fused(a, a, out=a)):
        with pytest.raises(ValueError):
            bad()
