"""The C ABI of the row, routing and epilogue operators without a GPU: every
argument check runs before any HIP call, and valid calls end at the missing
device."""
import ctypes
import os
import re

import pytest

import microscaled_block_scaled_amd as mxg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G = 1 << 20                       # a well aligned address that is never read
E = dict(fmt=mxg.MX_ERR_FORMAT, dt=mxg.MX_ERR_IN_DTYPE, shape=mxg.MX_ERR_ROW_SHAPE,
         null=mxg.MX_ERR_NULL, align=mxg.MX_ERR_ALIGN, ws=mxg.MX_ERR_WORKSPACE, ok=mxg.MX_OK)
DEV = (mxg.MX_ERR_NO_DEVICE, mxg.MX_ERR_ARCH)


def _call(name, defaults, over):
    assert set(over) <= set(defaults), over
    args = dict(defaults, **over)
    # no device here: a call that passes every check must not have a real one
    if _has_gpu():
        pytest.skip("a device is present: valid calls would launch on fake addresses")
    return getattr(mxg.lib(), name)(*args.values())


def _has_gpu():
    import torch
    return torch.cuda.is_available()


def _expect(rc, what):
    assert rc in DEV if what == "dev" else rc == E[what], (rc, what)


NORM = dict(fmt=2, dtype=2, w_dtype=1, rows=4, width=64, X=G, ldx=64, R=G, ldr=64, W=G, eps=1e-6,
            H=G, Y=G, Q=G, S=G, rstd=G, stream=None)


@pytest.mark.parametrize("over,what", [
    ({}, "dev"), (dict(fmt=0), "fmt"), (dict(fmt=6), "fmt"), (dict(fmt=0, Q=None, S=None), "dev"),
    (dict(dtype=0), "dt"), (dict(w_dtype=3), "dt"), (dict(rows=-1), "shape"),
    (dict(rows=(1 << 30) + 1), "shape"), (dict(width=48), "shape"), (dict(width=0), "shape"),
    (dict(width=65568, ldx=65568, ldr=65568), "shape"), (dict(ldx=63), "shape"),
    (dict(ldr=32), "shape"), (dict(R=None, ldr=0), "dev"), (dict(eps=-1.0), "shape"),
    (dict(eps=float("nan")), "shape"), (dict(rows=0, X=None, W=None), "ok"), (dict(X=None), "null"),
    (dict(W=None), "null"), (dict(H=None), "null"), (dict(H=None, R=None), "dev"),
    (dict(Q=None, Y=None), "null"), (dict(S=None), "null"), (dict(X=G + 8), "align"),
    (dict(ldx=68), "align"), (dict(ldx=68, dtype=1), "dev"), (dict(ldr=68), "align"),
    (dict(Q=G + 4), "align"), (dict(Y=G + 8), "align"), (dict(rstd=G + 2), "align"),
    (dict(rstd=None), "dev")])
def test_norm(over, what):
    _expect(_call("mx_rmsnorm_quantize", NORM, over), what)


NORM_B = dict(dtype=2, w_dtype=1, rows=4, width=64, dY=G, lddy=64, H=G, ldh=64, rstd=G, W=G, dH=G,
              lddh=64, dX=G, dW=G, ws=G, bytes=1 << 30, stream=None)


@pytest.mark.parametrize("over,what", [
    ({}, "dev"), (dict(dtype=7), "dt"), (dict(w_dtype=0), "dt"), (dict(width=33), "shape"),
    (dict(lddy=10), "shape"), (dict(ldh=10), "shape"), (dict(lddh=10), "shape"),
    (dict(dH=None, lddh=0), "dev"), (dict(rows=9000, bytes=256 * 64 * 4 - 1), "ws"),
    (dict(rows=9000, bytes=256 * 64 * 4), "dev"), (dict(rows=9000, ws=None), "null"),
    (dict(ws=None, bytes=0), "dev"), (dict(rows=9000, ws=None, dW=None, bytes=0), "dev"), (dict(rstd=None), "null"),
    (dict(dX=None), "null"), (dict(rows=0, dW=None, dY=None), "ok"),
    (dict(rows=0, dY=None, H=None, rstd=None, W=None, dX=None, ws=None, bytes=0), "dev"),
    (dict(dY=G + 2), "align"), (dict(ws=G + 4), "align"), (dict(lddy=65), "align")])
def test_norm_backward(over, what):
    _expect(_call("mx_rmsnorm_backward", NORM_B, over), what)


GLU = dict(fmt=2, dtype=2, rows=4, width=64, GU=G, ld=128, Q=G, S=G, stream=None)
GLU_B = dict(dtype=2, rows=4, width=64, dY=G, lddy=64, GU=G, ld=128, dGU=G, stream=None)


@pytest.mark.parametrize("name,base,over,what", [
    ("mx_swiglu_quantize", GLU, o, w) for o, w in (
        ({}, "dev"), (dict(fmt=9), "fmt"), (dict(dtype=3), "dt"), (dict(width=16), "shape"),
        (dict(ld=127), "shape"), (dict(rows=0, GU=None), "ok"), (dict(GU=None), "null"),
        (dict(S=None), "null"), (dict(Q=G + 4), "align"), (dict(ld=132), "align"))] + [
    ("mx_swiglu_backward", GLU_B, o, w) for o, w in (
        ({}, "dev"), (dict(dtype=3), "dt"), (dict(ld=64), "shape"), (dict(lddy=63), "shape"),
        (dict(rows=0, dY=None), "ok"), (dict(dGU=None), "null"), (dict(dGU=G + 8), "align"),
        (dict(lddy=66), "align"))])
def test_swiglu(name, base, over, what):
    _expect(_call(name, base, over), what)


SORT = dict(idb=8, tokens=100, top=2, experts=8, ids=G, rows=G, row_of=G, ws=G, bytes=1 << 20,
            stream=None)


@pytest.mark.parametrize("over,what", [
    ({}, "dev"), (dict(idb=4), "dev"), (dict(idb=2), "dt"), (dict(top=0), "shape"),
    (dict(top=65), "shape"), (dict(experts=0), "shape"), (dict(experts=257), "shape"),
    (dict(tokens=1 << 29, top=4), "shape"), (dict(tokens=-1), "shape"), (dict(rows=None), "null"),
    (dict(ids=None), "null"), (dict(tokens=0, ids=None, row_of=None), "dev"),
    (dict(ws=None, bytes=0), "dev"), (dict(tokens=1 << 20, ws=None), "null"),
    (dict(tokens=1 << 20, bytes=8), "ws"), (dict(ids=G + 4), "align"), (dict(rows=G + 4), "align")])
def test_sort(over, what):
    _expect(_call("mx_moe_sort", SORT, over), what)


GATHER = dict(tokens=10, top=2, row_of=G, X=G, rb=64, ldx=64, XS=G, sb=2, lds=2, out=G, outs=G,
              stream=None)


@pytest.mark.parametrize("over,what", [
    ({}, "dev"), (dict(X=G + 1, rb=3, ldx=5), "dev"), (dict(rb=0), "shape"), (dict(ldx=63), "shape"),
    (dict(lds=1), "shape"), (dict(sb=0), "shape"), (dict(XS=None, sb=0, lds=0, outs=None), "dev"),
    (dict(tokens=0, X=None), "ok"), (dict(out=None), "null"), (dict(outs=None), "null"),
    (dict(row_of=G + 2), "align"), (dict(top=0), "shape"), (dict(top=65), "shape")])
def test_gather(over, what):
    _expect(_call("mx_moe_gather", GATHER, over), what)


COMBINE = dict(dtype=2, tokens=10, top=2, width=64, row_of=G, Y=G, rows=20, ldy=64, w=G, R=G, ldr=64,
               out=G, stream=None)
COMBINE_B = dict(dtype=2, tokens=10, top=2, width=64, row_of=G, dO=G, lddo=64, Y=G, rows=20, ldy=64,
                 w=G, dY=G, dw=G, stream=None)


@pytest.mark.parametrize("name,base,over,what", [
    ("mx_moe_combine", COMBINE, o, w) for o, w in (
        ({}, "dev"), (dict(dtype=0), "dt"), (dict(width=60), "shape"), (dict(ldy=56), "shape"),
        (dict(rows=-1), "shape"), (dict(rows=0, Y=None), "dev"), (dict(Y=None), "null"),
        (dict(w=None, R=None, ldr=0), "dev"), (dict(out=None), "null"), (dict(tokens=0, Y=None), "ok"),
        (dict(Y=G + 8), "align"), (dict(ldy=68), "align"), (dict(ldr=68), "align"))] + [
    ("mx_moe_combine_backward", COMBINE_B, o, w) for o, w in (
        ({}, "dev"), (dict(dtype=0), "dt"), (dict(rows=21), "shape"), (dict(lddo=8), "shape"),
        (dict(rows=0, Y=None, dY=None), "dev"), (dict(w=None), "null"), (dict(dw=None), "null"),
        (dict(dY=G + 8), "align"), (dict(tokens=0), "shape"), (dict(tokens=0, rows=0, Y=None), "ok"))])
def test_combine(name, base, over, what):
    _expect(_call(name, base, over), what)


FUSED = dict(fa=2, fb=1, M=8, N=64, K=512, A=G, As=G, B=G, Bs=G, bias=G, bdt=1, act=2, res=G, ldr=64,
             C=G, out=2, ws=None, bytes=0, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(ws=G, bytes=1 << 30), None), (dict(ws=G + 8), mxg.MX_ERR_ALIGN),
    ({}, None), (dict(fa=1, fb=1), None), (dict(fa=2, fb=2), None), (dict(fa=1, fb=2), mxg.MX_ERR_FORMAT),
    (dict(fa=3, fb=3), mxg.MX_ERR_FORMAT), (dict(fa=0), mxg.MX_ERR_FORMAT),
    (dict(fb=6), mxg.MX_ERR_FORMAT), (dict(out=3), mxg.MX_ERR_OUT_DTYPE), (dict(K=192), mxg.MX_ERR_SHAPE),
    (dict(M=0), mxg.MX_ERR_SHAPE), (dict(act=5), mxg.MX_ERR_ACT), (dict(act=-1), mxg.MX_ERR_ACT),
    (dict(bdt=0), mxg.MX_ERR_IN_DTYPE), (dict(bdt=0, bias=None), None), (dict(ldr=63), mxg.MX_ERR_ROW_SHAPE),
    (dict(ldr=0, res=None), None), (dict(bias=G + 2), mxg.MX_ERR_ALIGN), (dict(bias=G + 2, bdt=2), None),
    (dict(res=G + 2), mxg.MX_ERR_ALIGN), (dict(A=None), mxg.MX_ERR_NULL), (dict(Bs=None), mxg.MX_ERR_NULL)])
def test_fused(over, code):
    rc = _call("mx_gemm_fused", FUSED, over)
    assert rc in DEV if code is None else rc == code, rc
    bf = {k: v for k, v in FUSED.items() if k not in ("fa", "fb", "As", "Bs")}
    over = {k: v for k, v in over.items() if k in bf}
    if code in (mxg.MX_ERR_ACT, mxg.MX_ERR_IN_DTYPE, mxg.MX_ERR_ROW_SHAPE, mxg.MX_ERR_ALIGN):
        assert _call("mx_gemm_bf16_fused", bf, over) == code


def test_fused_plans():
    """Every plan is a kernel that is compiled, covers C, and splits K into at
    most MAX_SPLIT_K slices with planes for each; huge problems are refused."""
    tiles = {(256, 256): 512, (256, 192): 512, (256, 128): 512, (128, 128): 512, (128, 64): 256,
             (64, 64): 256}
    for fmt, fmt_b in ((1, 1), (2, 2), (2, 1), (None, None)):
        for M in (1, 31, 33, 64, 65, 300, 2048, 100000, 1 << 30):
            for N in (1, 64, 1000, 8192, 1 << 20):
                for K in (128, 512, 640, 4096, 28672, 1 << 20):
                    try:
                        p = mxg.plan_fused(fmt, M, N, K, fmt_b=fmt_b)
                    except ValueError:
                        assert M * N >= 1 << 43
                        continue
                    if p["variant"] == mxg.VARIANT_DECODE:
                        assert fmt is not None and M <= 32 and K >= 512
                        continue
                    bm, bn = p["tile_m"], p["tile_n"]
                    assert tiles[bm, bn] == p["threads"]
                    assert p["workgroups"] == -(-M // bm) * -(-N // bn) * p["split_k"]
                    assert 1 <= p["split_k"] <= mxg.MAX_SPLIT_K and (p["split_k"] == 1 or K >= 2048)
                    need = p["split_k"] * -(-M * N // 64) * 256 if p["split_k"] > 1 else 0
                    assert p["workspace_bytes"] == need
    with pytest.raises(ValueError):
        mxg.plan_fused(3, 8, 64, 512)
    with pytest.raises(ValueError):
        mxg.plan_fused(None, 8, 64, 20)
    assert mxg.lib().mx_gemm_fused_plan(2, 2, 8, 64, 512, 2, None) == mxg.MX_ERR_NULL
    assert mxg.lib().mx_gemm_bf16_fused_plan(8, 64, 512, 2, None) == mxg.MX_ERR_NULL


def test_workspaces():
    L = mxg.lib()
    assert L.mx_rmsnorm_backward_workspace(0, 64) == 0
    assert L.mx_rmsnorm_backward_workspace(3, 64) == 0
    assert L.mx_rmsnorm_backward_workspace(3, 8224) == 3 * 8224 * 4
    assert L.mx_rmsnorm_backward_workspace(9000, 64) == 256 * 64 * 4
    big = L.mx_rmsnorm_backward_workspace(1 << 30, 65536)
    assert 0 < big <= 1024 * 65536 * 4
    assert L.mx_rmsnorm_backward_workspace(3, 65) == mxg.MX_ERR_ROW_SHAPE
    assert L.mx_moe_sort_workspace(0, 4, 8) == 0
    assert L.mx_moe_sort_workspace(16, 4, 8) == 0
    assert 0 < L.mx_moe_sort_workspace(1 << 24, 64, 256) <= 257 * 257 * 4
    assert L.mx_moe_sort_workspace(16, 65, 8) == mxg.MX_ERR_ROW_SHAPE


def test_new_codes_and_constants():
    for code in (mxg.MX_ERR_ROW_SHAPE, mxg.MX_ERR_WORKSPACE, mxg.MX_ERR_ACT):
        assert mxg.strerror(code) != mxg.strerror(-99)
    src = open(os.path.join(ROOT, "include", "mxgemm.h")).read()
    assert int(re.search(r"#define MX_ROW_MAX_WIDTH (\d+)", src).group(1)) == mxg.ROW_MAX_WIDTH
    assert int(re.search(r"#define MX_MOE_MAX_TOP (\d+)", src).group(1)) == mxg.MOE_MAX_TOP
    for name in ("NONE", "RELU", "SILU", "GELU", "GELU_TANH"):
        assert int(re.search(r"MX_ACT_%s = (\d)" % name, src).group(1)) == getattr(mxg, "ACT_" + name)


def test_every_declared_operator_is_bound():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxgemm.h")).read(), flags=re.S)
    for n in re.findall(r"\b(mx_(?:rmsnorm|swiglu|moe)[a-z_0-9]*|mx_gemm[a-z_0-9]*_fused|mx_gemm_fused)\s*\(",
                        src):
        assert getattr(mxg.lib(), n).argtypes, n
        assert isinstance(getattr(mxg.lib(), n).restype(), (ctypes.c_int, ctypes.c_int64)), n
