"""Python binding of the operators between two products of a transformer
block: row operators with MX outputs, expert routing around the grouped GEMM,
and products with a fused epilogue (include/mxgemm.h).

Like the rest of the binding it only marshals arguments; every result is
computed by the library's HIP kernels, on the current stream or on ``stream``
(a raw stream handle).  Outputs and workspaces of a call on another stream
than the current one are allocated for that stream.  Results carry no autograd
history, whatever their inputs carry: the backward functions are called by
name, as examples/moe_block.py does.

A call with plain tensors on the current device and stream is checked and
launched in one step by the compiled module _native (csrc/binding.cpp), which
halves its host time; every other call, wrong arguments among them, takes the
Python code below.

    o = mx_rmsnorm_quantize(x, weight, FMT_E4M3, residual=r)   # o.q, o.q_scale, o.h
    dx, dw = mx_rmsnorm_backward(dy, o.h, o.rstd, weight, dh=dh)
    q, q_scale = mx_swiglu_quantize(gate_up, FMT_E4M3)
    dgate_up = mx_swiglu_backward(dy, gate_up)
    plan = mx_moe_sort(ids, experts)
    xs, xs_scale = mx_moe_gather(plan, q, q_scale)
    out = mx_moe_combine(plan, y, weights, residual=h)
    dy, dweights = mx_moe_combine_backward(plan, dout, y, weights)
    c = mx_gemm_fused(a, a_scale, b, b_scale, FMT_E4M3, bias=bias, act=ACT_SILU, residual=r)
"""
import contextlib
import ctypes
from collections import namedtuple

import microscaled_block_scaled_amd as _m

ACT_NONE = 0
ACT_RELU = 1
ACT_SILU = 2
ACT_GELU = 3            # by erf
ACT_GELU_TANH = 4
ROW_MAX_WIDTH = 65536   # longest row of a row operator
MOE_MAX_TOP = 64        # most choices per token

NormOut = namedtuple("NormOut", "q q_scale h y rstd")
NormOut.__doc__ = """What mx_rmsnorm_quantize returns; None for what was not wanted."""

MoePlan = namedtuple("MoePlan", "group_rows row_of")
MoePlan.__doc__ = """Tokens sorted by expert (mx_moe_sort): rows per expert (int64, on the
device) and each (token, choice) pair's row in expert order (int32, -1 - row
for a pair without an expert)."""


# The library functions that _native calls, in the order it takes them.
_NATIVE_ORDER = ("mx_rmsnorm_quantize", "mx_rmsnorm_backward_workspace", "mx_rmsnorm_backward",
                 "mx_swiglu_quantize", "mx_swiglu_backward", "mx_moe_sort_workspace",
                 "mx_moe_sort", "mx_moe_gather", "mx_moe_combine", "mx_moe_combine_backward",
                 "mx_gemm_fused", "mx_gemm_bf16_fused", "mx_gemm_fused_plan",
                 "mx_gemm_bf16_fused_plan")
_native = None


def native():
    """The compiled module, bound to the loaded library (raises if it has not
    been built)."""
    global _native
    if _native is None:
        L = _m.lib()                         # loads torch, which _native links to
        try:
            from . import _native as module
        except ImportError as e:
            raise RuntimeError("_native.so is not built; run microscaled_block_scaled_amd/build.py "
                               "(or __graft_entry__.build()): %s" % e)
        module.bind(tuple(ctypes.cast(getattr(L, n), ctypes.c_void_p).value
                          for n in _NATIVE_ORDER))
        _native = module
    return _native


def _fast(name, stream, like, *args):
    """The operator's outputs from _native, or None where the call is not one
    it takes.  ``like`` is the tensor whose device the call runs on."""
    torch = _torch()
    if stream is not None or not isinstance(like, torch.Tensor):
        return None
    device = like.get_device()
    if device < 0 or device != torch._C._cuda_getDevice():
        return None
    r = getattr(_native or native(), name)(*args, device,
                                           torch._C._cuda_getCurrentRawStream(device))
    if r.__class__ is int:
        _m._raise(r)
    return r


def declare(L):
    """Argument types of the library functions bound here."""
    i64, vp, ci, cf = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    for name, res, args in (
            ("mx_rmsnorm_quantize", ci, [ci, ci, ci, i64, i64, vp, i64, vp, i64, vp, cf, vp, vp,
                                         vp, vp, vp, vp]),
            ("mx_rmsnorm_backward_workspace", i64, [i64, i64]),
            ("mx_rmsnorm_backward", ci, [ci, ci, i64, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp,
                                         vp, vp, i64, vp]),
            ("mx_swiglu_quantize", ci, [ci, ci, i64, i64, vp, i64, vp, vp, vp]),
            ("mx_swiglu_backward", ci, [ci, i64, i64, vp, i64, vp, i64, vp, vp]),
            ("mx_moe_sort_workspace", i64, [i64, i64, i64]),
            ("mx_moe_sort", ci, [ci, i64, i64, i64, vp, vp, vp, vp, i64, vp]),
            ("mx_moe_gather", ci, [i64, i64, vp, vp, i64, i64, vp, i64, i64, vp, vp, vp]),
            ("mx_moe_combine", ci, [ci, i64, i64, i64, vp, vp, i64, i64, vp, vp, i64, vp, vp]),
            ("mx_moe_combine_backward", ci, [ci, i64, i64, i64, vp, vp, i64, vp, i64, i64, vp, vp,
                                             vp, vp]),
            ("mx_gemm_fused", ci, [ci, ci, i64, i64, i64, vp, vp, vp, vp, vp, ci, ci, vp, i64, vp,
                                   ci, vp, i64, vp]),
            ("mx_gemm_bf16_fused", ci, [i64, i64, i64, vp, vp, vp, ci, ci, vp, i64, vp, ci, vp, i64,
                                        vp]),
            ("mx_gemm_fused_plan", ci, [ci, ci, i64, i64, i64, ci, vp]),
            ("mx_gemm_bf16_fused_plan", ci, [i64, i64, i64, ci, vp])):
        f = getattr(L, name)
        f.restype, f.argtypes = res, args


_torch_module = None
_codes = {}             # torch dtype -> MX_IN_* code


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _codes.update({torch.float32: _m.IN_FP32, torch.bfloat16: _m.IN_BF16})
        _byte_types.update((torch.uint8, torch.float8_e4m3fn, torch.float8_e8m0fnu))
        _torch_module = torch
    return _torch_module


_HERE = contextlib.nullcontext()


def _enter(device, stream):
    """(context, stream handle) of one call: inside the context the device is
    current, and allocations belong to ``stream`` when that is not the current
    one."""
    torch = _torch()
    index = device.index
    current = torch._C._cuda_getCurrentRawStream(index)
    if stream is not None and int(stream) != current:
        # handle 0 is the default stream; an external stream of 0 would be
        # some new stream, to which the allocations would belong
        on = torch.cuda.ExternalStream(int(stream), device) if int(stream) else \
            torch.cuda.default_stream(device)
        return torch.cuda.stream(on), int(stream) or None
    if torch._C._cuda_getDevice() != index:
        return torch.cuda.device(device), current or None
    return _HERE, current or None


def _dtype_code(t, name):
    code = _codes.get(t.dtype)
    if code is None:
        raise ValueError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    return code


def _tensor(t, name, device=None):
    if not isinstance(t, _torch().Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % name)
    if device is not None and t.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    return t


def _rows(t, name, width=None, rows=None, dtype=None, device=None):
    """A 2-D tensor of rows with contiguous elements (any row pitch): its
    pitch."""
    _tensor(t, name, device)
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be 2-D" % name)
    n, w = shape
    if (width is not None and w != width) or (rows is not None and n != rows):
        raise ValueError("%s has shape %s, expected (%s, %s)"
                         % (name, tuple(shape), rows if rows is not None else "rows",
                            width if width is not None else "width"))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    ld, one = t.stride()
    if one != 1 and w > 1:
        raise ValueError("%s must have contiguous rows" % name)
    if n <= 1:
        return w                             # the pitch of one row means nothing
    if ld < w:
        raise ValueError("%s must have rows that do not overlap" % name)
    return ld


_byte_types = set()     # torch types of packed elements and scales


def _bytes(t, name, device):
    """Shape of a contiguous 2-D tensor of bytes (packed elements, scales)."""
    if t.__class__ is not _torch().Tensor or not t.is_cuda or t.dtype not in _byte_types:
        _m._as_u8(t, name)                   # raises, or knows better
    shape = t.shape
    if len(shape) != 2 or not t.is_contiguous():
        raise ValueError("%s must be 2-D and contiguous" % name)
    if t.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    return shape


def _vector(t, name, n, device, dtypes):
    _tensor(t, name, device)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous vector of %d values" % (name, n))
    if t.dtype not in dtypes:
        raise ValueError("%s must be one of %s, got %s" % (name, dtypes, t.dtype))
    return t


def _fmt(fmt):
    if fmt not in (_m.FMT_E2M1, _m.FMT_E4M3, _m.FMT_E5M2, _m.FMT_E2M3, _m.FMT_E3M2):
        raise ValueError("fmt must be one of the MX element formats")
    return int(fmt)


def _act(act):
    if act not in (ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH):
        _m._raise(_m.MX_ERR_ACT)
    return int(act)


def _ptr(t):
    return None if t is None else t.data_ptr()


def mx_rmsnorm_quantize(x, weight, fmt, residual=None, eps=1e-6, need_y=False, need_rstd=False,
                        stream=None):
    """Residual addition, RMS norm and MX quantization of the rows of x
    (float32 or bfloat16, any row pitch that keeps rows 16-byte aligned):
    h = x + residual (rounded to x's type; x itself without a residual),
    y = h * rstd * weight, (q, q_scale) = MX(y) in mx_gemm's operand layout.
    ``fmt`` None gives no q.  ``need_y`` also returns y in x's type,
    ``need_rstd`` the float32 rstd that mx_rmsnorm_backward takes.  Returns
    NormOut(q, q_scale, h, y, rstd)."""
    r = _fast("rmsnorm_quantize", stream, x, x, weight, residual, fmt, eps, need_y, need_rstd)
    if r is not None:
        q, qs, h, y, rstd = r
        return NormOut(q, qs, x if h is None else h, y, rstd)
    torch = _torch()
    ldx = _rows(x, "x")
    rows, width = x.shape
    dev = x.device
    code = _dtype_code(x, "x")
    _vector(weight, "weight", width, dev, (torch.float32, torch.bfloat16))
    ldr = 0
    if residual is not None:
        ldr = _rows(residual, "residual", width, rows, x.dtype, dev)
    L = _m.lib()
    ctx, s = _enter(dev, stream)
    with ctx:
        h = x if residual is None else x.new_empty((rows, width))
        q = qs = y = rstd = None
        if fmt is not None:
            q = torch.empty((rows, _m._row_bytes(_fmt(fmt), width)), dtype=torch.uint8, device=dev)
            qs = torch.empty((rows, width // 32), dtype=torch.uint8, device=dev)
        if need_y:
            y = x.new_empty((rows, width))
        if need_rstd:
            rstd = torch.empty(rows, dtype=torch.float32, device=dev)
        rc = L.mx_rmsnorm_quantize(
            fmt or 0, code, _dtype_code(weight, "weight"), rows, width, x.data_ptr(), ldx,
            _ptr(residual), ldr, weight.data_ptr(), eps, h.data_ptr(), _ptr(y), _ptr(q), _ptr(qs),
            _ptr(rstd), s)
    if rc:
        _m._raise(rc)
    return NormOut(q, qs, h, y, rstd)


def mx_rmsnorm_backward(dy, h, rstd, weight, dh=None, need_dw=True, stream=None):
    """Gradient of mx_rmsnorm_quantize (the MX rounding passes gradients
    through): (dx, dw), dx in h's type for x and the residual alike, dw
    float32 (None without ``need_dw``).  ``dh`` is the gradient that reaches h
    from its other uses."""
    r = _fast("rmsnorm_backward", stream, h, dy, h, rstd, weight, dh, need_dw)
    if r is not None:
        return r
    torch = _torch()
    ldh = _rows(h, "h")
    rows, width = h.shape
    dev = h.device
    code = _dtype_code(h, "h")
    lddy = _rows(dy, "dy", width, rows, h.dtype, dev)
    lddh = 0 if dh is None else _rows(dh, "dh", width, rows, h.dtype, dev)
    _vector(weight, "weight", width, dev, (torch.float32, torch.bfloat16))
    _vector(rstd, "rstd", rows, dev, (torch.float32,))
    L = _m.lib()
    ctx, s = _enter(dev, stream)
    with ctx:
        dx = h.new_empty((rows, width))
        dw = ws = None
        nbytes = 0
        if need_dw:
            nbytes = L.mx_rmsnorm_backward_workspace(rows, width)
            if nbytes < 0:
                _m._raise(nbytes)
            dw = torch.empty(width, dtype=torch.float32, device=dev)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        rc = L.mx_rmsnorm_backward(
            code, _dtype_code(weight, "weight"), rows, width, dy.data_ptr(), lddy, h.data_ptr(),
            ldh, rstd.data_ptr(), weight.data_ptr(), _ptr(dh), lddh, dx.data_ptr(), _ptr(dw),
            _ptr(ws), nbytes, s)
    if rc:
        _m._raise(rc)
    return dx, dw


def mx_swiglu_quantize(gate_up, fmt, stream=None):
    """MX(silu(gate) * up) of rows holding gate then up (rows x 2*width):
    (q, q_scale) in mx_gemm's operand layout."""
    r = _fast("swiglu_quantize", stream, gate_up, gate_up, fmt)
    if r is not None:
        return r
    torch = _torch()
    ld = _rows(gate_up, "gate_up")
    rows, two = gate_up.shape
    if two % 2:
        raise ValueError("gate_up must have an even row length")
    width = two // 2
    dev = gate_up.device
    code = _dtype_code(gate_up, "gate_up")
    L = _m.lib()
    ctx, s = _enter(dev, stream)
    with ctx:
        q = torch.empty((rows, _m._row_bytes(_fmt(fmt), width)), dtype=torch.uint8, device=dev)
        qs = torch.empty((rows, width // 32), dtype=torch.uint8, device=dev)
        rc = L.mx_swiglu_quantize(fmt, code, rows, width, gate_up.data_ptr(), ld,
                                           q.data_ptr(), qs.data_ptr(), s)
    if rc:
        _m._raise(rc)
    return q, qs


def mx_swiglu_backward(dy, gate_up, stream=None):
    """Gradient of mx_swiglu_quantize with respect to gate_up (the MX rounding
    passes gradients through), in its type."""
    r = _fast("swiglu_backward", stream, gate_up, dy, gate_up)
    if r is not None:
        return r[0]
    torch = _torch()
    ld = _rows(gate_up, "gate_up")
    rows, two = gate_up.shape
    if two % 2:
        raise ValueError("gate_up must have an even row length")
    dev = gate_up.device
    code = _dtype_code(gate_up, "gate_up")
    lddy = _rows(dy, "dy", two // 2, rows, gate_up.dtype, dev)
    L = _m.lib()
    ctx, s = _enter(dev, stream)
    with ctx:
        dgu = gate_up.new_empty((rows, two))
        rc = L.mx_swiglu_backward(code, rows, two // 2, dy.data_ptr(), lddy,
                                           gate_up.data_ptr(), ld, dgu.data_ptr(), s)
    if rc:
        _m._raise(rc)
    return dgu


def mx_moe_sort(ids, experts, stream=None):
    """Sorts the (token, choice) pairs of ids (tokens x top, int32 or int64)
    by expert, in the order of the pairs within an expert.  An id outside 0 ..
    experts - 1 is no expert: its pair comes after all others.  Returns
    MoePlan(group_rows, row_of); ``group_rows.tolist()`` is what
    mx_gemm_grouped takes."""
    r = _fast("moe_sort", stream, ids, ids, experts)
    if r is not None:
        return MoePlan(*r)
    torch = _torch()
    _tensor(ids, "ids")
    if ids.dim() != 2 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous (tokens, top) tensor")
    if ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be int32 or int64, got %s" % ids.dtype)
    tokens, top = ids.shape
    dev = ids.device
    L = _m.lib()
    nbytes = L.mx_moe_sort_workspace(tokens, top, experts)
    if nbytes < 0:
        _m._raise(nbytes)
    ctx, s = _enter(dev, stream)
    with ctx:
        group_rows = torch.empty(experts, dtype=torch.int64, device=dev)
        row_of = torch.empty((tokens, top), dtype=torch.int32, device=dev)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        rc = L.mx_moe_sort(ids.element_size(), tokens, top, experts, ids.data_ptr(),
                             group_rows.data_ptr(), row_of.data_ptr(), _ptr(ws), nbytes, s)
    if rc:
        _m._raise(rc)
    return MoePlan(group_rows, row_of)


def _plan_rows(plan, device):
    row_of = _tensor(plan.row_of, "plan.row_of", device)
    if row_of.dim() != 2 or row_of.dtype != _torch().int32 or not row_of.is_contiguous():
        raise ValueError("plan.row_of must be a contiguous (tokens, top) int32 tensor")
    return row_of


def mx_moe_gather(plan, x, x_scale=None, stream=None):
    """Token rows in expert order: row t of x (any type, any row pitch) at the
    rows of its pairs, and likewise its rows of x_scale.  Returns
    (xs, xs_scale) of tokens * top rows (xs_scale None without x_scale); rows
    of pairs without an expert, which come last, are zeros."""
    r = _fast("moe_gather", stream, x, plan.row_of, x, x_scale)
    if r is not None:
        return r
    torch = _torch()
    ld = _rows(x, "x")
    dev = x.device
    row_of = _plan_rows(plan, dev)
    tokens, top = row_of.shape
    if x.shape[0] != tokens:
        raise ValueError("x has %d rows, the plan %d tokens" % (x.shape[0], tokens))
    size, lds, sbytes = x.element_size(), 0, 0
    if x_scale is not None:
        ssize = x_scale.element_size()
        lds = _rows(x_scale, "x_scale", rows=tokens, device=dev) * ssize
        sbytes = x_scale.shape[1] * ssize
    L = _m.lib()
    ctx, s = _enter(dev, stream)
    with ctx:
        xs = x.new_empty((tokens * top, x.shape[1]))
        ss = None
        if x_scale is not None:
            ss = x_scale.new_empty((tokens * top, x_scale.shape[1]))
        rc = L.mx_moe_gather(tokens, top, row_of.data_ptr(), x.data_ptr(),
                                      x.shape[1] * size, ld * size, _ptr(x_scale), sbytes, lds,
                                      xs.data_ptr(), _ptr(ss), s)
    if rc:
        _m._raise(rc)
    return xs, ss


def _weights(weights, row_of, device):
    _tensor(weights, "weights", device)
    if weights.dtype != _torch().float32 or weights.shape != row_of.shape or \
            not weights.is_contiguous():
        raise ValueError("weights must be a contiguous %s float32 tensor" % (tuple(row_of.shape),))
    return weights


def mx_moe_combine(plan, y, weights=None, residual=None, stream=None):
    """Expert rows back to their tokens: residual[t] + sum over choices j of
    weights[t, j] * y[row of (t, j)], in y's type; pairs without an expert add
    nothing.  ``weights`` (tokens x top, float32) None counts each row once,
    which is the gradient of mx_moe_gather.  y may leave out the rows of pairs
    without an expert."""
    r = _fast("moe_combine", stream, y, plan.row_of, y, weights, residual)
    if r is not None:
        return r[0]
    torch = _torch()
    ldy = _rows(y, "y")
    dev = y.device
    code = _dtype_code(y, "y")
    row_of = _plan_rows(plan, dev)
    tokens, top = row_of.shape
    width = y.shape[1]
    if weights is not None:
        _weights(weights, row_of, dev)
    ldr = 0 if residual is None else _rows(residual, "residual", width, tokens, y.dtype, dev)
    L = _m.lib()
    ctx, s = _enter(dev, stream)
    with ctx:
        out = y.new_empty((tokens, width))
        rc = L.mx_moe_combine(code, tokens, top, width, row_of.data_ptr(), y.data_ptr(),
                                       y.shape[0], ldy, _ptr(weights), _ptr(residual), ldr,
                                       out.data_ptr(), s)
    if rc:
        _m._raise(rc)
    return out


def mx_moe_combine_backward(plan, dout, y, weights, stream=None):
    """Gradient of mx_moe_combine: (dy, dweights).  dy has y's rows, zeros in
    those of pairs without an expert; dweights is (tokens, top) float32.  The
    residual's gradient is dout itself."""
    r = _fast("moe_combine_backward", stream, y, plan.row_of, dout, y, weights)
    if r is not None:
        return r
    torch = _torch()
    ldy = _rows(y, "y")
    dev = y.device
    code = _dtype_code(y, "y")
    row_of = _plan_rows(plan, dev)
    tokens, top = row_of.shape
    width = y.shape[1]
    lddo = _rows(dout, "dout", width, tokens, y.dtype, dev)
    _weights(weights, row_of, dev)
    L = _m.lib()
    ctx, s = _enter(dev, stream)
    with ctx:
        dy = y.new_empty((y.shape[0], width))
        dw = torch.empty((tokens, top), dtype=torch.float32, device=dev)
        rc = L.mx_moe_combine_backward(
            code, tokens, top, width, row_of.data_ptr(), dout.data_ptr(), lddo, y.data_ptr(),
            y.shape[0], ldy, weights.data_ptr(), dy.data_ptr(), dw.data_ptr(), s)
    if rc:
        _m._raise(rc)
    return dy, dw


def plan_fused(fmt, M, N, K, out_dtype=None, fmt_b=None):
    """How mx_gemm_fused would run this problem (a dict), or with ``fmt`` None
    mx_gemm_bf16_fused; host logic only."""
    p = _m.MxPlan()
    out = _m.OUT_BF16 if out_dtype is None else int(out_dtype)
    if fmt is None:
        rc = _m.lib().mx_gemm_bf16_fused_plan(M, N, K, out, ctypes.addressof(p))
    else:
        rc = _m.lib().mx_gemm_fused_plan(fmt, fmt if fmt_b is None else fmt_b, M, N, K, out,
                                         ctypes.addressof(p))
    if rc:
        _m._raise(rc)
    return p.as_dict()


def _epilogue(M, N, tdt, dev, bias, residual, out):
    """Checks bias, residual and out: (bias code, residual pitch)."""
    torch = _torch()
    code, ldr = 0, 0
    if bias is not None:
        _vector(bias, "bias", N, dev, (torch.float32, torch.bfloat16))
        code = _dtype_code(bias, "bias")
    if residual is not None:
        ldr = _rows(residual, "residual", N, M, tdt, dev)
    if out is not None and (out.dtype != tdt or tuple(out.shape) != (M, N)
                            or not out.is_contiguous() or out.device != dev):
        raise ValueError("out must be a contiguous (M, N) %s tensor on %s" % (tdt, dev))
    return code, ldr


def mx_gemm_fused(a, a_scale, b, b_scale, fmt, bias=None, act=ACT_NONE, residual=None,
                  out_dtype=None, out=None, stream=None, fmt_b=None):
    """C = residual + act(A * B^T + bias) with mx_gemm's operands, in E2M1,
    E4M3, or E4M3 (A) with E2M1 (B).  bias is N float32 or bfloat16 values,
    act an ACT_* code, residual (M, N) in C's type (any row pitch; may be
    ``out`` itself).  Everything is applied to the FP32 sums before C's one
    rounding to ``out_dtype`` (bfloat16 by default)."""
    code, tdt = _m._out_code(_torch().bfloat16 if out_dtype is None else out_dtype)
    r = _fast("gemm_fused", stream, a, fmt, fmt if fmt_b is None else fmt_b, a, a_scale, b, b_scale,
              bias, act, residual, code, out)
    if r is not None:
        return r[0] if out is None else out
    torch = _torch()
    fmt_b = fmt if fmt_b is None else fmt_b
    fmt, fmt_b, act = _fmt(fmt), _fmt(fmt_b), _act(act)
    dev = a.device if isinstance(a, torch.Tensor) else None
    M, row_a = _bytes(a, "a", dev)
    N, row_b = _bytes(b, "b", dev)
    K = _m._k_of(fmt, row_a)
    if _m._k_of(fmt_b, row_b) != K:
        raise ValueError("a and b disagree on K")
    if _bytes(a_scale, "a_scale", dev) != (M, K // 32) or \
            _bytes(b_scale, "b_scale", dev) != (N, K // 32):
        raise ValueError("scales must be (rows, K/32) = (%d, %d) and (%d, %d)"
                         % (M, K // 32, N, K // 32))
    bias_code, ldr = _epilogue(M, N, tdt, dev, bias, residual, out)
    L = _m.lib()
    ctx, s = _enter(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty((M, N), dtype=tdt, device=dev)
        nbytes = plan_fused(fmt, M, N, K, code, fmt_b)["workspace_bytes"]
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        rc = L.mx_gemm_fused(
            fmt, fmt_b, M, N, K, a.data_ptr(), a_scale.data_ptr(), b.data_ptr(),
            b_scale.data_ptr(), _ptr(bias), bias_code, act, _ptr(residual), ldr, out.data_ptr(),
            code, _ptr(ws), nbytes, s)
    if rc:
        _m._raise(rc)
    return out


def mx_gemm_bf16_fused(a, b, bias=None, act=ACT_NONE, residual=None, out_dtype=None, out=None,
                       stream=None):
    """mx_gemm_fused with mx_gemm_bf16's dense BF16 operands."""
    code, tdt = _m._out_code(_torch().bfloat16 if out_dtype is None else out_dtype)
    r = _fast("gemm_bf16_fused", stream, a, a, b, bias, act, residual, code, out)
    if r is not None:
        return r[0] if out is None else out
    torch = _torch()
    _m._as_bf16(a, "a"), _m._as_bf16(b, "b")
    act = _act(act)
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError("a and b disagree on K")
    dev = a.device
    if b.device != dev:
        raise ValueError("all operands must be on the same device")
    bias_code, ldr = _epilogue(M, N, tdt, dev, bias, residual, out)
    L = _m.lib()
    ctx, s = _enter(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty((M, N), dtype=tdt, device=dev)
        nbytes = plan_fused(None, M, N, K, code)["workspace_bytes"]
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        rc = L.mx_gemm_bf16_fused(M, N, K, a.data_ptr(), b.data_ptr(), _ptr(bias), bias_code, act,
                                  _ptr(residual), ldr, out.data_ptr(), code, _ptr(ws), nbytes, s)
    if rc:
        _m._raise(rc)
    return out
