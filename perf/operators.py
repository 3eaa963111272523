"""Cases of the transformer-block operators around the MX GEMM.

Four operators, each with its directions:

* norm       residual addition + root-mean-square norm + MX quantization of
             the normed rows, and its gradient;
* swiglu     silu(gate) * up of a fused gate/up product + MX quantization,
             and its gradient;
* moe        tokens sorted by expert and their rows gathered, expert rows
             combined with weights, and the gradient of the combination;
* gemm       C = residual + act(A * B^T + bias) with MX or BF16 operands.

``own`` False computes them from elementary torch operations in 32 bits;
``own`` True calls microscaled_block_scaled_amd.  8-bit results are returned
as float8 tensors (elements) and float8_e8m0fnu tensors (scales), so that
they compare as the values they hold.
"""
import math

import torch

own = False

E2M1, E4M3, E5M2 = 1, 2, 3                       # element format codes of the library
FMT = {"e2m1": E2M1, "e4m3": E4M3, "e5m2": E5M2}
EMAX = {"e2m1": 2, "e4m3": 8, "e5m2": 15}        # exponent of the largest element
TOP = {"e2m1": 6.0, "e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


def _mxg():
    import microscaled_block_scaled_amd as mxg
    return mxg


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # One decode step of a 70B-Llama-shaped layer, 8 requests: latency.
        dict(name="norm_decode", op="norm", rows=8, width=8192, dtype="bf16", fmt="e4m3",
             residual=True),
        # Prefill of 64 requests x 256 tokens at the same width: bandwidth.
        dict(name="norm_prefill", op="norm", rows=16384, width=8192, dtype="bf16", fmt="e4m3",
             residual=True),
        # Training step, a ragged batch at Qwen3-32B's width.
        dict(name="norm_grad", op="norm_grad", rows=4001, width=5120, dtype="bf16"),
        # A single token through an 8B-Llama MLP: the smallest call.
        dict(name="swiglu_decode", op="swiglu", rows=1, width=14336, dtype="bf16", fmt="e4m3"),
        # The 70B-Llama MLP between its two products, 2048 tokens.
        dict(name="swiglu_prefill", op="swiglu", rows=2048, width=28672, dtype="bf16",
             fmt="e4m3"),
        # Training step of the Qwen3-32B MLP, a ragged batch.
        dict(name="swiglu_grad", op="swiglu_grad", rows=1999, width=25600, dtype="bf16"),
        # 64 decoding requests on 8 experts, two per token: latency.
        dict(name="moe_dispatch_decode", op="dispatch", rows=64, top=2, experts=8, width=4096,
             fmt="e4m3", drop=0.0),
        # Prefill on many small experts, some padding tokens: bandwidth.
        dict(name="moe_dispatch_prefill", op="dispatch", rows=16384, top=8, experts=256,
             width=4096, fmt="e4m3", drop=0.03),
        # Expert rows back to their tokens and onto the residual stream.
        dict(name="moe_combine", op="combine", rows=8192, top=4, experts=64, width=4096,
             dtype="bf16", drop=0.03),
        # The same in training: gradients of the expert rows and the weights.
        dict(name="moe_combine_grad", op="combine_grad", rows=4095, top=4, experts=64,
             width=4096, dtype="bf16", drop=0.03),
        # 70B-Llama down projection onto the residual stream, batch 8, 8-bit
        # activations and 4-bit weights.
        dict(name="gemm_decode", op="gemm", m=8, n=8192, k=28672, fmt_a="e4m3", fmt_b="e2m1",
             out="bf16", act="none", bias=True, residual=True),
        # The same projection over 2048 tokens, MXFP4: the largest call.
        dict(name="gemm_prefill", op="gemm", m=2048, n=8192, k=28672, fmt_a="e2m1",
             fmt_b="e2m1", out="bf16", act="gelu", bias=True, residual=True),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in lo .. hi, spread over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "swiglu", "swiglu_grad", "dispatch", "combine",
                     "combine_grad", "gemm", "gemm"])
    if op in ("norm", "norm_grad"):
        width = _log(rng, 1024, 16384, 32)
        c = dict(op=op, rows=_log(rng, 1, min(16384, 2 ** 27 // width)), width=width,
                 dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "norm":
            c.update(fmt=rng.choice(["e4m3", "e5m2"]), residual=rng.random() < 0.75)
            if c["dtype"] == "f32":
                c["rows"] = max(1, c["rows"] // 2)
        else:
            c["rows"] = max(1, c["rows"] // 4)
    elif op in ("swiglu", "swiglu_grad"):
        width = _log(rng, 1024, 28672, 32)
        c = dict(op=op, rows=_log(rng, 1, min(8192, 2048 * 28672 // width)), width=width,
                 dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op == "swiglu":
            c["fmt"] = rng.choice(["e4m3", "e5m2"])
            if c["dtype"] == "f32":
                c["rows"] = max(1, c["rows"] // 2)
        else:
            c["rows"] = max(1, c["rows"] // 3)
    elif op in ("dispatch", "combine", "combine_grad"):
        experts = _log(rng, 4, 256)
        top = rng.choice([1, 2, 4, 6, 8])
        top = min(top, experts)
        width = _log(rng, 1024, 8192, 128)
        c = dict(op=op, rows=_log(rng, 1, min(16384, 2 ** 27 // (top * width))), top=top,
                 experts=experts, width=width, drop=rng.choice([0.0, 0.0, 0.05, 0.4]))
        if op == "dispatch":
            c["fmt"] = rng.choice(["e4m3", "e5m2"])
        else:
            c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
            if op == "combine_grad":
                c["rows"] = max(1, c["rows"] // 2)
    else:
        fa, fb, out = rng.choice([("e4m3", "e4m3", "bf16"), ("e2m1", "e2m1", "bf16"),
                                  ("e2m1", "e2m1", "f32"), ("e4m3", "e2m1", "bf16"),
                                  ("bf16", "bf16", "bf16"), ("bf16", "bf16", "f32")])
        n = _log(rng, 1000, 14336)
        k = _log(rng, 1024, 14336, 128)
        c = dict(op=op, m=_log(rng, 1, 2048), n=n, k=k, fmt_a=fa, fmt_b=fb, out=out,
                 act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                 bias=rng.random() < 0.6, residual=rng.random() < 0.6)
    return c


# ------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", dtype=torch.float32, generator=g)


def _rand(g, *shape):
    return torch.rand(shape, device="cuda", dtype=torch.float32, generator=g)


def _pow2(byte):
    """2^(byte - 127) as float32 for bytes 1 .. 254."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _mx_elements(x, fmt):
    """Scaled rows x (R, K) float32 -> (x / 2^X per 32 values, X + 127 bytes),
    X = floor(log2 amax) - emax, by the OCP Microscaling rule."""
    b = x.view(x.shape[0], -1, 32)
    amax = b.abs().amax(-1)
    byte = torch.frexp(amax).exponent - 1 - EMAX[fmt] + 127
    byte = torch.where(amax > 0, byte, 0).clamp(0, 254).to(torch.uint8)
    # the cases' blocks have scales far from both ends of the range
    y = b / _pow2(byte.clamp(1, 254)).unsqueeze(-1)
    return y.view(x.shape), byte


def _quantize(x, fmt):
    """x (R, K) float32 -> (float8 elements, float8_e8m0fnu scales)."""
    y, byte = _mx_elements(x, fmt)
    q = y.clamp(-TOP[fmt], TOP[fmt]).to(F8[fmt])
    return q, byte.view(torch.float8_e8m0fnu)


_E2M1_MIDS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _operand(g, rows, k, fmt, std):
    """A quantized GEMM operand as a user's program holds it: (bytes, scales)."""
    x = _randn(g, rows, k) * std
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    y, byte = _mx_elements(x, fmt)
    del x
    if fmt == "e2m1":
        mids = torch.tensor(_E2M1_MIDS, device="cuda")
        code = torch.bucketize(y.abs(), mids, out_int32=True).to(torch.uint8)
        code |= (y < 0).to(torch.uint8) << 3
        return code[:, 0::2] | (code[:, 1::2] << 4), byte
    return y.clamp(-TOP[fmt], TOP[fmt]).to(F8[fmt]).view(torch.uint8), byte


def _routing(g, case):
    """Expert ids (rows, top) int64, -1 for padding tokens, and the weights."""
    rows, top, experts = case["rows"], case["top"], case["experts"]
    logits = _randn(g, rows, experts) + 0.7 * _randn(g, 1, experts)     # uneven experts
    w, ids = torch.topk(logits, top, dim=-1)
    w = torch.softmax(w, -1)
    if case["drop"]:
        ids = torch.where(_rand(g, rows, 1) < case["drop"], -1, ids)
    return ids.contiguous(), w.contiguous()


def _sort(ids, experts):
    """Stable order of the (token, choice) pairs by expert, pairs without an
    expert last: rows per expert, and each pair's row (-1 - row without one)."""
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    order = torch.sort(key, stable=True).indices
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=ids.device)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    counts.scatter_add_(0, key, torch.ones_like(key))
    row = torch.where(key == experts, -1 - row, row)
    return counts[:experts], row.to(torch.int32).view(ids.shape), order


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op in ("norm", "norm_grad"):
        dt = DT[case["dtype"]]
        rows, width = case["rows"], case["width"]
        gain = 0.5 + _rand(g, rows, 1) * 2
        s["x"] = (_randn(g, rows, width) * gain).to(dt)
        s["w"] = (1 + 0.1 * _randn(g, width)).to(dt)
        if op == "norm":
            s["res"] = _randn(g, rows, width).to(dt) if case["residual"] else None
        else:
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(-1) + EPS)
            s["dy"] = (_randn(g, rows, width) * 0.01).to(dt)
            s["dh"] = (_randn(g, rows, width) * 0.01).to(dt)
    elif op in ("swiglu", "swiglu_grad"):
        dt = DT[case["dtype"]]
        s["gu"] = (_randn(g, case["rows"], 2 * case["width"]) * 1.5).to(dt)
        if op == "swiglu_grad":
            s["dy"] = (_randn(g, case["rows"], case["width"]) * 0.01).to(dt)
    elif op == "dispatch":
        s["ids"], _ = _routing(g, case)
        s["x"], s["x_scale"] = _operand(g, case["rows"], case["width"], case["fmt"], 1.0)
    elif op in ("combine", "combine_grad"):
        dt = DT[case["dtype"]]
        ids, s["weights"] = _routing(g, case)
        s["group_rows"], s["row_of"], _ = _sort(ids, case["experts"])
        s["y"] = _randn(g, case["rows"] * case["top"], case["width"]).to(dt)
        side = _randn(g, case["rows"], case["width"])
        if op == "combine":
            s["res"] = side.to(dt)
        else:
            s["dout"] = (side * 0.01).to(dt)
    else:
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["a_scale"] = _operand(g, m, k, case["fmt_a"], 1.0)
        s["b"], s["b_scale"] = _operand(g, n, k, case["fmt_b"], 1.0 / math.sqrt(k))
        s["bias_v"] = _randn(g, n) * 0.5 if case["bias"] else None
        s["res"] = _randn(g, m, n).to(DT[case["out"]]) if case["residual"] else None
    return s


# ----------------------------------------------------------- the plain forms

def _plain_norm(s):
    x = s["x"]
    h = x if s["res"] is None else (x.float() + s["res"].float()).to(x.dtype)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(-1, keepdim=True) + EPS)
    q, scale = _quantize(hf * rstd * s["w"].float(), s["fmt"])
    return {"q": q, "scale": scale, "h": h}


def _plain_norm_grad(s):
    r = s["rstd"][:, None]
    dy, xhat = s["dy"].float(), s["x"].float() * r
    wdy = dy * s["w"].float()
    c = (wdy * xhat).mean(-1, keepdim=True)
    dx = (wdy - xhat * c) * r + s["dh"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xhat).sum(0)}


def _plain_swiglu(s):
    f = s["width"]
    gate, up = s["gu"][:, :f].float(), s["gu"][:, f:].float()
    q, scale = _quantize(gate / (1 + torch.exp(-gate)) * up, s["fmt"])
    return {"q": q, "scale": scale}


def _plain_swiglu_grad(s):
    f = s["width"]
    gate, up, dy = s["gu"][:, :f].float(), s["gu"][:, f:].float(), s["dy"].float()
    sig = 1 / (1 + torch.exp(-gate))
    d_up = dy * gate * sig
    d_gate = dy * up * sig * (1 + gate * (1 - sig))
    return {"dgu": torch.cat([d_gate, d_up], 1).to(s["gu"].dtype)}


def _plain_dispatch(s):
    counts, row_of, order = _sort(s["ids"], s["experts"])
    token = torch.div(order, s["top"], rounding_mode="floor")
    live = torch.arange(order.numel(), device=order.device) < counts.sum()
    xs = torch.where(live[:, None], s["x"][token], 0)
    scales = torch.where(live[:, None], s["x_scale"][token], 0)
    return {"group_rows": counts, "row_of": row_of, "x": xs.view(F8[s["fmt"]]),
            "scale": scales.view(torch.float8_e8m0fnu)}


def _plain_combine(s):
    live = s["row_of"] >= 0
    w = torch.where(live, s["weights"], 0)
    picked = s["y"][s["row_of"].clamp(min=0).long()].float()
    picked = torch.where(live[..., None], picked, 0)
    out = (picked * w[..., None]).sum(1) + s["res"].float()
    return {"out": out.to(s["y"].dtype)}


def _plain_combine_grad(s):
    live = s["row_of"] >= 0
    w = torch.where(live, s["weights"], 0)
    row = torch.where(live, s["row_of"], -1 - s["row_of"]).long()
    dout = s["dout"].float()
    dy = torch.empty_like(s["y"])
    dy[row.view(-1)] = (dout[:, None, :] * w[..., None]).to(dy.dtype).view(-1, s["width"])
    picked = torch.where(live[..., None], s["y"][row].float(), 0)
    return {"dy": dy, "dw": (picked * dout[:, None, :]).sum(-1)}


def _decode_operand(q, scale, fmt):
    """Operand bytes and scales -> float32 values."""
    if fmt == "bf16":
        return q.float()
    if fmt == "e2m1":
        mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
        lut = torch.cat([mags, -mags])
        v = torch.stack([lut[(q & 15).int()], lut[(q >> 4).int()]], -1)
    else:
        v = q.view(F8[fmt]).float()
    v = v.view(q.shape[0], -1, 32) * _pow2(scale).unsqueeze(-1)
    return v.view(q.shape[0], -1)


def _act(v, act):
    if act == "relu":
        return torch.where(v > 0, v, 0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_gemm(s):
    c = _decode_operand(s["a"], s["a_scale"], s["fmt_a"]) @ \
        _decode_operand(s["b"], s["b_scale"], s["fmt_b"]).T
    if s["bias_v"] is not None:
        c = c + s["bias_v"]
    c = _act(c, s["act"])
    if s["res"] is not None:
        c = c + s["res"].float()
    return {"c": c.to(DT[s["out"]])}


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "swiglu": _plain_swiglu,
          "swiglu_grad": _plain_swiglu_grad, "dispatch": _plain_dispatch,
          "combine": _plain_combine, "combine_grad": _plain_combine_grad, "gemm": _plain_gemm}


# --------------------------------------------------- the framework's kernels

def _own_norm(s):
    o = _mxg().mx_rmsnorm_quantize(s["x"], s["w"], FMT[s["fmt"]], residual=s["res"], eps=EPS)
    return {"q": o.q.view(F8[s["fmt"]]), "scale": o.q_scale.view(torch.float8_e8m0fnu),
            "h": o.h}


def _own_norm_grad(s):
    dx, dw = _mxg().mx_rmsnorm_backward(s["dy"], s["x"], s["rstd"], s["w"], dh=s["dh"])
    return {"dx": dx, "dw": dw}


def _own_swiglu(s):
    q, scale = _mxg().mx_swiglu_quantize(s["gu"], FMT[s["fmt"]])
    return {"q": q.view(F8[s["fmt"]]), "scale": scale.view(torch.float8_e8m0fnu)}


def _own_swiglu_grad(s):
    return {"dgu": _mxg().mx_swiglu_backward(s["dy"], s["gu"])}


def _own_dispatch(s):
    mxg = _mxg()
    plan = mxg.mx_moe_sort(s["ids"], s["experts"])
    xs, scales = mxg.mx_moe_gather(plan, s["x"], s["x_scale"])
    return {"group_rows": plan.group_rows, "row_of": plan.row_of, "x": xs.view(F8[s["fmt"]]),
            "scale": scales.view(torch.float8_e8m0fnu)}


def _own_combine(s):
    mxg = _mxg()
    plan = mxg.MoePlan(s["group_rows"], s["row_of"])
    return {"out": mxg.mx_moe_combine(plan, s["y"], weights=s["weights"], residual=s["res"])}


def _own_combine_grad(s):
    mxg = _mxg()
    plan = mxg.MoePlan(s["group_rows"], s["row_of"])
    dy, dw = mxg.mx_moe_combine_backward(plan, s["dout"], s["y"], s["weights"])
    return {"dy": dy, "dw": dw}


def _own_gemm(s):
    mxg = _mxg()
    act = {"none": mxg.ACT_NONE, "relu": mxg.ACT_RELU, "silu": mxg.ACT_SILU,
           "gelu": mxg.ACT_GELU, "gelu_tanh": mxg.ACT_GELU_TANH}[s["act"]]
    if s["fmt_a"] == "bf16":
        c = mxg.mx_gemm_bf16_fused(s["a"], s["b"], bias=s["bias_v"], act=act, residual=s["res"],
                                   out_dtype=DT[s["out"]])
    else:
        c = mxg.mx_gemm_fused(s["a"], s["a_scale"], s["b"], s["b_scale"], FMT[s["fmt_a"]],
                              bias=s["bias_v"], act=act, residual=s["res"],
                              out_dtype=DT[s["out"]], fmt_b=FMT[s["fmt_b"]])
    return {"c": c}


_OWN = {"norm": _own_norm, "norm_grad": _own_norm_grad, "swiglu": _own_swiglu,
        "swiglu_grad": _own_swiglu_grad, "dispatch": _own_dispatch, "combine": _own_combine,
        "combine_grad": _own_combine_grad, "gemm": _own_gemm}


def run(state):
    return (_OWN if own else _PLAIN)[state["op"]](state)


# ------------------------------------------------------------------ the work

def work(case):
    """Each input read once, each output written once; the arithmetic of the
    definition."""
    op = case["op"]
    size = {"bf16": 2, "f32": 4}.get(case.get("dtype"), 0)
    if op == "norm":
        e = case["rows"] * case["width"]
        # without a residual h is x itself: neither read again nor written
        b = e * size * (3 if case["residual"] else 1) + e * 33 // 32 + case["width"] * size
        return {"bytes": b, "flops": 6 * e}
    if op == "norm_grad":
        e = case["rows"] * case["width"]
        return {"bytes": e * size * 4 + case["rows"] * 4 + case["width"] * (size + 4),
                "flops": 10 * e}
    if op == "swiglu":
        e = case["rows"] * case["width"]
        return {"bytes": e * size * 2 + e * 33 // 32, "flops": 6 * e}
    if op == "swiglu_grad":
        e = case["rows"] * case["width"]
        return {"bytes": e * size * 5, "flops": 12 * e}
    if op == "dispatch":
        pairs = case["rows"] * case["top"]
        row = case["width"] * 33 // 32
        return {"bytes": pairs * 12 + case["experts"] * 8 + (case["rows"] + pairs) * row,
                "flops": 0}
    if op == "combine":
        pairs = case["rows"] * case["top"]
        return {"bytes": pairs * 8 + (pairs + 2 * case["rows"]) * case["width"] * size,
                "flops": 2 * pairs * case["width"]}
    if op == "combine_grad":
        pairs = case["rows"] * case["top"]
        return {"bytes": pairs * 12 + (2 * pairs + case["rows"]) * case["width"] * size,
                "flops": 3 * pairs * case["width"]}
    bits = {"e2m1": 4.25, "e4m3": 8.25, "bf16": 16}
    m, n, k = case["m"], case["n"], case["k"]
    out = {"bf16": 2, "f32": 4}[case["out"]] * m * n
    return {"bytes": (m * bits[case["fmt_a"]] + n * bits[case["fmt_b"]]) * k / 8
            + out * (2 if case["residual"] else 1) + (4 * n if case["bias"] else 0),
            "flops": 2 * m * n * k}


# ---------------------------------------------------- the definitions, 64 bits

def _exact_quantize(y, fmt):
    """OCP rule in float64: element grid of the block's scale, nearest with
    ties to the even multiple, saturating."""
    b = y.view(y.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    shared = torch.floor(torch.log2(amax))
    # log2 may round across a power of two: put it right by comparison
    shared = shared - (torch.exp2(shared) > amax).double()
    shared = shared + (torch.exp2(shared + 1) <= amax).double()
    scale = torch.exp2(shared - EMAX[fmt])
    v = b / scale
    man, emin = (3, -6) if fmt == "e4m3" else (2, -14)
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -40)))
    e = e - (torch.exp2(e) > v.abs()).double()
    e = e + (torch.exp2(e + 1) <= v.abs()).double()
    step = torch.exp2(e.clamp(min=emin) - man)
    q = (torch.round(v / step) * step).clamp(-TOP[fmt], TOP[fmt])
    return q.view(y.shape), scale.squeeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = torch.float64
    if op == "norm":
        x = s["x"].to(d)
        h = x if s["res"] is None else x + s["res"].to(d)
        # the norm's input is h as it is handed on, in the rows' own type
        hr = h.to(s["x"].dtype).to(d)
        y = hr / torch.sqrt((hr * hr).sum(-1, keepdim=True) / case["width"] + EPS) * s["w"].to(d)
        q, scale = _exact_quantize(y, case["fmt"])
        return {"q": q, "scale": scale, "h": h}
    if op == "norm_grad":
        x, dy, w, r = s["x"].to(d), s["dy"].to(d), s["w"].to(d), s["rstd"].to(d)[:, None]
        dot = (dy * w * x).sum(-1, keepdim=True)
        dx = r * dy * w - r ** 3 * x * dot / case["width"] + s["dh"].to(d)
        return {"dx": dx, "dw": (dy * x * r).sum(0)}
    if op in ("swiglu", "swiglu_grad"):
        gate, up = s["gu"].to(d).split(case["width"], 1)
        sig = torch.sigmoid(gate)
        if op == "swiglu":
            q, scale = _exact_quantize(gate * sig * up, case["fmt"])
            return {"q": q, "scale": scale}
        dy = s["dy"].to(d)
        return {"dgu": torch.cat([dy * up * (sig + gate * sig * torch.sigmoid(-gate)),
                                  dy * gate * sig], 1)}
    if op == "dispatch":
        ids = s["ids"].reshape(-1).tolist()
        lists = [[] for _ in range(case["experts"])]
        rest = []
        for i, e in enumerate(ids):
            (lists[e] if 0 <= e < case["experts"] else rest).append(i)
        order = [i for one in lists for i in one]
        token = torch.tensor(order, dtype=torch.int64, device="cuda") // case["top"]
        pad = torch.zeros((len(rest), case["width"]), dtype=torch.float32, device="cuda")
        xs = torch.cat([s["x"].view(F8[case["fmt"]])[token].float(), pad]).to(d)
        scale = torch.exp2(s["x_scale"][token].to(d) - 127)
        low = torch.full((len(rest), case["width"] // 32), 2.0 ** -127, dtype=d, device="cuda")
        return {"group_rows": None, "row_of": None, "x": xs, "scale": torch.cat([scale, low])}
    if op == "combine":
        live = s["row_of"] >= 0
        out = s["res"].to(d)
        for j in range(case["top"]):
            rows = s["y"].to(d)[s["row_of"][:, j].clamp(min=0).long()]
            out = out + rows * torch.where(live[:, j], s["weights"][:, j].to(d), 0)[:, None]
        return {"out": out}
    if op == "combine_grad":
        dout = s["dout"].to(d)
        dy = torch.zeros(s["y"].shape, dtype=d, device="cuda")
        dw = torch.zeros(s["weights"].shape, dtype=d, device="cuda")
        for j in range(case["top"]):
            at = torch.nonzero(s["row_of"][:, j] >= 0).view(-1)
            rows = s["row_of"][at, j].long()
            dy[rows] = dout[at] * s["weights"][at, j].to(d)[:, None]
            dw[at, j] = (dout[at] * s["y"][rows].to(d)).sum(-1)
        return {"dy": dy, "dw": dw}

    def values(q, scale, fmt):
        if fmt == "bf16":
            return q.to(d)
        if fmt == "e2m1":
            code = torch.stack([q & 15, q >> 4], -1).view(q.shape[0], -1).int()
            mag, e = (code & 1).to(d), (code >> 1) & 3
            v = torch.where(e == 0, mag * 0.5, (1 + mag * 0.5) * torch.exp2((e - 1).to(d)))
            v = torch.where((code & 8) != 0, -v, v)
        else:
            v = q.view(F8[fmt]).to(d)
        return v * torch.exp2(scale.to(d) - 127).repeat_interleave(32, 1)

    c = values(s["a"], s["a_scale"], case["fmt_a"]) @ \
        values(s["b"], s["b_scale"], case["fmt_b"]).T.contiguous()
    if s["bias_v"] is not None:
        c = c + s["bias_v"].to(d)
    if case["act"] == "relu":
        c = c.clamp(min=0)
    elif case["act"] == "silu":
        c = c * torch.sigmoid(c)
    elif case["act"] == "gelu":
        c = c * torch.special.ndtr(c)
    elif case["act"] == "gelu_tanh":
        c = c * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (c + 0.044715 * c ** 3))
    if s["res"] is not None:
        c = c + s["res"].to(d)
    return {"c": c}
