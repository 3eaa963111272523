"""A mixture-of-experts block from the library's operators, as a model runs it.

    python examples/moe_block.py [--tokens 256] [--hidden 1024] [--ffn 2048]
                                 [--experts 8] [--top 2]

serve() is one inference pass: residual and norm to 8-bit rows in one kernel,
router logits, tokens sorted by expert and gathered, two grouped products with
4-bit weights around the gated activation, the rows combined back onto the
residual stream, and a dense shared expert whose second product adds its
result to that stream in its epilogue.

train() is the forward and backward pass of the routed part with BF16 experts
(no shared expert, no 8-bit rounding): the library's gradients of the
combination, the gated activation, the gather and the norm, and torch's
products where a gradient needs an operand transposed, which the library's
A * B^T does not take.
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import microscaled_block_scaled_amd as mxg  # noqa: E402

EPS = 1e-5


def make_weights(hidden, ffn, experts, seed=0):
    """Random weights: BF16, and the same quantized to MXFP4 for serving."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, device="cuda", generator=g)

    w = {"norm": 1 + 0.1 * rand(hidden),
         "router": (rand(experts, hidden) / hidden ** 0.5).to(torch.bfloat16),
         "router_bias": 0.1 * rand(experts),
         "up": (rand(experts, 2 * ffn, hidden) / hidden ** 0.5).to(torch.bfloat16),
         "down": (rand(experts, hidden, ffn) / ffn ** 0.5).to(torch.bfloat16),
         "shared_up": (rand(2 * ffn, hidden) / hidden ** 0.5).to(torch.bfloat16),
         "shared_down": (rand(hidden, ffn) / ffn ** 0.5).to(torch.bfloat16),
         "shared_bias": 0.1 * rand(hidden)}
    for name in ("up", "down", "shared_up", "shared_down"):
        rows = w[name].reshape(-1, w[name].shape[-1])
        w[name + "_q"], w[name + "_s"] = mxg.mx_quantize(rows, mxg.FMT_E2M1)
    return w


def route(logits, top):
    """Expert ids and weights of each token."""
    value, ids = torch.topk(logits, top, dim=-1)
    return ids.contiguous(), torch.softmax(value, -1).contiguous()


def serve(x, residual, w, top):
    """The block's output, the new residual stream, for tokens x."""
    a, b = mxg.FMT_E4M3, mxg.FMT_E2M1
    o = mxg.mx_rmsnorm_quantize(x, w["norm"], a, residual=residual, eps=EPS, need_y=True)
    logits = mxg.mx_gemm_bf16_fused(o.y, w["router"], bias=w["router_bias"],
                                    out_dtype=torch.float32)
    ids, weights = route(logits, top)
    plan = mxg.mx_moe_sort(ids, w["router"].shape[0])
    xs, xs_scale = mxg.mx_moe_gather(plan, o.q, o.q_scale)
    rows = plan.group_rows.tolist()               # the grouped products take host counts
    gu = mxg.mx_gemm_grouped(xs, xs_scale, w["up_q"], w["up_s"], rows, a, fmt_b=b)
    q, s = mxg.mx_swiglu_quantize(gu, a)
    y = mxg.mx_gemm_grouped(q, s, w["down_q"], w["down_s"], rows, a, fmt_b=b)
    out = mxg.mx_moe_combine(plan, y, weights, residual=o.h)
    gu = mxg.mx_gemm_fused(o.q, o.q_scale, w["shared_up_q"], w["shared_up_s"], a, fmt_b=b)
    q, s = mxg.mx_swiglu_quantize(gu, a)
    return mxg.mx_gemm_fused(q, s, w["shared_down_q"], w["shared_down_s"], a, fmt_b=b,
                             bias=w["shared_bias"], residual=out, out=out)


def train(x, residual, w, ids, weights, dout):
    """(out, gradients) of the routed part for given routing: gradients of x
    (and the residual), of the routing weights, and of norm, up and down."""
    experts = w["router"].shape[0]
    o = mxg.mx_rmsnorm_quantize(x, w["norm"], None, residual=residual, eps=EPS, need_y=True,
                                need_rstd=True)
    plan = mxg.mx_moe_sort(ids, experts)
    xs, _ = mxg.mx_moe_gather(plan, o.y)
    rows = plan.group_rows.tolist()
    n = sum(rows)
    xs = xs[:n]
    up, down = (w[k].view(-1, w[k].shape[-1]) for k in ("up", "down"))
    gu = mxg.mx_gemm_grouped_bf16(xs, up, rows)
    gate, lin = gu.float().chunk(2, 1)
    act = (torch.nn.functional.silu(gate) * lin).to(torch.bfloat16)
    y = mxg.mx_gemm_grouped_bf16(act, down, rows)
    out = mxg.mx_moe_combine(plan, y, weights, residual=o.h)

    dy, dweights = mxg.mx_moe_combine_backward(plan, dout, y, weights)
    dact, dxs = torch.empty_like(act), torch.empty_like(xs)
    d_up, d_down = torch.zeros_like(w["up"]), torch.zeros_like(w["down"])
    at = [0]
    for r in rows:
        at.append(at[-1] + r)
    for e in range(experts):
        r = slice(at[e], at[e + 1])
        dact[r] = dy[r] @ w["down"][e]
        d_down[e] = dy[r].t() @ act[r]
    dgu = mxg.mx_swiglu_backward(dact, gu)
    for e in range(experts):
        r = slice(at[e], at[e + 1])
        dxs[r] = dgu[r] @ w["up"][e]
        d_up[e] = dgu[r].t() @ xs[r]
    # the gather's gradient: a token's rows back, each once
    dnormed = mxg.mx_moe_combine(plan, dxs)
    # dout reaches h directly too, through the combination's residual
    dx, d_norm = mxg.mx_rmsnorm_backward(dnormed, o.h, o.rstd, w["norm"], dh=dout)
    return out, {"x": dx, "weights": dweights, "norm": d_norm, "up": d_up, "down": d_down}


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 256), ("hidden", 1024), ("ffn", 2048), ("experts", 8),
                          ("top", 2)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    w = make_weights(a.hidden, a.ffn, a.experts)
    x, r, dout = (torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
                  for _ in range(3))
    out = serve(x, r, w, a.top)
    ids, weights = route(torch.randn((a.tokens, a.experts), device="cuda"), a.top)
    _, grads = train(x, r, w, ids, weights, dout * 0.01)
    torch.cuda.synchronize()
    print("served %s, rms %.3f" % (tuple(out.shape), out.float().square().mean().sqrt().item()))
    for name, g in grads.items():
        print("gradient of %-8s %-18s rms %.3g" % (name, tuple(g.shape),
                                                 g.float().square().mean().sqrt().item()))


if __name__ == "__main__":
    main()
