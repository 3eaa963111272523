"""The example block end to end: serving against a float32 model of the same
quantized values, training gradients against autograd in float32."""
import os
import sys

import pytest

import microscaled_block_scaled_amd as mxg
from gpu_util import log

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def _rel(a, b):
    return ((a.float() - b.float()).norm() / b.float().norm()).item()


def _dequant(q, s, fmt):
    import torch
    if fmt == mxg.FMT_E2M1:
        m = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=q.device)
        lut = torch.cat([m, -m])
        v = torch.stack([lut[(q & 15).long()], lut[(q >> 4).long()]], -1).view(q.shape[0], -1)
    else:
        v = q.view(torch.float8_e4m3fn).float()
    return v * torch.exp2(s.float() - 127).repeat_interleave(32, 1)


@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_serve(tokens):
    """Each stage's output is within BF16 and E4M3 rounding of float32: 8-bit
    rows 2^-4 relative per value and 4 stages of them, so 0.1 overall."""
    import torch
    import moe_block as mb
    hidden, ffn, experts, top = 512, 768, 8, 2
    log("moe block serving %d tokens" % tokens)
    w = mb.make_weights(hidden, ffn, experts, seed=tokens)
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    x, r = (torch.randn((tokens, hidden), device="cuda", generator=g).to(torch.bfloat16)
            for _ in range(2))
    out = mb.serve(x, r, w, top)
    h = (x.float() + r.float()).to(torch.bfloat16).float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + mb.EPS) * w["norm"]
    logits = y.to(torch.bfloat16).float() @ w["router"].float().t() + w["router_bias"]
    ids, weights = mb.route(logits, top)
    dq = {k: _dequant(w[k + "_q"], w[k + "_s"], mxg.FMT_E2M1)
          for k in ("up", "down", "shared_up", "shared_down")}

    def mlp(v, up, down):
        a, b = (v @ up.t()).chunk(2, 1)
        return (torch.nn.functional.silu(a) * b) @ down.t()

    want = h + mlp(y, dq["shared_up"], dq["shared_down"]) + w["shared_bias"]
    up, down = dq["up"].view(experts, 2 * ffn, hidden), dq["down"].view(experts, hidden, ffn)
    for e in range(experts):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t):
            want.index_add_(0, t, mlp(y[t], up[e], down[e]) * weights[t, j][:, None])
    assert torch.isfinite(out).all()
    assert _rel(out, want) < 0.1


def test_train_gradients_match_autograd():
    """Against float32 autograd of the same block; BF16 activations and
    gradients of 6 stages, 2^-8 each: 0.03 in the 2-norm."""
    import torch
    import moe_block as mb
    tokens, hidden, ffn, experts, top = 200, 256, 384, 6, 3
    log("moe block training gradients")
    w = mb.make_weights(hidden, ffn, experts, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x, r, dout = (torch.randn((tokens, hidden), device="cuda", generator=g).to(torch.bfloat16)
                  for _ in range(3))
    ids, weights = mb.route(torch.randn((tokens, experts), device="cuda", generator=g), top)
    ids[::9] = -1                                      # padding tokens
    out, got = mb.train(x, r, w, ids, weights, dout)

    leaf = {"x": x.float(), "weights": weights.clone(), "norm": w["norm"].clone(),
            "up": w["up"].float(), "down": w["down"].float()}
    for v in leaf.values():
        v.requires_grad_(True)
    h = leaf["x"] + r.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + mb.EPS) * leaf["norm"]
    want = h
    for e in range(experts):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        a, b = (y[t] @ leaf["up"][e].t()).chunk(2, 1)
        rows = (torch.nn.functional.silu(a) * b) @ leaf["down"][e].t()
        want = want.index_add(0, t, rows * leaf["weights"][t, j][:, None])
    want.backward(dout.float())
    assert _rel(out, want) < 0.03
    for name, v in leaf.items():
        err = _rel(got[name], v.grad)
        log("  gradient of %s: %.4f" % (name, err))
        assert err < 0.03, name
