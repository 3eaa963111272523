"""Plain 64-bit references of the operators between two products of a
transformer block, and the rounding units of their tolerances."""
import math

import numpy as np

U32 = 2.0 ** -24          # FP32 unit roundoff
UBF = 2.0 ** -8           # BF16, 8 significant bits: half of the spacing 2^-7 of [1, 2)


def norm(h, w, eps):
    """(y, rstd) of the RMS norm of the rows of h."""
    rstd = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h * rstd[:, None] * w, rstd


def norm_grad(dy, h, w, eps, dh=None):
    """(dx, dw, |dx| terms, |dw| terms): the gradient and the sums of the
    magnitudes of its terms, which its rounding errors scale with."""
    rstd = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    xhat = h * rstd
    g = dy * w
    dx = rstd * (g - xhat * (g * xhat).mean(-1, keepdims=True))
    mag = rstd * (abs(g) + abs(xhat) * abs(g * xhat).mean(-1, keepdims=True))
    if dh is not None:
        dx, mag = dx + dh, mag + abs(dh)
    return dx, (dy * xhat).sum(0), mag, abs(dy * xhat).sum(0)


def sigmoid(x):
    return np.where(x >= 0, 1 / (1 + np.exp(-abs(x))), np.exp(-abs(x)) / (1 + np.exp(-abs(x))))


def swiglu(gu):
    g, u = np.split(gu, 2, 1)
    return g * sigmoid(g) * u


def swiglu_grad(dy, gu):
    g, u = np.split(gu, 2, 1)
    s = sigmoid(g)
    return np.concatenate([dy * u * s * (1 + g * (1 - s)), dy * g * s], 1)


def sort(ids, experts):
    """(group_rows, row_of) of the stable sort of the pairs by expert."""
    flat = [int(i) for i in np.asarray(ids).reshape(-1)]
    lists = [[] for _ in range(experts + 1)]
    for i, e in enumerate(flat):
        lists[e if 0 <= e < experts else experts].append(i)
    row_of = np.empty(len(flat), np.int64)
    at = 0
    for e, one in enumerate(lists):
        for i in one:
            row_of[i] = at if e < experts else -1 - at
            at += 1
    return (np.array([len(one) for one in lists[:experts]], np.int64),
            row_of.reshape(np.asarray(ids).shape))


def gather(row_of, x):
    out = np.zeros((row_of.size,) + x.shape[1:], x.dtype)
    for t in range(row_of.shape[0]):
        for r in row_of[t]:
            if r >= 0:
                out[r] = x[t]
    return out


def combine(row_of, y, w=None, res=None):
    """(out, sum of the magnitudes of its terms)."""
    tokens, top = row_of.shape
    out = np.zeros((tokens, y.shape[1])) if res is None else res.astype(np.float64).copy()
    mag = abs(out)
    for t in range(tokens):
        for j in range(top):
            r = row_of[t, j]
            if 0 <= r < y.shape[0]:
                term = y[r] * (1.0 if w is None else w[t, j])
                out[t] += term
                mag[t] += abs(term)
    return out, mag


def combine_grad(row_of, dout, y, w):
    """(dy, dw, magnitudes of dw's terms)."""
    dy, dw, mag = np.zeros(y.shape), np.zeros(row_of.shape), np.zeros(row_of.shape)
    for t in range(row_of.shape[0]):
        for j in range(row_of.shape[1]):
            r = row_of[t, j]
            if 0 <= r < y.shape[0]:
                dy[r] = w[t, j] * dout[t]
                dw[t, j] = (dout[t] * y[r]).sum()
                mag[t, j] = abs(dout[t] * y[r]).sum()
    return dy, dw, mag


ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def act(v, name):
    if name == "relu":
        return np.maximum(v, 0)
    if name == "silu":
        return v * sigmoid(v)
    if name == "gelu":
        return 0.5 * v * (1 + np.vectorize(math.erf)(v / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v
