"""The 64-bit references of tests/block_ref.py: gradients against central
differences, the sort against numpy, the activations at known values."""
import math

import numpy as np
import pytest

import block_ref as ref


def _difference(f, x, step=1e-5):
    """Gradient of the scalar f by central differences."""
    g = np.empty_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        at = it.multi_index
        old = x[at]
        x[at] = old + step
        up = f()
        x[at] = old - step
        down = f()
        x[at] = old
        g[at] = (up - down) / (2 * step)
    return g


# central differences with step 1e-5 of smooth functions of order 1: error
# step^2 times a third derivative of order 10, plus 2^-53 / step
TOL = 1e-8


@pytest.mark.parametrize("eps", [0.0, 1e-5, 0.5])
def test_norm_gradient_matches_differences(eps):
    rng = np.random.default_rng(1)
    h, dy, dh = (rng.standard_normal((3, 16)) for _ in range(3))
    w = rng.standard_normal(16)
    loss = lambda: (ref.norm(h, w, eps)[0] * dy).sum() + (h * dh).sum()  # noqa: E731
    dx, dw, _, _ = ref.norm_grad(dy, h, w, eps, dh)
    assert abs(_difference(loss, h) - dx).max() < TOL
    assert abs(_difference(loss, w) - dw).max() < TOL


def test_swiglu_gradient_matches_differences():
    rng = np.random.default_rng(2)
    gu, dy = rng.standard_normal((4, 12)) * 2, rng.standard_normal((4, 6))
    assert abs(_difference(lambda: (ref.swiglu(gu) * dy).sum(), gu)
               - ref.swiglu_grad(dy, gu)).max() < TOL


def test_combine_gradients_match_differences():
    rng = np.random.default_rng(3)
    ids = np.array([[0, 2], [2, -1], [-1, -1], [1, 0]])
    _, row_of = ref.sort(ids, 3)
    y, w = rng.standard_normal((8, 5)), rng.standard_normal((4, 2))
    dout = rng.standard_normal((4, 5))
    loss = lambda: (ref.combine(row_of, y, w)[0] * dout).sum()  # noqa: E731
    dy, dw, _ = ref.combine_grad(row_of, dout, y, w)
    assert abs(_difference(loss, y) - dy).max() < TOL
    assert abs(_difference(loss, w) - dw).max() < TOL
    # the gather's gradient is the combination without weights
    x = rng.standard_normal((4, 5))
    dxs = rng.standard_normal((8, 5))
    got = _difference(lambda: (ref.gather(row_of, x) * dxs).sum(), x)
    assert abs(got - ref.combine(row_of, dxs)[0]).max() < TOL


def test_sort_is_numpys_stable_sort():
    rng = np.random.default_rng(4)
    ids = rng.integers(-2, 9, (37, 3))
    rows, row_of = ref.sort(ids, 7)
    key = np.where((ids >= 0) & (ids < 7), ids, 7).reshape(-1)
    order = np.argsort(key, kind="stable")
    place = np.where(row_of >= 0, row_of, -1 - row_of).reshape(-1)
    assert (place[order] == np.arange(111)).all()
    assert (rows == np.bincount(key, minlength=8)[:7]).all()
    assert ((row_of.reshape(-1) < 0) == (key == 7)).all()


def test_activations_at_known_values():
    v = np.array([-1.0, 0.0, 1.0])
    assert (ref.act(v, "relu") == [0, 0, 1]).all() and (ref.act(v, "none") == v).all()
    assert np.allclose(ref.act(v, "silu"), [-1 / (1 + math.e), 0, 1 / (1 + 1 / math.e)])
    assert np.allclose(ref.act(v, "gelu"), [-0.15865525393, 0, 0.84134474607], atol=1e-10)
    assert np.allclose(ref.act(v, "gelu_tanh"), [-0.15880801, 0, 0.84119199], atol=1e-7)


def test_rounding_units():
    """The units of the tolerances: the largest relative error of rounding to
    FP32 and BF16, met just above a power of two."""
    import torch
    x = torch.tensor([1 + 2.0 ** -8 * 0.999], dtype=torch.float64)
    assert abs(x - x.to(torch.bfloat16).double()).item() > 0.99 * ref.UBF
    v = torch.linspace(1, 2, 100001, dtype=torch.float64)
    assert (abs(v - v.to(torch.bfloat16).double()) <= ref.UBF * v).all()
    assert (abs(v - v.float().double()) <= ref.U32 * v).all()
