"""The 64-bit forms of tests/dense_oracle.py: the recurrence's and the norms'
gradients by their formulas against central differences of the forward."""
import math

import pytest
import torch

from tests import dense_oracle as O


def _difference(f, x, i, h=1e-5):
    """Central difference of f() by element i of x."""
    flat = x.view(-1)
    old = flat[i].item()
    flat[i] = old + h
    up = f()
    flat[i] = old - h
    down = f()
    flat[i] = old
    return (up - down) / (2 * h)


@pytest.mark.parametrize("reset", [False, True])
def test_linear_gradients_by_differences(reset):
    r = torch.Generator().manual_seed(1)
    randn = lambda *s: torch.randn(s, generator=r, dtype=torch.float64)  # noqa: E731
    B, H, Hk, T, dk, dv = 2, 4, 2, 6, 3, 5
    q, k, v = randn(B, Hk, T, dk), randn(B, Hk, T, dk), randn(B, H, T, dv)
    S, dout, G = randn(B, H, dk, dv), randn(B, H, T, dv), randn(B, H, dk, dv)
    g = -randn(B, H, T).abs()
    if reset:
        g[:, :, 3] = -math.inf

    def loss():
        out, end, _ = O.linear_forward(S, q, k, v, g)
        return float((out * dout).sum() + (end * G).sum())

    grads = O.linear_reverse(S, q, k, v, g, dout, G)
    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("G", S)):
        for i in range(0, x.numel(), 7):
            if name == "dg" and math.isinf(x.view(-1)[i]):
                assert grads["dg"].reshape(-1)[i] == 0
                continue
            want = _difference(loss, x, i)
            assert abs(grads[name].reshape(-1)[i].item() - want) < 1e-7 * (1 + abs(want)), name


@pytest.mark.parametrize("heads", [False, True])
@pytest.mark.parametrize("gate", [False, True])
def test_norm_gradients_by_differences(heads, gate):
    r = torch.Generator().manual_seed(2)
    randn = lambda *s: torch.randn(s, generator=r, dtype=torch.float64)  # noqa: E731
    y = randn(2, 3, 4, 8) if heads else randn(5, 8)
    shape = (2, 4, 24) if heads else (5, 8)
    w, z, dout = randn(8), randn(*shape) if gate else None, randn(*shape)
    skip = randn(*y.shape)

    def loss():
        out = O.norm_forward(y, w, z, scale=0.7, heads=heads)
        return float((out * dout).sum() + (skip * y).sum())

    grads = O.norm_reverse(dout, y, w, z, scale=0.7, skip=skip, heads=heads)
    for name, x in (("dy", y), ("dw", w), ("dz", z)):
        if x is None:
            continue
        for i in range(0, x.numel(), 5):
            want = _difference(loss, x, i)
            assert abs(grads[name].reshape(-1)[i].item() - want) < 1e-7 * (1 + abs(want)), name


def test_sizes_cover_the_values():
    r = torch.Generator().manual_seed(3)
    randn = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    a = (randn(1, 2, 4, 4), randn(1, 1, 9, 4), randn(1, 1, 9, 4), randn(1, 2, 9, 4),
         -randn(1, 2, 9).abs())
    more = (randn(1, 2, 9, 4), randn(1, 2, 4, 4))
    out, S, _ = O.linear_forward(*a)
    sout, sS, _ = O.sizes_forward(*a)
    assert (out.abs() <= sout * (1 + 1e-12)).all() and (S.abs() <= sS * (1 + 1e-12)).all()
    grads, sizes = O.linear_reverse(*a, *more), O.sizes_reverse(*a, *more)
    for n in grads:
        assert (grads[n].abs() <= sizes[n] * (1 + 1e-12)).all(), n
