"""How near the dense recurrence's results come to its 64-bit form, where the
bounds of tests/test_gpu_linear.py would let fewer bits pass.

bf16 outputs and gradients are sums in fp32, rounded once: half a step, 2^-8 of
the value.  What fp32 holds (the state, its gradient, products of steps) enters
them with two bf16 parts, off by half a step of the second at most, 2^-16 of
the magnitudes that are summed; the sums by n * 2^-24 of them."""
import pytest
import torch

from tests import dense_oracle as O
from tests.test_gpu_linear import BF16, ORDER, make, run_scan, run_train

pytestmark = pytest.mark.gpu

HEADS = [(32, 32), (64, 64), (128, 128), (32, 128), (128, 64)]


def rounded_once(want, size, n):
    """The bound of a bf16 output: `want` with sums of n terms of size `size`."""
    return want.abs() * 2.0 ** -8 + size * (2.0 ** -16 + n * O.U32) * (1 + 2.0 ** -8) + 1e-30


@pytest.mark.parametrize("dk,dv", HEADS)
@pytest.mark.parametrize("T", [1, 33, 101])
def test_outputs_are_rounded_once(T, dk, dv):
    a = make(2, 2, 1, T, dk, dv, BF16, seed=40 + T + dk, resets=True)
    out, _ = run_scan(a)
    want = O.linear_forward(*(a[n] for n in ORDER))[0]
    size = O.sizes_forward(*(a[n] for n in ORDER))[0]
    O.check("out", out, want, rounded_once(want, size, O.terms(a["q"], a["v"])))


def test_outputs_behind_segments_are_rounded_once():
    a = make(1, 2, 2, 600, 64, 64, BF16, seed=41)
    out, _ = run_scan(a)
    want = O.linear_forward(*(a[n] for n in ORDER))[0]
    size = O.sizes_forward(*(a[n] for n in ORDER))[0]
    O.check("out", out, want, rounded_once(want, size, O.terms(a["q"], a["v"])))


@pytest.mark.parametrize("dk,dv", HEADS)
@pytest.mark.parametrize("T", [1, 33, 101])
def test_gradients_are_rounded_once(T, dk, dv):
    a = make(2, 2, 2, T, dk, dv, BF16, seed=50 + T + dv, resets=True, grads=True)
    _, _, _, grads, _ = run_train(a)
    args = [a[n] for n in ORDER] + [a["dout"], a["G"]]
    want, size = O.linear_reverse(*args), O.sizes_reverse(*args)
    for name in ("dq", "dk", "dv"):
        O.check(name, grads[name], want[name],
                rounded_once(want[name], size[name], O.terms(a["q"], a["v"])))


@pytest.mark.parametrize("T", [70, 600])
def test_gradients_of_shared_keys_are_rounded_once(T):
    a = make(1, 4, 2, T, 64, 64, BF16, seed=52, grads=True)
    _, _, _, grads, _ = run_train(a)
    args = [a[n] for n in ORDER] + [a["dout"], a["G"]]
    want, size = O.linear_reverse(*args), O.sizes_reverse(*args)
    for name in ("dq", "dk", "dv"):
        O.check(name, grads[name], want[name],
                rounded_once(want[name], size[name], O.terms(a["q"], a["v"]) + 4))
