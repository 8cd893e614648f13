"""Steps that forget the state (g <= -128) in front of steps whose decay is
above 1: nothing from before the reset comes back, in the scan, in its reverse
pass and token by token.  The steps behind a reset write nothing (k = 0) and
grow by exp(20) each, exp(80) in all, so that what should be gone would show:
their outputs are exactly 0, within the 1e-30 that every bound allows."""
import math

import pytest
import torch

from tests import dense_oracle as O
from tests.test_gpu_linear import (BF16, F32, ORDER, check_forward, check_reverse, dev, forward_bounds,
                                   make, run_scan, run_train)

pytestmark = pytest.mark.gpu

KINDS = [-128.0, -200.0, -1e30, -math.inf]


def growing(a, at, kind):
    """Step `at` forgets; four steps grow, then one takes the growth back."""
    a["g"][:, :, at] = kind
    a["g"][:, :, at + 1:at + 5] = 20.0
    a["g"][:, :, at + 5] = -80.0
    a["k"][:, :, at:at + 5] = 0
    # gradients that would have to come through these steps stay in range
    a["q"][:, :, at:at + 5] = a["q"][:, :, at:at + 5].sign()
    return a


def meant(a):
    """The same with every reset written as -infinity: exp(-128) is 0 here."""
    return dict(a, g=torch.where(a["g"] <= -128, -math.inf, a["g"]))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kind", KINDS)
def test_scan_of_growth_behind_a_reset(kind, dtype):
    a = make(1, 2, 1, 150, 32, 64, dtype, seed=60)
    for at in (3, 29, 60, 70, 126, 140):
        growing(a, at, kind)
    out, S = run_scan(a)
    assert not out[:, :, 3:8].any() and not out[:, :, 140:145].any()
    check_forward(meant(a), out, S)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [40, 150, 600])
def test_backward_of_growth_behind_a_reset(T, dtype):
    a = make(1, 2, 2, T, 64, 32, dtype, seed=61, grads=True)
    for at in range(2, T - 10, 23):
        growing(a, at, -math.inf)
    out, S, _, grads, G = run_train(a)
    check_forward(meant(a), out, S)
    check_reverse(meant(a), grads, G)
    assert not grads["dg"][:, :, 2].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [20, 600])
def test_growth_without_a_reset(T, dtype):
    """Decays above 1, their products over any stretch in range."""
    a = make(1, 2, 1, T, 32, 32, dtype, seed=62, grads=True)
    for at in range(4, T - 10, 17):
        a["g"][:, :, at:at + 4] = 2.0
        a["g"][:, :, at + 4] = -8.0
    out, S, _, grads, G = run_train(a)
    check_forward(meant(a), out, S)
    check_reverse(meant(a), grads, G)


@pytest.mark.parametrize("kind", KINDS)
def test_steps_of_growth_behind_a_reset(kind):
    import sparse_memory_linear_sdm_amd as sdm

    a = growing(make(2, 2, 1, 8, 32, 32, F32, seed=63), 2, kind)
    d = dev(a)
    outs = [sdm.linear_step(d["S"], *(d[n][:, :, t].contiguous() for n in ORDER[1:])) for t in range(8)]
    a = meant(a)
    want, _, S, slim, _ = forward_bounds(a)
    size = O.sizes_forward(*(a[n] for n in ORDER))[0]
    O.check("out", torch.stack(outs, 2), want, O.bound(size, F32, O.terms(a["q"], a["v"])))
    O.check("S", d["S"], S, slim)
