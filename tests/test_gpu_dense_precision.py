"""The state, its gradient, the tape and the decays' gradient hold fp32's
precision for both types: results that stand on one product or on few, in half
steps of fp32 (tests/dense_precision.py; tests/test_dense_precision.py shows
that fewer bits exceed these bounds)."""
import pytest
import torch

from tests import dense_oracle as O
from tests import dense_precision as P
from tests.test_gpu_linear import BF16, F32, ORDER, run_scan, run_train

pytestmark = pytest.mark.gpu

HEADS = [(32, 32), (64, 32), (64, 64), (32, 128), (128, 64), (128, 128)]


def at_most(name, got, want, size, half_steps):
    off = P.off_in_half_steps(got, want, size)
    assert off <= half_steps, f"{name}: {off} half steps, {half_steps} allowed"


def reverse(a):
    args = [a[n] for n in ORDER] + [a["dout"], a["G"]]
    return O.linear_reverse(*args), O.sizes_reverse(*args)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", HEADS)
def test_states_of_one_chunk(dk, dv, dtype):
    a = P.one_row_each(64 if dtype == BF16 else 32, dk, dv, dtype, dk + dv)
    _, S, _, _, G = run_train(a)
    want = O.linear_forward(*(a[n] for n in ORDER))[1]
    at_most("S", S, want, want.abs(), P.HALF_STEPS)
    want, _ = reverse(a)
    at_most("G", G, want["G"], want["G"].abs(), P.HALF_STEPS)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [100, 190])
def test_states_of_chunks_and_the_tape(T, dtype):
    a = P.one_row_each(T, 64, 64, dtype, T)
    chunk = 64 if dtype == BF16 else 32
    _, S, tape, _, G = run_train(a)
    _, want, before = O.linear_forward(*(a[n] for n in ORDER))
    hops = -(-T // chunk)
    at_most("S", S, want, want.abs(), P.HALF_STEPS + 4 * hops)
    for c in range(1, hops):
        at_most(f"tape {c}", tape[:, :, c], before[c * chunk], before[c * chunk].abs(), P.HALF_STEPS + 4 * c)
    want, _ = reverse(a)
    at_most("G", G, want["G"], want["G"].abs(), P.HALF_STEPS + 4 * hops)


@pytest.mark.parametrize("dtype,T", [(F32, 300), (BF16, 600), (BF16, 1500)])
def test_states_of_segments(T, dtype):
    import sparse_memory_linear_sdm_amd as sdm

    assert sdm.lib().sdm_linear_scan_workspace_size(int(dtype == BF16), 1, 2, 64, 64, T) > 0
    writes = [3 + (T - 7) * i // 64 for i in range(64)]
    a = P.one_row_each(T, 64, 64, dtype, T, writes=writes)
    hops = -(-T // (64 if dtype == BF16 else 32))
    _, S, tape, _, G = run_train(a)
    want = O.linear_forward(*(a[n] for n in ORDER))[1]
    at_most("S", S, want, want.abs(), P.HALF_STEPS + 4 * hops)
    want, _ = reverse(a)
    at_most("G", G, want["G"], want["G"].abs(), P.HALF_STEPS + 4 * hops)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("state", ["S", "G"])
@pytest.mark.parametrize("dk,dv", HEADS)
def test_decays_gradients_through_one_element(dk, dv, state, dtype):
    """Eight paths at most, each through one element of the state."""
    a = P.one_path_through(state, 8, dk, dv, dtype, dk - dv + 200)
    _, _, _, grads, _ = run_train(a)
    want, size = reverse(a)
    at_most("dg", grads["dg"], want["dg"], size["dg"], P.HALF_STEPS + 8)


@pytest.mark.parametrize("T,first", [(32, 20), (64, 20), (64, 44), (150, 120)])
def test_decays_behind_many_resets(T, first):
    a = P.many_resets(T, first, F32, T + first)
    out, S = run_scan(a)
    want = O.linear_forward(*(a[n] for n in ORDER))[0]
    assert not out[:, :, :first].any()
    at_most("out", out, want, want.abs(), P.HALF_STEPS + 8)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,first", [(32, 20), (64, 20), (64, 44)])
def test_gradients_of_decays_behind_many_resets(T, first, dtype):
    """One path: from the key's step to the last one."""
    a = P.many_resets(T, first, dtype, T + first)
    a["v"].zero_()
    a["dout"].zero_()
    a["v"][:, :, first, 5] = 1
    a["dout"][:, :, -1, 5] = 1
    _, _, _, grads, _ = run_train(a)
    want, size = reverse(a)
    assert (want["dg"][:, :, first + 1:] != 0).all()
    at_most("dg", grads["dg"], want["dg"], size["dg"], P.HALF_STEPS + 8)
