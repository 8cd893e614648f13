"""The bounds of tests/test_gpu_dense_precision.py tell a state of fp32's
precision from one of fewer bits: the same results computed here with three and
with two bf16 parts, and with sums of logarithms kept as two floats and as one."""
import pytest
import torch

from tests import dense_oracle as O
from tests import dense_precision as P


@pytest.mark.parametrize("dk,dv,seed", [(32, 32, 1), (64, 64, 2), (128, 128, 3)])
def test_two_parts_of_a_scaled_operand_are_seen(dk, dv, seed):
    a = P.one_row_each(64, dk, dv, P.BF16, seed)
    want = O.linear_forward(*(a[n] for n in ("S", "q", "k", "v", "g")))[1]
    off = {n: P.off_in_half_steps(P.scaled_rows(a, n), want, want.abs()) for n in (2, 3)}
    assert off[3] <= P.HALF_STEPS and off[2] > 4 * P.HALF_STEPS, off


@pytest.mark.parametrize("state", ["S", "G"])
def test_two_parts_of_a_state_are_seen(state):
    """What a state of two parts would be off by, where dg stands on one element."""
    a = P.one_path_through(state, 8, 64, 64, P.BF16, 4)
    S = a[state]
    off = {n: P.off_in_half_steps(P.bf16_parts(S, n), S.double(), S.double().abs()) for n in (2, 3)}
    assert off[3] <= 1 and off[2] > 4 * (P.HALF_STEPS + 8), off


@pytest.mark.parametrize("reset", [-1024.0, -184.6649652337873])
@pytest.mark.parametrize("T,first", [(32, 20), (64, 20), (64, 44)])
def test_sums_of_logarithms_in_one_float_are_seen(reset, T, first):
    a = P.many_resets(T, first, P.F32, T + first)
    want = O.linear_forward(*(a[n] for n in ("S", "q", "k", "v", "g")))[0][:, :, first:]
    off = {n: P.off_in_half_steps(P.decayed_values(a, first, reset, n)[:, :, first:], want, want.abs())
           for n in (1, 2)}
    assert off[2] <= P.HALF_STEPS and off[1] > 20 * P.HALF_STEPS, off
