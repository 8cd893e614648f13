"""The dense recurrence keeps a tape only where its reverse pass takes one: both
refuse the same sizes, the forward before any work."""
import pytest

import sparse_memory_linear_sdm_amd as sdm

FAKE = 1 << 20  # a non-null, aligned address that is never dereferenced
MOST = (1 << 26) - 4


def _scan(B, H, T, tape, out):
    status = sdm.lib().sdm_linear_scan(FAKE, 1, B, H, H, 32, 32, T, FAKE, FAKE, FAKE, FAKE, out, tape,
                                       FAKE, 1 << 50, None)
    return status, sdm.lib().sdm_last_error().decode()


def _backward(B, H, T, dg):
    status = sdm.lib().sdm_linear_backward(1, B, H, H, 32, 32, T, *[FAKE] * 10, dg, FAKE, 1 << 50, None)
    return status, sdm.lib().sdm_last_error().decode()


@pytest.mark.parametrize("B,H,T", [(1, 1, MOST + 1), (64, 1, 1 << 20), (1, 2, MOST // 2 + 1),
                                   (1 << 10, 1 << 10, 64)])
def test_a_tape_that_no_call_takes_is_not_made(B, H, T):
    assert _scan(B, H, T, FAKE, FAKE) == (2, _backward(B, H, T, FAKE)[1])
    assert "2^26 - 4" in sdm.lib().sdm_last_error().decode()
    # without a tape the scan goes on to its next argument
    status, message = _scan(B, H, T, None, None)
    assert status == 1 and "out is NULL" in message


@pytest.mark.parametrize("B,H,T", [(1, 1, MOST), (2, 1, MOST // 2), (4, 4, MOST // 16)])
def test_the_largest_tape_is_taken(B, H, T):
    status, message = _scan(B, H, T, FAKE, None)
    assert status == 1 and "out is NULL" in message
    status, message = _backward(B, H, T, None)
    assert status == 1 and "dg is NULL" in message
