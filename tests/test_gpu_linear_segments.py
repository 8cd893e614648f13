"""Heads of 64 x 64 and more are cut into segments from five chunks on, where
there are at most 64 memories (four segments of each or more)."""
import pytest

from tests.test_gpu_linear import BF16, F32, check_forward, check_reverse, make, run_scan, run_train

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (32, 128), (128, 32)])
@pytest.mark.parametrize("H,chunks", [(3, 4), (3, 5), (65, 5)])
def test_heads_of_few_chunks(H, chunks, dk, dv, dtype):
    import sparse_memory_linear_sdm_amd as sdm

    T = (64 if dtype == BF16 else 32) * chunks - 7
    need = sdm.lib().sdm_linear_scan_workspace_size(int(dtype == BF16), 1, H, dk, dv, T)
    assert (need > 0) == (H <= 64 and chunks >= 5)
    a = make(1, H, H, T, dk, dv, dtype, seed=T + dk, resets=True, grads=H == 3)
    if H == 3:
        out, S, _, grads, G = run_train(a)
        check_reverse(a, grads, G)
    else:
        out, S = run_scan(a)
    check_forward(a, out, S)
