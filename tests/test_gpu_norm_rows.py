"""A row's values do not depend on how many rows the call has, bit for bit:
short calls give a long row one vector of 8 values a thread, others two."""
import pytest
import torch

from tests.test_gpu_norm import BF16, F32, dev, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [128, 520, 1000, 1032, 4096, 5128, 8192, 8200])
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("gate", [False, True])
def test_a_row_alone_and_among_others(d, gate, dtype, out_dtype):
    import sparse_memory_linear_sdm_amd as sdm

    a = dev(make((700, d), dtype, out_dtype, False, d + 1, gate=gate))
    out, behind = sdm.norm(a["y"], a["w"], z=a["z"], x=a["x"], scale=0.5, next_w=a["next_w"])
    plain = sdm.norm(a["y"], a["w"])
    for lo, hi in ((0, 1), (3, 40), (188, 700)):
        part = {n: None if x is None else x[lo:hi].contiguous() for n, x in a.items() if n not in ("w", "next_w")}
        o, n = sdm.norm(part["y"], a["w"], z=part["z"], x=part["x"], scale=0.5, next_w=a["next_w"])
        assert torch.equal(o, out[lo:hi]) and torch.equal(n, behind[lo:hi])
        assert torch.equal(sdm.norm(part["y"], a["w"]), plain[lo:hi])
    grads = sdm.norm_backward(a["dout"], a["y"], a["w"], z=a["z"], skip=a["skip"])
    few = {n: None if x is None else x[5:9].contiguous() for n, x in a.items() if n not in ("w", "next_w")}
    got = sdm.norm_backward(few["dout"], few["y"], a["w"], z=few["z"], skip=few["skip"])
    for n in got:
        if n != "dw":
            assert torch.equal(got[n], grads[n][5:9]), n
