"""Every combination of a norm's optional arrays, the next block's norm where
the output takes the residual's place, and heads that are one."""
import pytest
import torch

from tests import dense_oracle as O
from tests.test_gpu_norm import BF16, F32, check_forward, dev, make

pytestmark = pytest.mark.gpu


def next_bounds(a, want, size, d, dtype):
    """The next norm of `want`, as in tests/test_gpu_norm.py: a relative error of
    out's size moves its root by as much at most, twice."""
    root = 1 / (want.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    n = want * root
    ratio = size.square().mean(-1, keepdim=True).sqrt() * root
    off = (size * root + n.abs() * ratio * 2) * a["next_w"].abs() * (d + 40) * O.U32
    return n * a["next_w"], off + (n * a["next_w"]).abs() * O.HALF[dtype] + 1e-30


@pytest.mark.parametrize("d", [64, 520, 8200])
@pytest.mark.parametrize("gate,residual", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF16, BF16), (F32, BF16)])
def test_next_with_and_without_the_others(d, gate, residual, dtype, out_dtype):
    import sparse_memory_linear_sdm_amd as sdm

    a = make((37, d), dtype, out_dtype, False, d + gate, gate=gate, residual=residual)
    g = dev(a)
    got, behind = sdm.norm(g["y"], g["w"], z=g["z"], x=g["x"], scale=-0.7, next_w=g["next_w"], dtype=out_dtype)
    want, size = check_forward(a, got, False, -0.7, d)
    O.check("next", behind, *next_bounds(a, want, size, d, out_dtype))
    alone = sdm.norm(g["y"], g["w"], z=g["z"], x=g["x"], scale=-0.7, dtype=out_dtype)
    assert torch.equal(alone, got)
    if residual:
        x, n = g["x"].clone(), torch.empty_like(g["x"])
        sdm.norm(g["y"], g["w"], z=g["z"], x=x, scale=-0.7, next_w=g["next_w"], out=(x, n))
        assert torch.equal(x, got) and torch.equal(n, behind)


@pytest.mark.parametrize("shape", [(2, 1, 9, 128), (1, 1, 1, 8)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_head_is_whole_rows(shape, dtype):
    import sparse_memory_linear_sdm_amd as sdm

    a = dev(make(shape, dtype, dtype, True, 9))
    rows = {n: None if x is None else x.reshape(-1, shape[-1]) if n in ("y", "skip") else x for n, x in a.items()}
    z = a["z"].reshape(-1, shape[-1])
    got = sdm.norm(a["y"], a["w"], z=a["z"], heads=True)
    assert got.shape == (shape[0], shape[2], shape[3])
    assert torch.equal(got.reshape(-1, shape[-1]), sdm.norm(rows["y"], a["w"], z=z))
    grads = sdm.norm_backward(a["dout"], a["y"], a["w"], z=a["z"], skip=a["skip"], heads=True)
    flat = sdm.norm_backward(a["dout"].reshape(-1, shape[-1]), rows["y"], a["w"], z=z, skip=rows["skip"])
    for n in grads:
        assert torch.equal(grads[n].reshape(flat[n].shape), flat[n])
