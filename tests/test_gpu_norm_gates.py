"""Gates far from zero: silu(z) and its gradient keep fp32's precision relative
to themselves.  Of rows of 8 values: squares, their sum, mean and root (7
roundings, the ones under the root halved), quotient, product with the row, w,
the scale, z and the sigmoid (6); the sigmoid itself 1 + exp(-z) within 8
half steps; the gradient's own factors 4 more.  24 half steps cover both.  Below
2^-126 fp32 holds no more than absolute values."""
import pytest
import torch

from tests import dense_oracle as O

pytestmark = pytest.mark.gpu


def _inputs(lo, hi, seed):
    r = torch.Generator().manual_seed(seed)
    z = lo + (hi - lo) * torch.rand(4000, 8, generator=r)
    return torch.randn(4000, 8, generator=r), 1 + 0.2 * torch.randn(8, generator=r), z


@pytest.mark.parametrize("lo,hi", [(-86, -40), (-40, -10), (-10, 10), (10, 90), (-3000, -80)])
def test_far_gates(lo, hi):
    import sparse_memory_linear_sdm_amd as sdm

    y, w, z = _inputs(lo, hi, 70)
    got = sdm.norm(y.cuda(), w.cuda(), z=z.cuda())
    want = O.norm_forward(y, w, z)
    tiny = 200 * 2.0 ** -126
    O.check("out", got, want, want.abs() * 24 * O.U32 + tiny)
    dout = torch.randn(4000, 8, generator=torch.Generator().manual_seed(71))
    grads = sdm.norm_backward(dout.cuda(), y.cuda(), w.cuda(), z=z.cuda())
    want = O.norm_reverse(dout, y, w, z)["dz"]
    # 1 + z (1 - sigmoid) may cancel: its terms' magnitudes
    s = torch.sigmoid(z.double())
    n = y.double() / (y.double().square().mean(-1, keepdim=True) + 1e-6).sqrt()
    size = (dout.double() * n * w.double() * s).abs() * (1 + (z.double() * (1 - s)).abs())
    O.check("dz", grads["dz"], want, size * 24 * O.U32 + tiny * 50)


def test_gates_at_the_ends():
    import sparse_memory_linear_sdm_amd as sdm

    z = torch.tensor([[-3e38, -1e30, -88.8, -87.4, 88.8, 1e30, 3e38, 0.0]])
    y = torch.ones(1, 8)
    got = sdm.norm(y.cuda(), torch.ones(8).cuda(), z=z.cuda(), eps=0.0).cpu()
    want = torch.nn.functional.silu(z.double())
    assert torch.isfinite(got).all()
    O.check("out", got, want, want.abs() * 24 * O.U32 + 200 * 2.0 ** -126)
