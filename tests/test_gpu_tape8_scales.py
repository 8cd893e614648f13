"""The reverse pass from an 8-bit tape over the whole range of its scales and
of fp32: it agrees with the rows that sdm_tape8_read gives, also where the
sums come near fp32's largest value and for every scale byte.

Every output here is a sum of terms of one sign, so it is within n roundings
of 2^-24 of the float64 form, relative to itself; n is at most the number of
terms, W * d_v, and 64 for the products and the steps that G is carried over."""
import numpy as np
import pytest

from tests import mx_oracle as O

pytestmark = pytest.mark.gpu

GRADS = ("dv", "dwk", "drw", "dalpha", "dbeta")
T, W, R, N = 3, 2, 2, 40

# memories and columns: reverse tiles of 8 columns, of 16, and pairs of 16
SIZES = [(1, 16), (2, 128), (40, 128), (80, 128)]


def _sdm():
    import sparse_memory_linear_sdm_amd as sdm

    return sdm


def _step(rng, H, d_v, v, alpha):
    """Selections without repeats, small weights, constant v and alpha."""
    pick = np.argsort(rng.random((1, H, T, N)), -1).astype(np.int32)
    f = np.float32
    return dict(widx=pick[..., :W].copy(), wk=rng.uniform(.01, .02, (1, H, T, W)).astype(f),
                ridx=pick[..., W - 1:W - 1 + R].copy(),  # one row is written and read
                rw=rng.uniform(.005, .01, (1, H, T, R)).astype(f),
                v=np.full((1, H, T, d_v), v, f), alpha=np.full((1, H, T), alpha, f),
                beta=rng.uniform(.4, .5, (1, H, T)).astype(f))


def _run(s, codes, scales, dout, G):
    import torch

    sdm = _sdm()
    dev = {k: torch.from_numpy(x).cuda() for k, x in s.items()}
    Gd = torch.from_numpy(G).cuda()
    tape = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    got = sdm.scan_backward8(*dev.values(), tape, torch.from_numpy(dout).cuda(), Gd)
    return {**{k: x.cpu().numpy()[0] for k, x in got.items()}, "G": Gd.cpu().numpy()[0]}


def _want(s, codes, scales, dout, G):
    H, d_v = G.shape[1], G.shape[3]
    rows = O.int8_values(codes, scales)[0].transpose(0, 2, 3, 1, 4).reshape(H, T, W + R, d_v)
    out = {k: [] for k in (*GRADS, "G")}
    for h in range(H):
        Gh = G[0, h].astype(np.float64)
        g = O.backward(Gh, *(x[0, h].astype(np.int64 if x.dtype == np.int32 else np.float64)
                             for x in s.values()), rows[h], dout[0, h].astype(np.float64))
        for k in GRADS:
            out[k].append(g[k])
        out["G"].append(Gh)
    return {k: np.array(x) for k, x in out.items()}


def _check(got, want, d_v):
    tol = (W * d_v + 64) * 2.0 ** -24
    for k in (*GRADS, "G"):
        err = np.abs(got[k].astype(np.float64) - want[k])
        assert np.all(err <= tol * np.abs(want[k])), (k, got[k], want[k])


@pytest.mark.parametrize("H,d_v", SIZES)
def test_sums_near_the_largest_value(H, d_v):
    """Rows of about 1 and gradients of 2^119: finite sums, although the rows'
    whole numbers (127, in scales of 2^-7) times the gradients are not."""
    rng = np.random.default_rng(H + d_v)
    s = _step(rng, H, d_v, 2.0, 0.99)
    shape = (1, H, d_v // 16, T, W + R)
    codes, scales = np.full((*shape, 16), 127, np.int8), np.full(shape, 120, np.uint8)
    big = np.float32(2.0 ** 119)
    dout = rng.uniform(1.06, 1.1, (1, H, T, d_v)).astype(np.float32) * big
    G = rng.uniform(1.06, 1.1, (1, H, N, d_v)).astype(np.float32) * big
    want = _want(s, codes, scales, dout, G)
    assert all(np.all(np.abs(x) < 2.0 ** 128) for x in want.values())
    _check(_run(s, codes, scales, dout, G), want, d_v)


@pytest.mark.parametrize("H,d_v", SIZES)
def test_the_smallest_scale_bytes(H, d_v):
    """Bytes 0 (2^-127) to 3 in turn; v = 0, so that d(beta k) is the rows' part alone."""
    rng = np.random.default_rng(H * d_v)
    s = _step(rng, H, d_v, 0.0, 0.5)
    shape = (1, H, d_v // 16, T, W + R)
    codes = rng.integers(1, 128, (*shape, 16)).astype(np.int8)
    big = np.float32(2.0 ** 100)
    dout = rng.uniform(.5, 1, (1, H, T, d_v)).astype(np.float32) * big
    G = rng.uniform(.5, 1, (1, H, N, d_v)).astype(np.float32) * big
    for byte in range(4):
        scales = np.full(shape, byte, np.uint8)
        _check(_run(s, codes, scales, dout, G), _want(s, codes, scales, dout, G), d_v)


@pytest.mark.parametrize("H,d_v", SIZES)
def test_a_marked_block_is_nan_whatever_its_codes(H, d_v):
    """Byte 255 on one block of one write slot and of one read slot: the sums
    that take these rows are NaN, the others as without the mark."""
    rng = np.random.default_rng(H * d_v + 1)
    s = _step(rng, H, d_v, 2.0, 0.5)
    shape = (1, H, d_v // 16, T, W + R)
    codes = rng.integers(1, 128, (*shape, 16)).astype(np.int8)
    scales = np.full(shape, 120, np.uint8)
    scales[:, :, -1, 1, 0] = 255  # step 1: write slot 0 and read slot 1
    scales[:, :, 0, 1, W + 1] = 255
    dout = rng.uniform(.5, 1, (1, H, T, d_v)).astype(np.float32)
    G = rng.uniform(.5, 1, (1, H, N, d_v)).astype(np.float32)
    got, want = _run(s, codes, scales, dout, G), _want(s, codes, scales, dout, G)
    for k in (*GRADS, "G"):
        nan = np.isnan(want[k])
        assert np.array_equal(np.isnan(got[k]), nan), k
        got[k], want[k] = np.where(nan, 0, got[k]), np.where(nan, 0, want[k])
    assert np.isnan(_want(s, codes, scales, dout, G)["drw"]).sum() == H
    _check(got, want, d_v)
