"""Pins of the microscaled formats' plain form: closed cases, the error bound
of half a step, and the scale rule by brute force."""
import numpy as np
import pytest

from tests import mx_oracle as O


def _block(values, width):
    x = np.zeros((1, width))
    x[0, :len(values)] = values
    return x


def test_e2m1_borders_tie_to_even():
    # the first value fixes the scale at 1 (its floor(log2) is 2)
    x = _block([4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 7, -.25, -.75, -5, .2500001, 3.4999], 128)
    v = O.mx4_values(*O.mx4_quantize(x))[0, :14]
    assert v.tolist() == [4, 0, 1, 1, 2, 2, 4, 4, 6, 0, -1, -4, .5, 3]


def test_e2m1_error_is_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((50, 256)) * np.exp(rng.standard_normal((50, 1)) * 20)
    codes, scales = O.mx4_quantize(x)
    v = O.mx4_values(codes, scales)
    s = np.ldexp(1.0, scales.transpose(1, 0, 2).reshape(50, -1).astype(int) - 127)
    y = np.abs(x.reshape(50, -1, 32) / s[..., None])
    assert y.max(-1).min() >= 4 and y.max() < 8  # the scale rule
    half = np.where(y < 2, .25, np.where(y < 4, .5, np.where(y < 6, 1, 2)))
    assert np.all(np.abs((v - x).reshape(50, -1, 32)) / s[..., None] <= half)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_block_that_is_not_finite_reads_as_nan(bad):
    x = np.ones((1, 128))
    x[0, 40] = bad
    codes, scales = O.mx4_quantize(x)
    v = O.mx4_values(codes, scales)
    assert scales.ravel().tolist() == [125, 255, 125, 125]
    assert np.all(np.isnan(v[0, 32:64])) and np.all(v[0, :32] == 1) and np.all(v[0, 64:] == 1)
    q, b = O.int8_quantize(x[:, 32:48])
    assert b[0] == 255 and not q.any() and np.all(np.isnan(O.int8_values(q, b)))


def test_int8_scale_is_the_smallest_that_fits():
    rng = np.random.default_rng(2)
    tops = np.concatenate([127.5 * 2.0 ** np.arange(-8, 8), 127.49 * 2.0 ** np.arange(-8, 8),
                           2.0 ** np.arange(-20, 20), np.exp(rng.uniform(-40, 40, 200))])
    x = tops[:, None] * np.concatenate([np.ones((1, 1)), rng.uniform(-1, 1, (1, 15))], 1)
    q, b = O.int8_quantize(x)
    e = b.astype(int) - 127
    assert np.abs(q).max() <= 127
    assert np.all(np.rint(np.ldexp(tops, 1 - e)) > 127)  # half the scale would not fit
    assert np.all(np.abs(O.int8_values(q, b) - x) <= np.ldexp(.5, e)[:, None])


def test_zero_and_tiny_blocks_take_the_smallest_scale():
    for x in (np.zeros((1, 128)), np.full((1, 128), 2.0 ** -149)):
        codes, scales = O.mx4_quantize(x)
        assert np.all(scales == 2) and not codes.any()
    q, b = O.int8_quantize(np.full((1, 16), 2.0 ** -126))
    assert b[0] == 2 and np.all(q == 0)  # half of 2^-125: ties to even


def test_plain_backward_against_differences():
    """The plain reverse pass (unrounded tape) against central differences of
    the plain forward, in every input.  The forward is a polynomial in each
    input, so with h = 1e-4 the differences are within h^2 of third derivatives
    of order one, plus 2^-52 / h of rounding: 1e-7 holds both."""
    rng = np.random.default_rng(7)
    N, d_v, T, W, R = 10, 3, 6, 4, 3
    widx = np.array([rng.permutation(N)[:W] for _ in range(T)])
    ridx = np.array([rng.permutation(N)[:R] for _ in range(T)])
    widx[2, 1], ridx[3, 0], ridx[4, 2] = -1, N, 1 << 30  # skipped rows
    x = dict(M=rng.standard_normal((N, d_v)), wk=rng.random((T, W)), rw=rng.random((T, R)),
             v=rng.standard_normal((T, d_v)), alpha=rng.random(T), beta=rng.random(T))
    dout, dM = rng.standard_normal((T, d_v)), rng.standard_normal((N, d_v))

    def run(y):
        M = y["M"].copy()
        out, tape = O.forward(M, widx, y["wk"], ridx, y["rw"], y["v"], y["alpha"], y["beta"])
        return M, out, tape

    def loss(y):
        M, out, _ = run(y)
        return (out * dout).sum() + (M * dM).sum()

    G = dM.copy()
    g = O.backward(G, widx, x["wk"], ridx, x["rw"], x["v"], x["alpha"], x["beta"], run(x)[2], dout)
    want = dict(M=G, wk=g["dwk"], rw=g["drw"], v=g["dv"], alpha=g["dalpha"], beta=g["dbeta"])
    for name, grad in want.items():
        for i in np.ndindex(grad.shape):
            up, down = ({k: v.copy() for k, v in x.items()} for _ in range(2))
            up[name][i] += 1e-4
            down[name][i] -= 1e-4
            assert abs((loss(up) - loss(down)) / 2e-4 - grad[i]) <= 1e-7, (name, i)
