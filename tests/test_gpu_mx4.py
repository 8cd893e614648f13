"""GPU parity of the 4-bit microscaled calls (sdm_mx4_quantize,
sdm_mx4_dequantize, sdm_project_mx4) against the plain form in float64.

Bars.  Quantising and reading back are exact operations followed by one
defined rounding: codes, scales and values equal bit for bit.  Projections:
the products of two e2m1 values and their powers of two are exact, so each
output is a binary32 sum of d_model exact terms, as in sdm_project, with its
bound: (d_model - 1) * 2^-23 * sum |x_i w_i| for any order of additions, also
ones rounded toward zero; the gates bound/4 + 2^-21 (the logistic function's
slope is at most 1/4, plus a few ulps of expf and division)."""
import numpy as np
import pytest

from tests import mx_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
GATE_ATOL = 2.0 ** -21


def _sdm():
    import sparse_memory_linear_sdm_amd as sdm

    return sdm


def _cuda(x, dtype=None):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def _inputs(rows, cols, seed, dtype):
    """Values of many magnitudes, with borders, zeros, subnormals, huge values,
    infinities and NaN in some blocks; as the dtype holds them."""
    import torch

    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-12, 12, (rows, 1)))
    flat = x.reshape(-1, 32)
    n = flat.shape[0]
    borders = np.array([4, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 7.96875, -.25, -2.5, -7, 0, -0.])
    for i in rng.permutation(n)[:max(1, n // 4)]:
        flat[i, :16] = borders * np.exp2(rng.integers(-100, 100))
        flat[i, 16:] = 0
    special = [0.0, 2.0 ** -149, 2.0 ** -127, 1.5 * 2.0 ** -127, 2.0 ** -126, 3e38, -3e38,
               np.inf, -np.inf, np.nan]
    for i, v in zip(rng.permutation(n), special):
        flat[i] = rng.standard_normal(32) * 2.0 ** -126 if 0 < abs(v) < 1e-37 else flat[i]
        flat[i, rng.integers(32)] = v
        if v == 0:
            flat[i] = 0
    with np.errstate(over="ignore"):
        t = torch.from_numpy(x).float().to(dtype)
    return t, t.double().numpy()


SHAPES = [(1, 128), (3, 128), (4, 512), (5, 640), (33, 384), (130, 1152),
          (2049, 4224)]  # the last: 257 x 9 tiles of 8 rows


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_quantize_bitwise(rows, cols, dtype):
    import torch

    sdm = _sdm()
    t, x = _inputs(rows, cols, rows + cols, getattr(torch, dtype))
    codes, scales = sdm.mx4_quantize(t.cuda())
    oc, os_ = O.mx4_quantize(x)
    assert np.array_equal(scales.cpu().numpy(), os_)
    assert np.array_equal(codes.cpu().numpy(), oc)
    for out in (torch.float32, torch.bfloat16):
        v = sdm.mx4_dequantize(codes, scales, out).double().cpu().numpy()
        assert np.array_equal(v, O.mx4_values(oc, os_), equal_nan=True)


def test_dequantize_every_code_and_scale():
    import torch

    sdm = _sdm()
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))[:, :64]  # low nibbles all, high 0..3
    codes = (codes & 15) | ((codes + 5 * np.arange(256, dtype=np.uint8)[:, None]) << 4).astype(np.uint8)
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 4, 1)[None]
    want = O.mx4_values(codes, scales)
    for out in (torch.float32, torch.bfloat16):
        with np.errstate(over="ignore"):
            w = torch.from_numpy(want).to(torch.float32).to(out).float().numpy()
        v = sdm.mx4_dequantize(_cuda(codes), _cuda(scales), out).float().cpu().numpy()
        assert np.array_equal(v, w, equal_nan=True)
        assert np.array_equal(np.signbit(v[:255]), np.signbit(w[:255]))


def test_quantize_leading_dimensions_and_out():
    import torch

    sdm = _sdm()
    x = torch.randn(2, 3, 256, device="cuda")
    codes, scales = sdm.mx4_quantize(x)
    assert codes.shape == (2, 3, 128) and scales.shape == (2, 6, 4)
    out = (torch.zeros_like(codes), torch.zeros_like(scales))
    got = sdm.mx4_quantize(x, out=out)
    assert got[0] is out[0] and torch.equal(out[0], codes) and torch.equal(out[1], scales)
    flat = sdm.mx4_quantize(x.view(6, 256))
    assert torch.equal(flat[0].view_as(codes), codes) and torch.equal(flat[1], scales)
    v = torch.empty(2, 3, 256, dtype=torch.bfloat16, device="cuda")
    assert sdm.mx4_dequantize(codes, scales, out=v) is v
    assert torch.equal(v.float(), sdm.mx4_dequantize(codes, scales))


def test_quantize_writes_nothing_behind_its_rows():
    import torch

    sdm = _sdm()
    rows, cols = 5, 384
    x = torch.randn(rows, cols, device="cuda")
    codes = torch.full((rows * cols // 2 + 64,), 171, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows * cols // 32 + 64,), 171, dtype=torch.uint8, device="cuda")
    sdm.mx4_quantize(x, out=(codes[:rows * cols // 2].view(rows, -1),
                             scales[:rows * cols // 32].view(cols // 128, rows, 4)))
    assert torch.all(codes[rows * cols // 2:] == 171) and torch.all(scales[rows * cols // 32:] == 171)


# ------------------------------------------------------------- projections

def _operands(B, T, d_model, H, n, d_v, seed, spread=3):
    rng = np.random.default_rng(seed)
    rows, cols = B * T, H * (4 * n + d_v + 2)

    def one(r):
        codes = rng.integers(0, 256, (r, d_model // 2), dtype=np.uint8)
        scales = (127 - spread + rng.integers(0, 2 * spread + 1, (d_model // 128, r, 4))).astype(np.uint8)
        return codes, scales

    return one(rows), one(cols)


def _project(ops, B, T, d_model, H, n, d_v, **kw):
    sdm = _sdm()
    (xq, xs), (wq, ws) = ops
    P = 4 * n + d_v + 2
    return sdm.project_mx4(_cuda(xq).view(B, T, -1), _cuda(xs), _cuda(wq).view(H, P, -1),
                           _cuda(ws), n, **kw)


def _check(ops, got, B, T, d_model, H, n, d_v, tokens=None):
    (xq, xs), (wq, ws) = ops
    toks = np.arange(B * T) if tokens is None else np.asarray(tokens)
    x = O.mx4_values(xq[toks], xs[:, toks])
    w = O.mx4_values(wq, ws)
    y = (x @ w.T).reshape(len(toks), H, -1)
    lim = (d_model - 1) * U * (np.abs(x) @ np.abs(w).T).reshape(y.shape)
    b, t = toks // T, toks % T
    at = 0
    worst = 0.0
    for part in got[:5]:
        g = part.cpu().numpy()[b, :, t].astype(np.float64)
        width = g.shape[-1]
        want, bound = y[..., at:at + width], lim[..., at:at + width]
        assert np.array_equal(np.isnan(g), np.isnan(want))
        err = np.where(np.isnan(want), 0.0, np.abs(g - want))
        assert np.all(err <= np.where(np.isnan(bound), 0.0, bound)), f"columns {at}.."
        worst = max(worst, float(np.max(err / np.where(bound > 0, bound, 1.0))))
        at += width
    for gate in got[5:]:
        g = gate.cpu().numpy()[b, :, t].astype(np.float64)
        want = 1 / (1 + np.exp(-y[..., at]))
        ok = np.abs(g - want) <= lim[..., at] / 4 + GATE_ATOL
        assert np.all(ok | (np.isnan(g) & np.isnan(want)))
        at += 1
    return worst


PROJECT = [
    # the few-token kernel: 1, 2 and 4 token fragments, 1 to 9 column fragments,
    # one block of tokens and several, K shorter than its wavefronts' first turns
    (1, 1, 128, 1, 1, 1), (1, 1, 128, 1, 64, 16), (16, 1, 256, 2, 37, 32), (17, 1, 384, 1, 16, 16),
    (3, 11, 640, 3, 37, 32), (1, 47, 1152, 2, 128, 64), (64, 1, 4480, 1, 64, 128),
    (32, 2, 8192, 1, 5, 16), (5, 1, 1024, 5, 1024, 64), (1, 64, 1408, 3, 2048, 16),
    (30, 1, 1152, 6, 1024, 100), (10, 1, 256, 9, 1024, 128), (63, 1, 1280, 8, 1024, 128),
    (65, 1, 128, 1, 16, 16), (2, 150, 384, 3, 64, 16), (1, 257, 256, 1, 37, 32),
    (300, 1, 640, 1, 8, 16), (37, 3, 128, 2, 16, 16), (2, 700, 1024, 1, 128, 128),
    (1, 300, 512, 2, 256, 64),
    # tiles, of both sizes: one stage of K and several, ragged rows and columns,
    # T = 1, 3, 4 and long, gates and array borders inside a wavefront's columns
    (300, 4, 640, 3, 333, 40), (1, 1025, 128, 4, 256, 66), (3, 401, 1152, 2, 512, 17),
    (1203, 1, 384, 1, 1024, 16), (401, 3, 256, 1, 1024, 16), (1, 2048, 512, 1, 1020, 14),
    (130, 1, 8192, 1, 1024, 128), (9, 60, 8192, 1, 512, 64), (1, 640, 4096, 2, 256, 30),
    (2, 1100, 1024, 7, 5, 3), (3000, 1, 128, 30, 1, 1), (60, 200, 128, 2, 64, 16),
    (1, 2050, 4096, 2, 512, 64), (7, 117, 16384, 1, 512, 16), (7, 4681, 128, 1, 64, 16),
    (3, 5461, 384, 1, 128, 20), (1, 16384, 128, 4, 30, 8), (777, 21, 256, 2, 64, 64),
    # the few-token kernel's wide column blocks
    (2, 7, 128, 8, 1024, 128), (3, 7, 384, 8, 1024, 128), (17, 1, 256, 4, 1024, 128),
    (9, 2, 128, 1, 1024, 128), (21, 1, 128, 2, 1024, 128), (33, 1, 2048, 8, 1024, 128),
    (5, 410, 1024, 1, 60, 30), (63, 1, 2176, 8, 1024, 128),
]


@pytest.mark.parametrize("B,T,d_model,H,n,d_v", PROJECT)
def test_project_mx4_parity(B, T, d_model, H, n, d_v):
    ops = _operands(B, T, d_model, H, n, d_v, seed=B * 1000 + T + n)
    got = _project(ops, B, T, d_model, H, n, d_v)
    worst = _check(ops, got, B, T, d_model, H, n, d_v)
    again = _project(ops, B, T, d_model, H, n, d_v)
    import torch

    assert all(torch.equal(a, b) for a, b in zip(got, again))
    print(f"worst |err| / bound = {worst:.3e}")


@pytest.mark.parametrize("B,T,H,n", [(1, 40, 2, 32), (2, 100, 2, 32), (2, 600, 1, 1024)])
def test_project_mx4_wide_scales(B, T, H, n):
    """Block scales over 40 powers of two: sums of terms of very unequal size."""
    ops = _operands(B, T, 1024, H, n, 32, seed=9, spread=20)
    _check(ops, _project(ops, B, T, 1024, H, n, 32), B, T, 1024, H, n, 32)


@pytest.mark.parametrize("tokens", [3, 33, 1200])
def test_project_mx4_writes_nothing_beside_its_outputs(tokens):
    """Ragged last blocks: guard words around every output stay as they were."""
    import torch

    B, T, d_model, H, n, d_v = 1, tokens, 256, 1, 1025, 20
    ops = _operands(B, T, d_model, H, n, d_v, seed=tokens)
    shapes = [(B, H, T, n)] * 4 + [(B, H, T, d_v), (B, H, T), (B, H, T)]
    bufs = [torch.full((64 + int(np.prod(s)) + 64,), 5.0, device="cuda") for s in shapes]
    out = tuple(b[64:-64].view(s) for b, s in zip(bufs, shapes))
    got = _project(ops, B, T, d_model, H, n, d_v, out=out)
    assert all(a is b for a, b in zip(got, out))
    _check(ops, got, B, T, d_model, H, n, d_v)
    assert all(torch.all(b[:64] == 5) and torch.all(b[-64:] == 5) for b in bufs)


@pytest.mark.parametrize("B,T,H,n", [(5, 9, 2, 16), (3, 100, 2, 16), (4, 300, 1, 1024)])
def test_project_mx4_nan_blocks_stay_in_their_rows(B, T, H, n):
    d_model, d_v = 512, 16
    ops = _operands(B, T, d_model, H, n, d_v, seed=4)
    (xq, xs), (wq, ws) = ops
    xs[2, 7, 1] = 255
    ws[0, 50, 3] = 255
    got = _project(ops, B, T, d_model, H, n, d_v)
    _check(ops, got, B, T, d_model, H, n, d_v)
    assert all(np.isnan(g.cpu().numpy()[7 // T, :, 7 % T]).all() for g in got)


def test_project_mx4_zero_blocks_and_smallest_scales():
    """All-zero tokens (scale byte 2 everywhere) give zeros and gates of 1/2."""
    import torch

    sdm = _sdm()
    x = torch.zeros(1, 70, 256, device="cuda")
    w = torch.randn(1, 4 * 4 + 2 + 2, 256, device="cuda")
    for rows in (70, 3):
        got = sdm.project_mx4(*sdm.mx4_quantize(x[:, :rows].contiguous()), *sdm.mx4_quantize(w), 4)
        assert all(torch.all(g == 0) for g in got[:5]) and all(torch.all(g == .5) for g in got[5:])


def test_project_mx4_close_to_bf16_project_of_the_same_values():
    """Values that 4 bits hold exactly: both projections see the same numbers,
    so they differ by their two summation orders at most."""
    import torch

    sdm = _sdm()
    g = torch.Generator(device="cuda").manual_seed(3)
    B, T, d_model, H, n, d_v = 2, 90, 512, 2, 32, 16
    q = [sdm.mx4_quantize(torch.randn(s, generator=g, device="cuda"))
         for s in ((B, T, d_model), (H, 4 * n + d_v + 2, d_model))]
    x, w = (sdm.mx4_dequantize(*o, torch.bfloat16) for o in q)
    a, b = sdm.project_mx4(*q[0], *q[1], n), sdm.project(x, w, n)
    lim = 2 * (d_model - 1) * U * (x.double().abs().view(-1, d_model) @
                                   w.double().abs().view(-1, d_model).t()).max().item()
    assert all((i - j).abs().max().item() <= lim for i, j in zip(a, b))


def test_project_mx4_full_width_sampled():
    """The mid workload's widths (d_model 16384, H = 8, n = 1024, d_v = 128):
    prompts through the tiles, a decode step through the few-token kernel."""
    H, n, d_v, d_model = 8, 1024, 128, 16384
    for B, T, toks in ((2, 300, [0, 255, 256, 300, 511, 599]), (48, 1, [0, 15, 16, 33, 47]),
                       (9, 1, [0, 4, 8])):
        ops = _operands(B, T, d_model, H, n, d_v, seed=T)
        got = _project(ops, B, T, d_model, H, n, d_v)
        _check(ops, got, B, T, d_model, H, n, d_v, tokens=toks)


def test_empty_batches_are_no_ops():
    import torch

    sdm = _sdm()
    codes, scales = sdm.mx4_quantize(torch.empty(0, 4, 256, device="cuda"))
    assert codes.shape == (0, 4, 128) and scales.shape == (2, 0, 4)
    assert sdm.mx4_dequantize(codes, scales).shape == (0, 4, 256)
    wq, ws = sdm.mx4_quantize(torch.randn(1, 4 * 2 + 3 + 2, 256, device="cuda"))
    assert sdm.project_mx4(codes, scales, wq, ws, 2)[0].shape == (0, 1, 4, 2)


def test_calls_on_another_stream_and_captured():
    """A side stream, and a graph of quantise + project replayed on changed
    inputs, give the bits of plain calls."""
    import torch

    sdm = _sdm()
    x = torch.randn(3, 40, 384, device="cuda")
    w = sdm.mx4_quantize(torch.randn(2, 4 * 16 + 16 + 2, 384, device="cuda"))
    small = torch.randn(3, 1, 384, device="cuda")
    side = torch.cuda.Stream()
    for inp in (x, small):
        want = sdm.project_mx4(*sdm.mx4_quantize(inp), *w, 16)
        side.wait_stream(torch.cuda.current_stream())
        got = sdm.project_mx4(*sdm.mx4_quantize(inp, stream=side), *w, 16, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = sdm.project_mx4(*sdm.mx4_quantize(inp), *w, 16)
        for k in range(3):
            inp.copy_(torch.randn_like(inp))
            graph.replay()
            want = sdm.project_mx4(*sdm.mx4_quantize(inp), *w, 16)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, held)), k


@pytest.mark.parametrize("B,T,n", [(1, 1, 8), (2, 35, 8), (3, 400, 256)])
def test_project_mx4_widest_rows(B, T, n):
    """d_model 65536, the largest."""
    ops = _operands(B, T, 65536, 1, n, 16, seed=T)
    _check(ops, _project(ops, B, T, 65536, 1, n, 16), B, T, 65536, 1, n, 16,
           tokens=None if B * T < 100 else [0, 255, 256, 700, B * T - 1])


def test_two_streams_project_at_once():
    """Prompt tiles on one stream beside decode steps on another."""
    import torch

    sdm = _sdm()
    w = sdm.mx4_quantize(torch.randn(2, 4 * 256 + 64 + 2, 1024, device="cuda"))
    xs = [sdm.mx4_quantize(torch.randn(B, T, 1024, device="cuda")) for B, T in ((4, 500), (7, 1))]
    want = [sdm.project_mx4(*x, *w, 256) for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [sdm.project_mx4(*x, *w, 256, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refusals_on_the_gpu():
    import torch

    sdm = _sdm()
    with pytest.raises(sdm.SDMError, match="multiple of 128"):
        sdm.mx4_quantize(torch.zeros(4, 96, device="cuda"))
    buf = torch.zeros(4 * 128 + 4, device="cuda")
    with pytest.raises(sdm.SDMError, match="16-byte"):
        sdm.mx4_quantize(buf[1:1 + 4 * 128].view(4, 128))
    with pytest.raises(ValueError, match="contiguous"):
        sdm.mx4_quantize(torch.zeros(256, 4, device="cuda").t())
