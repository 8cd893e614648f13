"""Norms before and after a block against their 64-bit form.  Bounds: the root
and the gate are within a few fp32 roundings, the sums over d values within
d * 2^-24 of their size; each output is rounded once."""
import pytest
import torch

from tests import dense_oracle as O

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def make(shape, dtype, out_dtype, heads, seed, gate=True, residual=True):
    r = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    d = shape[-1]
    wide = (shape[0], shape[2], shape[1] * d) if heads else shape
    return dict(y=(randn(*shape) * torch.exp(randn(*shape[:-1], 1))).to(dtype), w=1 + 0.3 * randn(d),
                z=(2 * randn(*wide)).to(out_dtype) if gate else None,
                x=randn(*wide).to(out_dtype) if residual else None,
                dout=randn(*wide).to(out_dtype), skip=randn(*shape).to(dtype), next_w=randn(d))


def dev(a):
    return {n: None if x is None else x.cuda() for n, x in a.items()}


def limit(size, dtype, d):
    return size * (O.HALF[dtype] + (d + 40) * O.U32) + 1e-30


def check_forward(a, got, heads, scale, d):
    args = dict(scale=scale, heads=heads)
    want = O.norm_forward(a["y"], a["w"], a["z"], a["x"], **args)
    part = O.norm_forward(a["y"], a["w"], a["z"], None, **args)
    size = part.abs() + (0 if a["x"] is None else a["x"].double().abs())
    O.check("out", got, want, limit(size, got.dtype, d))
    return want, size


@pytest.mark.parametrize("d", [8, 16, 24, 64, 128, 136, 256, 504, 512, 520, 1024, 4096, 5128, 8192,
                               8200, 16376, 16384])
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_norm_every_width(d, dtype, out_dtype):
    import sparse_memory_linear_sdm_amd as sdm

    a = make((3, 5, d), dtype, out_dtype, False, d)
    g = dev(a)
    got, behind = sdm.norm(g["y"], g["w"], z=g["z"], x=g["x"], scale=0.5, next_w=g["next_w"])
    assert got.dtype == out_dtype and got.shape == (3, 5, d)
    want, size = check_forward(a, got, False, 0.5, d)
    # a relative error of out's size moves its root by as much at most, twice
    n = want / (want.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    ratio = (size.square().mean(-1, keepdim=True) / (want.square().mean(-1, keepdim=True) + 1e-6)).sqrt()
    root = 1 / (want.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    off = (size * root + n.abs() * ratio * 2) * a["next_w"].abs() * (d + 40) * O.U32
    O.check("next", behind, n * a["next_w"], off + (n * a["next_w"]).abs() * O.HALF[out_dtype] + 1e-30)
    plain = sdm.norm(g["y"], g["w"])
    assert plain.dtype == dtype
    want = O.norm_forward(a["y"], a["w"])
    O.check("plain", plain, want, limit(want.abs(), dtype, d))


@pytest.mark.parametrize("shape", [(1, 1, 1, 16), (2, 3, 7, 32), (1, 5, 33, 128), (3, 2, 9, 520),
                                   (2, 7, 1, 64), (1, 64, 3, 8)])
@pytest.mark.parametrize("dtype,out_dtype", [(F32, BF16), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("gate", [False, True])
def test_norm_per_head(shape, dtype, out_dtype, gate):
    import sparse_memory_linear_sdm_amd as sdm

    a = make(shape, dtype, out_dtype, True, 3, gate=gate, residual=not gate)
    g = dev(a)
    got = sdm.norm(g["y"], g["w"], z=g["z"], x=g["x"], heads=True, dtype=out_dtype)
    assert got.shape == (shape[0], shape[2], shape[1] * shape[3])
    check_forward(a, got, True, 1.0, shape[-1])


def check_backward(a, got, heads, scale, d, skip):
    args = (a["dout"], a["y"], a["w"], a["z"])
    want = O.norm_reverse(*args, scale=scale, skip=a["skip"] if skip else None, heads=heads)
    # sums of magnitudes: the mean over a row enters with its terms' magnitudes
    y = a["y"].double()
    r = 1 / (y.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    rows = lambda t: t.double().unflatten(-1, (-1, d)).transpose(1, 2) if heads else t.double()  # noqa: E731
    D = rows(a["dout"]).abs() * abs(scale)
    gate = 1.0 if a["z"] is None else (rows(a["z"]) * torch.sigmoid(rows(a["z"]))).abs()
    m, n = D * gate * a["w"].double().abs(), (y * r).abs()
    size = r * (m + n * (m * n).mean(-1, keepdim=True) * 2)
    if skip:
        size = size + a["skip"].double().abs()
    O.check("dy", got["dy"], want["dy"], limit(size, got["dy"].dtype, 2 * d))
    terms = y.numel() // d + d
    O.check("dw", got["dw"], want["dw"], limit((D * gate * n).flatten(0, -2).sum(0), F32, terms))
    if a["z"] is not None:
        z = rows(a["z"])
        s = torch.sigmoid(z)
        size = D * n * a["w"].double().abs() * s * (1 + (z * (1 - s)).abs())
        size = size.transpose(1, 2).flatten(2) if heads else size
        O.check("dz", got["dz"], want["dz"], limit(size, got["dz"].dtype, d))
    else:
        assert "dz" not in got


@pytest.mark.parametrize("d", [8, 24, 128, 504, 512, 520, 4096, 4104, 8192, 8200, 16384])
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("gate,skip", [(True, False), (False, True)])
def test_norm_backward_every_width(d, dtype, out_dtype, gate, skip):
    import sparse_memory_linear_sdm_amd as sdm

    a = make((2, 7, d), dtype, out_dtype, False, d, gate=gate)
    g = dev(a)
    got = sdm.norm_backward(g["dout"], g["y"], g["w"], z=g["z"], scale=0.5,
                            skip=g["skip"] if skip else None)
    check_backward(a, got, False, 0.5, d, skip)


@pytest.mark.parametrize("shape", [(1, 1, 1, 16), (2, 3, 7, 32), (1, 5, 333, 128), (3, 2, 9, 520),
                                   (4, 16, 300, 8)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("gate,skip", [(True, True), (False, False)])
def test_norm_backward_per_head(shape, dtype, gate, skip):
    import sparse_memory_linear_sdm_amd as sdm

    a = make(shape, dtype, BF16, True, 4, gate=gate)
    g = dev(a)
    got = sdm.norm_backward(g["dout"], g["y"], g["w"], z=g["z"], skip=g["skip"] if skip else None,
                            heads=True)
    check_backward(a, got, True, 1.0, shape[-1], skip)


@pytest.mark.parametrize("rows,d", [(511, 520), (512, 520), (513, 520), (1300, 1024), (8200, 512),
                                    (20000, 64)])
def test_norm_backward_many_rows(rows, d):
    """More rows than workgroups: each takes several, and dw sums over all."""
    import sparse_memory_linear_sdm_amd as sdm

    a = make((rows, d), F32, F32, False, 5)
    g = dev(a)
    got = sdm.norm_backward(g["dout"], g["y"], g["w"], z=g["z"])
    check_backward(a, got, False, 1.0, d, False)
    again = sdm.norm_backward(g["dout"], g["y"], g["w"], z=g["z"])
    assert all(torch.equal(got[n], again[n]) for n in got)


def test_norm_of_no_rows():
    import sparse_memory_linear_sdm_amd as sdm

    y, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    assert sdm.norm(y, w).shape == (0, 64)
    got = sdm.norm_backward(y, y, w)
    assert got["dy"].shape == (0, 64) and not got["dw"].any()


def test_rows_of_zeros_and_far_gates():
    """A row of zeros gives zeros (eps keeps the root); silu(-1e30) is 0, not NaN;
    a row with an infinity or a NaN spoils itself alone."""
    import sparse_memory_linear_sdm_amd as sdm

    a = make((6, 128), F32, F32, False, 6)
    a["y"][0] = 0
    a["z"][1] = -1e30
    a["z"][2] = 1e30
    a["y"][3, 5] = float("inf")
    a["y"][4, 7] = float("nan")
    g = dev(a)
    got = sdm.norm(g["y"], g["w"], z=g["z"]).cpu()
    assert not got[0].any() and not got[1].any()
    assert torch.isfinite(got[2]).all() and got[4].isnan().all() and got[3, 5].isnan()
    one = {n: None if x is None or n in ("w", "next_w") else x[5:] for n, x in a.items()}
    one["w"] = a["w"]
    check_forward(dict(one, x=None), got[5:], False, 1.0, 128)
    grads = sdm.norm_backward(g["dout"], g["y"], g["w"], z=g["z"])
    assert torch.isfinite(grads["dy"][:3]).all() and torch.isfinite(grads["dy"][5]).all()
    assert not grads["dz"][1].any()


def test_norm_in_place():
    """out may be the residual, dy may be skip."""
    import sparse_memory_linear_sdm_amd as sdm

    a = dev(make((9, 1000), BF16, BF16, False, 7))
    want = sdm.norm(a["y"], a["w"], z=a["z"], x=a["x"], scale=0.3)
    x = a["x"].clone()
    assert sdm.norm(a["y"], a["w"], z=a["z"], x=x, scale=0.3, out=x) is x and torch.equal(x, want)
    ref = sdm.norm_backward(a["dout"], a["y"], a["w"], skip=a["skip"])
    skip = a["skip"].clone()
    sdm.norm_backward(a["dout"], a["y"], a["w"], skip=skip,
                      out=dict(dy=skip, dw=torch.empty(1000, device="cuda")))
    assert torch.equal(skip, ref["dy"])


def test_norm_captured_and_replayed():
    import sparse_memory_linear_sdm_amd as sdm

    a = dev(make((40, 1024), BF16, BF16, False, 8))

    def step():
        out, behind = sdm.norm(a["y"], a["w"], z=a["z"], x=a["x"], scale=0.3, next_w=a["next_w"])
        return [out, behind, *sdm.norm_backward(a["dout"], a["y"], a["w"], z=a["z"]).values()]

    want = [x.clone() for x in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        step()
