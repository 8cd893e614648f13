"""GPU parity of the 8-bit training tape (sdm_scan_train8, sdm_tape8_read,
sdm_scan_backward8).

Bars.  M and out: bit for bit those of sdm_scan_train.  The tape: its fp32
tape's rows through one defined rounding, so codes and scale bytes equal the
plain form's bit for bit; reading back is exact.  The reverse pass: G bit for
bit as sdm_scan_backward leaves it, and every gradient within 1e-5 normwise of
the float64 reverse pass from the same rows -- sums of at most a few hundred
fp32 products per step, carried over the steps by factors alpha*(1 - beta*k)
<= 1, as for sdm_scan_backward."""
import numpy as np
import pytest

from tests import mx_oracle as O

pytestmark = pytest.mark.gpu

GRAD_REL = 1e-5
STEP = ("widx", "wk", "ridx", "rw", "v", "alpha", "beta")


def _sdm():
    import sparse_memory_linear_sdm_amd as sdm

    return sdm


def _inputs(B, H, N, d_v, T, W, R, seed, strays=True):
    """A step's inputs on the GPU.  Few rows are picked much more often than
    the others, read rows often coincide with write rows, and with `strays`
    some row numbers lie outside the table."""
    import torch

    rng = np.random.default_rng(seed)

    def rows(K):
        p = rng.random((B, H, T, N)) * np.where(np.arange(N) < 2 * K, 3.0, 1.0)
        i = np.argsort(-p, -1)[..., :K].astype(np.int32)
        if strays and K > 1:
            bad = rng.random(i.shape) < 0.05
            i = np.where(bad, rng.choice([-1, N, N + 5, 1 << 30, -(1 << 31)], i.shape), i)
        return torch.from_numpy(i.astype(np.int32)).cuda()

    def f(x):
        return torch.from_numpy(x.astype(np.float32)).cuda()

    def weights(K):
        w = rng.random((B, H, T, K)) + 0.01
        return f(w / w.sum(-1, keepdims=True))

    d = dict(widx=rows(W), wk=weights(W), ridx=rows(R), rw=weights(R),
             v=f(rng.standard_normal((B, H, T, d_v))), alpha=f(rng.uniform(.9, 1, (B, H, T))),
             beta=f(rng.random((B, H, T))))
    d["M"] = f(rng.standard_normal((B, H, N, d_v)) * np.exp2(rng.integers(-9, 3, (B, H, N, 1))))
    d["dout"] = f(rng.standard_normal((B, H, T, d_v)))
    return d


def _step(d):
    return [d[k] for k in STEP]


# (B, H, N, d_v, T, W, R): forward tiles of 16 columns with two row shards, 16
# unsharded and 32, reverse tiles of 8 and 16; one tile, one step, one slot, the
# widest rows
CASES = [
    (1, 2, 70, 16, 77, 8, 5), (2, 2, 200, 64, 61, 32, 32), (3, 7, 100, 128, 45, 16, 9),
    (5, 8, 90, 128, 33, 13, 64), (1, 3, 128, 128, 60, 64, 64), (1, 1, 40, 16, 1, 1, 1),
    (2, 5, 64, 256, 19, 7, 33), (1, 1, 5, 32, 40, 3, 2), (9, 4, 50, 256, 9, 11, 1),
    (8, 8, 70, 128, 18, 9, 12),  # 64 memories: cache lines of G shared by two wavefronts
]


def _known(rows_idx, N):
    """Slots [B, H, T, S] whose rows lie in the table."""
    return (rows_idx >= 0) & (rows_idx < N)


def _valid(d, N):
    import torch

    return torch.cat([_known(d["widx"], N), _known(d["ridx"], N)], -1).cpu().numpy()


@pytest.mark.parametrize("B,H,N,d_v,T,W,R", CASES)
def test_train8_parity(B, H, N, d_v, T, W, R):
    import torch

    sdm = _sdm()
    d = _inputs(B, H, N, d_v, T, W, R, seed=B * 100 + T)
    Ma, Mb = d["M"].clone(), d["M"].clone()
    out, tape = sdm.scan_train(Ma, *_step(d), tape=torch.zeros(B, H, T, W + R, d_v, device="cuda"))
    held = (torch.full((B, H, d_v // 16, T, W + R, 16), 77, dtype=torch.int8, device="cuda"),
            torch.full((B, H, d_v // 16, T, W + R), 99, dtype=torch.uint8, device="cuda"))
    out8, got = sdm.scan_train8(Mb, *_step(d), tape=held)
    assert torch.equal(Ma, Mb) and torch.equal(out, out8)
    assert got[0] is held[0] and got[1] is held[1]
    rows = tape.cpu().numpy().reshape(B, H, T, W + R, d_v // 16, 16).transpose(0, 1, 4, 2, 3, 5)
    codes, scales = O.int8_quantize(rows)
    ok = np.broadcast_to(_valid(d, N)[:, :, None], scales.shape)
    gc, gs = (x.cpu().numpy() for x in got)
    assert np.array_equal(gs[ok], scales[ok]) and np.array_equal(gc[ok], codes[ok])
    assert np.all(gc[~ok] == 77) and np.all(gs[~ok] == 99)  # skipped rows: left as they were
    want = O.int8_values(codes, scales).transpose(0, 1, 3, 4, 2, 5).reshape(B, H, T, W + R, d_v)
    for dt in (torch.float32, torch.bfloat16):
        back = sdm.tape8_read(got, dt).double().cpu().numpy()
        assert np.array_equal(back[_valid(d, N)], want[_valid(d, N)])


def test_train8_values_that_are_not_finite_or_tiny():
    """Rows with NaN, infinities, zeros, subnormals and the largest values."""
    import torch

    sdm = _sdm()
    B, H, N, d_v, T, W, R = 1, 2, 40, 32, 12, 4, 6
    d = _inputs(B, H, N, d_v, T, W, R, seed=3, strays=False)
    d["v"].zero_()
    for i, x in enumerate([np.nan, np.inf, -np.inf, 0.0, 2.0 ** -149, 2.0 ** -127, 3.3e38, -3e38,
                           127.5, 127.49]):
        d["M"][:, :, i, :16] = x
        d["M"][:, :, i, 16:] *= 0
        d["M"][:, :, i, 20] = x
    Ma = d["M"].clone()
    _, tape = sdm.scan_train(Ma, *_step(d))
    Mb = d["M"].clone()
    _, got = sdm.scan_train8(Mb, *_step(d))
    rows = tape.cpu().numpy().reshape(B, H, T, W + R, 2, 16).transpose(0, 1, 4, 2, 3, 5)
    codes, scales = O.int8_quantize(rows)
    assert (scales == 255).any() and (scales == 2).any() and (scales > 240).any()
    assert np.array_equal(got[1].cpu().numpy(), scales)
    assert np.array_equal(got[0].cpu().numpy(), codes)
    want = O.int8_values(codes, scales).transpose(0, 1, 3, 4, 2, 5).reshape(B, H, T, W + R, d_v)
    back = sdm.tape8_read(got).double().cpu().numpy()
    assert np.array_equal(back, want, equal_nan=True)
    # The reverse pass: a block that reads as NaN reaches the sums over it, and
    # sums without one, and without a row of ~3e38 (whose products overflow),
    # are the plain form's.
    rows = sdm.tape8_read(got)
    b = sdm.scan_backward8(*_step(d), got, d["dout"], torch.zeros_like(d["M"]))
    nan = torch.isnan(rows).any(-1).cpu().numpy()
    bad = nan | (rows.abs() > 1e30).any(-1).cpu().numpy()
    h = {k: d[k].double().cpu().numpy() for k in ("wk", "rw", "v", "alpha", "beta", "dout")}
    rows = np.where(bad[..., None], 0.0, rows.double().cpu().numpy())
    assert nan[..., :W].any() and nan[..., W:].any()
    for m in np.ndindex(B, H):
        g = O.backward(np.zeros((N, d_v)), d["widx"][m].cpu().numpy(), h["wk"][m],
                       d["ridx"][m].cpu().numpy(), h["rw"][m], h["v"][m], h["alpha"][m],
                       h["beta"][m], rows[m], h["dout"][m])
        x = {k: b[k][m].cpu().numpy() for k in b}
        _close(x["dv"], g["dv"], "dv")
        for k, off in (("dwk", slice(0, W)), ("drw", slice(W, W + R))):
            assert np.isnan(x[k][nan[m][:, off]]).all()
            ok = ~bad[m][:, off]
            _close(x[k][ok], g[k][ok], k)
        for k in ("dalpha", "dbeta"):
            assert np.isnan(x[k][nan[m][:, :W].any(-1)]).all()
            ok = ~bad[m][:, :W].any(-1)
            if ok.any():
                _close(x[k][ok], g[k][ok], k)


def test_tape8_read_every_code_and_scale():
    import torch

    sdm = _sdm()
    codes = np.arange(-128, 128).astype(np.int8).reshape(1, 1, 1, 1, 16, 16)
    codes = np.ascontiguousarray(np.broadcast_to(codes, (256, 1, 1, 1, 16, 16)))
    scales = np.broadcast_to(np.arange(256, dtype=np.uint8)[:, None], (256, 16)).reshape(256, 1, 1, 1, 16)
    want = O.int8_values(codes, scales).reshape(256, 1, 1, 16, 16)
    t = (torch.from_numpy(codes).cuda(), torch.from_numpy(np.ascontiguousarray(scales)).cuda())
    for dt in (torch.float32, torch.bfloat16):
        with np.errstate(over="ignore"):
            w = torch.from_numpy(want).float().to(dt).float().numpy()
        assert np.array_equal(sdm.tape8_read(t, dt).float().cpu().numpy(), w, equal_nan=True)


def _close(got, want, what):
    scale = max(1.0, float(np.abs(want).max()))
    err = float(np.abs(got - want).max())
    assert err <= GRAD_REL * scale, f"{what}: {err} against {scale}"


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("B,H,N,d_v,T,W,R", CASES)
def test_backward8_parity(B, H, N, d_v, T, W, R, sparse):
    import torch

    sdm = _sdm()
    d = _inputs(B, H, N, d_v, T, W, R, seed=B * 77 + T)
    M = d["M"].clone()
    # slots of skipped rows hold NaN blocks: they must not be read
    tape = (torch.zeros(B, H, d_v // 16, T, W + R, 16, dtype=torch.int8, device="cuda"),
            torch.full((B, H, d_v // 16, T, W + R), 255, dtype=torch.uint8, device="cuda"))
    sdm.scan_train8(M, *_step(d), tape=tape)
    rows = torch.nan_to_num(sdm.tape8_read(tape))
    first = sdm.touch_prepare(d["widx"], d["ridx"], N)[1] if sparse else None
    G0 = torch.full_like(M, 7.0) if sparse else torch.randn_like(M)
    Ga, Gb = G0.clone(), G0.clone()
    sdm.scan_backward(*_step(d), rows, d["dout"], Ga, first=first)
    b = sdm.scan_backward8(*_step(d), tape, d["dout"], Gb, first=first)
    assert torch.equal(Ga, Gb)
    again = sdm.scan_backward8(*_step(d), tape, d["dout"], G0.clone(), first=first)
    assert all(torch.equal(again[k], b[k]) for k in b)  # the same bits every time
    h = {k: d[k].double().cpu().numpy() for k in ("wk", "rw", "v", "alpha", "beta", "dout")}
    wi, ri, rows = (x.cpu().numpy() for x in (d["widx"], d["ridx"], rows.double()))
    for m in np.ndindex(B, H):
        G = G0[m].double().cpu().numpy()
        seen = np.unique(np.concatenate([wi[m].ravel(), ri[m].ravel()]))
        seen = seen[(seen >= 0) & (seen < N)]
        if sparse:
            G[seen] = 0
        g = O.backward(G, wi[m], h["wk"][m], ri[m], h["rw"][m], h["v"][m], h["alpha"][m],
                       h["beta"][m], rows[m], h["dout"][m])
        for k in g:
            _close(b[k][m].cpu().numpy(), g[k], k)
        _close(Gb[m].cpu().numpy(), G, "G")


def test_gradients_from_the_8_bit_tape_against_the_exact_ones():
    """How far the rounding of the tape moves the gradients: a row's value is
    off by at most half its block's scale; G does not read the rows, and
    dr_l = <dout, row> moves by at most sum |dout| * off."""
    import torch

    sdm = _sdm()
    B, H, N, d_v, T, W, R = 1, 2, 90, 64, 40, 16, 12
    d = _inputs(B, H, N, d_v, T, W, R, seed=11, strays=False)
    Ma, Mb = d["M"].clone(), d["M"].clone()
    _, tape = sdm.scan_train(Ma, *_step(d))
    _, tape8 = sdm.scan_train8(Mb, *_step(d))
    Ga, Gb = (torch.zeros_like(Ma) for _ in range(2))
    a = sdm.scan_backward(*_step(d), tape, d["dout"], Ga)
    b = sdm.scan_backward8(*_step(d), tape8, d["dout"], Gb)
    assert torch.equal(Ga, Gb)  # does not read the rows
    half = torch.ldexp(torch.tensor(0.5, device="cuda"), tape8[1].int() - 127)
    off = (half.permute(0, 1, 3, 4, 2).unsqueeze(-1).expand(*tape.shape[:4], d_v // 16, 16)
           .reshape(tape.shape).double())
    assert torch.all((sdm.tape8_read(tape8).double() - tape.double()).abs() <= off)
    # plus the rounding of both sums of d_v products
    lim = (d["dout"].double().abs().unsqueeze(3) * off[..., W:, :]).sum(-1)
    lim = lim + 2 * d_v * 2.0 ** -24 * (d["dout"].abs().unsqueeze(3) * tape[..., W:, :].abs()).sum(-1)
    assert torch.all((a["drw"] - b["drw"]).abs() <= lim)


def test_small_shapes_chunks_and_empty_calls():
    """Consecutive calls give the tape and state of one; T = 0 changes nothing."""
    import torch

    sdm = _sdm()
    B, H, N, d_v, T, W, R = 2, 2, 50, 32, 21, 6, 7
    d = _inputs(B, H, N, d_v, T, W, R, seed=5, strays=False)
    M = d["M"].clone()
    out, tape = sdm.scan_train8(M, *_step(d))
    Mc = d["M"].clone()
    parts = []
    for lo, hi in ((0, 1), (1, 1), (1, 9), (9, 21)):
        part = [d[k][:, :, lo:hi].contiguous() for k in STEP]
        parts.append(sdm.scan_train8(Mc, *part))
    assert torch.equal(M, Mc) and torch.equal(out, torch.cat([p[0] for p in parts], 2))
    assert torch.equal(tape[0], torch.cat([p[1][0] for p in parts], 3))
    assert torch.equal(tape[1], torch.cat([p[1][1] for p in parts], 3))
    empty = [d[k][:, :, :0].contiguous() for k in STEP]
    G = torch.randn_like(M)
    keep = G.clone()
    g = sdm.scan_backward8(*empty, parts[1][1], d["dout"][:, :, :0].contiguous(), G)
    assert torch.equal(G, keep) and g["dwk"].shape == (B, H, 0, W)
    assert sdm.tape8_read(parts[1][1]).shape == (B, H, 0, W + R, d_v)


def test_on_another_stream_and_captured():
    """A side stream, and one graph of the training step replayed on changed
    inputs with eager work in between, give the bits of plain calls."""
    import torch

    sdm = _sdm()
    B, H, N, d_v, T, W, R = 2, 3, 60, 64, 17, 8, 8
    d = _inputs(B, H, N, d_v, T, W, R, seed=8, strays=False)
    start = d["M"].clone()

    def run(stream=None):
        M = start.clone()
        G = torch.zeros_like(M)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        out, tape = sdm.scan_train8(M, *_step(d), stream=stream)
        rows = sdm.tape8_read(tape, torch.bfloat16, stream=stream)
        g = sdm.scan_backward8(*_step(d), tape, d["dout"], G, stream=stream)
        return [out, M, G, rows, *g.values()]

    want = run()
    side = torch.cuda.Stream()
    got = run(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for k in range(3):
        d["v"].copy_(torch.randn_like(d["v"]))
        d["dout"].copy_(torch.randn_like(d["dout"]))
        graph.replay()
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held)), k


def test_backward8_without_allocation():
    """With out and a workspace the call makes no tensors and gives the same bits."""
    import torch

    sdm = _sdm()
    B, H, N, d_v, T, W, R = 1, 2, 40, 32, 9, 5, 6
    d = _inputs(B, H, N, d_v, T, W, R, seed=2, strays=False)
    _, tape = sdm.scan_train8(d["M"].clone(), *_step(d))
    Ga, Gb = (torch.zeros_like(d["M"]) for _ in range(2))
    a = sdm.scan_backward8(*_step(d), tape, d["dout"], Ga)
    out = {k: torch.full_like(x, 3.0) for k, x in a.items()}
    ws = torch.full((sdm.lib().sdm_scan_backward8_workspace_size(B, H, d_v, T, W, R),), 1,
                    dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    b = sdm.scan_backward8(*_step(d), tape, d["dout"], Gb, workspace=ws, out=out)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    assert b is out and torch.equal(Ga, Gb) and all(torch.equal(a[k], out[k]) for k in a)


def test_a_side_stream_owns_what_the_call_makes():
    """Called on a side stream with nothing passed in, and with the current stream
    filling fresh memory of the workspace's size right after: the workspace the
    call made must not be among it."""
    import torch

    sdm = _sdm()
    B, H, N, d_v, T, W, R = 2, 2, 300, 64, 400, 32, 32
    d = _inputs(B, H, N, d_v, T, W, R, seed=12, strays=False)
    _, tape = sdm.scan_train8(d["M"].clone(), *_step(d))
    G0 = torch.randn_like(d["M"])
    Ga = G0.clone()
    want = sdm.scan_backward8(*_step(d), tape, d["dout"], Ga)
    size = sdm.lib().sdm_scan_backward8_workspace_size(B, H, d_v, T, W, R)
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        Gb = G0.clone()
        torch.cuda.synchronize()
        got = sdm.scan_backward8(*_step(d), tape, d["dout"], Gb, stream=handle)
        for _ in range(3):
            torch.full((size // 4,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        assert torch.equal(Ga, Gb) and all(torch.equal(want[k], got[k]) for k in want)


def test_two_streams_at_once():
    """Two training steps side by side on two streams, each with its own workspace."""
    import torch

    sdm = _sdm()
    size = (2, 4, 120, 128, 150, 16, 16)
    B, H, N, d_v, T, W, R = size
    ds = [_inputs(*size, seed=k, strays=False) for k in (20, 21)]

    def run(d, stream):
        M, G = d["M"].clone(), torch.zeros_like(d["M"])
        out, tape = sdm.scan_train8(M, *_step(d), stream=stream)
        g = sdm.scan_backward8(*_step(d), tape, d["dout"], G, stream=stream)
        return [M, out, *tape, G, *g.values()]

    want = [run(d, None) for d in ds]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                got.append(run(d, s))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_two_graphs_share_a_workspace():
    """Reverse passes of two sizes captured into two graphs over one workspace,
    replayed in turn on one stream."""
    import torch

    sdm = _sdm()
    sizes = [(1, 2, 50, 64, 30, 8, 8), (4, 4, 90, 128, 21, 12, 16)]
    ds = [_inputs(*z, seed=k, strays=False) for k, z in enumerate(sizes)]
    need = max(sdm.lib().sdm_scan_backward8_workspace_size(z[0], z[1], *z[3:]) for z in sizes)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for d in ds:
        _, tape = sdm.scan_train8(d["M"].clone(), *_step(d))
        G0 = torch.randn_like(d["M"])
        Gw = G0.clone()
        want = sdm.scan_backward8(*_step(d), tape, d["dout"], Gw)
        G, out = G0.clone(), {k: torch.empty_like(x) for k, x in want.items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            G.copy_(G0)
            sdm.scan_backward8(*_step(d), tape, d["dout"], G, workspace=ws, out=out)
        graphs.append((graph, G, Gw, out, want, G0, tape))
    for k in range(4):
        graphs[k % 2][0].replay()
        graphs[1 - k % 2][0].replay()
        torch.cuda.synchronize()
        for _, G, Gw, out, want, *_ in graphs:
            assert torch.equal(G, Gw) and all(torch.equal(out[n], want[n]) for n in want), k
            G.fill_(5.0)
            for x in out.values():
                x.fill_(5.0)


def test_the_layer_in_4_and_8_bits():
    """A training step as it would be used: tokens and weights in 4 bits through
    the projections, both selections, the forward with its 8-bit tape, the
    reverse pass and the gradients of the halves and of M0 -- against the plain
    chain in float64, from the projected halves the GPU gave (selections are
    discontinuous in them)."""
    import torch

    import oracle

    sdm = _sdm()
    B, T, d_model, H, n, d_v, K = 2, 25, 256, 2, 16, 32, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(B, T, d_model, generator=g, device="cuda").bfloat16()
    Wt = torch.randn(H, 4 * n + d_v + 2, d_model, generator=g, device="cuda") / d_model ** .5
    s1, s2, q1, q2, v, alpha, beta = sdm.project_mx4(*sdm.mx4_quantize(X), *sdm.mx4_quantize(Wt), n)
    M0 = 0.02 * torch.randn(H, n * n, d_v, generator=g, device="cuda")
    M = sdm.state_init(M0, B)
    widx, _, wk = sdm.select(s1, s2, K)
    ridx, _, rw = sdm.select(q1, q2, K)
    out, tape = sdm.scan_train8(M, widx, wk, ridx, rw, v, alpha, beta)
    dout = torch.randn(B, H, T, d_v, generator=g, device="cuda")
    seen, first = sdm.touch_prepare(widx, ridx, n * n)
    G = torch.empty_like(M)
    gr = sdm.scan_backward8(widx, wk, ridx, rw, v, alpha, beta, tape, dout, G, first=first)
    ds1, ds2 = sdm.select_backward(widx, wk, gr["dwk"], n)
    dM0 = sdm.state_init_backward(G, seen=seen)
    rows = sdm.tape8_read(tape).double().cpu().numpy()
    x = {k: t.double().cpu().numpy() for k, t in
         dict(wk=wk, rw=rw, v=v, alpha=alpha, beta=beta, dout=dout, M0=M0).items()}
    wi, ri = widx.cpu().numpy(), ridx.cpu().numpy()
    total = np.zeros((H, n * n, d_v))
    for b, h in np.ndindex(B, H):
        Mo = x["M0"][h].copy()
        a = (wi[b, h], x["wk"][b, h], ri[b, h], x["rw"][b, h], x["v"][b, h], x["alpha"][b, h],
             x["beta"][b, h])
        oo, _ = O.forward(Mo, *a)
        assert np.abs(oo - out[b, h].cpu().numpy()).max() <= 1e-5
        Go = np.zeros((n * n, d_v))
        go = O.backward(Go, *a, rows[b, h], x["dout"][b, h])
        for k in go:
            _close(gr[k][b, h].cpu().numpy(), go[k], k)
        total[h] += Go
        d1, d2 = oracle.select_backward(wi[b, h], wk[b, h].cpu().numpy(), go["dwk"].astype(np.float32), n)
        _close(ds1[b, h].cpu().numpy(), d1, "ds1")
        _close(ds2[b, h].cpu().numpy(), d2, "ds2")
    _close(dM0.cpu().numpy(), total, "dM0")
