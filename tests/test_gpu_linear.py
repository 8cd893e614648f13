"""The dense recurrence with a decay for each head against its 64-bit form,
step by step.  Bounds: sums of n terms in 32 bits; bf16 outputs are rounded
once, and their operands (the state, the products q.k, and in the reverse pass
those and the state's gradient) once more."""
import math

import pytest
import torch

from tests import dense_oracle as O

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def make(B, H, Hk, T, dk, dv, dtype, seed=0, resets=False, grads=False):
    """Inputs on the CPU: dict S, q, k, v, g (and dout, G)."""
    r = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    a = dict(S=randn(B, H, dk, dv), q=(randn(B, Hk, T, dk) / math.sqrt(dk)).to(dtype),
             k=randn(B, Hk, T, dk).to(dtype), v=randn(B, H, T, dv).to(dtype),
             g=-torch.exp(randn(B, H, T) - 2.5))
    if resets and T:
        hit = torch.rand(B, H, T, generator=r) < 0.05
        kinds = torch.tensor([-math.inf, -128.0, -1e30])
        a["g"] = torch.where(hit, kinds[torch.randint(0, 3, (B, H, T), generator=r)], a["g"])
    if grads:
        a["dout"], a["G"] = randn(B, H, T, dv).to(dtype), randn(B, H, dk, dv)
    return a


def dev(a):
    return {n: x.cuda() for n, x in a.items()}


ORDER = ("S", "q", "k", "v", "g")


def forward_bounds(a):
    out, S, before = O.linear_forward(*(a[n] for n in ORDER))
    sout, sS, _ = O.sizes_forward(*(a[n] for n in ORDER))
    n, dtype = O.terms(a["q"], a["v"]), a["q"].dtype
    return (out, O.bound(sout, dtype, n, operands=dtype == BF16),
            S, O.bound(sS, F32, n), before)


def check_forward(a, out, S):
    want, wlim, wS, slim, _ = forward_bounds(a)
    O.check("out", out, want, wlim)
    O.check("S", S, wS, slim)


def check_reverse(a, got, G):
    args = [a[n] for n in ORDER] + [a["dout"], a["G"]]
    want, size = O.linear_reverse(*args), O.sizes_reverse(*args)
    n, dtype = O.terms(a["q"], a["v"]) + a["v"].shape[1], a["q"].dtype
    for name in ("dq", "dk", "dv"):
        O.check(name, got[name], want[name],
                O.bound(size[name], dtype, n, operands=dtype == BF16))
    O.check("dg", got["dg"], want["dg"], O.bound(size["dg"], F32, n + a["q"].shape[-1] * 2))
    O.check("G", G, want["G"], O.bound(size["G"], F32, n))


def run_scan(a, **kw):
    import sparse_memory_linear_sdm_amd as sdm

    d = dev(a)
    out = sdm.linear_scan(*(d[n] for n in ORDER), **kw)
    return out, d["S"]


def run_train(a):
    import sparse_memory_linear_sdm_amd as sdm

    d = dev(a)
    out, tape = sdm.linear_scan_train(*(d[n] for n in ORDER))
    grads = sdm.linear_backward(d["q"], d["k"], d["v"], d["g"], tape, d["dout"], d["G"])
    return out, d["S"], tape, grads, d["G"]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_scan_every_head_size(dk, dv, dtype):
    a = make(2, 4, 2, 101, dk, dv, dtype, seed=dk + dv, resets=True)
    check_forward(a, *run_scan(a))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129])
def test_scan_every_tail(T, dtype):
    a = make(1, 3, 1, T, 64, 64, dtype, seed=T, resets=True)
    check_forward(a, *run_scan(a))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [255, 256, 300, 513, 1000])
def test_scan_in_segments(T, dtype):
    """One memory: the steps are cut into segments, joined by their states."""
    import sparse_memory_linear_sdm_amd as sdm

    need = sdm.lib().sdm_linear_scan_workspace_size(int(dtype == BF16), 1, 2, 64, 32, T)
    assert (need > 0) == (T >= (512 if dtype == BF16 else 256) - 63)
    a = make(1, 2, 2, T, 64, 32, dtype, seed=T)
    check_forward(a, *run_scan(a))


@pytest.mark.parametrize("dtype,H,T", [(F32, 64, 300), (BF16, 64, 600), (F32, 40, 430), (F32, 128, 2080),
                                      (BF16, 128, 4100)])
def test_segments_of_several_chunks(dtype, H, T):
    a = make(1, H, H // 4, T, 32, 32, dtype, seed=T, grads=T < 1000)
    if T < 1000:
        out, S, _, grads, G = run_train(a)
        check_reverse(a, grads, G)
    else:
        out, S = run_scan(a)
    check_forward(a, out, S)


@pytest.mark.parametrize("dtype,H,T", [(F32, 2, 128), (F32, 2, 129), (F32, 5, 200), (BF16, 2, 256),
                                      (BF16, 2, 257), (BF16, 5, 400), (BF16, 65, 300)])
def test_wide_heads_of_few_chunks(dtype, H, T):
    """Heads of 128 x 128 are cut from five chunks on, for up to 64 memories."""
    import sparse_memory_linear_sdm_amd as sdm

    chunk = 64 if dtype == BF16 else 32
    need = sdm.lib().sdm_linear_scan_workspace_size(int(dtype == BF16), 1, H, 128, 128, T)
    assert (need > 0) == (H <= 64 and T > 4 * chunk)
    a = make(1, H, H, T, 128, 128, dtype, seed=T, resets=True, grads=H < 65)
    if H < 65:
        out, S, _, grads, G = run_train(a)
        check_reverse(a, grads, G)
    else:
        out, S = run_scan(a)
    check_forward(a, out, S)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("g", [0.0, -0.0, -1e-6, -100.0, -127.9, -math.inf, -3e38])
def test_scan_of_one_decay(g, dtype):
    a = make(1, 2, 1, 150, 32, 64, dtype, seed=5)
    a["g"].fill_(g)
    check_forward(a, *run_scan(a))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_steps_that_forget_leave_nothing(dtype):
    """Packed sequences: behind a reset the outputs do not depend on what came
    before, bit for bit."""
    a = make(1, 2, 2, 200, 64, 64, dtype, seed=6)
    for at in (70, 128, 150):
        a["g"][:, :, at] = -math.inf
    b = {n: x.clone() for n, x in a.items()}
    b["S"] *= 3
    for n in ("k", "v", "q"):
        b[n][:, :, :128] *= -2
    (x, Sx), (y, Sy) = run_scan(a), run_scan(b)
    assert torch.equal(x[:, :, 128:], y[:, :, 128:]) and torch.equal(Sx, Sy)
    assert not torch.equal(x[:, :, :70], y[:, :, :70])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cut", [1, 64, 77])
def test_scan_in_two_calls(cut, dtype):
    import sparse_memory_linear_sdm_amd as sdm

    a = make(2, 2, 1, 150, 64, 128, dtype, seed=7)
    d = dev(a)
    outs = []
    for lo, hi in ((0, cut), (cut, 150)):
        part = [d[n][:, :, lo:hi].contiguous() for n in ORDER[1:]]
        outs.append(sdm.linear_scan(d["S"], *part))
    check_forward(a, torch.cat(outs, 2), d["S"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_steps_one_by_one(dk, dv, dtype):
    """linear_step: fp32 throughout, outputs rounded once."""
    import sparse_memory_linear_sdm_amd as sdm

    a = make(3, 4, 2, 5, dk, dv, dtype, seed=8, resets=True)
    d = dev(a)
    outs = [sdm.linear_step(d["S"], *(d[n][:, :, t].contiguous() for n in ORDER[1:]))
            for t in range(5)]
    want, _, S, slim, _ = forward_bounds(a)
    sout = O.sizes_forward(*(a[n] for n in ORDER))[0]
    O.check("out", torch.stack(outs, 2), want, O.bound(sout, dtype, O.terms(a["q"], a["v"])))
    O.check("S", d["S"], S, slim)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [0, 1, 63, 130])
def test_train_is_the_scan_and_its_tape_the_states(T, dtype):
    import sparse_memory_linear_sdm_amd as sdm

    a = make(1, 2, 1, T, 64, 32, dtype, seed=9)
    d, e = dev(a), dev(a)
    out, tape = sdm.linear_scan_train(*(d[n] for n in ORDER))
    again = sdm.linear_scan(*(e[n] for n in ORDER))
    assert torch.equal(out, again) and torch.equal(d["S"], e["S"])
    chunk = 64 if dtype == BF16 else 32
    assert tape.shape == (1, 2, -(-T // chunk), 64, 32)
    if T:
        _, _, _, slim, before = forward_bounds(a)
        for c in range(tape.shape[2]):
            sS = O.sizes_forward(a["S"], *(a[n][:, :, :c * chunk] for n in ORDER[1:]))[1]
            O.check(f"tape {c}", tape[:, :, c], before[c * chunk],
                    O.bound(sS, F32, O.terms(a["q"], a["v"])))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk", [32, 64, 128])
@pytest.mark.parametrize("dv", [32, 64, 128])
def test_backward_every_head_size(dk, dv, dtype):
    a = make(2, 2, 2, 101, dk, dv, dtype, seed=dk - dv, resets=True, grads=True)
    out, S, _, grads, G = run_train(a)
    check_forward(a, out, S)
    check_reverse(a, grads, G)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 2, 16, 17, 31, 32, 33, 48, 63, 64, 65, 128, 129])
def test_backward_every_tail(T, dtype):
    a = make(1, 3, 3, T, 64, 32, dtype, seed=T, resets=True, grads=True)
    _, _, _, grads, G = run_train(a)
    check_reverse(a, grads, G)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,Hk", [(4, 1), (6, 2), (3, 3)])
def test_backward_of_shared_keys(H, Hk, dtype):
    a = make(2, H, Hk, 70, 64, 64, dtype, seed=H, grads=True)
    _, _, _, grads, G = run_train(a)
    check_reverse(a, grads, G)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [256, 600, 1030])
@pytest.mark.parametrize("Hk", [1, 2])
def test_backward_in_segments(T, Hk, dtype):
    a = make(1, 2, Hk, T, 32, 64, dtype, seed=T, resets=T == 600, grads=True)
    out, S, _, grads, G = run_train(a)
    check_forward(a, out, S)
    check_reverse(a, grads, G)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv,T,Hk", [(32, 32, 64, 2), (64, 128, 150, 1), (128, 64, 97, 2),
                                        (32, 64, 700, 2)])
def test_gradients_of_gates_that_forget_much(dk, dv, T, Hk, dtype):
    """dg of a step is the sum of the paths across it, in fp32's precision of
    those: steps that leave 1e-2 to 1e-26 of the state have paths that are as
    much smaller than the ones beside them."""
    a = make(1, 2, Hk, T, dk, dv, dtype, seed=T, grads=True)
    r = torch.Generator().manual_seed(T + dk)
    hit = torch.rand(a["g"].shape, generator=r) < 0.1
    a["g"] = torch.where(hit, -5 - 55 * torch.rand(a["g"].shape, generator=r), a["g"])
    _, _, _, grads, G = run_train(a)
    check_reverse(a, grads, G)


def test_no_steps():
    import sparse_memory_linear_sdm_amd as sdm

    a = dev(make(1, 2, 1, 0, 32, 32, F32, grads=True))
    S, G = a["S"].clone(), a["G"].clone()
    out, tape = sdm.linear_scan_train(*(a[n] for n in ORDER))
    grads = sdm.linear_backward(a["q"], a["k"], a["v"], a["g"], tape, a["dout"], a["G"])
    assert out.shape == (1, 2, 0, 32) and grads["dq"].shape == (1, 1, 0, 32)
    assert torch.equal(a["S"], S) and torch.equal(a["G"], G)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_twice_the_same_bits(dtype):
    a = make(1, 4, 2, 700, 64, 64, dtype, seed=11, grads=True)
    x, y = run_train(a), run_train(a)
    for u, v in zip(x, y):
        for n in (u if isinstance(u, dict) else [None]):
            p, q = (u, v) if n is None else (u[n], v[n])
            assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nothing_outside_the_outputs_is_written(dtype):
    import sparse_memory_linear_sdm_amd as sdm

    B, H, Hk, T, dk, dv = 1, 2, 1, 333, 64, 32
    d = dev(make(B, H, Hk, T, dk, dv, dtype, seed=12, grads=True))
    chunks = -(-T // (64 if dtype == BF16 else 32))
    guarded = {}

    def guard(name, shape, t, content=None):
        n = math.prod(shape)
        buf = torch.full((n + 128,), 7.0, dtype=t, device="cuda")
        guarded[name] = (buf, n)
        view = buf[64:64 + n].view(shape)
        if content is not None:
            view.copy_(content)
        return view

    S, G = guard("S", d["S"].shape, F32, d["S"]), guard("G", d["G"].shape, F32, d["G"])
    out, tape = guard("out", (B, H, T, dv), dtype), guard("tape", (B, H, chunks, dk, dv), F32)
    ins = [d[n] for n in ORDER[1:]]
    ws = {}
    for n, need in (("w1", sdm.lib().sdm_linear_scan_workspace_size(int(dtype == BF16), B, H, dk, dv, T)),
                    ("w2", sdm.lib().sdm_linear_backward_workspace_size(int(dtype == BF16), B, H, Hk, dk, dv, T))):
        buf = torch.full((need + 512,), 9, dtype=torch.uint8, device="cuda")
        ws[n] = (buf, need)
    sdm.linear_scan_train(S, *ins, out=out, tape=tape, workspace=ws["w1"][0][256:256 + ws["w1"][1]])
    o = dict(dq=guard("dq", (B, Hk, T, dk), dtype), dk=guard("dk", (B, Hk, T, dk), dtype),
             dv=guard("dv", (B, H, T, dv), dtype), dg=guard("dg", (B, H, T), F32))
    sdm.linear_backward(*ins, tape, d["dout"], G, out=o, workspace=ws["w2"][0][256:256 + ws["w2"][1]])
    torch.cuda.synchronize()
    for name, (buf, n) in guarded.items():
        assert (buf[:64] == 7).all() and (buf[64 + n:] == 7).all(), name
    for name, (buf, n) in ws.items():
        assert (buf[:256] == 9).all() and (buf[256 + n:] == 9).all(), name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_and_replayed(dtype):
    """A training step (segments, shared keys) and a token in one graph, replayed
    between eager calls on the same inputs."""
    import sparse_memory_linear_sdm_amd as sdm

    a = dev(make(1, 2, 1, 600, 64, 64, dtype, seed=13, grads=True))
    ins = [a[n] for n in ORDER[1:]]
    token = [x[:, :, 0].contiguous() for x in ins]
    S, G = a["S"].clone(), a["G"].clone()

    def step():
        out, tape = sdm.linear_scan_train(S, *ins)
        grads = sdm.linear_backward(*ins, tape, a["dout"], G)
        return [out, sdm.linear_step(S, *token), *grads.values()]

    want, wS, wG = [x.clone() for x in step()], S.clone(), G.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        S.copy_(a["S"])
        G.copy_(a["G"])
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        assert torch.equal(S, wS) and torch.equal(G, wG)
        S.copy_(a["S"])
        G.copy_(a["G"])
        assert torch.equal(step()[0], want[0])


def test_two_streams_at_once():
    import sparse_memory_linear_sdm_amd as sdm

    runs = [dev(make(1, 4, 4, 1500, 64, 64, BF16, seed=s)) for s in (20, 21)]
    want = []
    for d in runs:
        S = d["S"].clone()
        want.append((sdm.linear_scan(S, *(d[n] for n in ORDER[1:])), S))
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(3):
        states = [d["S"].clone() for d in runs]
        torch.cuda.synchronize()
        got = [sdm.linear_scan(S, *(d[n] for n in ORDER[1:]), stream=s)
               for d, S, s in zip(runs, states, streams)]
        torch.cuda.synchronize()
        for g, S, (w, wS) in zip(got, states, want):
            assert torch.equal(g, w) and torch.equal(S, wS)
