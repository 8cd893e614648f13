"""One layer as a user strings it together: the norm before a block, the token
projections, the dense recurrence with the projections' forget gate as its
decay, the heads' norm with its gate, and the norm after the block with
residual scale and the next block's norm; then the gradients back through all
of it, and a token by token run that continues a prompt's state.

Bound for fp32: each of the five stages keeps its values within n * 2^-24 of
the magnitudes they are summed from, n < 500 (d_k + d_v + 2 T + 64 for the
recurrence, d + 40 for a norm); these magnitudes are at most about ten times
the values' norm, so a chain is within 5 * 500 * 10 * 2^-24 = 1.5e-3 of it."""
import pytest
import torch

from tests import dense_oracle as O

pytestmark = pytest.mark.gpu

CHAIN = 1.5e-3
B, H, T, n, d_v = 2, 3, 90, 64, 32
D = H * d_v  # the layer's width after the heads' norm


def _near(name, got, want, bound=CHAIN):
    got, want = got.double().cpu(), want.detach().double().cpu()
    off = float((got - want).norm() / want.norm())
    assert off <= bound, f"{name}: {off}"


def _inputs():
    r = torch.Generator().manual_seed(31)
    randn = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    P = 4 * n + d_v + 2
    Wt = randn(H, P, 128) / 11
    Wt[:, -2] += 0.3  # forget gates mostly open
    return dict(x0=randn(B, T, 128), w0=1 + 0.1 * randn(128), Wt=Wt, z=randn(B, T, D), w1=1 + 0.1 * randn(d_v),
                x=randn(B, T, D), w2=1 + 0.1 * randn(D), w3=1 + 0.1 * randn(D), S=0.3 * randn(B, H, n, d_v),
                dx=randn(B, T, D), dnext=randn(B, T, D), dS=0.1 * randn(B, H, n, d_v))


def _front(a):
    import sparse_memory_linear_sdm_amd as sdm

    h = sdm.norm(a["x0"].cuda(), a["w0"].cuda())
    s1, _, q1, _, v, alpha, _ = sdm.project(h.bfloat16(), a["Wt"].cuda().bfloat16(), n)
    want = O.norm_forward(a["x0"], a["w0"])
    O.check("h", h, want, want.abs() * (128 + 41) * O.U32 + 1e-30)
    return s1 / 8, q1 / 8, v, alpha


def test_a_layer_and_its_gradients():
    import sparse_memory_linear_sdm_amd as sdm

    a = _inputs()
    k, q, v, alpha = _front(a)
    g = alpha.log()
    d = {m: t.cuda() for m, t in a.items()}
    S = d["S"].clone()
    out, tape = sdm.linear_scan_train(S, q, k, v, g)
    y = sdm.norm(out, d["w1"], z=d["z"], heads=True)
    x, behind = sdm.norm(y, d["w2"], x=d["x"], scale=0.5, next_w=d["w3"])

    back = sdm.norm_backward(d["dnext"], x, d["w3"], skip=d["dx"])
    dx = back["dy"]  # the residual's gradient as well
    after = sdm.norm_backward(dx, y, d["w2"], scale=0.5)
    heads = sdm.norm_backward(after["dy"], out, d["w1"], z=d["z"], heads=True)
    G = d["dS"].clone()
    grads = sdm.linear_backward(q, k, v, g, tape, heads["dy"], G)

    # the same in 64 bits, by automatic differentiation
    leaf = {m: t.double().cpu().requires_grad_() for m, t in
            dict(q=q, k=k, v=v, g=g, S=a["S"], z=a["z"], w1=a["w1"], x=a["x"], w2=a["w2"], w3=a["w3"]).items()}
    state, outs = leaf["S"], []
    for t in range(T):
        state = torch.exp(leaf["g"][:, :, t, None, None]) * state + \
            leaf["k"][:, :, t, :, None] * leaf["v"][:, :, t, None, :]
        outs.append((state * leaf["q"][:, :, t, :, None]).sum(-2))
    w_out = torch.stack(outs, 2)
    rms = lambda u: u / (u.square().mean(-1, keepdim=True) + 1e-6).sqrt()  # noqa: E731
    w_y = (rms(w_out) * leaf["w1"]).transpose(1, 2).flatten(2) * leaf["z"] * torch.sigmoid(leaf["z"])
    w_x = leaf["x"] + 0.5 * rms(w_y) * leaf["w2"]
    w_next = rms(w_x) * leaf["w3"]
    for name, got, want in (("out", out, w_out), ("S", S, state), ("y", y, w_y), ("x", x, w_x),
                            ("next", behind, w_next)):
        _near(name, got, want)
    loss = (w_x * a["dx"].double()).sum() + (w_next * a["dnext"].double()).sum() + \
        (state * a["dS"].double()).sum()
    want = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    for name, got in (("q", grads["dq"]), ("k", grads["dk"]), ("v", grads["dv"]), ("g", grads["dg"]),
                      ("S", G), ("z", heads["dz"]), ("w1", heads["dw"]), ("x", dx), ("w2", after["dw"]),
                      ("w3", back["dw"])):
        _near("gradient of " + name, got, want[name])


def test_a_prompt_then_tokens():
    """A prompt's state goes on with single tokens: equal to one longer prompt."""
    import sparse_memory_linear_sdm_amd as sdm

    a = _inputs()
    k, q, v, alpha = _front(a)
    g, w, z = alpha.log(), a["w1"].cuda(), a["z"].cuda()
    whole = a["S"].cuda()
    want = sdm.norm(sdm.linear_scan(whole, q, k, v, g), w, z=z, heads=True)
    S, cut = a["S"].cuda(), T - 5
    part = lambda lo, hi: [t[:, :, lo:hi].contiguous() for t in (q, k, v, g)]  # noqa: E731
    got = [sdm.norm(sdm.linear_scan(S, *part(0, cut)), w, z=z[:, :cut].contiguous(), heads=True)]
    for t in range(cut, T):
        o = sdm.linear_step(S, *(u.squeeze(2) for u in part(t, t + 1)))
        got.append(sdm.norm(o.unsqueeze(2), w, z=z[:, t:t + 1].contiguous(), heads=True))
    _near("outputs", torch.cat(got, 1), want)
    _near("state", S, whole)


def test_a_forgetting_gate():
    """A forget gate of exactly 0 (its logarithm -inf) starts the state anew."""
    import sparse_memory_linear_sdm_amd as sdm

    a = _inputs()
    k, q, v, alpha = _front(a)
    alpha[:, :, 40] = 0
    S, T0 = a["S"].cuda(), 40
    out = sdm.linear_scan(S, q, k, v, alpha.log())
    empty = torch.zeros_like(S)
    tail = [t[:, :, T0:].contiguous() for t in (q, k, v, alpha.log())]
    _near("out", out[:, :, T0:], sdm.linear_scan(empty, *tail))
    _near("S", S, empty)
