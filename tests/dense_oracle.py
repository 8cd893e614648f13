"""Plain 64-bit forms of the dense recurrence and the norms, and bounds on how
far a 32-bit computation may be off.

Run on the absolute values of the inputs, each form gives the sum of the
magnitudes that enter an output (its "size").  A sum of n products in 32 bits is
within about n * 2^-24 of its size, whatever the order."""
import torch

U32 = 2.0 ** -24  # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def repeat(x, H):
    """[B, Hk, ...] keys or queries for each of H heads."""
    return x.double().repeat_interleave(H // x.shape[1], 1)


def decays(g):
    return torch.exp(g.double())  # exp(-inf) is 0


def linear_forward(S, q, k, v, g):
    """Step by step: (out, S after the last step, S before every step [T, ...])."""
    H = v.shape[1]
    q, k, v, a = repeat(q, H), repeat(k, H), v.double(), decays(g)
    S = S.double()
    out, before = torch.empty_like(v), []
    for t in range(v.shape[2]):
        before.append(S)
        S = a[:, :, t, None, None] * S + k[:, :, t, :, None] * v[:, :, t, None, :]
        out[:, :, t] = (S * q[:, :, t, :, None]).sum(-2)
    return out, S, before


def linear_reverse(S, q, k, v, g, dout, G):
    """The gradients, from the states step by step: dict dq, dk, dv, dg, G."""
    Hk, H = q.shape[1], v.shape[1]
    _, _, before = linear_forward(S, q, k, v, g)
    q, k, v, a, do = repeat(q, H), repeat(k, H), v.double(), decays(g), dout.double()
    G = G.double()
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty_like(a)
    for t in reversed(range(v.shape[2])):
        kt, vt, qt, dot = (x[:, :, t] for x in (k, v, q, do))
        decayed = a[:, :, t, None, None] * before[t]
        after = decayed + kt.unsqueeze(-1) * vt.unsqueeze(-2)
        dq[:, :, t] = (after * dot.unsqueeze(-2)).sum(-1)
        G = G + qt.unsqueeze(-1) * dot.unsqueeze(-2)  # of the state after step t
        dk[:, :, t] = (G * vt.unsqueeze(-2)).sum(-1)
        dv[:, :, t] = (G * kt.unsqueeze(-1)).sum(-2)
        dg[:, :, t] = (G * decayed).sum((-1, -2))
        G = a[:, :, t, None, None] * G
    share = (Hk, H // Hk)
    return dict(dq=dq.unflatten(1, share).sum(2), dk=dk.unflatten(1, share).sum(2), dv=dv, dg=dg,
                G=G)


def sizes_forward(S, q, k, v, g):
    return linear_forward(S.abs(), q.abs(), k.abs(), v.abs(), g)


def sizes_reverse(S, q, k, v, g, dout, G):
    """The sums of magnitudes of the gradients."""
    return linear_reverse(S.abs(), q.abs(), k.abs(), v.abs(), g, dout.abs(), G.abs())


def terms(q, v):
    """Additions on the way to one output, at most: the inner sizes, the steps
    (each scaled once), parts of operands and a few roundings of decays."""
    return q.shape[-1] + v.shape[-1] + 2 * v.shape[2] + 64


def bound(size, dtype, n, operands=0):
    """Of an output of `dtype` whose sums are 32-bit and whose operands were
    rounded `operands` times to dtype."""
    return size * (HALF[dtype] * (1 + operands) * (1 + HALF[dtype]) + n * U32) + 1e-30


def check(name, got, want, limit):
    got, want, limit = got.double().cpu(), want.cpu(), limit.cpu()
    assert got.shape == want.shape, name
    off = (got - want).abs()
    bad = ~(off <= limit)  # NaN is bad
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off; worst "
                           f"{(off / limit).nan_to_num(1e9).max():.3g} of its bound")


# ---- norms

def norm_forward(y, w, z=None, x=None, scale=1.0, eps=1e-6, heads=False):
    y = y.double()
    out = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double() * scale
    if heads:
        out = out.transpose(1, 2).flatten(2)
    if z is not None:
        out = out * z.double() * torch.sigmoid(z.double())
    return out if x is None else x.double() + out


def norm_reverse(dout, y, w, z=None, scale=1.0, eps=1e-6, skip=None, heads=False):
    """By the formulas: dict dy, dw, dz."""
    d = y.shape[-1]
    y = y.double()
    rows = lambda t: t.double().unflatten(-1, (-1, d)).transpose(1, 2) if heads else t.double()  # noqa: E731
    back = lambda t: t.transpose(1, 2).flatten(2) if heads else t  # noqa: E731
    D, r = rows(dout) * scale, 1 / (y.square().mean(-1, keepdim=True) + eps).sqrt()
    n, w = y * r, w.double()
    grads = {}
    a = torch.ones_like(y)
    if z is not None:
        zr = rows(z)
        s = torch.sigmoid(zr)
        a = zr * s
        grads["dz"] = back(D * n * w * s * (1 + zr * (1 - s)))
    grads["dw"] = (D * a * n).flatten(0, -2).sum(0)
    m = D * a * w
    grads["dy"] = r * (m - n * (m * n).mean(-1, keepdim=True))
    if skip is not None:
        grads["dy"] = grads["dy"] + skip.double()
    return grads
