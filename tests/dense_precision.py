"""Inputs whose results each stand on one product or on few, so that an operand
held in fewer bits shows in full, with bounds counted in half steps of fp32
(2^-24 of the result), and the same results as a computation would have them that
splits operands into fewer bf16 parts or keeps sums of logarithms as one float.

Keys (or queries) that are rows of the identity put one scaled row v_t into one
row of the state (one row dout_t into the state's gradient).  Roundings on the way:
the decay's exponent x, half a step of it: |x| ln 2 <= 4.2 half steps for |x| <= 6;
the power 2; its product with v 1; what three bf16 parts leave 1; the sums of
the parts 3; the decays of further chunks and segments and their sums 4 each."""
import math

import torch

from tests import dense_oracle as O

F32, BF16 = torch.float32, torch.bfloat16
HALF_STEPS = 4.2 + 2 + 1 + 1 + 3


def gentle(shape, r, total):
    """Decays that leave exp(-total) at least over all steps (the last axis)."""
    return -torch.rand(shape, generator=r) * (total / shape[-1])


def one_row_each(T, dk, dv, dtype, seed, writes=None):
    """Key t (of the first min(T, dk) steps, or of `writes`) is row i of the
    identity, query likewise; v, dout and the decays are dense."""
    r = torch.Generator().manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=r)  # noqa: E731
    at = torch.arange(min(T, dk)) if writes is None else torch.tensor(writes)
    keys = torch.zeros(1, 2, T, dk)
    keys[:, :, at, torch.arange(len(at))] = 1
    return dict(S=torch.zeros(1, 2, dk, dv), q=keys.to(dtype), k=keys.to(dtype).clone(),
                v=randn(1, 2, T, dv).to(dtype), g=gentle((1, 2, T), r, 4.0),
                dout=randn(1, 2, T, dv).to(dtype), G=torch.zeros(1, 2, dk, dv))


def one_path_through(state, T, dk, dv, dtype, seed):
    """dg through one element of a state of all 24 bits a step: the state before
    the first step (q and dout rows of the identity, k = v = 0) or the gradient of
    the one behind the last (k and v; q = dout = 0)."""
    r = torch.Generator().manual_seed(seed)
    a = one_row_each(T, dk, dv, dtype, seed)
    rows, cols = (torch.zeros(1, 2, T, d) for d in (dk, dv))
    for t in range(T):
        rows[:, :, t, torch.randint(0, dk, (), generator=r)] = 1
        cols[:, :, t, torch.randint(0, dv, (), generator=r)] = 1
    zk, zv = torch.zeros_like(rows), torch.zeros_like(cols)
    dense = torch.randn(1, 2, dk, dv, generator=r)
    a.update(S=dense, G=torch.zeros_like(dense), q=rows, dout=cols, k=zk, v=zv)
    if state == "G":
        a.update(S=torch.zeros_like(dense), G=dense, q=zk, dout=zv, k=rows, v=cols)
    for n in ("q", "k", "v", "dout"):
        a[n] = a[n].to(dtype)
    return a


def many_resets(T, first, dtype, seed):
    """Steps before `first` forget the state, the others do not; one key, at
    `first`, and queries of all ones in its direction: output t is the decay
    from there to t times v."""
    r = torch.Generator().manual_seed(seed)
    a = one_row_each(T, 32, 32, dtype, seed)
    a["g"][:, :, :first] = -math.inf
    a["g"][:, :, first:] = -0.3 * torch.rand(1, 2, T - first, generator=r)
    a["k"], a["q"] = torch.zeros_like(a["k"]), torch.zeros_like(a["q"])
    a["k"][:, :, first, 3] = 1
    a["q"][:, :, :, 3] = 1
    return a


def bf16_parts(x, n):
    """x (float32) as the sum of n bf16 numbers."""
    total, rest = torch.zeros_like(x, dtype=torch.float64), x.clone()
    for _ in range(n):
        part = rest.bfloat16().float()
        total += part.double()
        rest = rest - part
    return total


def scaled_rows(a, parts):
    """The state behind the last step of one_row_each (one chunk): v times its
    decay in 32 bits, the product in `parts` bf16 parts."""
    L = a["g"].double().cumsum(-1)
    decay = torch.exp(L[..., -1:] - L).float()
    rows = bf16_parts(decay.unsqueeze(-1) * a["v"].float(), parts)
    return a["k"].double().mT @ rows


def decayed_values(a, first, reset, floats):
    """Outputs of many_resets: log2 decays, `reset` for a step that forgets,
    summed in 64 bits and kept as one float or two."""
    x = torch.where(a["g"] <= -128, reset, a["g"].double() * 1.4426950408889634).cumsum(-1)
    hi = x.float()
    lo = (x - hi.double()).float() if floats == 2 else torch.zeros_like(hi)
    e = (hi - hi[..., first:first + 1]) + (lo - lo[..., first:first + 1])
    return torch.exp2(e.double()).unsqueeze(-1) * a["v"][:, :, first:first + 1].double()


def off_in_half_steps(got, want, size):
    """The largest |got - want| in half steps of fp32 of `size`, where it is not 0."""
    off = (got.double().cpu() - want).abs()
    assert not off[size == 0].any()
    return float((off / size.clamp(min=1e-300)).max() / O.U32)
