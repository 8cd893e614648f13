"""The dense recurrence and the norms on arrays past 2^32 bytes: their ends
against small calls on the same values.  Behind a step that forgets the state
nothing depends on what came before, so the tail of a long stream stands alone
(up to the order of 32-bit sums: other chunk borders)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

# sums of at most d_k + d_v + 2 * 300 + 64 terms in 32 bits, about ten times
# below their magnitudes; bf16 operands and outputs half a step (2^-8) each
F32_REL, BF16_REL = 1000 * 10 * 2.0 ** -24, 2 * 2.0 ** -8


def _near(name, got, want, rel):
    off = float((got.double() - want.double()).norm() / want.double().norm())
    assert off <= rel, f"{name}: {off}"


def _stream(B, H, T, d, dtype, seed):
    r = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, scale=1.0):
        x = torch.empty(shape, dtype=dtype, device="cuda")
        flat = x.view(-1)
        for at in range(0, flat.numel(), 1 << 28):  # a bounded fp32 copy at a time
            part = flat[at:at + (1 << 28)]
            part.copy_(torch.randn(part.shape, generator=r, device="cuda") * scale)
        return x

    q, k, v = randn(B, H, T, d, scale=1 / math.sqrt(d)), randn(B, H, T, d), randn(B, H, T, d)
    g = torch.nn.functional.logsigmoid(3 + torch.randn(B, H, T, generator=r, device="cuda"))
    return q, k, v, g, randn


def test_a_scan_past_4_gib():
    import sparse_memory_linear_sdm_amd as sdm

    B, H, T, d = 1, 5, (1 << 22) + 37, 128  # 5.4 GB an array
    q, k, v, g, _ = _stream(B, H, T, d, torch.bfloat16, 1)
    at = T - 230
    g[:, :, at] = -math.inf
    S = torch.ones(B, H, d, d, device="cuda")
    out = sdm.linear_scan(S, q, k, v, g)
    assert out.numel() * 2 > 1 << 32
    tail, end = [x[:, :, at:].contiguous() for x in (q, k, v, g)], torch.zeros_like(S)
    want = sdm.linear_scan(end, *tail)
    _near("out", out[:, :, at:], want, BF16_REL)
    _near("S", S, end, F32_REL)
    head = [x[:, :, :300].contiguous() for x in (q, k, v, g)]
    _near("first", out[:, :, :300], sdm.linear_scan(torch.ones_like(S), *head), BF16_REL)


def test_a_backward_past_4_gib():
    import sparse_memory_linear_sdm_amd as sdm

    B, H, T, d = 1, 1, (1 << 25) + 1001, 32  # 4.3 GB an array and the tape
    q, k, v, g, randn = _stream(B, H, T, d, torch.float32, 2)
    at = T - 230
    g[:, :, at] = -math.inf
    dout, S = randn(B, H, T, d), torch.ones(B, H, d, d, device="cuda")
    G = torch.randn(B, H, d, d, device="cuda")
    end = G.clone()
    _, tape = sdm.linear_scan_train(S, q, k, v, g)
    assert tape.numel() * 4 > 1 << 32
    grads = sdm.linear_backward(q, k, v, g, tape, dout, G)
    tail = [x[:, :, at:].contiguous() for x in (q, k, v, g)]
    _, tape = sdm.linear_scan_train(torch.zeros_like(S), *tail)
    want = sdm.linear_backward(*tail, tape, dout[:, :, at:].contiguous(), end)
    for n in want:
        _near(n, grads[n][:, :, at:], want[n], F32_REL)
    # the first steps see nothing of the last ones either
    g2 = g[:, :, :4000].contiguous()
    g2[:, :, 3000] = -math.inf
    g[:, :, 3000] = -math.inf
    S = torch.ones(B, H, d, d, device="cuda")
    _, tape = sdm.linear_scan_train(S, q, k, v, g)
    G = torch.randn(B, H, d, d, device="cuda")
    grads = sdm.linear_backward(q, k, v, g, tape, dout, G)
    head = [x[:, :, :4000].contiguous() for x in (q, k, v)] + [g2]
    _, tape = sdm.linear_scan_train(torch.ones(B, H, d, d, device="cuda"), *head)
    first = torch.zeros(B, H, d, d, device="cuda")
    want = sdm.linear_backward(*head, tape, dout[:, :, :4000].contiguous(), first)
    for n in want:
        _near(n, grads[n][:, :, :3000], want[n][:, :, :3000], F32_REL)
    _near("G", G, first, F32_REL)


@pytest.mark.parametrize("heads", [False, True])
def test_a_norm_past_4_gib(heads):
    import sparse_memory_linear_sdm_amd as sdm

    d = 128 if heads else 4096
    shape = (2, 8, (1 << 20) + 3, d) if heads else ((1 << 19) + 5, d)  # 8.6 GB
    y = torch.empty(shape, device="cuda").normal_()
    w = torch.rand(d, device="cuda")
    out = sdm.norm(y, w, heads=heads, dtype=torch.bfloat16)
    if heads:
        tail = y[1:, :, -40:].contiguous()
        assert torch.equal(out[1:, -40:], sdm.norm(tail, w, heads=True, dtype=torch.bfloat16))
    else:
        assert torch.equal(out[-40:], sdm.norm(y[-40:], w, dtype=torch.bfloat16))
    grads = sdm.norm_backward(out, y, w, heads=heads)
    if heads:
        want = sdm.norm_backward(out[1:, -40:].contiguous(), tail, w, heads=True)
        assert torch.equal(grads["dy"][1:, :, -40:], want["dy"])
    else:
        want = sdm.norm_backward(out[-40:].contiguous(), y[-40:], w)
        assert torch.equal(grads["dy"][-40:], want["dy"])
    # dw: the rows' products summed, block by block, in 64 bits
    total = torch.zeros(d, dtype=torch.float64, device="cuda")
    rows = y.transpose(1, 2).reshape(-1, d) if heads else y
    o = out.view(-1, d)
    for at in range(0, rows.shape[0], 1 << 17):
        part = rows[at:at + (1 << 17)].double()
        total += (part / (part.square().mean(-1, keepdim=True) + 1e-6).sqrt() * o[at:at + (1 << 17)].double()).sum(0)
    _near("dw", grads["dw"], total, F32_REL)
