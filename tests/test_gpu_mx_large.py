"""The microscaled operators past 2^31 and 2^32: element counts, byte offsets and
row records that need 64-bit arithmetic, and tapes close to 2 GiB a memory.
Expected values come from the same calls on small pieces (whose own tests hold
them to the plain forms), so everything is compared bit for bit on the GPU."""
import pytest

pytestmark = pytest.mark.gpu


def _sdm():
    import sparse_memory_linear_sdm_amd as sdm

    return sdm


@pytest.fixture(autouse=True)
def _give_memory_back():
    import torch

    yield
    torch.cuda.empty_cache()


def test_mx4_matrix_above_2_34_elements():
    """[2^18 + 16, 65536] bf16 (34 GB): read back from 4 bits and quantised again.
    A quantised matrix's values have that very quantised form."""
    import torch

    sdm = _sdm()
    piece, cols, times = 2048, 65536, 128
    rows = piece * times + 16
    x = torch.randn(piece, cols, device="cuda", dtype=torch.bfloat16)
    c, s = sdm.mx4_quantize(x)
    want = sdm.mx4_dequantize(c, s, torch.bfloat16)
    codes = torch.empty(rows, cols // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(cols // 128, rows, 4, dtype=torch.uint8, device="cuda")
    for k in range(times + 1):
        at = slice(k * piece, min((k + 1) * piece, rows))
        codes[at] = c[:at.stop - at.start]
        scales[:, at] = s[:, :at.stop - at.start]
    big = sdm.mx4_dequantize(codes, scales, torch.bfloat16)
    assert big.numel() > 1 << 34
    for k in range(times + 1):
        got = big[k * piece:(k + 1) * piece]
        assert torch.equal(got, want[:got.shape[0]]), k
    codes2, scales2 = sdm.mx4_quantize(big)
    assert torch.equal(scales2, scales)
    for k in range(times + 1):
        got = codes2[k * piece:(k + 1) * piece]
        assert torch.equal(got, c[:got.shape[0]]), k


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_tape8_of_more_than_2_29_records(dtype):
    """Five memories of 2^27 - 64 records each: rows as from one memory's call."""
    import torch

    sdm = _sdm()
    B, d_v, S = 5, 16, 64
    T = (1 << 21) - 1
    codes = torch.randint(-127, 128, (B, 1, 1, T, S, 16), dtype=torch.int8, device="cuda")
    scales = torch.randint(2, 250, (B, 1, 1, T, S), dtype=torch.uint8, device="cuda")
    assert B * T * S > 1 << 29
    dtype, bits = getattr(torch, dtype), torch.int16 if dtype == "bfloat16" else torch.int32
    rows = sdm.tape8_read((codes, scales), dtype)
    for b in range(B):
        one = sdm.tape8_read((codes[b:b + 1], scales[b:b + 1]), dtype)
        assert torch.equal(one[0].view(bits), rows[b].view(bits)), b


def test_project_mx4_outputs_above_2_31_values():
    """2^21 + 5 tokens x 1024 half scores: every output's first, last and middle
    tokens as in calls on those tokens alone (one block of 128 columns of K: each
    value is one exact sum of products rounded once per block of the matrix
    instruction, the same in every tile)."""
    import torch

    sdm = _sdm()
    T, n, d_v, d_model = (1 << 21) + 5, 1024, 16, 128
    P = 4 * n + d_v + 2
    xq, xs = sdm.mx4_quantize(torch.randn(1, T, d_model, device="cuda", dtype=torch.bfloat16))
    w = sdm.mx4_quantize(torch.randn(1, P, d_model, device="cuda", dtype=torch.bfloat16))
    got = sdm.project_mx4(xq, xs, *w, n)
    assert got[0].numel() > 1 << 31
    for t0 in (0, (T // 2) // 256 * 256, (1 << 21) - 512):
        part = slice(t0, min(t0 + 768, T))
        one = sdm.project_mx4(xq[:, part].contiguous(), xs[:, part].contiguous(), *w, n)
        for a, b in zip(one, got):
            assert torch.equal(a, b[:, :, part]), t0


def _long_inputs(T, N, d_v, W, R):
    import torch

    g = torch.Generator(device="cuda").manual_seed(3)

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def rows(K):  # distinct within a step: an odd stride over a power-of-two table
        start = torch.randint(0, N, (1, 1, T, 1), generator=g, device="cuda")
        stride = 2 * torch.randint(0, N // 2, (1, 1, T, 1), generator=g, device="cuda") + 1
        return ((start + stride * torch.arange(K, device="cuda")) % N).int()

    wk, rw = rand(1, 1, T, W), rand(1, 1, T, R)
    step = [rows(W), wk / wk.sum(-1, keepdim=True), rows(R), rw / rw.sum(-1, keepdim=True),
            rand(1, 1, T, d_v) - 0.5, 0.9 + 0.1 * rand(1, 1, T), rand(1, 1, T)]
    return step, rand(1, 1, N, d_v) - 0.5, rand(1, 1, T, d_v) - 0.5


def test_tape_just_below_2_gib_a_memory():
    """131071 steps of 128 rows of 128 values: forward and reverse pass in one call
    against the same steps in five."""
    import torch

    sdm = _sdm()
    T, N, d_v, W, R = (1 << 17) - 1, 4096, 128, 64, 64
    step, M0, dout = _long_inputs(T, N, d_v, W, R)
    M = M0.clone()
    out, tape = sdm.scan_train8(M, *step)
    assert tape[0].numel() > (1 << 31) - (1 << 15)
    G = torch.zeros_like(M0)
    g = sdm.scan_backward8(*step, tape, dout, G)
    cuts = [0, 1, 40000, 77777, 131064, T]
    Mc, Gc = M0.clone(), torch.zeros_like(M0)
    parts = []
    for lo, hi in zip(cuts, cuts[1:]):
        part = [a[:, :, lo:hi].contiguous() for a in step]
        o, tp = sdm.scan_train8(Mc, *part)
        assert torch.equal(o, out[:, :, lo:hi])
        assert torch.equal(tp[0], tape[0][:, :, :, lo:hi])
        assert torch.equal(tp[1], tape[1][:, :, :, lo:hi])
        parts.append((lo, hi, part, tp))
    assert torch.equal(M, Mc)
    for lo, hi, part, tp in reversed(parts):
        h = sdm.scan_backward8(*part, tp, dout[:, :, lo:hi].contiguous(), Gc)
        for k in h:
            assert torch.equal(h[k], g[k][:, :, lo:hi]), (k, lo)
    assert torch.equal(G, Gc)
