"""Measured cases of the microscaled operators: 4-bit projections and the
8-bit training tape.

  quantize   mx4_quantize of a matrix, read back with mx4_dequantize
  project    a prompt's or a decode step's tokens quantised (mx4_quantize) and
             projected with 4-bit weights that were laid out once (project_mx4)
  train      scan_train8: the training forward with its tape in 8 bits, the
             tape read back (tape8_read)
  backward   scan_backward8: the reverse pass from such a tape

`own` false: plain torch operations in 32 bits; `own` true: the calls a user
makes.  exact() is the operators' definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step's activations of the decode workload (64 sequences, d_model = 2nH = 8192)
        dict(name="quantize decode tokens", op="quantize", rows=64, cols=8192, dtype="bf16"),
        # one head's fp32 master weights after an optimiser step (P = 4n + d_v + 2 rows)
        dict(name="quantize head weights f32", op="quantize", rows=4226, cols=16384, dtype="f32"),
        # one token through a small layer: the smallest call, latency only
        dict(name="project one token", op="project", B=1, T=1, H=1, n=64, d_v=16, d_model=128),
        # a decode step: 64 sequences, one token each, weights streamed from memory
        dict(name="project decode", op="project", B=64, T=1, H=4, n=1024, d_v=128, d_model=8192),
        # a ragged batch: odd token count, odd n, d_model not a multiple of 256
        dict(name="project ragged", op="project", B=3, T=37, H=3, n=37, d_v=32, d_model=640),
        # a prompt batch of the mid workload at the layer's full width
        dict(name="project prompts", op="project", B=8, T=4096, H=8, n=1024, d_v=128,
             d_model=16384),
        # the tiny workload: one memory, one column block
        dict(name="train tiny", op="train", B=1, H=1, n=64, d_v=16, T=256, W=8, R=8),
        # few memories and odd counts of steps and slots
        dict(name="train few", op="train", B=1, H=4, n=256, d_v=64, T=301, W=32, R=29),
        # the mid workload's memories and slots over 1024 steps
        dict(name="train mid", op="train", B=8, H=8, n=512, d_v=128, T=1024, W=64, R=64),
        # loss reads the final state: the gradient table comes in filled (dense mode)
        dict(name="backward dense few", op="backward", B=1, H=4, n=256, d_v=64, T=301, W=32, R=29,
             sparse=False),
        dict(name="backward dense mid", op="backward", B=8, H=8, n=512, d_v=128, T=512, W=64,
             R=64, sparse=False),
        # loss reads the outputs only: first touches skip the gradient table (sparse mode)
        dict(name="backward sparse mid", op="backward", B=8, H=8, n=512, d_v=128, T=1024, W=64,
             R=64, sparse=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "project", "project", "train", "backward"])
    if op == "quantize":
        cols = 128 * _log_int(rng, 1, 128)
        return dict(op=op, rows=_log_int(rng, 1, min(33808, (1 << 26) // cols)), cols=cols,
                    dtype=rng.choice(["bf16", "f32"]))
    d_v = rng.choice([16, 32, 64, 128, 256])
    if op == "project":
        while True:
            B, T = _log_int(rng, 1, 64), _log_int(rng, 1, 4096)
            H, n, d_model = _log_int(rng, 1, 8), _log_int(rng, 1, 1024), 128 * _log_int(rng, 1, 128)
            cols = H * (4 * n + d_v + 2)
            if B * T <= 32768 and B * T * cols * d_model < 2e12:
                return dict(op=op, B=B, T=T, H=H, n=n, d_v=d_v, d_model=d_model)
    while True:
        n = rng.choice([rng.randint(16, 64), 128, 256, 512])
        B, H = _log_int(rng, 1, 8), _log_int(rng, 1, 16)
        W, R = rng.randint(1, min(n, 64)), rng.randint(1, min(n, 64))
        T = _log_int(rng, 1, 512)
        if B * H <= 64 and B * H * n * n * d_v < (1 << 31):
            case = dict(op=op, B=B, H=H, n=n, d_v=d_v, T=T, W=W, R=R)
            if op == "backward":
                case["sparse"] = rng.random() < 0.5
            return case


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device=DEV)


def _topk_slots(x1, x2, K):
    """Product-key selection: slots a*n + b of the K largest sums, softmax weights."""
    n = x1.shape[-1]
    v1, a = x1.topk(K)
    v2, b = x2.topk(K)
    s, f = (v1.unsqueeze(-1) + v2.unsqueeze(-2)).flatten(-2).topk(K)
    slot = a.gather(-1, f // K) * n + b.gather(-1, f % K)
    return slot.int().contiguous(), s.softmax(-1).contiguous()


def _selections(g, mem, T, n, K):
    """[mem, T, K] slots and weights, a bounded number of scores at a time."""
    step = max(1, (1 << 27) // (mem * max(n, K * K)))
    parts = [_topk_slots(_randn(g, mem, min(step, T - t), n), _randn(g, mem, min(step, T - t), n), K)
             for t in range(0, T, step)]
    return torch.cat([p[0] for p in parts], 1), torch.cat([p[1] for p in parts], 1)


def _last_touch_masks(widx, ridx, N):
    """[mem, T, 2] int64: bit j of word 0 (1) is set when write (read) slot j's
    row is selected for the last time at that step."""
    mem, T = widx.shape[:2]
    t = torch.arange(T, device=DEV, dtype=torch.int32)[None, :, None]
    last = torch.full((mem, N), -1, dtype=torch.int32, device=DEV)
    for idx in (widx, ridx):
        last.scatter_reduce_(1, idx.flatten(1).long(), t.expand_as(idx).reshape(mem, -1), "amax")
    words = []
    for idx in (widx, ridx):
        hit = last.gather(1, idx.flatten(1).long()).view_as(idx) == t
        bits = torch.arange(idx.shape[-1], device=DEV)
        words.append((hit.long() << bits).sum(-1))
    return torch.stack(words, -1).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    c = case
    if c["op"] == "quantize":
        # channels of unequal size, as activations and weights have
        x = _randn(g, c["rows"], c["cols"]) * torch.exp(_randn(g, c["cols"]))
        return dict(case=c, x=x.bfloat16() if c["dtype"] == "bf16" else x)
    B, H, n, d_v, T = c["B"], c["H"], c["n"], c["d_v"], c["T"]
    if c["op"] == "project":
        P, d = 4 * n + d_v + 2, c["d_model"]
        x = (_randn(g, B, T, d) * torch.exp(0.5 * _randn(g, d))).bfloat16()
        codes, scales = _mx4_codes(_randn(g, H * P, d) / math.sqrt(d))
        return dict(case=c, x=x, wq=codes.view(H, P, d // 2), ws=scales)
    N, W, R = n * n, c["W"], c["R"]
    widx, wk = _selections(g, B * H, T, n, W)
    ridx, rw = _selections(g, B * H, T, n, R)
    s = dict(case=c, widx=widx.view(B, H, T, W), wk=wk.view(B, H, T, W),
             ridx=ridx.view(B, H, T, R), rw=rw.view(B, H, T, R), v=_randn(g, B, H, T, d_v),
             alpha=0.9 + 0.1 * _rand(g, B, H, T), beta=_rand(g, B, H, T))
    if c["op"] == "train":
        s["M"] = 0.02 * _randn(g, B, H, N, d_v)
        return s
    s["dout"] = _randn(g, B, H, T, d_v)
    # rows a state holds after some writes, as the forward's tape keeps them
    nb = d_v // 16
    s["codes"] = torch.empty(B, H, nb, T, W + R, 16, dtype=torch.int8, device=DEV)
    s["scales"] = torch.empty(B, H, nb, T, W + R, dtype=torch.uint8, device=DEV)
    for b in range(B):
        rows = 0.5 * _randn(g, H, nb, T, W + R, 16) * _rand(g, H, 1, T, W + R, 1)
        s["codes"][b], s["scales"][b] = _int8_codes(rows)
    if c["sparse"]:
        s["first"] = _last_touch_masks(widx, ridx, N).view(B, H, T, 2)
        s["G"] = torch.zeros(B, H, N, d_v, device=DEV)
    else:
        s["first"] = None
        s["G"] = 0.1 * _randn(g, B, H, N, d_v)
    return s


# ------------------------------------------------------------------ formats

def _pow2(biased):
    """2^(biased - 127) as float32, biased in [1, 254]."""
    return (biased << 23).view(torch.float32)


def _mx4_blocks(x):
    """x [rows, cols] -> (e2m1 values in units of the block scale [rows, cols/32, 32],
    biased scale exponents [rows, cols/32])."""
    y = x.float().view(x.shape[0], -1, 32)
    e = (y.abs().amax(-1).view(torch.int32) >> 23).sub(2).clamp(min=2)
    y = y * _pow2(254 - e).unsqueeze(-1)
    a = y.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.round(y / step).mul_(step).clamp_(-6, 6), e


def _mx4_codes(x):
    """Packed codes [rows, cols/2] (even column in the low nibble) and scale
    bytes [cols/128, rows, 4] of finite x."""
    q, e = _mx4_blocks(x)
    a = q.abs()
    mag = torch.where(a <= 2, 2 * a, torch.where(a < 6, a + 2, 7)).to(torch.uint8)
    code = (mag | ((q < 0).to(torch.uint8) << 3)).view(x.shape[0], -1, 2)
    scales = e.to(torch.uint8).view(x.shape[0], -1, 4).transpose(0, 1).contiguous()
    return code[..., 0] | (code[..., 1] << 4), scales


def _mx4_values(codes, scales):
    """float32 values [rows, cols] of packed codes and scale bytes."""
    rows = codes.shape[0]
    code = torch.stack((codes & 15, codes >> 4), -1).view(rows, -1, 32)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=DEV)
    e = scales.transpose(0, 1).reshape(rows, -1).int()
    return (table[code.int()] * _pow2(e).unsqueeze(-1)).view(rows, -1)


def _int8_codes(x):
    """x [..., 16] finite -> (int8 codes, biased scale exponents [...])."""
    e = ((x.abs().amax(-1).view(torch.int32) + 0x10000) >> 23).sub(6).clamp(min=2)
    return torch.round(x * _pow2(254 - e).unsqueeze(-1)).to(torch.int8), e.to(torch.uint8)


# ------------------------------------------------------------------ one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import sparse_memory_linear_sdm_amd as sdm

    c = s["case"]
    if c["op"] == "quantize":
        codes, scales = sdm.mx4_quantize(s["x"])
        return sdm.mx4_dequantize(codes, scales, s["x"].dtype)
    if c["op"] == "project":
        xq, xs = sdm.mx4_quantize(s["x"])
        return sdm.project_mx4(xq, xs, s["wq"], s["ws"], c["n"])
    step = [s[k] for k in ("widx", "wk", "ridx", "rw", "v", "alpha", "beta")]
    if c["op"] == "train":
        out, tape = sdm.scan_train8(s["M"], *step)
        return dict(out=out, M=s["M"], tape=sdm.tape8_read(tape, torch.bfloat16))
    grads = sdm.scan_backward8(*step, (s["codes"], s["scales"]), s["dout"], s["G"],
                               first=s["first"])
    return dict(grads, G=s["G"])


def _run_plain(s):
    return {"quantize": _plain_quantize, "project": _plain_project, "train": _plain_train,
            "backward": _plain_backward}[s["case"]["op"]](s)


def _plain_quantize(s):
    q, e = _mx4_blocks(s["x"])
    return (q * _pow2(e).unsqueeze(-1)).view_as(s["x"]).to(s["x"].dtype)


def _split(y, c, sigmoid):
    """y [B*T, H*P] -> s1, s2, q1, q2, v, alpha, beta in the step's layouts."""
    n, d_v = c["n"], c["d_v"]
    y = y.view(c["B"], c["T"], c["H"], -1).transpose(1, 2)
    parts = y.split([n, n, n, n, d_v, 1, 1], -1)
    return ([p.contiguous() for p in parts[:5]] +
            [sigmoid(p.squeeze(-1)).contiguous() for p in parts[5:]])


def _plain_project(s):
    c = s["case"]
    q, e = _mx4_blocks(s["x"].view(-1, c["d_model"]))
    x = (q * _pow2(e).unsqueeze(-1)).view(-1, c["d_model"])
    w = _mx4_values(s["wq"].view(-1, c["d_model"] // 2), s["ws"])
    return _split(x @ w.t(), c, lambda y: 1 / (1 + torch.exp(-y)))


def _rows(idx, N):
    """[mem, T, K] row numbers in the flattened [mem * N] table, time first."""
    mem = torch.arange(idx.shape[0], device=DEV)[:, None, None] * N
    return (idx.long() + mem).transpose(0, 1).contiguous()


def _time_first(s, *names):
    """Tensors [B, H, T, ...] as [T, B*H, ...]."""
    return [s[k].flatten(0, 1).transpose(0, 1) for k in names]


def _plain_train(s):
    c = s["case"]
    W, R, d_v, T, N = c["W"], c["R"], c["d_v"], c["T"], c["n"] ** 2
    M = s["M"].view(-1, d_v)
    fw, fr = (_rows(s[k].flatten(0, 1), N) for k in ("widx", "ridx"))
    wk, rw, v, alpha, beta = _time_first(s, "wk", "rw", "v", "alpha", "beta")
    out = torch.empty(T, fw.shape[1], d_v, device=DEV)
    tape = torch.empty(T, fw.shape[1], W + R, d_v, dtype=torch.bfloat16, device=DEV)
    for t in range(T):
        old = M[fw[t]]
        a, k = alpha[t][:, None, None], (beta[t][:, None] * wk[t]).unsqueeze(-1)
        # each sum with a product rounded once, in 64 bits: the tape's rounding
        # borders turn on the rows' last bits
        diff = (v[t][:, None].double() - a.double() * old.double()).float()
        M[fw[t]] = ((a * old).double() + k.double() * diff.double()).float()
        read = M[fr[t]]
        out[t] = (rw[t].unsqueeze(-1) * read).sum(1)
        q, e = _int8_codes(torch.cat((old, read), 1).unflatten(-1, (-1, 16)))
        tape[t] = (q.float() * _pow2(e.int()).unsqueeze(-1)).flatten(-2)
    shape = (c["B"], c["H"])
    return dict(out=out.transpose(0, 1).unflatten(0, shape).contiguous(), M=s["M"],
                tape=tape.transpose(0, 1).unflatten(0, shape).contiguous())


def _plain_backward(s):
    c = s["case"]
    W, R, d_v, T, N = c["W"], c["R"], c["d_v"], c["T"], c["n"] ** 2
    mem = c["B"] * c["H"]
    G = s["G"].view(-1, d_v)
    fw, fr = (_rows(s[k].flatten(0, 1), N) for k in ("widx", "ridx"))
    wk, rw, v, alpha, beta, dout = _time_first(s, "wk", "rw", "v", "alpha", "beta", "dout")
    codes = s["codes"].flatten(0, 1)
    scales = s["scales"].flatten(0, 1)
    dv = torch.empty(T, mem, d_v, device=DEV)
    dwk, drw = torch.empty(T, mem, W, device=DEV), torch.empty(T, mem, R, device=DEV)
    dalpha, dbeta = torch.empty(T, mem, device=DEV), torch.empty(T, mem, device=DEV)
    bw, br = torch.arange(W, device=DEV), torch.arange(R, device=DEV)
    for t in range(T - 1, -1, -1):
        rows = codes[:, :, t].float() * _pow2(scales[:, :, t].int()).unsqueeze(-1)
        rows = rows.transpose(1, 2).flatten(-2)  # [mem, W + R, d_v]
        pre, read = rows[:, :W], rows[:, W:]
        gw, gr = G[fw[t]], G[fr[t]]
        if s["first"] is not None:
            first = s["first"].flatten(0, 1)[:, t]
            gw = torch.where(((first[:, :1] >> bw) & 1).bool().unsqueeze(-1), 0.0, gw)
            gr = torch.where(((first[:, 1:] >> br) & 1).bool().unsqueeze(-1), 0.0, gr)
        d = dout[t][:, None]
        drw[t] = (d * read).sum(-1)
        same = fw[t].unsqueeze(-1) == fr[t].unsqueeze(-2)
        gw = gw + (same * rw[t][:, None]).sum(-1, keepdim=True) * d
        k = (beta[t][:, None] * wk[t]).unsqueeze(-1)
        a = alpha[t][:, None, None]
        dv[t] = (k * gw).sum(1)
        dalpha[t] = ((1 - k) * gw * pre).sum((1, 2))
        dk = (gw * (v[t][:, None] - a * pre)).sum(-1)
        dwk[t] = beta[t][:, None] * dk
        dbeta[t] = (wk[t] * dk).sum(-1)
        G[fr[t]] = gr + rw[t].unsqueeze(-1) * d
        G[fw[t]] = a * (1 - k) * gw
    back = lambda x: x.transpose(0, 1).unflatten(0, (c["B"], c["H"])).contiguous()  # noqa: E731
    return dict(dv=back(dv), dwk=back(dwk), drw=back(drw), dalpha=back(dalpha), dbeta=back(dbeta),
                G=s["G"])


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "quantize":
        n, size = c["rows"] * c["cols"], 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=n * (2 * size + 0.5 + 1 / 32), flops=0)
    mem_tokens = c["B"] * c["T"]
    if c["op"] == "project":
        cols, d = c["H"] * (4 * c["n"] + c["d_v"] + 2), c["d_model"]
        return dict(bytes=mem_tokens * d * 2 + cols * d * (0.5 + 1 / 32) + mem_tokens * cols * 4,
                    flops=2 * mem_tokens * cols * d)
    W, R, d_v, steps = c["W"], c["R"], c["d_v"], mem_tokens * c["H"]
    meta = 8 * (W + R) + 4 * d_v + 8  # indices, weights, v and gates of a step
    tape = (W + R) * d_v * (1 + 1 / 16)
    if c["op"] == "train":
        state = (2 * W + R) * d_v * 4
        return dict(bytes=steps * (meta + state + tape + 2 * (W + R) * d_v + 4 * d_v),
                    flops=steps * d_v * (4 * W + 2 * R))
    grads = 4 * (d_v + W + R + 2)
    table = (W + R) * d_v * 4 * (1 if c["sparse"] else 2)  # sparse: most rows are first touches
    return dict(bytes=steps * (meta + 4 * d_v + tape + table + grads),
                flops=steps * d_v * (16 * W + 4 * R))


# ------------------------------------------------------------------ 64 bits

def _exact_e2m1(x):
    """Nearest of the 15 values +-{0, .5, 1, 1.5, 2, 3, 4, 6} times the block
    scale 2^(floor(log2 max|x|) - 2), ties to the even code; x [rows, cols]."""
    y = x.double().view(x.shape[0], -1, 32)
    top = y.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -125).clamp(min=-125)  # top = m 2^k, m in [.5, 1)
    scale = torch.ldexp(torch.ones_like(top), e)
    mag = y.abs() / scale
    out = torch.zeros_like(mag)
    # each border: values above it (or at it, where the next code is even) move up
    for border, up, even in ((.25, .5, False), (.75, 1., True), (1.25, 1.5, False),
                             (1.75, 2., True), (2.5, 3., False), (3.5, 4., True), (5., 6., False)):
        out = torch.where(mag >= border if even else mag > border, up, out)
    return (torch.copysign(out, y) * scale).view(x.shape)


def _exact_int8(x):
    """x [..., d_v] double: blocks of 16 columns rounded to whole multiples, at
    most 127, of the smallest power of two (from 2^-125) that allows it."""
    y = x.unflatten(-1, (-1, 16))
    top = y.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top)[1] - 7, -125)
    e = torch.where(torch.ldexp(top, -e) >= 127.5, e + 1, e).clamp(min=-125)
    return torch.ldexp(torch.round(torch.ldexp(y, -e)), e).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "quantize":
        return _exact_e2m1(s["x"])
    if c["op"] == "project":
        x = _exact_e2m1(s["x"].view(-1, c["d_model"]))
        code = torch.stack((s["wq"] & 15, s["wq"] >> 4), -1).flatten(-2).flatten(0, 1).long()
        mag, neg = code & 7, code >> 3
        # exponent field mag >> 1, mantissa bit mag & 1: (1 + m/2) 2^(e-1), or m/2 at e = 0
        ex, m = mag >> 1, (mag & 1).double()
        w = torch.where(ex > 0, torch.ldexp(1 + m / 2, ex - 1), m / 2) * (1 - 2 * neg)
        sc = s["ws"].permute(1, 0, 2).flatten(1).int() - 127
        w = torch.ldexp(w.unflatten(-1, (-1, 32)), sc.unsqueeze(-1)).flatten(-2)
        del code, mag, neg, ex, m
        return _split(x @ w.t(), c, torch.sigmoid)
    return _exact_train(s) if c["op"] == "train" else _exact_backward(s)


def _exact_train(s):
    c = s["case"]
    M = s["M"].flatten(0, 1).double()
    each = torch.arange(M.shape[0], device=DEV)[:, None]
    widx, ridx = s["widx"].flatten(0, 1).long(), s["ridx"].flatten(0, 1).long()
    wk, rw, v, alpha, beta = (s[k].flatten(0, 1).double()
                              for k in ("wk", "rw", "v", "alpha", "beta"))
    out, tape = [], []
    for t in range(c["T"]):
        # a (1 - b k) M + b k v, the write's two steps taken together
        bk = (beta[:, t, None] * wk[:, t]).unsqueeze(-1)
        old = M[each, widx[:, t]]
        M[each, widx[:, t]] = alpha[:, t, None, None] * (1 - bk) * old + bk * v[:, t, None]
        read = M[each, ridx[:, t]]
        out.append((read * rw[:, t].unsqueeze(-1)).sum(1))
        tape.append(_exact_int8(torch.cat((old, read), 1)))
    shape = (c["B"], c["H"])
    return dict(out=torch.stack(out, 1).unflatten(0, shape), M=M.unflatten(0, shape),
                tape=torch.stack(tape, 1).unflatten(0, shape))


def _exact_backward(s):
    c = s["case"]
    G = s["G"].flatten(0, 1).double()
    each = torch.arange(G.shape[0], device=DEV)[:, None]
    widx, ridx = s["widx"].flatten(0, 1).long(), s["ridx"].flatten(0, 1).long()
    wk, rw, v, alpha, beta, dout = (s[k].flatten(0, 1).double()
                                    for k in ("wk", "rw", "v", "alpha", "beta", "dout"))
    if s["first"] is not None:  # the final state has no gradient: touched rows start at zero
        for idx in (widx, ridx):
            G[each, idx.flatten(1)] = 0
    codes, scales = s["codes"].flatten(0, 1), s["scales"].flatten(0, 1)
    grads = {k: [] for k in ("dv", "dwk", "drw", "dalpha", "dbeta")}
    for t in reversed(range(c["T"])):
        rows = torch.ldexp(codes[:, :, t].double(), scales[:, :, t].int().unsqueeze(-1) - 127)
        rows = rows.transpose(1, 2).flatten(2)
        pre, read = rows[:, :c["W"]], rows[:, c["W"]:]
        d = dout[:, t, None]
        grads["drw"].append((read * d).sum(-1))
        G[each, ridx[:, t]] += rw[:, t].unsqueeze(-1) * d
        g = G[each, widx[:, t]]
        a, bk = alpha[:, t, None], beta[:, t, None] * wk[:, t]
        g_pre, g_v = (g * pre).sum(-1), (g * v[:, t, None]).sum(-1)
        d_bk = g_v - a * g_pre
        grads["dv"].append((bk.unsqueeze(-1) * g).sum(1))
        grads["dalpha"].append(((1 - bk) * g_pre).sum(-1))
        grads["dwk"].append(beta[:, t, None] * d_bk)
        grads["dbeta"].append((wk[:, t] * d_bk).sum(-1))
        G[each, widx[:, t]] = (a * (1 - bk)).unsqueeze(-1) * g
    shape = (c["B"], c["H"])
    return dict({k: torch.stack(x[::-1], 1).unflatten(0, shape) for k, x in grads.items()},
                G=G.unflatten(0, shape))
