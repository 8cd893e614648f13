"""Plain numpy form, in float64, of the microscaled formats (include/sdm.h):
4-bit e2m1 blocks of 32 and 8-bit integer blocks of 16, one power-of-two scale
per block.  Written from the definitions, value by value."""
import numpy as np

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], np.float64)


def _nearest_e2m1(mag):
    """Index 0..7 of the nearest magnitude, ties to the even index, 6 above it."""
    mag = np.minimum(mag, 6.0)
    hi = np.searchsorted(E2M1, mag, side="left").clip(1, 7)
    lo = hi - 1
    dl, dh = mag - E2M1[lo], E2M1[hi] - mag
    even_hi = hi % 2 == 0
    return np.where((dh < dl) | ((dh == dl) & even_hi), hi, lo)


def mx4_quantize(x):
    """x [rows, cols] -> codes uint8 [rows, cols/2], scales uint8 [cols/128, rows, 4]."""
    rows, cols = x.shape
    y = np.asarray(x, np.float64).reshape(rows, cols // 32, 32)
    with np.errstate(invalid="ignore"):
        top = np.abs(y).max(-1)
    finite = np.isfinite(top)
    e = np.frexp(np.where(finite & (top > 0), top, 1.0))[1] - 1  # floor(log2 top)
    e = np.where(finite & (top > 0), np.maximum(e - 2, -125), -125)
    y = np.where(finite[..., None], y, 0.0)
    code = _nearest_e2m1(np.abs(np.ldexp(y, -e[..., None])))
    code = code | (np.signbit(y) << 3)
    code = np.where(finite[..., None], code, 0).reshape(rows, cols // 2, 2).astype(np.uint8)
    scale = np.where(finite, e + 127, 255).astype(np.uint8)
    return (code[..., 0] | (code[..., 1] << 4),
            np.ascontiguousarray(scale.reshape(rows, cols // 128, 4).transpose(1, 0, 2)))


def mx4_values(codes, scales):
    """float64 [rows, cols] of codes and scales (NaN where the scale byte is 255)."""
    rows = codes.shape[0]
    code = np.stack((codes & 15, codes >> 4), -1).reshape(rows, -1, 32)
    val = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    b = scales.transpose(1, 0, 2).reshape(rows, -1).astype(np.int64)
    out = np.ldexp(val, (b - 127)[..., None])
    out[b == 255] = np.nan
    return out.reshape(rows, -1)


def int8_quantize(x):
    """x [..., 16] -> codes int8 [..., 16], scale bytes uint8 [...]."""
    y = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        top = np.abs(y).max(-1)
    finite = np.isfinite(top)
    top = np.where(finite, top, 0.0)
    e = np.full(top.shape, -125)
    # the smallest scale whose rounded codes stay within 127
    grow = np.rint(np.ldexp(top, -e)) > 127
    k = np.frexp(np.where(grow, top, 1.0))[1]
    e = np.where(grow, np.maximum(k - 7, -125), e)
    e = np.where(np.rint(np.ldexp(top, -e)) > 127, e + 1, e)
    q = np.rint(np.ldexp(np.where(finite[..., None], y, 0.0), -e[..., None])).astype(np.int8)
    return q, np.where(finite, e + 127, 255).astype(np.uint8)


def int8_values(codes, scales):
    b = scales.astype(np.int64)
    out = np.ldexp(codes.astype(np.float64), (b - 127)[..., None])
    out[b == 255] = np.nan
    return out


# --------------------------------------------- the step on one memory, in float64

def forward(M, widx, wk, ridx, rw, v, alpha, beta):
    """T steps on M [N, d_v] (updated): out [T, d_v] and the tape rows
    [T, W + R, d_v] (write rows before the step's write, read rows after it).
    Row numbers outside [0, N) are skipped."""
    out, tape = [], []
    N = M.shape[0]
    for t in range(len(v)):
        wv, rv = (widx[t] >= 0) & (widx[t] < N), (ridx[t] >= 0) & (ridx[t] < N)
        pre = np.where(wv[:, None], M[np.where(wv, widx[t], 0)], 0.0)
        k = (beta[t] * wk[t])[:, None]
        M[widx[t][wv]] = (alpha[t] * (1 - k) * pre + k * v[t])[wv]
        read = np.where(rv[:, None], M[np.where(rv, ridx[t], 0)], 0.0)
        out.append((rw[t][:, None] * read).sum(0))
        tape.append(np.concatenate([pre, read]))
    return np.array(out), np.array(tape)


def backward(G, widx, wk, ridx, rw, v, alpha, beta, tape, dout):
    """Gradients at the tape's rows; G [N, d_v] in: of the state after the last
    step, out: before the first."""
    T, W = wk.shape
    N = G.shape[0]
    g = {"dv": np.zeros(v.shape), "dwk": np.zeros(wk.shape), "drw": np.zeros(rw.shape),
         "dalpha": np.zeros(T), "dbeta": np.zeros(T)}
    for t in reversed(range(T)):
        wv, rv = (widx[t] >= 0) & (widx[t] < N), (ridx[t] >= 0) & (ridx[t] < N)
        pre = np.where(wv[:, None], tape[t, :W], 0.0)
        read = np.where(rv[:, None], tape[t, W:], 0.0)
        g["drw"][t] = read @ dout[t]
        G[ridx[t][rv]] += np.outer(rw[t], dout[t])[rv]
        gr = np.where(wv[:, None], G[np.where(wv, widx[t], 0)], 0.0)
        k = beta[t] * wk[t]
        d = (gr * (v[t] - alpha[t] * pre)).sum(1)
        g["dv"][t] = k @ gr
        g["dalpha"][t] = ((1 - k) * (gr * pre).sum(1)).sum()
        g["dwk"][t] = beta[t] * d
        g["dbeta"][t] = wk[t] @ d
        G[widx[t][wv]] = ((alpha[t] * (1 - k))[:, None] * gr)[wv]
    return g
