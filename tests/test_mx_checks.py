"""The microscaled calls refuse bad arguments before any launch: the C entry
points by status and message, the binding by ValueError (CPU tensors; no
kernel is reached)."""
import pytest
import torch

import sparse_memory_linear_sdm_amd as sdm

FAKE = 1 << 20  # a non-null, aligned address that is never dereferenced
u8, f32 = torch.uint8, torch.float32


def _err():
    return sdm.lib().sdm_last_error().decode()


def _each(fn, ok, bad):
    for at, value, status, word in bad:
        a = list(ok)
        a[at] = value
        assert fn(*a) == status, (at, value, _err())
        assert word in _err(), _err()


def test_mx4_entry_points():
    L = sdm.lib()
    ok = (FAKE, 0, 10, 256, FAKE, FAKE, None)  # x, dtype, rows, cols, codes, scales, stream
    _each(L.sdm_mx4_quantize, ok, [
        (0, None, 1, "x is NULL"), (0, FAKE + 4, 1, "16-byte"), (1, 2, 1, "dtype"),
        (2, -1, 1, "rows"), (2, 1 << 31, 2, "tiles"), (3, 96, 2, "multiple of 128"),
        (3, 0, 2, "multiple of 128"), (3, 65536 + 128, 2, "multiple of 128"),
        (4, None, 1, "codes"), (4, FAKE + 8, 1, "16-byte"), (5, None, 1, "scales"),
        (5, FAKE + 2, 1, "4-byte")])
    assert L.sdm_mx4_quantize(None, 0, 0, 256, None, None, None) == 0
    # one tile of 512 columns per 8 rows: 2^24 - 1 tiles is the largest grid
    assert L.sdm_mx4_quantize(FAKE, 0, 1 << 30, 512, FAKE, FAKE, None) == 2 and "tiles" in _err()
    ok = (FAKE, FAKE, 0, 10, 256, FAKE, None)  # codes, scales, dtype, rows, cols, x, stream
    _each(L.sdm_mx4_dequantize, ok, [
        (0, None, 1, "codes"), (1, None, 1, "codes and scales"), (2, 2, 1, "dtype"),
        (3, -1, 1, "rows"), (4, 64, 2, "multiple of 128"), (5, None, 1, "x is NULL"),
        (5, FAKE + 2, 1, "16-byte")])
    assert L.sdm_mx4_dequantize(None, None, 1, 0, 128, None, None) == 0
    # fp32 is written in tiles of half as many columns
    assert L.sdm_mx4_dequantize(FAKE, FAKE, 0, 1 << 27, 384, FAKE, None) == 2 and "256" in _err()


def test_project_mx4_entry_point():
    L = sdm.lib()
    ok = (FAKE,) * 4 + (2, 100, 256, 2, 64, 16) + (FAKE,) * 7 + (None,)
    _each(L.sdm_project_mx4, ok, [
        (0, None, 1, "NULL"), (1, None, 1, "NULL"), (2, None, 1, "NULL"), (3, None, 1, "NULL"),
        (0, FAKE + 8, 1, "16-byte"), (2, FAKE + 4, 1, "16-byte"), (1, FAKE + 2, 1, "4-byte"),
        (3, FAKE + 1, 1, "4-byte"), (4, -1, 1, "B and T"), (6, 64, 2, "multiple of 128"),
        (6, 192, 2, "multiple of 128"), (6, 65536 + 128, 2, "multiple of 128"),
        (7, 0, 1, "H, n and d_v"), (8, 0, 1, "H, n and d_v"), (14, None, 1, "v is NULL"),
        (10, FAKE + 2, 1, "s1 must be 4-byte")])
    a = list(ok)
    a[4] = a[5] = 1 << 30
    assert L.sdm_project_mx4(*a) == 2 and "tiles" in _err()
    a = list(ok)
    a[7] = a[8] = 1 << 20
    assert L.sdm_project_mx4(*a) == 2 and "2^31" in _err()
    assert L.sdm_project_mx4(*[None] * 4, 0, 100, 256, 2, 64, 16, *[None] * 8) == 0


def _expect(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def _z(*shape, dtype=u8):
    return torch.zeros(shape, dtype=dtype)


def test_mx4_binding():
    x = _z(3, 5, 256, dtype=f32)
    _expect("on the GPU", sdm.mx4_quantize, x)
    _expect("float32 or bfloat16", sdm.mx4_quantize, x.half())
    _expect("last dimension", sdm.mx4_quantize, torch.zeros(()))
    _expect("contiguous", sdm.mx4_quantize, x.transpose(0, 1))
    _expect("codes must have shape", sdm.mx4_quantize, x, out=(_z(3, 5, 127), _z(2, 15, 4)))
    _expect("scales must have shape", sdm.mx4_quantize, x, out=(_z(3, 5, 128), _z(2, 14, 4)))
    _expect("scales must be", sdm.mx4_quantize, x, out=(_z(3, 5, 128), _z(2, 15, 4, dtype=f32)))
    codes, scales = _z(3, 5, 128), _z(2, 15, 4)
    _expect("on the GPU", sdm.mx4_dequantize, codes, scales)
    _expect("scales must have shape", sdm.mx4_dequantize, codes, _z(15, 2, 4))
    _expect("float32 or bfloat16", sdm.mx4_dequantize, codes, scales, torch.float64)
    _expect("out must have shape", sdm.mx4_dequantize, codes, scales, out=_z(15, 256, dtype=f32))
    _expect("out must be", sdm.mx4_dequantize, codes, scales, torch.bfloat16, out=x)


def test_project_mx4_binding():
    B, T, d, H, n, d_v = 2, 5, 256, 3, 8, 16
    P = 4 * n + d_v + 2
    xq, xs, wq, ws = _z(B, T, d // 2), _z(2, B * T, 4), _z(H, P, d // 2), _z(2, H * P, 4)
    _expect("on the GPU", sdm.project_mx4, xq, xs, wq, ws, n)
    _expect("Xq must be", sdm.project_mx4, xq.view(B * T, -1), xs, wq, ws, n)
    _expect("Xs must have shape", sdm.project_mx4, xq, xs[:1], wq, ws, n)
    _expect("Wq must have shape", sdm.project_mx4, xq, xs, _z(H, P, d), ws, n)
    _expect("Ws must be", sdm.project_mx4, xq, xs, wq, ws.int(), n)
    _expect("too few", sdm.project_mx4, xq, xs, wq, ws, P)
    _expect("7 tensors", sdm.project_mx4, xq, xs, wq, ws, n, out=(xq,))


# ------------------------------------------------------------- 8-bit tape

def test_train8_entry_point():
    L = sdm.lib()
    # M, B, H, N, d_v, T, W, R, 7 inputs, out, tape, tape_scale, stream
    ok = [FAKE, 1, 1, 4096, 16, 8, 8, 8] + [FAKE] * 10 + [None]
    _each(L.sdm_scan_train8, ok, [
        (0, None, 1, "M is NULL"), (1, 0, 1, "B and H"), (3, 4, 1, "exceed N"),
        (4, 24, 2, "d_v=24"), (5, -1, 1, "T must"), (6, 65, 2, "64"), (8, None, 1, "NULL"),
        (15, FAKE + 8, 1, "16-byte"), (16, None, 1, "tape"), (16, FAKE + 4, 1, "tape"),
        (17, None, 1, "tape_scale")])
    a = list(ok)
    a[4], a[5], a[6], a[7] = 128, 1 << 17, 64, 64  # exactly 2 GiB of codes
    assert L.sdm_scan_train8(*a) == 2 and "2 GiB" in _err()
    a[4], a[5], a[6], a[7] = 16, 1 << 32, 1, 1
    assert L.sdm_scan_train8(*a) == 2
    assert L.sdm_scan_train8(FAKE, 1, 1, 4096, 16, 0, 8, 8, *[None] * 11) == 0


def test_tape8_read_entry_point():
    L = sdm.lib()
    ok = [FAKE, FAKE, 2, 3, 64, 10, 12, 0, FAKE, None]  # codes, scales, B, H, d_v, T, S, dtype, rows
    _each(L.sdm_tape8_read, ok, [
        (0, None, 1, "NULL"), (1, None, 1, "NULL"), (8, None, 1, "NULL"), (0, FAKE + 8, 1, "16-byte"),
        (8, FAKE + 8, 1, "16-byte"), (2, 0, 1, "B and H"), (2, 1 << 20, 2, "2^20"),
        (4, 48, 2, "d_v=48"), (5, -1, 1, "T must"), (5, 1 << 40, 2, "2 GiB"), (6, 0, 1, "S (rows"),
        (6, 129, 1, "S (rows"), (7, 2, 1, "dtype")])
    assert L.sdm_tape8_read(None, None, 1, 1, 16, 0, 2, 1, None, None) == 0


def test_backward8_entry_point():
    L = sdm.lib()
    size = L.sdm_scan_backward8_workspace_size
    # 16 padded steps' records of 5 x 64 + 4 words, and 8 steps' sums of W + 1 per tile
    # (8 columns where there is a compute unit for each, else 16)
    ws = size(1, 1, 16, 8, 8, 8)
    assert ws == 16 * 1296 + 8 * 2 * 9 * 4
    assert size(8, 8, 128, 7, 64, 1) == 64 * (8 * 1296 + 7 * 8 * 65 * 4)
    for bad in ((0, 1, 16, 8, 8, 8), (1, 1, 24, 8, 8, 8), (1, 1, 16, -1, 8, 8), (1, 1, 16, 8, 65, 8),
                (1, 1, 16, 8, 8, 0), (1 << 11, 1 << 10, 16, 8, 8, 8), (1, 1, 16, 1 << 40, 8, 8)):
        assert size(*bad) == 0, bad
    # B, H, N, d_v, T, W, R, 7 inputs, tape, tape_scale, dout, G, dv, dwk, drw, dalpha, dbeta,
    # first, workspace, bytes, stream
    ok = [1, 1, 4096, 16, 8, 8, 8] + [FAKE] * 18 + [ws, None]
    _each(L.sdm_scan_backward8, ok, [
        (14, None, 1, "NULL"), (14, FAKE + 4, 1, "16-byte"), (15, None, 1, "tape_scale"),
        (16, None, 1, "NULL"), (17, None, 1, "M is NULL"), (23, FAKE + 4, 1, "first"),
        (24, None, 1, "workspace"), (24, FAKE + 4, 1, "workspace"), (25, ws - 4, 1, "workspace"),
        (4, 1 << 26, 2, "2^26"), (3, 24, 2, "d_v=24"), (6, 65, 2, "64")])
    a = list(ok)
    a[3], a[4], a[5], a[6] = 128, 1 << 17, 64, 64
    assert L.sdm_scan_backward8(*a) == 2 and "2 GiB" in _err()
    a = list(ok)
    a[0], a[1], a[4], a[25] = 1 << 10, 1 << 10, 63, 1 << 50  # padded: 2^20 * 64 wavefronts
    assert L.sdm_scan_backward8(*a) == 2 and "T + 8" in _err()
    args = [1, 1, 4096, 16, 0, 8, 8] + [None] * 10 + [FAKE] + [None] * 7 + [0, None]
    assert L.sdm_scan_backward8(*args) == 0


def test_tape8_binding():
    B, H, N, d_v, T, W, R = 2, 3, 64, 32, 5, 4, 3
    i32, i8 = torch.int32, torch.int8
    step = dict(widx=_z(B, H, T, W, dtype=i32), wk=_z(B, H, T, W, dtype=f32),
                ridx=_z(B, H, T, R, dtype=i32), rw=_z(B, H, T, R, dtype=f32),
                v=_z(B, H, T, d_v, dtype=f32), alpha=_z(B, H, T, dtype=f32),
                beta=_z(B, H, T, dtype=f32))
    M = _z(B, H, N, d_v, dtype=f32)
    codes, scales = _z(B, H, 2, T, W + R, 16, dtype=i8), _z(B, H, 2, T, W + R)
    _expect("on the GPU", sdm.scan_train8, M, **step)
    _expect("M must be", sdm.scan_train8, M.bfloat16(), **step)
    _expect("wk must have shape", sdm.scan_train8, M, **{**step, "wk": step["rw"]})
    _expect("tape codes must be", sdm.scan_train8, M, **step, tape=(codes.view(u8), scales))
    _expect("tape scales must have shape", sdm.scan_train8, M, **step, tape=(codes, scales[:, :, :1]))
    _expect("out must have shape", sdm.scan_train8, M, **step, out=_z(B, H, T, 16, dtype=f32))
    _expect("on the GPU", sdm.tape8_read, (codes, scales))
    _expect("tape codes must be", sdm.tape8_read, (codes[0], scales))
    _expect("tape codes must have shape", sdm.tape8_read, (codes[..., :8].contiguous(), scales))
    _expect("float32 or bfloat16", sdm.tape8_read, (codes, scales), torch.float16)
    _expect("out must have shape", sdm.tape8_read, (codes, scales), out=M)
    dout = step["v"]
    _expect("on the GPU", sdm.scan_backward8, **step, tape=(codes, scales), dout=dout, G=M)
    _expect("tape scales must have shape", sdm.scan_backward8, **step, tape=(codes, scales[:1]),
            dout=dout, G=M)
    _expect("first must be", sdm.scan_backward8, **step, tape=(codes, scales), dout=dout, G=M,
            first=_z(B, H, T, 2, dtype=i32))
    bad = dict(dv=step["v"], dwk=step["wk"], drw=step["wk"], dalpha=step["alpha"], dbeta=step["beta"])
    _expect("drw must have shape", sdm.scan_backward8, **step, tape=(codes, scales), dout=dout, G=M,
            out=bad)


def test_projection_launches_stay_below_2_to_the_32_work_items():
    """Tiles are workgroups of 512 threads, so 2^23 - 1 of them at most."""
    L = sdm.lib()
    for call, ptrs in ((L.sdm_project, 2), (L.sdm_project_mx4, 4)):
        a = [FAKE] * ptrs + [1 << 15, 1 << 16, 256, 1, 64, 16] + [FAKE] * 7 + [None]
        assert call(*a) == 2 and "2^23 - 1" in _err()  # 2^23 row tiles x 2


def test_backward8_workspace_size_is_0_where_the_call_refuses():
    """Its limits on steps and on a memory's tape: the last size inside, the first outside."""
    L = sdm.lib()
    size = L.sdm_scan_backward8_workspace_size
    ok = [1, 1, 4096, 16, 8, 8, 8] + [FAKE] * 18 + [1 << 60, None]
    for inside, outside, word in [
            # B*H*(T + 8) <= 2^26 - 4
            ((8, 8, 16, (1 << 20) - 9, 1, 1), (8, 8, 16, (1 << 20) - 8, 1, 1), "T + 8"),
            ((1 << 10, 1 << 10, 16, 55, 1, 1), (1 << 10, 1 << 10, 16, 56, 1, 1), "T + 8"),
            # T*(W + R)*d_v < 2^31
            ((1, 1, 128, (1 << 17) - 1, 64, 64), (1, 1, 128, 1 << 17, 64, 64), "2 GiB"),
            ((8, 8, 256, 1 << 18, 16, 15), (8, 8, 256, 1 << 18, 16, 16), "2 GiB")]:
        assert size(*inside) > 0, inside
        assert size(*outside) == 0, outside
        B, H, d_v, T, W, R = outside
        a = list(ok)
        a[0], a[1], a[3], a[4], a[5], a[6] = B, H, d_v, T, W, R
        assert L.sdm_scan_backward8(*a) == 2 and word in _err()
    # 164 GiB of workspace for a call that refuses
    assert size(8, 8, 16, 1 << 21, 1, 1) == 0
