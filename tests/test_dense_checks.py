"""The dense recurrence's and the norms' calls refuse bad arguments before any
launch: the C entry points by status and message, the binding by ValueError
(CPU tensors; no kernel is reached)."""
import pytest
import torch

import sparse_memory_linear_sdm_amd as sdm

FAKE = 1 << 20  # a non-null, aligned address that is never dereferenced
f32, bf16 = torch.float32, torch.bfloat16


def _err():
    return sdm.lib().sdm_last_error().decode()


def _each(fn, ok, bad):
    for at, value, status, word in bad:
        a = list(ok)
        a[at] = value
        assert fn(*a) == status, (at, value, _err())
        assert word in _err(), _err()


# sizes: dtype, B, H, Hk, d_k, d_v, T at `first` and on
def _size_refusals(first):
    return [(first, 2, 1, "dtype"), (first + 1, 0, 1, "B, H and Hk"), (first + 2, 0, 1, "B, H and Hk"),
            (first + 3, 0, 1, "B, H and Hk"), (first + 3, 3, 1, "multiple of Hk"),
            (first + 1, 1 << 20, 2, "2^20"), (first + 4, 16, 2, "d_k=16"), (first + 4, 256, 2, "d_k=256"),
            (first + 5, 96, 2, "d_v=96"), (first + 5, 0, 2, "d_v=0")]


def test_linear_scan_entry_point():
    L = sdm.lib()
    ok = (FAKE, 1, 2, 4, 2, 64, 128, 100) + (FAKE,) * 7 + (1 << 40, None)
    assert len(ok) == 17
    _each(L.sdm_linear_scan, ok, _size_refusals(1) + [
        (0, None, 1, "S is NULL"), (0, FAKE + 8, 1, "S must be 16-byte"), (7, -1, 1, "T must"),
        (7, 1 << 31, 2, "2^31"), (8, None, 1, "q is NULL"), (9, FAKE + 2, 1, "k must be 16-byte"),
        (10, None, 1, "v is NULL"), (11, FAKE + 2, 1, "g must be 4-byte"), (12, None, 1, "out is NULL"),
        (13, FAKE + 4, 1, "tape must be 16-byte")])
    need = L.sdm_linear_scan_workspace_size(1, 1, 2, 64, 128, 100000)
    assert need > 0
    ok = (FAKE, 1, 1, 2, 2, 64, 128, 100000) + (FAKE,) * 5 + (None, FAKE, need, None)
    _each(L.sdm_linear_scan, ok, [(14, None, 1, "workspace is NULL"), (14, FAKE + 16, 1, "256-byte"),
                                  (15, need - 1, 1, "below the")])
    assert L.sdm_linear_scan(FAKE, 0, 1, 1, 1, 32, 32, 0, *[None] * 7, 0, None) == 0


def test_linear_workspace_sizes():
    L = sdm.lib()
    assert L.sdm_linear_scan_workspace_size(1, 64, 16, 128, 128, 4096) == 0  # many memories
    assert L.sdm_linear_scan_workspace_size(1, 1, 1, 128, 128, 100) == 0     # few steps
    one = L.sdm_linear_backward_workspace_size(1, 1, 4, 4, 64, 64, 100)
    assert one == 0
    assert L.sdm_linear_backward_workspace_size(1, 1, 4, 2, 64, 64, 100) == 2 * 4 * 100 * 64 * 4
    for bad in ((2, 1, 1, 64, 64, 9), (0, 0, 1, 64, 64, 9), (0, 1, 0, 64, 64, 9), (0, 1, 1, 48, 64, 9),
                (0, 1, 1, 64, 8, 9), (0, 1, 1, 64, 64, -1), (0, 1, 1, 64, 64, 1 << 31),
                (0, 1 << 20, 2, 64, 64, 9)):
        assert L.sdm_linear_scan_workspace_size(*bad) == 0
        assert L.sdm_linear_backward_workspace_size(*bad[:3], 1, *bad[3:]) == 0
    assert L.sdm_linear_backward_workspace_size(0, 1, 4, 3, 64, 64, 100) == 0
    assert L.sdm_linear_backward_workspace_size(0, 1, 2, 1, 64, 64, 1 << 25) == 0  # B*H*T


def test_linear_step_entry_point():
    L = sdm.lib()
    ok = (FAKE, 0, 2, 4, 2, 64, 128) + (FAKE,) * 5 + (None,)
    _each(L.sdm_linear_step, ok, _size_refusals(1) + [
        (0, None, 1, "S is NULL"), (7, None, 1, "q is NULL"), (8, None, 1, "k is NULL"),
        (9, FAKE + 8, 1, "v must be 16-byte"), (10, None, 1, "g is NULL"),
        (11, None, 1, "out is NULL")])


def test_linear_backward_entry_point():
    L = sdm.lib()
    ok = (1, 2, 4, 2, 64, 128, 100) + (FAKE,) * 12 + (1 << 40, None)
    assert len(ok) == 21
    _each(L.sdm_linear_backward, ok, _size_refusals(0) + [
        (6, -1, 1, "T must"), (6, 1 << 24, 2, "2^26 - 4"), (7, None, 1, "q is NULL"),
        (10, None, 1, "g is NULL"), (11, None, 1, "tape is NULL"), (12, FAKE + 8, 1, "dout must be"),
        (13, None, 1, "G is NULL"), (14, None, 1, "dq is NULL"), (15, None, 1, "dk is NULL"),
        (16, FAKE + 4, 1, "dv must be 16-byte"), (17, FAKE + 2, 1, "dg must be 4-byte"),
        (18, None, 1, "workspace is NULL"), (18, FAKE + 128, 1, "256-byte")])
    a = list(ok)
    a[19] = 2 * 8 * 100 * 64 * 4 - 1
    assert L.sdm_linear_backward(*a) == 1 and "below the" in _err()
    assert L.sdm_linear_backward(1, 2, 4, 2, 64, 128, 0, *[None] * 6, FAKE, *[None] * 5, 0, None) == 0


def test_norm_entry_points():
    L = sdm.lib()
    ok = (FAKE, 0, FAKE, FAKE, FAKE, 1.0, 1e-6, 2, 1, 5, 64, FAKE, 1, FAKE, FAKE, None)
    sizes = lambda B, d: [(B, -1, 1, "B and T"), (B + 1, 0, 1, "H >= 1"), (B + 2, -1, 1, "B and T"),  # noqa: E731
                          (B + 2, 1 << 31, 2, "2^31"), (B, 1 << 30, 2, "2^31"), (d, 12, 2, "multiple of 8"),
                          (d, 0, 2, "multiple of 8"), (d, 16392, 2, "multiple of 8")]
    _each(L.sdm_norm, ok, sizes(7, 10) + [
        (0, None, 1, "y is NULL"), (0, FAKE + 8, 1, "y must be 16-byte"), (1, 2, 1, "dtypes"),
        (2, None, 1, "w is NULL"), (3, FAKE + 2, 1, "16-byte"), (4, FAKE + 2, 1, "16-byte"),
        (6, -1.0, 1, "eps"), (6, float("nan"), 1, "eps"), (8, 2, 1, "H = 1"), (11, None, 1, "out is NULL"),
        (12, 3, 1, "dtypes"), (13, None, 1, "together"), (14, None, 1, "together"),
        (14, FAKE + 4, 1, "16-byte")])
    assert L.sdm_norm(*[None, 0, None, None, None, 1.0, 0.0, 0, 1, 5, 64, None, 1, None, None, None]) == 0
    need = L.sdm_norm_backward_workspace_size(2, 1, 5, 64)
    assert need > 0
    for bad in ((-1, 1, 5, 64), (1, 0, 5, 64), (1, 1, -5, 64), (1, 1, 5, 12), (1, 1, 1 << 31, 64), (0, 1, 5, 64)):
        assert L.sdm_norm_backward_workspace_size(*bad) == 0
    ok = (FAKE, 1, FAKE, 0, FAKE, FAKE, FAKE, 1.0, 1e-6, 2, 1, 5, 64, FAKE, FAKE, FAKE, FAKE, need, None)
    _each(L.sdm_norm_backward, ok, sizes(9, 12) + [
        (0, None, 1, "dout is NULL"), (1, 2, 1, "dtypes"), (2, FAKE + 8, 1, "y must be 16-byte"),
        (3, 2, 1, "dtypes"), (4, None, 1, "w is NULL"), (5, None, 1, "together"), (6, FAKE + 2, 1, "16-byte"),
        (8, -1.0, 1, "eps"), (13, None, 1, "dy is NULL"), (14, None, 1, "dw is NULL"),
        (14, FAKE + 4, 1, "dw must be 16-byte"), (15, None, 1, "together"), (16, None, 1, "workspace is NULL"),
        (16, FAKE + 16, 1, "256-byte"), (17, need - 1, 1, "below the")])


def _expect(match, fn, *a, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*a, **kw)


def _z(*shape, dtype=f32):
    return torch.zeros(shape, dtype=dtype)


def _linear():
    return dict(S=_z(2, 4, 32, 64), q=_z(2, 2, 9, 32), k=_z(2, 2, 9, 32), v=_z(2, 4, 9, 64), g=_z(2, 4, 9))


@pytest.mark.parametrize("name,bad,match", [
    ("S", _z(2, 4, 32), "S must be"), ("S", _z(2, 4, 32, 64, dtype=bf16), "S must be"),
    ("S", _z(2, 3, 32, 64), "multiple of q's 2"), ("q", _z(2, 2, 32), "q and k must be"),
    ("q", _z(2, 0, 9, 32), "multiple of q's 0"), ("q", _z(2, 2, 9, 64), "q must have shape"),
    ("q", _z(2, 2, 9, 32, dtype=bf16), "k must be"), ("k", _z(2, 1, 9, 32), "k must have shape"),
    ("v", _z(2, 4, 9, 32), "v must have shape"), ("v", _z(2, 4, 9, 64, dtype=bf16), "v must be"),
    ("g", _z(2, 4, 8), "g must have shape"), ("g", _z(2, 4, 9, dtype=bf16), "g must be"),
    ("v", _z(2, 4, 64, 9).transpose(2, 3), "v must be contiguous")])
def test_linear_binding_refuses(name, bad, match):
    a = dict(_linear(), **{name: bad})
    for fn in (sdm.linear_scan, sdm.linear_scan_train):
        _expect(match, fn, **a)
    G = a.pop("S")
    _expect(match.replace("S must", "G must"), sdm.linear_backward, **a, G=G, tape=_z(2, 4, 1, 32, 64),
            dout=_z(2, 4, 9, 64))


def test_linear_binding_outputs():
    a = _linear()
    _expect("on the GPU", sdm.linear_scan, **a)
    _expect("out must have shape", sdm.linear_scan, **a, out=_z(2, 4, 8, 64))
    _expect("out must be", sdm.linear_scan, **a, out=_z(2, 4, 9, 64, dtype=bf16))
    _expect("tape must have shape", sdm.linear_scan_train, **a, tape=_z(2, 4, 2, 32, 64))
    _expect("workspace must be contiguous", sdm.linear_scan, **a, workspace=_z(8, 8).t())
    half = {n: x.half() if n in "qkv" else x for n, x in a.items()}
    _expect("float32 or bfloat16", sdm.linear_scan, **half)
    step = dict(a, **{n: a[n][:, :, 0].contiguous() for n in "qkvg"})
    _expect("on the GPU", sdm.linear_step, **step)
    _expect(r"\[B, Hk, d_k\]", sdm.linear_step, **a)
    _expect("out must have shape", sdm.linear_step, **step, out=_z(2, 4, 32))
    G = a.pop("S")
    more = dict(G=G, tape=_z(2, 4, 1, 32, 64), dout=_z(2, 4, 9, 64))
    _expect("on the GPU", sdm.linear_backward, **a, **more)
    _expect("tape must have shape", sdm.linear_backward, **a, **dict(more, tape=_z(2, 4, 2, 32, 64)))
    _expect("dout must be", sdm.linear_backward, **a, **dict(more, dout=_z(2, 4, 9, 64, dtype=bf16)))
    out = dict(dq=_z(2, 2, 9, 32), dk=_z(2, 2, 9, 32), dv=_z(2, 4, 9, 64), dg=_z(2, 4, 8))
    _expect("dg must have shape", sdm.linear_backward, **a, **more, out=out)


def test_norm_binding():
    y, w = _z(3, 5, 64), _z(64)
    _expect("on the GPU", sdm.norm, y, w)
    _expect("last dimension", sdm.norm, torch.zeros(()), w)
    _expect("w must have shape", sdm.norm, y, _z(63))
    _expect("w must be", sdm.norm, y, _z(64, dtype=bf16))
    _expect("float32 or bfloat16", sdm.norm, y.half(), w)
    _expect("z must be", sdm.norm, y, w, z=_z(3, 5, 64, dtype=bf16), dtype=f32)
    _expect("z must be", sdm.norm, y, w, z=_z(3, 5, 64, dtype=bf16), x=_z(3, 5, 64))
    _expect("x must have shape", sdm.norm, y, w, x=_z(3, 64))
    _expect("y must be contiguous", sdm.norm, y.transpose(0, 1), w)
    _expect("out must have shape", sdm.norm, y, w, out=_z(3, 5, 63))
    _expect("next must have shape", sdm.norm, y, w, next_w=w, out=(y, _z(3, 64)))
    _expect("next_w must have shape", sdm.norm, y, w, next_w=_z(32))
    _expect(r"\[B, H, T, d\]", sdm.norm, y, w, heads=True)
    _expect("whole rows", sdm.norm, _z(2, 3, 5, 64), w, next_w=w, heads=True)
    _expect("z must have shape", sdm.norm, _z(2, 3, 5, 64), w, z=_z(2, 3, 5, 64), heads=True)
    _expect("on the GPU", sdm.norm_backward, y, y, w)
    _expect("dout must have shape", sdm.norm_backward, _z(3, 64), y, w)
    _expect("z must be", sdm.norm_backward, y, y, w, z=_z(3, 5, 64, dtype=bf16))
    _expect("skip must be", sdm.norm_backward, y, y, w, skip=_z(3, 5, 64, dtype=bf16))
    _expect("dw must have shape", sdm.norm_backward, y, y, w, out=dict(dy=y, dw=_z(63)))
