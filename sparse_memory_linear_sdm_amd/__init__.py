"""Sparse Delta Memory (SDM) step on AMD Instinct MI355X (gfx950).

Thin Python binding over the C ABI of libsdm.so (include/sdm.h): it checks
tensor devices, dtypes and contiguity, passes raw device pointers and the
current HIP stream, and raises on a non-zero status.  Every step of the
computation runs in the library's HIP kernels; there is no CPU path and no
fallback -- importing works without the library, but every call raises if
libsdm.so is not built.  PyTorch is used only for device memory and streams.

Calls (same names as the C ABI without the "sdm_" prefix):
  project(X, Wt, n)                      -> (s1, s2, q1, q2, v, alpha, beta)
  mx4_quantize(x)                        -> (codes, scales)   (4-bit, blocks of 32)
  mx4_dequantize(codes, scales, dtype)   -> x
  project_mx4(Xq, Xs, Wq, Ws, n)         -> as project, from 4-bit operands
  select(x1, x2, K)                      -> (idx, score, weight)
  state_init(M0, B, dtype)               -> M
  scan(M, widx, wk, ridx, rw, v, alpha, beta) -> out      (M updated in place)
  step_decode(M, s1, s2, q1, q2, v, alpha, beta, W, R) -> (out, widx, ridx)
Training (fp32 state; selections held fixed):
  scan_train(M, widx, wk, ridx, rw, v, alpha, beta) -> (out, tape)
  scan_backward(widx, wk, ridx, rw, v, alpha, beta, tape, dout, G) -> dict
  scan_backward_noalloc(..., G, out) -> out   (no workspace, no allocation)
  scan_train8(M, widx, wk, ridx, rw, v, alpha, beta) -> (out, (codes, scales))
  tape8_read((codes, scales), dtype) -> tape  (the 8-bit tape's rows)
  scan_backward8(widx, wk, ridx, rw, v, alpha, beta, (codes, scales), dout, G) -> dict
Planned scan (fp32 state; few memories, long sequences):
  scan_plan(widx, wk, ridx, rw, N, d_v) -> workspace
  scan_planned(M, v, alpha, beta, workspace) -> out       (M updated in place)
  touch_prepare(widx, ridx, N) -> (seen, first)
  select_backward(idx, weight, dweight, n) -> (dx1, dx2)
  state_init_backward(G) -> dM0
Dense recurrence with a decay for each head (fp32 or bf16; fp32 state):
  linear_scan(S, q, k, v, g) -> out                       (S updated in place)
  linear_step(S, q, k, v, g) -> out                       (one token)
  linear_scan_train(S, q, k, v, g) -> (out, tape)
  linear_backward(q, k, v, g, tape, dout, G) -> dict      (G updated in place)
Norms before and after a block (fp32 or bf16):
  norm(y, w, z, x, scale, eps) -> out, or (out, next) with next_w
  norm_backward(dout, y, w, z, scale, eps, skip) -> dict

stream= is a torch stream or a raw handle (None: the current stream).  Tensors
that a call makes are allocated for that stream and marked as used by the
current one; tensors passed in have to stay allocated until the stream has run
the call.  A call runs on its tensors' GPU, whichever is current; a stream of
another GPU is refused.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsdm.so")
ABI_VERSION = 6  # the library's sdm_abi_version() this binding is written for

SDM_F32 = 0
SDM_BF16 = 1
SDM_FP8 = 2
STATUS = {0: "SDM_OK", 1: "SDM_ERR_INVALID", 2: "SDM_ERR_UNSUPPORTED", 3: "SDM_ERR_HIP"}

# Every symbol include/sdm.h declares.
EXPORTS = ("sdm_project", "sdm_mx4_quantize", "sdm_mx4_dequantize", "sdm_project_mx4", "sdm_select", "sdm_state_init", "sdm_scan", "sdm_step_decode", "sdm_scan_train",
           "sdm_scan_backward_workspace_size", "sdm_scan_backward", "sdm_scan_backward_noalloc",
           "sdm_select_backward", "sdm_scan_plan_workspace_size", "sdm_scan_plan",
           "sdm_scan_planned", "sdm_state_init_backward", "sdm_touch_prepare", "sdm_scan_train8", "sdm_tape8_read",
           "sdm_scan_backward8", "sdm_scan_backward8_workspace_size", "sdm_linear_scan_workspace_size", "sdm_linear_scan",
           "sdm_linear_step", "sdm_linear_backward_workspace_size", "sdm_linear_backward", "sdm_norm",
           "sdm_norm_backward_workspace_size", "sdm_norm_backward", "sdm_status_string", "sdm_last_error",
           "sdm_abi_version")

_lib = None


class SDMError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


def lib():
    """Load libsdm.so (raises if it is not built, or built from other sources
    than this binding's)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m sparse_memory_linear_sdm_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        missing = [e for e in EXPORTS if not hasattr(L, e)]
        if "sdm_abi_version" not in missing and L.sdm_abi_version() != ABI_VERSION:
            raise RuntimeError(f"{LIB_PATH} has ABI {L.sdm_abi_version()}, this binding "
                               f"expects {ABI_VERSION}: rebuild it")
        if missing:
            raise RuntimeError(f"{LIB_PATH} lacks {', '.join(missing)}: rebuild it")
        p, i32, i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
        L.sdm_project.argtypes = [p, p, i32, i32, i32, i32, i32, i32] + [p] * 8
        L.sdm_mx4_quantize.argtypes = [p, i32, i64, i64, p, p, p]
        L.sdm_mx4_dequantize.argtypes = [p, p, i32, i64, i64, p, p]
        L.sdm_project_mx4.argtypes = [p] * 4 + [i32] * 6 + [p] * 8
        L.sdm_select.argtypes = [p, p, i64, i32, i32, p, p, p, p]
        L.sdm_state_init.argtypes = [p, i32, p, i32, i32, i64, i32, p]
        L.sdm_scan.argtypes = [p, i32, i32, i32, i64, i32, i64, i32, i32] + [p] * 9
        L.sdm_step_decode.argtypes = [p, i32, i32, i32, i32, i32, i32, i32] + [p] * 11
        L.sdm_scan_train.argtypes = [p, i32, i32, i64, i32, i64, i32, i32] + [p] * 10
        L.sdm_scan_backward_workspace_size.argtypes = [i32, i32, i32, i64, i32, i32]
        L.sdm_scan_backward_workspace_size.restype = ctypes.c_size_t
        L.sdm_scan_backward.argtypes = ([i32, i32, i64, i32, i64, i32, i32] + [p] * 17 +
                                        [ctypes.c_size_t, p])
        L.sdm_scan_backward_noalloc.argtypes = [i32, i32, i64, i32, i64, i32, i32] + [p] * 17
        L.sdm_scan_train8.argtypes = [p, i32, i32, i64, i32, i64, i32, i32] + [p] * 11
        L.sdm_tape8_read.argtypes = [p, p, i32, i32, i32, i64, i32, i32, p, p]
        L.sdm_scan_backward8_workspace_size.argtypes = [i32, i32, i32, i64, i32, i32]
        L.sdm_scan_backward8_workspace_size.restype = ctypes.c_size_t
        L.sdm_scan_backward8.argtypes = ([i32, i32, i64, i32, i64, i32, i32] + [p] * 18 +
                                         [ctypes.c_size_t, p])
        L.sdm_touch_prepare.argtypes = [i32, i32, i64, i64, i32, i32, p, p, p, p, p]
        L.sdm_scan_plan_workspace_size.argtypes = [i32, i32, i32, i64]
        L.sdm_scan_plan_workspace_size.restype = ctypes.c_size_t
        L.sdm_scan_plan.argtypes = [i32, i32, i64, i32, i64, i32, i32] + [p] * 5 + [ctypes.c_size_t, p]
        L.sdm_scan_planned.argtypes = [p, i32, i32, i64, i32, i64] + [p] * 5 + [ctypes.c_size_t, p]
        L.sdm_select_backward.argtypes = [p, p, p, i64, i32, i32, p, p, p]
        L.sdm_state_init_backward.argtypes = [p, i32, i32, i64, i32, p, p, p]
        f32, size = ctypes.c_float, ctypes.c_size_t
        L.sdm_linear_scan_workspace_size.argtypes = [i32] * 5 + [i64]
        L.sdm_linear_scan_workspace_size.restype = size
        L.sdm_linear_scan.argtypes = [p] + [i32] * 6 + [i64] + [p] * 7 + [size, p]
        L.sdm_linear_step.argtypes = [p] + [i32] * 6 + [p] * 6
        L.sdm_linear_backward_workspace_size.argtypes = [i32] * 6 + [i64]
        L.sdm_linear_backward_workspace_size.restype = size
        L.sdm_linear_backward.argtypes = [i32] * 6 + [i64] + [p] * 12 + [size, p]
        L.sdm_norm.argtypes = ([p, i32, p, p, p, f32, f32, i32, i32, i64, i32, p, i32] + [p] * 3)
        L.sdm_norm_backward_workspace_size.argtypes = [i32, i32, i64, i32]
        L.sdm_norm_backward_workspace_size.restype = size
        L.sdm_norm_backward.argtypes = ([p, i32, p, i32, p, p, p, f32, f32, i32, i32, i64, i32] +
                                        [p] * 4 + [size, p])
        for f in ("sdm_project", "sdm_mx4_quantize", "sdm_mx4_dequantize", "sdm_project_mx4",
                  "sdm_select", "sdm_state_init", "sdm_scan", "sdm_step_decode",
                  "sdm_abi_version", "sdm_scan_train", "sdm_scan_backward",
                  "sdm_scan_backward_noalloc",
                  "sdm_select_backward", "sdm_state_init_backward", "sdm_touch_prepare",
                  "sdm_scan_plan", "sdm_scan_planned", "sdm_scan_train8", "sdm_tape8_read",
                  "sdm_scan_backward8", "sdm_linear_scan", "sdm_linear_step",
                  "sdm_linear_backward", "sdm_norm", "sdm_norm_backward"):
            getattr(L, f).restype = ctypes.c_int
        L.sdm_status_string.argtypes = [i32]
        L.sdm_status_string.restype = ctypes.c_char_p
        L.sdm_last_error.argtypes = []
        L.sdm_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(rc: int):
    if rc != 0:
        raise SDMError(rc, lib().sdm_last_error().decode())


def _arg(t, dtype, shape, name):
    """Check one tensor argument: type, exact shape (the one the call derives
    from its other arguments), dtype (one dtype or a tuple of allowed ones;
    None = any) and contiguity.  Returns (name, tensor) for _gpu().  A
    mismatch raises ValueError (TypeError for a non-tensor): the kernels
    index every buffer by sizes taken from other arguments, so a short or
    strided buffer must never reach them.  Every argument of a call passes
    these checks before any device check, so a call fails on the first bad
    shape whatever device its tensors are on."""
    try:  # the common case first: small calls cost about as much as their checks
        if t.dtype is dtype and t.shape == shape and t.is_contiguous():
            return (name, t)
    except AttributeError:
        pass
    import torch

    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    allowed = dtype if isinstance(dtype, tuple) else (dtype,)
    if dtype is not None and t.dtype not in allowed:
        raise ValueError(f"{name} must be {' or '.join(map(str, allowed))}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return (name, t)


def _gpu(*args):
    """Device pointers of checked arguments ((name, tensor) pairs from _arg,
    or None for an absent optional one): every tensor must be on the GPU, all
    on the same device."""
    dev = -1
    ptrs = []
    for a in args:
        if a is None:
            ptrs.append(None)
            continue
        name, t = a
        if not t.is_cuda:
            raise ValueError(f"{name} must be on the GPU")
        at = t.get_device()
        if at != dev:
            if dev >= 0:
                raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{dev}")
            dev = at
        ptrs.append(t.data_ptr())
    return ptrs


def _call(fn, t, stream, *args):
    """fn(*args, stream handle) for a call on tensor t's GPU, with that GPU
    current while the call runs: on the caller's stream, or on t's GPU's
    current one.  A stream of another GPU is refused."""
    import torch

    index = t.get_device()
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _call(fn, t, stream, *args)
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, the call's tensors on {t.device}")
        handle = stream.cuda_stream
    else:
        handle = int(stream)
    _check(fn(*args, handle))


def _empty_on(stream, device):
    """torch.empty(shape, dtype) for the tensors a call makes.  The call's
    stream is the first to write them, so they are that stream's memory (what
    the allocator hands out for another stream may still be in use there), and
    those the caller gets are marked as used by the current stream too."""
    import torch

    if stream is None or device.type != "cuda":
        return lambda shape, dtype, mine=False: torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                  else torch.cuda.default_stream(device))

    def make(shape, dtype, mine=False):
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=device)
        if not mine and stream != current:
            t.record_stream(current)
        return t

    return make


def _state_dtype(M):
    import torch

    if M.dtype == torch.float32:
        return SDM_F32
    if M.dtype == torch.bfloat16:
        return SDM_BF16
    if M.dtype == torch.float8_e4m3fn:
        return SDM_FP8
    raise ValueError(f"state must be float32, bfloat16 or float8_e4m3fn, got {M.dtype}")


def _state_types():
    import torch

    return (torch.float32, torch.bfloat16, torch.float8_e4m3fn)


def _units(lead):
    units = 1
    for s in lead:
        units *= s
    return units


def _project_out(B, T, H, P, n, weights, out, stream, device):
    """The projections' 7 output tensors, made unless the caller gives them,
    and their checked arguments."""
    import torch

    f32 = torch.float32
    d_v = P - 4 * n - 2
    if n < 1 or d_v < 1:
        raise ValueError(f"{weights} has P={P} rows per head: too few for n={n} "
                         "(P = 4n + d_v + 2)")
    names = ("s1", "s2", "q1", "q2", "v", "alpha", "beta")
    if out is None:
        empty = _empty_on(stream, device)
        s1, v, alpha = empty((B, H, T, n), f32), empty((B, H, T, d_v), f32), empty((B, H, T), f32)
        like = torch.empty_like if stream is None else lambda t: empty(t.shape, f32)
        out = (s1, like(s1), like(s1), like(s1), v, alpha, like(alpha))
        return out, list(zip(names, out))
    shapes = [(B, H, T, n)] * 4 + [(B, H, T, d_v), (B, H, T), (B, H, T)]
    if len(out) != 7:
        raise ValueError("out must hold 7 tensors (s1, s2, q1, q2, v, alpha, beta)")
    return tuple(out), [_arg(t, f32, sh, nm) for t, sh, nm in zip(out, shapes, names)]


def project(X, Wt, n: int, out=None, stream=None):
    """Token projections on the matrix cores: X [B, T, d_model] bfloat16,
    Wt [H, P, d_model] bfloat16 with P = 4n + d_v + 2 (rows s1, s2, q1, q2,
    v, alpha, beta of each head).  Returns fp32 (s1, s2, q1, q2) [B, H, T, n],
    v [B, H, T, d_v], alpha, beta [B, H, T] (the gates through the logistic
    function).  out = that 7-tuple writes into caller tensors."""
    import torch

    bf16 = torch.bfloat16
    if X.dim() != 3 or Wt.dim() != 3:
        raise ValueError("X must be [B, T, d_model] and Wt [H, P, d_model]")
    B, T, d_model = X.shape
    H, P = Wt.shape[0], Wt.shape[1]
    out, outs = _project_out(B, T, H, P, n, "Wt", out, stream, X.device)
    ptrs = _gpu(_arg(X, bf16, (B, T, d_model), "X"), _arg(Wt, bf16, (H, P, d_model), "Wt"), *outs)
    _call(lib().sdm_project, X, stream, *ptrs[:2], B, T, d_model, H, n, P - 4 * n - 2, *ptrs[2:])
    return out


def _value_dtype(dtype):
    import torch

    if dtype == torch.float32:
        return SDM_F32
    if dtype == torch.bfloat16:
        return SDM_BF16
    raise ValueError(f"values must be float32 or bfloat16, got {dtype}")


def _mx4_args(codes, scales, shape, names=("codes", "scales")):
    """Checked codes and scales of a 4-bit matrix of the given shape
    [..., cols] (its leading dimensions flattened are the rows)."""
    import torch

    *lead, cols = shape
    return [_arg(codes, torch.uint8, (*lead, cols // 2), names[0]),
            _arg(scales, torch.uint8, (cols // 128, _units(lead), 4), names[1])]


def mx4_quantize(x, out=None, stream=None):
    """4-bit microscaled form of x [..., cols] (fp32 or bf16): returns codes
    uint8 [..., cols/2] (two columns a byte) and scales uint8
    [cols/128, rows, 4] (one byte per 32 columns; rows: the leading dimensions
    together).  out = (codes, scales) writes into caller tensors."""
    import torch

    if x.dim() < 1:
        raise ValueError("x must have a last dimension cols")
    shape = tuple(x.shape)
    *lead, cols = shape
    rows, dtype = _units(lead), _value_dtype(x.dtype)
    if out is None:
        empty = _empty_on(stream, x.device)
        codes = empty((*lead, cols // 2), torch.uint8)
        scales = empty((cols // 128, rows, 4), torch.uint8)
        outs = (("codes", codes), ("scales", scales))
    else:
        codes, scales = out
        outs = _mx4_args(codes, scales, shape)
    px, pc, ps = _gpu(_arg(x, x.dtype, shape, "x"), *outs)
    _call(lib().sdm_mx4_quantize, x, stream, px, dtype, rows, cols, pc, ps)
    return codes, scales


def mx4_dequantize(codes, scales, dtype=None, out=None, stream=None):
    """Values [..., cols] (float32 unless dtype or out says bfloat16; exact in
    both) of a 4-bit matrix from mx4_quantize."""
    import torch

    if codes.dim() < 1:
        raise ValueError("codes must have a last dimension cols/2")
    shape = (*codes.shape[:-1], 2 * codes.shape[-1])
    if out is None:
        out = _empty_on(stream, codes.device)(shape, torch.float32 if dtype is None else dtype)
    elif dtype is not None and dtype != out.dtype:
        raise ValueError(f"out must be {dtype}, got {out.dtype}")
    dt = _value_dtype(out.dtype)
    pc, ps, px = _gpu(*_mx4_args(codes, scales, shape), _arg(out, out.dtype, shape, "out"))
    _call(lib().sdm_mx4_dequantize, codes, stream, pc, ps, dt, _units(shape[:-1]), shape[-1], px)
    return out


def project_mx4(Xq, Xs, Wq, Ws, n: int, out=None, stream=None):
    """project() from 4-bit operands (mx4_quantize of X and of Wt): Xq
    [B, T, d_model/2], Xs [d_model/128, B*T, 4], Wq [H, P, d_model/2], Ws
    [d_model/128, H*P, 4], all uint8.  Returns (or writes into out)
    project()'s 7 tensors."""
    if Xq.dim() != 3 or Wq.dim() != 3:
        raise ValueError("Xq must be [B, T, d_model/2] and Wq [H, P, d_model/2]")
    B, T, half = Xq.shape
    H, P = Wq.shape[0], Wq.shape[1]
    d_model = 2 * half
    out, outs = _project_out(B, T, H, P, n, "Wq", out, stream, Xq.device)
    ptrs = _gpu(*_mx4_args(Xq, Xs, (B, T, d_model), ("Xq", "Xs")),
                *_mx4_args(Wq, Ws, (H, P, d_model), ("Wq", "Ws")), *outs)
    _call(lib().sdm_project_mx4, Xq, stream, *ptrs[:4], B, T, d_model, H, n, P - 4 * n - 2, *ptrs[4:])
    return out


def select(x1, x2, K: int, out=None, stream=None):
    """Top-K slots of the product-key table for every leading index of
    x1, x2 [..., n]: returns idx int32, score fp32, weight fp32 [..., K].
    out = (idx, score, weight) writes into caller tensors (score may be
    None)."""
    import torch

    f32 = torch.float32
    shape = tuple(x1.shape)
    if len(shape) < 1:
        raise ValueError("x1 and x2 must have a last dimension n")
    n, lead = shape[-1], shape[:-1]
    if out is None:
        empty = _empty_on(stream, x1.device)
        idx, score, weight = (empty(lead + (K,), dt) for dt in (torch.int32, f32, f32))
    else:
        idx, score, weight = out
    p1, p2, pi, ps, pw = _gpu(
        _arg(x1, f32, shape, "x1"), _arg(x2, f32, shape, "x2"),
        _arg(idx, torch.int32, lead + (K,), "idx"),
        None if score is None else _arg(score, f32, lead + (K,), "score"),
        _arg(weight, f32, lead + (K,), "weight"))
    _call(lib().sdm_select, x1, stream, p1, p2, _units(lead), n, K, pi, ps, pw)
    return idx, score, weight


def state_init(M0, B: int, dtype=None, out=None, stream=None):
    """M [B,H,N,d_v] = M0 [H,N,d_v] for every b (fp32, bf16 or fp8 E4M3 state).
    out = an existing state tensor to fill (its dtype is the state type)."""
    import torch

    if M0.dim() != 3:
        raise ValueError(f"M0 must be [H, N, d_v], got {tuple(M0.shape)}")
    H, N, d_v = M0.shape
    a0 = _arg(M0, torch.float32, (H, N, d_v), "M0")
    if out is None:
        dtype = torch.float32 if dtype is None else dtype
        M = _empty_on(stream, M0.device)((B, H, N, d_v), dtype)
    else:
        M = out
    p0, pm = _gpu(a0, _arg(M, _state_types(), (B, H, N, d_v), "M"))
    _call(lib().sdm_state_init, M, stream, pm, _state_dtype(M), p0, B, H, N, d_v)
    return M


def _scan_shapes(M, widx, ridx):
    if M.dim() != 4:
        raise ValueError(f"the state must be [B, H, N, d_v], got {tuple(M.shape)}")
    if widx.dim() != 4 or ridx.dim() != 4:
        raise ValueError("widx and ridx must be [B, H, T, W] and [B, H, T, R]")
    B, H, N, d_v = M.shape
    T, W = widx.shape[2], widx.shape[3]
    R = ridx.shape[3]
    return B, H, N, d_v, T, W, R


def _scan_args(B, H, T, W, R, d_v, widx, wk, ridx, rw, v, alpha, beta):
    import torch

    f32 = torch.float32
    return [_arg(widx, torch.int32, (B, H, T, W), "widx"), _arg(wk, f32, (B, H, T, W), "wk"),
            _arg(ridx, torch.int32, (B, H, T, R), "ridx"), _arg(rw, f32, (B, H, T, R), "rw"),
            _arg(v, f32, (B, H, T, d_v), "v"), _arg(alpha, f32, (B, H, T), "alpha"),
            _arg(beta, f32, (B, H, T), "beta")]


def scan(M, widx, wk, ridx, rw, v, alpha, beta, out=None, stream=None):
    """T steps of write + read on M [B,H,N,d_v] in place.  widx, wk
    [B,H,T,W]; ridx, rw [B,H,T,R]; v [B,H,T,d_v]; alpha, beta [B,H,T].
    Returns out [B,H,T,d_v] fp32."""
    import torch

    B, H, N, d_v, T, W, R = _scan_shapes(M, widx, ridx)
    am = _arg(M, _state_types(), (B, H, N, d_v), "M")
    ins = _scan_args(B, H, T, W, R, d_v, widx, wk, ridx, rw, v, alpha, beta)
    if out is None:
        out = _empty_on(stream, M.device)((B, H, T, d_v), torch.float32)
    pm, *ptrs = _gpu(am, *ins, _arg(out, torch.float32, (B, H, T, d_v), "out"))
    _call(lib().sdm_scan, M, stream, pm, _state_dtype(M), B, H, N, d_v, T, W, R, *ptrs)
    return out


def step_decode(M, s1, s2, q1, q2, v, alpha, beta, W: int, R: int, out=None, want_idx=True,
                stream=None):
    """One token per (b,h): selections, write and read fused.  s1.. [B,H,n];
    v [B,H,d_v]; alpha, beta [B,H].  Returns (out [B,H,d_v], widx, ridx)."""
    import torch

    if M.dim() != 4:
        raise ValueError(f"the state must be [B, H, N, d_v], got {tuple(M.shape)}")
    B, H, N, d_v = M.shape
    n = s1.shape[-1]
    if n * n != N:
        raise ValueError(f"M has {N} rows but the halves give n*n = {n * n}")
    f32 = torch.float32
    ins = [_arg(M, _state_types(), (B, H, N, d_v), "M")]
    ins += [_arg(t, f32, (B, H, n), nm) for nm, t in
            (("s1", s1), ("s2", s2), ("q1", q1), ("q2", q2))]
    ins += [_arg(v, f32, (B, H, d_v), "v"), _arg(alpha, f32, (B, H), "alpha"),
            _arg(beta, f32, (B, H), "beta")]
    empty = _empty_on(stream, M.device) if out is None or want_idx else None
    if out is None:
        out = empty((B, H, d_v), f32)
    ins.append(_arg(out, f32, (B, H, d_v), "out"))
    widx = ridx = None
    if want_idx:
        widx, ridx = empty((B, H, W), torch.int32), empty((B, H, R), torch.int32)
    pm, *ptrs = _gpu(*ins)
    _call(lib().sdm_step_decode, M, stream, pm, _state_dtype(M), B, H, n, d_v, W, R, *ptrs,
          widx.data_ptr() if widx is not None else None,
          ridx.data_ptr() if ridx is not None else None)
    return out, widx, ridx


def scan_train(M, widx, wk, ridx, rw, v, alpha, beta, out=None, tape=None, stream=None):
    """scan() on an fp32 state that also keeps, per step, the W pre-write rows
    and the R rows the read used: returns (out [B,H,T,d_v],
    tape [B,H,T,W+R,d_v])."""
    import torch

    f32 = torch.float32
    B, H, N, d_v, T, W, R = _scan_shapes(M, widx, ridx)
    am = _arg(M, f32, (B, H, N, d_v), "M")
    ins = _scan_args(B, H, T, W, R, d_v, widx, wk, ridx, rw, v, alpha, beta)
    empty = _empty_on(stream, M.device)
    if out is None:
        out = empty((B, H, T, d_v), f32)
    if tape is None:
        tape = empty((B, H, T, W + R, d_v), f32)
    pm, *ptrs = _gpu(am, *ins, _arg(out, f32, (B, H, T, d_v), "out"),
                     _arg(tape, f32, (B, H, T, W + R, d_v), "tape"))
    _call(lib().sdm_scan_train, M, stream, pm, B, H, N, d_v, T, W, R, *ptrs)
    return out, tape


def scan_backward(widx, wk, ridx, rw, v, alpha, beta, tape, dout, G, workspace=None,
                  first=None, stream=None):
    """Reverse pass from the tape of scan_train (the state is not needed):
    G (dL/d final state, [B,H,N,d_v]) becomes dL/d initial state in place.
    With first (from touch_prepare) the final-state gradient is taken as
    zero and G need not be cleared; only the rows the steps select are
    written.  Returns dict dv [B,H,T,d_v], dwk [B,H,T,W], drw [B,H,T,R],
    dalpha, dbeta [B,H,T]."""
    import torch

    f32 = torch.float32
    B, H, N, d_v, T, W, R = _scan_shapes(G, widx, ridx)
    ins = _scan_args(B, H, T, W, R, d_v, widx, wk, ridx, rw, v, alpha, beta)
    ins += [_arg(tape, f32, (B, H, T, W + R, d_v), "tape"),
            _arg(dout, f32, (B, H, T, d_v), "dout"), _arg(G, f32, (B, H, N, d_v), "G")]
    af = None if first is None else _arg(first, torch.int64, (B, H, T, 2), "first")
    empty = _empty_on(stream, G.device)
    shapes = {"dv": (B, H, T, d_v), "dwk": (B, H, T, W), "drw": (B, H, T, R),
              "dalpha": (B, H, T), "dbeta": (B, H, T)}
    o = {k: empty(shp, f32) for k, shp in shapes.items()}
    if workspace is None:
        need = int(lib().sdm_scan_backward_workspace_size(B, H, d_v, T, W, R))
        workspace = empty(((max(need, 16) + 3) // 4,), f32, mine=True)
    ptrs = _gpu(*ins, *o.items(), af, _arg(workspace, None, None, "workspace"))
    nbytes = workspace.numel() * workspace.element_size()
    _call(lib().sdm_scan_backward, G, stream, B, H, N, d_v, T, W, R, *ptrs, nbytes)
    return o


def scan_backward_noalloc(widx, wk, ridx, rw, v, alpha, beta, tape, dout, G, out, first=None,
                          stream=None):
    """scan_backward() without a workspace and without any allocation: the
    library's per-GPU static scratch buffer (64 MiB) holds the partial sums,
    and out is a dict of caller tensors dv [B,H,T,d_v], dwk [B,H,T,W],
    drw [B,H,T,R], dalpha, dbeta [B,H,T] (fp32).  Calls on one GPU share the
    buffer and must not overlap in time.  Returns out."""
    import torch

    f32 = torch.float32
    B, H, N, d_v, T, W, R = _scan_shapes(G, widx, ridx)
    ins = _scan_args(B, H, T, W, R, d_v, widx, wk, ridx, rw, v, alpha, beta)
    ins += [_arg(tape, f32, (B, H, T, W + R, d_v), "tape"),
            _arg(dout, f32, (B, H, T, d_v), "dout"), _arg(G, f32, (B, H, N, d_v), "G")]
    shapes = {"dv": (B, H, T, d_v), "dwk": (B, H, T, W), "drw": (B, H, T, R),
              "dalpha": (B, H, T), "dbeta": (B, H, T)}
    ins += [_arg(out[k], f32, shp, k) for k, shp in shapes.items()]
    af = None if first is None else _arg(first, torch.int64, (B, H, T, 2), "first")
    ptrs = _gpu(*ins, af)
    _call(lib().sdm_scan_backward_noalloc, G, stream, B, H, N, d_v, T, W, R, *ptrs)
    return out


def _tape8_args(tape, B, H, T, S, d_v):
    import torch

    codes, scales = tape
    return [_arg(codes, torch.int8, (B, H, d_v // 16, T, S, 16), "tape codes"),
            _arg(scales, torch.uint8, (B, H, d_v // 16, T, S), "tape scales")]


def scan_train8(M, widx, wk, ridx, rw, v, alpha, beta, out=None, tape=None, stream=None):
    """scan_train() with its tape in 8 bits: returns (out [B,H,T,d_v],
    (codes int8 [B,H,d_v/16,T,W+R,16], scales uint8 [B,H,d_v/16,T,W+R])).
    M and out are scan_train()'s bit for bit."""
    import torch

    f32 = torch.float32
    B, H, N, d_v, T, W, R = _scan_shapes(M, widx, ridx)
    am = _arg(M, f32, (B, H, N, d_v), "M")
    ins = _scan_args(B, H, T, W, R, d_v, widx, wk, ridx, rw, v, alpha, beta)
    empty = _empty_on(stream, M.device)
    if out is None:
        out = empty((B, H, T, d_v), f32)
    if tape is None:
        tape = (empty((B, H, d_v // 16, T, W + R, 16), torch.int8),
                empty((B, H, d_v // 16, T, W + R), torch.uint8))
    pm, *ptrs = _gpu(am, *ins, _arg(out, f32, (B, H, T, d_v), "out"),
                     *_tape8_args(tape, B, H, T, W + R, d_v))
    _call(lib().sdm_scan_train8, M, stream, pm, B, H, N, d_v, T, W, R, *ptrs)
    return out, tuple(tape)


def tape8_read(tape, dtype=None, out=None, stream=None):
    """The rows [B,H,T,W+R,d_v] (float32 unless dtype or out says bfloat16;
    exact in both) of an 8-bit tape."""
    import torch

    codes, scales = tape
    if codes.dim() != 6:
        raise ValueError("tape codes must be [B, H, d_v/16, T, W+R, 16]")
    B, H, nb, T, S = codes.shape[:5]
    shape = (B, H, T, S, 16 * nb)
    if out is None:
        out = _empty_on(stream, codes.device)(shape, torch.float32 if dtype is None else dtype)
    elif dtype is not None and dtype != out.dtype:
        raise ValueError(f"out must be {dtype}, got {out.dtype}")
    dt = _value_dtype(out.dtype)
    pc, ps, po = _gpu(*_tape8_args(tape, B, H, T, S, 16 * nb), _arg(out, out.dtype, shape, "out"))
    _call(lib().sdm_tape8_read, codes, stream, pc, ps, B, H, 16 * nb, T, S, dt, po)
    return out


def scan_backward8(widx, wk, ridx, rw, v, alpha, beta, tape, dout, G, workspace=None, first=None,
                   out=None, stream=None):
    """scan_backward() from the 8-bit tape (codes, scales) of scan_train8.
    out = a dict of dv, dwk, drw, dalpha, dbeta writes into caller tensors;
    with it and a workspace the call allocates nothing."""
    import torch

    f32 = torch.float32
    B, H, N, d_v, T, W, R = _scan_shapes(G, widx, ridx)
    ins = _scan_args(B, H, T, W, R, d_v, widx, wk, ridx, rw, v, alpha, beta)
    ins += _tape8_args(tape, B, H, T, W + R, d_v)
    ins += [_arg(dout, f32, (B, H, T, d_v), "dout"), _arg(G, f32, (B, H, N, d_v), "G")]
    shapes = {"dv": (B, H, T, d_v), "dwk": (B, H, T, W), "drw": (B, H, T, R),
              "dalpha": (B, H, T), "dbeta": (B, H, T)}
    empty = _empty_on(stream, G.device)
    if out is None:
        out = {k: empty(shp, f32) for k, shp in shapes.items()}
    ins += [_arg(out[k], f32, shp, k) for k, shp in shapes.items()]
    af = None if first is None else _arg(first, torch.int64, (B, H, T, 2), "first")
    if workspace is None:
        need = int(lib().sdm_scan_backward8_workspace_size(B, H, d_v, T, W, R))
        workspace = empty(((max(need, 16) + 3) // 4,), f32, mine=True)
    ptrs = _gpu(*ins, af, _arg(workspace, None, None, "workspace"))
    nbytes = workspace.numel() * workspace.element_size()
    _call(lib().sdm_scan_backward8, G, stream, B, H, N, d_v, T, W, R, *ptrs, nbytes)
    return out


def touch_prepare(widx, ridx, N: int, seen=None, first=None, stream=None):
    """Bookkeeping of the sparse training mode: seen [B,H,ceil(N/32)] int32
    (the bits of the uint32 words: row r is selected at some step) and first
    [B,H,T,2] int64 (the bits of the uint64 masks of slots whose row is
    selected for the last time at that step).  N <= 2^20."""
    import torch

    if widx.dim() != 4 or ridx.dim() != 4:
        raise ValueError("widx and ridx must be [B, H, T, W] and [B, H, T, R]")
    B, H, T, W = widx.shape
    R = ridx.shape[3]
    ins = [_arg(widx, torch.int32, (B, H, T, W), "widx"),
           _arg(ridx, torch.int32, (B, H, T, R), "ridx")]
    empty = _empty_on(stream, widx.device)
    if seen is None:
        seen = empty((B, H, (N + 31) // 32), torch.int32)
    if first is None:
        first = empty((B, H, T, 2), torch.int64)
    ptrs = _gpu(*ins, _arg(seen, torch.int32, (B, H, (N + 31) // 32), "seen"),
                _arg(first, torch.int64, (B, H, T, 2), "first"))
    _call(lib().sdm_touch_prepare, widx, stream, B, H, N, T, W, R, *ptrs)
    return seen, first


def seen_rows(seen, N: int):
    """The seen bitmap of touch_prepare as a [B,H,N] bool tensor."""
    import torch

    shifts = torch.arange(32, dtype=torch.int32, device=seen.device)
    bits = (seen.unsqueeze(-1) >> shifts) & 1
    return bits.reshape(seen.shape[0], seen.shape[1], -1)[:, :, :N].bool()


def select_backward(idx, weight, dweight, n: int, stream=None):
    """Gradient of the selection weights back to the halves: idx, weight,
    dweight [..., K] -> (dx1, dx2) [..., n] fp32."""
    import torch

    f32 = torch.float32
    shape = tuple(idx.shape)
    if len(shape) < 1:
        raise ValueError("idx must have a last dimension K")
    K, lead = shape[-1], shape[:-1]
    ins = [_arg(idx, torch.int32, shape, "idx"), _arg(weight, f32, shape, "weight"),
           _arg(dweight, f32, shape, "dweight")]
    empty = _empty_on(stream, idx.device)
    dx1, dx2 = empty(lead + (n,), f32), empty(lead + (n,), f32)
    ptrs = _gpu(*ins, ("dx1", dx1), ("dx2", dx2))
    _call(lib().sdm_select_backward, idx, stream, *ptrs[:3], _units(lead), n, K, *ptrs[3:])
    return dx1, dx2


def state_init_backward(G, out=None, seen=None, stream=None):
    """dM0 [H,N,d_v] = sum over b of G [B,H,N,d_v]; with seen (from
    touch_prepare) only the rows each sequence selected count."""
    import torch

    f32 = torch.float32
    if G.dim() != 4:
        raise ValueError(f"G must be [B, H, N, d_v], got {tuple(G.shape)}")
    B, H, N, d_v = G.shape
    ag = _arg(G, f32, (B, H, N, d_v), "G")
    as_ = None if seen is None else _arg(seen, torch.int32, (B, H, (N + 31) // 32), "seen")
    dM0 = _empty_on(stream, G.device)((H, N, d_v), f32) if out is None else out
    pg, ps, po = _gpu(ag, as_, _arg(dM0, f32, (H, N, d_v), "dM0"))
    _call(lib().sdm_state_init_backward, G, stream, pg, B, H, N, d_v, ps, po)
    return dM0


def scan_plan_workspace_size(B: int, H: int, d_v: int, T: int) -> int:
    """Bytes of workspace scan_plan / scan_planned need on the current GPU (0: unsupported)."""
    return int(lib().sdm_scan_plan_workspace_size(B, H, d_v, T))


def scan_plan(widx, wk, ridx, rw, N: int, d_v: int, workspace=None, stream=None):
    """Plan the steps of a planned scan on memories of N rows of d_v fp32
    columns: widx, wk [B,H,T,W]; ridx, rw [B,H,T,R].  Returns the workspace
    (a uint8 device tensor, allocated when None) for scan_planned."""
    import torch

    if widx.dim() != 4 or ridx.dim() != 4:
        raise ValueError("widx and ridx must be [B, H, T, W] and [B, H, T, R]")
    B, H, T, W = widx.shape
    R = ridx.shape[3]
    f32 = torch.float32
    ins = [_arg(widx, torch.int32, (B, H, T, W), "widx"), _arg(wk, f32, (B, H, T, W), "wk"),
           _arg(ridx, torch.int32, (B, H, T, R), "ridx"), _arg(rw, f32, (B, H, T, R), "rw")]
    if workspace is None:
        with torch.cuda.device(widx.get_device()) if widx.is_cuda else contextlib.nullcontext():
            need = scan_plan_workspace_size(B, H, d_v, T)
        workspace = _empty_on(stream, widx.device)((max(need, 256),), torch.uint8)
    ptrs = _gpu(*ins, _arg(workspace, None, None, "workspace"))
    nbytes = workspace.numel() * workspace.element_size()
    _call(lib().sdm_scan_plan, widx, stream, B, H, N, d_v, T, W, R, *ptrs, nbytes)
    return workspace


def scan_planned(M, v, alpha, beta, workspace, out=None, stream=None):
    """Run the steps scan_plan wrote into workspace on the fp32 state M
    [B,H,N,d_v] in place; v [B,H,T,d_v]; alpha, beta [B,H,T].  Returns out
    [B,H,T,d_v] fp32."""
    import torch

    if M.dim() != 4 or v.dim() != 4:
        raise ValueError("M and v must be [B, H, N, d_v] and [B, H, T, d_v]")
    B, H, N, d_v = M.shape
    T = v.shape[2]
    f32 = torch.float32
    if out is None:
        out = _empty_on(stream, M.device)((B, H, T, d_v), f32)
    ptrs = _gpu(_arg(M, f32, (B, H, N, d_v), "M"), _arg(v, f32, (B, H, T, d_v), "v"),
                _arg(alpha, f32, (B, H, T), "alpha"), _arg(beta, f32, (B, H, T), "beta"),
                _arg(out, f32, (B, H, T, d_v), "out"), _arg(workspace, None, None, "workspace"))
    nbytes = workspace.numel() * workspace.element_size()
    _call(lib().sdm_scan_planned, M, stream, ptrs[0], B, H, N, d_v, T, *ptrs[1:], nbytes)
    return out


def _linear_args(S, name, q, k, v, g, time):
    """Checked arguments of a call on the dense recurrence's state S (or its
    gradient), named `name`: dtype code, sizes and the tensors' pairs."""
    import torch

    f32 = torch.float32
    if S.dim() != 4:
        raise ValueError(f"{name} must be [B, H, d_k, d_v], got {tuple(S.shape)}")
    if q.dim() != 3 + time:
        raise ValueError("q and k must be " + ("[B, Hk, T, d_k]" if time else "[B, Hk, d_k]"))
    B, H, d_k, d_v = S.shape
    Hk = q.shape[1]
    T = (q.shape[2],) if time else ()
    if Hk < 1 or H % Hk:
        raise ValueError(f"{name} has {H} heads, not a multiple of q's {Hk}")
    args = [_arg(S, f32, (B, H, d_k, d_v), name), _arg(q, q.dtype, (B, Hk, *T, d_k), "q"),
            _arg(k, q.dtype, (B, Hk, *T, d_k), "k"), _arg(v, q.dtype, (B, H, *T, d_v), "v"),
            _arg(g, f32, (B, H, *T), "g")]
    return _value_dtype(q.dtype), (B, H, Hk, d_k, d_v, *T), args


def _workspace(workspace, need, empty):
    """(name, tensor) and bytes of a call's workspace, made unless the caller
    gives one; (None, 0) where the call needs none."""
    import torch

    if workspace is None:
        if need == 0:
            return None, 0
        workspace = empty((need,), torch.uint8, mine=True)
    return (_arg(workspace, None, None, "workspace"),
            workspace.numel() * workspace.element_size())


def _linear_tape(dtype, T):
    """Chunks of T steps (one state of the tape each)."""
    chunk = 64 if dtype == SDM_BF16 else 32
    return (T + chunk - 1) // chunk


def _linear_scan(S, q, k, v, g, out, tape, want_tape, workspace, stream):
    import torch

    dt, sizes, args = _linear_args(S, "S", q, k, v, g, True)
    B, H, Hk, d_k, d_v, T = sizes
    empty = _empty_on(stream, S.device)
    if out is None:
        out = empty((B, H, T, d_v), q.dtype)
    outs = [_arg(out, q.dtype, (B, H, T, d_v), "out"), None]
    if want_tape:
        shape = (B, H, _linear_tape(dt, T), d_k, d_v)
        if tape is None:
            tape = empty(shape, torch.float32)
        outs[1] = _arg(tape, torch.float32, shape, "tape")
    ws, nbytes = _workspace(
        workspace, int(lib().sdm_linear_scan_workspace_size(dt, B, H, d_k, d_v, T)), empty)
    pS, *ptrs = _gpu(*args, *outs, ws)
    _call(lib().sdm_linear_scan, S, stream, pS, dt, *sizes, *ptrs, nbytes)
    return out, tape


def linear_scan(S, q, k, v, g, out=None, workspace=None, stream=None):
    """T steps of the dense recurrence S_t = exp(g_t) S_{t-1} + k_t v_t^T,
    out_t = S_t^T q_t on S [B,H,d_k,d_v] (fp32, in place).  q, k [B,Hk,T,d_k]
    (Hk divides H: heads share them in order) and v [B,H,T,d_v], float32 or
    bfloat16; g [B,H,T] float32, normally <= 0 (-inf: the step forgets the
    state).  Returns out [B,H,T,d_v] of q's type."""
    return _linear_scan(S, q, k, v, g, out, None, False, workspace, stream)[0]


def linear_scan_train(S, q, k, v, g, out=None, tape=None, workspace=None, stream=None):
    """linear_scan() that also keeps the state before each chunk of C steps (64
    for bfloat16, 32 for float32): returns (out, tape [B,H,ceil(T/C),d_k,d_v]).
    B*H*T at most 2^26 - 4, as linear_backward takes."""
    return _linear_scan(S, q, k, v, g, out, tape, True, workspace, stream)


def linear_step(S, q, k, v, g, out=None, stream=None):
    """One token of every memory: linear_scan() without a time axis (q, k
    [B,Hk,d_k]; v [B,H,d_v]; g [B,H]).  Returns out [B,H,d_v]."""
    dt, sizes, args = _linear_args(S, "S", q, k, v, g, False)
    shape = (sizes[0], sizes[1], sizes[4])
    if out is None:
        out = _empty_on(stream, S.device)(shape, q.dtype)
    pS, *ptrs = _gpu(*args, _arg(out, q.dtype, shape, "out"))
    _call(lib().sdm_linear_step, S, stream, pS, dt, *sizes, *ptrs)
    return out


def linear_backward(q, k, v, g, tape, dout, G, workspace=None, out=None, stream=None):
    """Reverse pass of linear_scan_train: G [B,H,d_k,d_v] (dL/d final state)
    becomes dL/d initial state in place.  Returns a dict dq, dk [B,Hk,T,d_k], dv
    [B,H,T,d_v] of q's type and dg [B,H,T] float32.  out = such a dict writes
    into caller tensors."""
    import torch

    f32 = torch.float32
    dt, sizes, (aG, *ins) = _linear_args(G, "G", q, k, v, g, True)
    B, H, Hk, d_k, d_v, T = sizes
    ins += [_arg(tape, f32, (B, H, _linear_tape(dt, T), d_k, d_v), "tape"),
            _arg(dout, q.dtype, (B, H, T, d_v), "dout"), aG]
    shapes = {"dq": (q.dtype, (B, Hk, T, d_k)), "dk": (q.dtype, (B, Hk, T, d_k)),
              "dv": (q.dtype, (B, H, T, d_v)), "dg": (f32, (B, H, T))}
    empty = _empty_on(stream, G.device)
    if out is None:
        out = {n: empty(shape, t) for n, (t, shape) in shapes.items()}
    ins += [_arg(out[n], t, shape, n) for n, (t, shape) in shapes.items()]
    ws, nbytes = _workspace(
        workspace, int(lib().sdm_linear_backward_workspace_size(dt, *sizes)), empty)
    ptrs = _gpu(*ins, ws)
    _call(lib().sdm_linear_backward, G, stream, dt, *sizes, *ptrs, nbytes)
    return out


def _norm_sizes(y, heads):
    """(B, H, T, d) and the shape of the outputs of rows y."""
    if heads:
        if y.dim() != 4:
            raise ValueError(f"y must be [B, H, T, d], got {tuple(y.shape)}")
        B, H, T, d = y.shape
        return (B, H, T, d), (B, T, H * d)
    if y.dim() < 1:
        raise ValueError("y must have a last dimension d")
    return (1, 1, _units(y.shape[:-1]), y.shape[-1]), tuple(y.shape)


def norm(y, w, z=None, x=None, scale: float = 1.0, eps: float = 1e-6, dtype=None, next_w=None,
         heads: bool = False, out=None, stream=None):
    """x + scale * silu(z) * w * y / sqrt(mean(y^2) + eps) per row of y [..., d]
    (float32 or bfloat16); w [d] float32; gate z and residual x may be None.
    heads=True: y is [B,H,T,d], normalised per head, and z, x and out are
    [B,T,H*d]; otherwise they are shaped as y.  They have one type: dtype, or
    x's, z's or y's.  With next_w [d] (not with heads=True) returns (out, next):
    the next block's norm of the same rows.  out = a tensor (or that pair)
    writes into caller tensors; it may be x."""
    import torch

    sizes, shape = _norm_sizes(y, heads)
    B, H, T, d = sizes
    if next_w is not None and heads:
        raise ValueError("next_w needs whole rows (heads=False)")
    if dtype is None:
        dtype = next((t.dtype for t in (x, z) if t is not None), y.dtype)
    ty, to = _value_dtype(y.dtype), _value_dtype(dtype)
    behind = None
    if out is None:
        empty = _empty_on(stream, y.device)
        out = empty(shape, dtype)
        behind = empty(shape, dtype) if next_w is not None else None
    elif next_w is not None:
        out, behind = out
    like = [None if t is None else _arg(t, dtype, shape, n) for n, t in (("z", z), ("x", x))]
    py, pw, pz, px, po, pnw, pn = _gpu(
        _arg(y, y.dtype, tuple(y.shape), "y"), _arg(w, torch.float32, (d,), "w"), *like,
        _arg(out, dtype, shape, "out"),
        None if next_w is None else _arg(next_w, torch.float32, (d,), "next_w"),
        None if next_w is None else _arg(behind, dtype, shape, "next"))
    _call(lib().sdm_norm, y, stream, py, ty, pw, pz, px, scale, eps, B, H, T, d, po, to, pnw, pn)
    return out if next_w is None else (out, behind)


def norm_backward(dout, y, w, z=None, scale: float = 1.0, eps: float = 1e-6, skip=None,
                  heads: bool = False, workspace=None, out=None, stream=None):
    """Gradients of norm(): a dict dy (like y), dw [d] float32 and, with a gate,
    dz (like z); the residual's is dout itself.  skip (like y) is a gradient
    that reaches y past the norm, added to dy.  dout and z have one type.
    out = such a dict writes into caller tensors."""
    import torch

    sizes, shape = _norm_sizes(y, heads)
    B, H, T, d = sizes
    ty, to = _value_dtype(y.dtype), _value_dtype(dout.dtype)
    at = tuple(y.shape)
    ins = [_arg(dout, dout.dtype, shape, "dout"), _arg(y, y.dtype, at, "y"),
           _arg(w, torch.float32, (d,), "w"),
           None if z is None else _arg(z, dout.dtype, shape, "z"),
           None if skip is None else _arg(skip, y.dtype, at, "skip")]
    empty = _empty_on(stream, y.device)
    shapes = {"dy": (y.dtype, at), "dw": (torch.float32, (d,))}
    if z is not None:
        shapes["dz"] = (dout.dtype, shape)
    if out is None:
        out = {n: empty(s, t) for n, (t, s) in shapes.items()}
    outs = [_arg(out[n], t, s, n) for n, (t, s) in shapes.items()]
    if z is None:
        outs.append(None)
    ws, nbytes = _workspace(
        workspace, int(lib().sdm_norm_backward_workspace_size(B, H, T, d)), empty)
    po, py, pw, pz, pskip, *outs = _gpu(*ins, *outs, ws)
    _call(lib().sdm_norm_backward, y, stream, po, to, py, ty, pw, pz, pskip, scale, eps, B, H, T,
          d, *outs, nbytes)
    return out
