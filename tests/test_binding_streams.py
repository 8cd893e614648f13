"""Calls of the binding on a stream given by the caller.  What a call makes is
that stream's memory: the current stream may still be using what the allocator
would hand out for it, and may be handed the call's own workspace as soon as
the call returns."""
import pytest
import torch

import sparse_memory_linear_sdm_amd as sdm

f32, i32, i64, u8 = torch.float32, torch.int32, torch.int64, torch.uint8
B, H, N, n, d_v, T, W, R, d_model = 2, 3, 64, 8, 32, 5, 4, 3, 128
P = 4 * n + d_v + 2


def _calls(device):
    """name -> (call with only a stream left out, how many tensors it makes)."""
    def z(*shape, dtype=f32):
        return torch.zeros(shape, dtype=dtype, device=device)

    sel = dict(widx=torch.arange(W, dtype=i32, device=device).expand(B, H, T, W).contiguous(),
               wk=z(B, H, T, W) + 1 / W,
               ridx=torch.arange(R, dtype=i32, device=device).expand(B, H, T, R).contiguous(),
               rw=z(B, H, T, R) + 1 / R)
    gates = dict(v=z(B, H, T, d_v) + 1, alpha=z(B, H, T) + 1, beta=z(B, H, T) + .5)
    step = {**sel, **gates}
    M, x, dout = z(B, H, N, d_v), torch.rand(B, H, T, n, device=device), z(B, H, T, d_v) + 1
    half, vec, one = torch.rand(B, H, n, device=device), z(B, H, d_v), z(B, H)
    M0, rows = z(H, N, d_v), z(6, d_model)
    X, Wt = z(B, T, d_model, dtype=torch.bfloat16), z(H, P, d_model, dtype=torch.bfloat16)
    tape = z(B, H, T, W + R, d_v)
    tape8 = (z(B, H, 2, T, W + R, 16, dtype=torch.int8), z(B, H, 2, T, W + R, dtype=u8) + 127)
    xq, xs = z(B, T, d_model // 2, dtype=u8), z(1, B * T, 4, dtype=u8) + 127
    wq, ws = z(H, P, d_model // 2, dtype=u8), z(1, H * P, 4, dtype=u8) + 127
    plan = sdm.scan_plan(**sel, N=N, d_v=d_v) if device == "cuda" else z(256, dtype=u8)
    return {
        "project": (lambda s: sdm.project(X, Wt, n, stream=s), 7),
        "mx4_quantize": (lambda s: sdm.mx4_quantize(rows, stream=s), 2),
        "mx4_dequantize": (lambda s: sdm.mx4_dequantize(xq, xs, stream=s), 1),
        "project_mx4": (lambda s: sdm.project_mx4(xq, xs, wq, ws, n, stream=s), 7),
        "select": (lambda s: sdm.select(x, x, W, stream=s), 3),
        "state_init": (lambda s: sdm.state_init(M0, B, stream=s), 1),
        "scan": (lambda s: sdm.scan(M, **step, stream=s), 1),
        "step_decode": (lambda s: sdm.step_decode(M, half, half, half, half, vec, one, one,
                                                  W, R, stream=s), 3),
        "scan_train": (lambda s: sdm.scan_train(M, **step, stream=s), 2),
        "scan_backward": (lambda s: sdm.scan_backward(**step, tape=tape, dout=dout, G=M, stream=s), 6),
        "scan_train8": (lambda s: sdm.scan_train8(M, **step, stream=s), 3),
        "tape8_read": (lambda s: sdm.tape8_read(tape8, stream=s), 1),
        "scan_backward8": (lambda s: sdm.scan_backward8(**step, tape=tape8, dout=dout, G=M, stream=s), 6),
        "touch_prepare": (lambda s: sdm.touch_prepare(sel["widx"], sel["ridx"], N, stream=s), 2),
        "select_backward": (lambda s: sdm.select_backward(sel["widx"], sel["wk"], sel["wk"], n,
                                                          stream=s), 2),
        "state_init_backward": (lambda s: sdm.state_init_backward(M, stream=s), 1),
        "scan_plan": (lambda s: sdm.scan_plan(**sel, N=N, d_v=d_v, stream=s), 1),
        "scan_planned": (lambda s: sdm.scan_planned(M, **gates, workspace=plan, stream=s), 1),
    }


NAMES = sorted(_calls("cpu"))
DROPPED = {"scan_backward": 1, "scan_backward8": 1}  # workspaces that end with the call


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_makes_is_its_streams(name, monkeypatch):
    """Every tensor a call makes is asked for on its stream, workspaces as the
    call's own (CPU tensors: the call stops at the device check)."""
    call, count = _calls("cpu")[name]
    made = []

    def empty_on(stream, device):
        def make(shape, dtype, mine=False):
            made.append((stream, mine))
            return torch.zeros(shape, dtype=dtype)
        return make

    def refuse(*a, **k):
        raise AssertionError("made on the current stream")

    stream = object()
    monkeypatch.setattr(sdm, "_empty_on", empty_on)
    monkeypatch.setattr(torch, "empty", refuse)
    monkeypatch.setattr(torch, "empty_like", refuse)
    with pytest.raises(ValueError, match="on the GPU"):
        call(stream)
    assert [s for s, _ in made] == [stream] * count
    assert sum(mine for _, mine in made) == DROPPED.get(name, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_the_memory_belongs_to_the_stream(name, monkeypatch):
    """The same on the GPU, by the allocator's record of each tensor's segment."""
    call, count = _calls("cuda")[name]
    made = []
    inner = sdm._empty_on

    def empty_on(stream, device):
        make = inner(stream, device)

        def keep(*a, **k):
            made.append(make(*a, **k))
            return made[-1]
        return keep

    monkeypatch.setattr(sdm, "_empty_on", empty_on)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle in (side, side.cuda_stream):
        call(handle)
    side.synchronize()
    assert len(made) == 2 * count
    segments = torch.cuda.memory_snapshot()
    for t in made:
        at = t.data_ptr()
        of = [g["stream"] for g in segments if g["address"] <= at < g["address"] + g["total_size"]]
        assert of == [side.cuda_stream]


# ------------------------------------------------------- the GPU a call runs on

class _On:
    """Stands for a tensor or a stream of GPU `index`."""

    def __init__(self, index):
        self.device = torch.device("cuda", index)
        self.cuda_stream = 1000 + index

    def get_device(self):
        return self.device.index


@pytest.fixture
def two_gpus(monkeypatch):
    """GPU 0 current, of two; the current stream of GPU i has handle 10 + i."""
    now = [0]

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *_):
            now[0] = self.before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 10 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "Stream", _On)
    return now


def test_a_call_runs_on_its_tensors_gpu(two_gpus):
    seen = []

    def fn(*args):
        seen.append((two_gpus[0], *args))
        return 0

    sdm._call(fn, _On(0), None, 5)
    sdm._call(fn, _On(1), None, 6)
    sdm._call(fn, _On(1), _On(1), 7)
    sdm._call(fn, _On(1), 99, 8)
    assert seen == [(0, 5, 10), (1, 6, 11), (1, 7, 1001), (1, 8, 99)] and two_gpus[0] == 0
    with pytest.raises(ValueError, match="the stream is on cuda:0, the call's tensors on cuda:1"):
        sdm._call(fn, _On(1), _On(0), 9)
    assert len(seen) == 4 and two_gpus[0] == 0


@pytest.mark.parametrize("name", NAMES + ["scan_backward_noalloc"])
def test_every_call_runs_on_its_tensors_gpu(name, monkeypatch):
    """Each launch goes through the one place that makes the tensors' GPU current."""
    calls = _calls("cpu")
    if name in calls:
        call = calls[name][0]
    else:
        z = torch.zeros
        out = dict(dv=z(B, H, T, d_v), dwk=z(B, H, T, W), drw=z(B, H, T, R), dalpha=z(B, H, T),
                   dbeta=z(B, H, T))
        i = [z(B, H, T, K, dtype=i32) for K in (W, R)]
        call = lambda s: sdm.scan_backward_noalloc(  # noqa: E731
            i[0], out["dwk"], i[1], out["drw"], out["dv"], out["dalpha"], out["dbeta"],
            z(B, H, T, W + R, d_v), out["dv"], z(B, H, N, d_v), out, stream=s)
    seen = []

    def launched(rc):
        raise AssertionError("launched on whatever GPU is current")

    def at(fn, t, stream, *args):
        assert isinstance(t, torch.Tensor)
        seen.append((fn.__name__, stream))

    monkeypatch.setattr(sdm, "_gpu", lambda *args: [None] * len(args))
    monkeypatch.setattr(sdm, "_check", launched)
    monkeypatch.setattr(sdm, "_call", at)
    stream = object()
    call(stream)
    call(None)
    assert seen == [("sdm_" + name, stream), ("sdm_" + name, None)]


def test_a_plan_is_sized_for_its_tensors_gpu(two_gpus, monkeypatch):
    """Shards, and so the workspace, are chosen from the GPU's compute units."""
    asked = []

    def size(*args):
        asked.append((two_gpus[0], *args))
        return 0

    class On1(torch.Tensor):
        """A CPU tensor that says it is on GPU 1."""
        is_cuda = True

        def get_device(self):
            return 1

    def on1(x):
        return x.as_subclass(On1)

    monkeypatch.setattr(sdm, "scan_plan_workspace_size", size)
    monkeypatch.setattr(sdm, "_call", lambda *a: None)
    monkeypatch.setattr(sdm, "_gpu", lambda *a: [None] * len(a))
    i, w = torch.zeros(B, H, T, W, dtype=i32), torch.zeros(B, H, T, W)
    sdm.scan_plan(on1(i), on1(w), on1(i), on1(w), N, d_v)
    assert asked == [(1, B, H, d_v, T)] and two_gpus[0] == 0
