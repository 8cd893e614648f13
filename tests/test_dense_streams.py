"""The dense recurrence's and the norms' calls on a stream given by the caller,
as tests/test_binding_streams.py has it for the others."""
import pytest
import torch

import sparse_memory_linear_sdm_amd as sdm

f32 = torch.float32


def _calls(device):
    """name -> (call with only a stream left out, tensors it makes, workspaces
    among them)."""
    def z(*shape):
        return torch.zeros(shape, dtype=f32, device=device)

    B, H, Hk, T, d = 1, 2, 1, 600, 32  # few memories, many steps: segments
    S, q, v, g = z(B, H, d, d), z(B, Hk, T, d) + 1, z(B, H, T, d) + 1, z(B, H, T) - 1
    tape, y, w = z(B, H, 19, d, d), z(7, 64) + 1, z(64) + 1
    one = [x[:, :, 0].contiguous() for x in (q, q, v, g)]
    return {
        "linear_scan": (lambda s: sdm.linear_scan(S, q, q, v, g, stream=s), 2, 1),
        "linear_scan_train": (lambda s: sdm.linear_scan_train(S, q, q, v, g, stream=s), 3, 1),
        "linear_backward": (lambda s: sdm.linear_backward(q, q, v, g, tape, v, S, stream=s), 5, 1),
        "linear_step": (lambda s: sdm.linear_step(S, *one, stream=s), 1, 0),
        "norm": (lambda s: sdm.norm(y, w, next_w=w, stream=s), 2, 0),
        "norm_backward": (lambda s: sdm.norm_backward(y, y, w, z=y, stream=s), 4, 1),
    }


NAMES = sorted(_calls("cpu"))


@pytest.mark.parametrize("name", NAMES)
def test_what_a_call_makes_is_its_streams(name, monkeypatch):
    call, count, dropped = _calls("cpu")[name]
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
    assert sum(mine for _, mine in made) == dropped


@pytest.mark.parametrize("name", NAMES)
def test_every_call_runs_on_its_tensors_gpu(name, monkeypatch):
    call = _calls("cpu")[name][0]
    seen = []
    monkeypatch.setattr(sdm, "_gpu", lambda *args: [None] * len(args))
    monkeypatch.setattr(sdm, "_check", lambda rc: pytest.fail("launched on whatever GPU is current"))
    monkeypatch.setattr(sdm, "_call", lambda fn, t, stream, *a: seen.append((fn.__name__, stream)))
    stream = object()
    call(stream)
    call(None)
    fn = "sdm_" + name.replace("_scan_train", "_scan")
    assert seen == [(fn, stream), (fn, None)]


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_the_memory_belongs_to_the_stream(name, monkeypatch):
    call, count, _ = _calls("cuda")[name]
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
