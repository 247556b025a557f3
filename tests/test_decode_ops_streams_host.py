"""A call on a stream of its own makes everything that it makes there (host, with stand-ins for tensors and streams)."""
import contextlib
import types

import pytest
import torch

import combine_ep_get_dispatch_gb300 as ep


class Fake:
    """What the page-level calls ask of a tensor, and the streams it was made on and is recorded for."""

    def __init__(self, shape, dtype, on=None):
        self.shape, self.dtype, self.device, self.on, self.recorded = torch.Size(shape), dtype, "device", on, []

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def record_stream(self, stream):
        self.recorded.append(stream)


@pytest.fixture
def world(monkeypatch):
    """current: the innermost stream; made: tensors made by the calls; launched: (call, stream) pairs."""
    w = types.SimpleNamespace(current="caller", made=[], launched=[])

    @contextlib.contextmanager
    def stream(s):
        outer, w.current = w.current, s
        try:
            yield
        finally:
            w.current = outer

    def make(*shape, dtype=None, device=None):
        shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
        w.made.append(Fake(shape, dtype, w.current))
        return w.made[-1]

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw: ("external", raw))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.current)
    monkeypatch.setattr(ep, "torch", types.SimpleNamespace(
        cuda=torch.cuda, Tensor=torch.Tensor, Size=torch.Size, zeros=make, empty=make, bfloat16=torch.bfloat16,
        float32=torch.float32, int32=torch.int32, uint8=torch.uint8))
    for name in ("ep_kv_append", "ep_kv_attention", "ep_expert_linear"):
        takes_stream = {"ep_kv_append": 10, "ep_kv_attention": 10, "ep_expert_linear": 14}[name]

        def launch(*args, name=name, at=takes_stream):
            given = args[at] if len(args) > at else None
            w.launched.append((name, w.current if given is None else given))
        monkeypatch.setattr(ep, name, launch)
    monkeypatch.setattr(ep, "ep_kv_attention_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(ep, "ep_expert_linear_workspace_bytes", lambda *a: 4096)
    w.side = Stream()
    return w


def append(stream):
    q, kv = Fake((3, 8, 64), torch.bfloat16), Fake((3, 2, 64), torch.bfloat16)
    return [ep.kv_append(kv, kv, object(), object(), q=q, stream=stream)]


def attend(stream):
    cache = types.SimpleNamespace(k=Fake((5, 2, 16, 64), torch.uint8))
    return list(ep.kv_attention(Fake((3, 8, 64), torch.bfloat16), cache, object(), return_lse=True, stream=stream))


def experts(stream):
    x = Fake((4, 6, 256), torch.bfloat16)
    return [ep.expert_linear(x, Fake((4, 64, 128), torch.uint8), Fake((4, 64, 8), torch.uint8), Fake((4,), torch.int32),
                             stream=stream)]


CALLS = pytest.mark.parametrize("call,makes", [(append, 1), (attend, 3), (experts, 2)])


@CALLS
def test_on_a_stream_of_its_own(world, call, makes):
    results = call(world.side)
    assert len(world.made) == makes and all(t.on is world.side for t in world.made)
    assert [s for _, s in world.launched] == [world.side] and world.current == "caller"
    # results are the caller's to use, a workspace is not
    assert all(t.recorded == ["caller"] for t in results)
    assert all(t.recorded == [] for t in world.made if not any(t is r for r in results))


@CALLS
@pytest.mark.parametrize("raw", [77, types.SimpleNamespace(cuda_stream=77)])
def test_on_a_raw_handle(world, call, makes, raw):
    call(raw)
    assert len(world.made) == makes and all(t.on == ("external", 77) for t in world.made)
    assert [s for _, s in world.launched] == [("external", 77)]


@CALLS
def test_on_the_current_stream(world, call, makes):
    results = call(None)
    assert len(world.made) == makes and all(t.on == "caller" and not t.recorded for t in world.made)
    assert [s for _, s in world.launched] == ["caller"] and len(results) >= 1
    world.current = world.side
    assert all(t.on is world.side and not t.recorded for t in call(world.side))
