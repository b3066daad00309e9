"""The serving operators' Python calls on the host: stand-ins for device tensors, streams and the
library show what is recorded and which device is current, without a GPU."""
import contextlib

import pytest
import torch


class FakeTensor:
    """A CPU tensor that says it lies on device `dev` and keeps the streams it was recorded on."""

    def __init__(self, t, dev):
        self.t, self.dev, self.recorded = t, dev, []
        self.is_cuda, self.dtype, self.shape = True, t.dtype, t.shape
        self.device = torch.device("cuda", dev)

    def get_device(self):
        return self.dev

    def record_stream(self, stream):
        self.recorded.append(stream)

    def __getattr__(self, name):
        return getattr(self.t, name)


class FakeStream:
    cuda_stream = 77


class FakeLib:
    """Every function answers 0 and notes its name and the device that was current."""

    def __init__(self, cuda):
        self.cuda, self.calls = cuda, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.cuda["current"], args))
            if name.endswith("_scratch_bytes"):
                args[-1]._obj.value = 1000 + self.cuda["current"]
            return 0
        return call


@pytest.fixture
def world(monkeypatch):
    from looped_transformer_self_b200 import binding as B
    cuda = {"current": 0, "dev": 0}

    @contextlib.contextmanager
    def device(d):
        before = cuda["current"]
        cuda["current"] = d if isinstance(d, int) else d.index
        yield
        cuda["current"] = before

    lib = FakeLib(cuda)
    monkeypatch.setattr(B, "lib", lambda: lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: cuda["current"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 5, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    empty = torch.empty
    monkeypatch.setattr(B.torch, "empty", lambda shape, dtype, device: FakeTensor(empty(shape, dtype=dtype),
                                                                                 device.index))
    return B, lib, cuda


NAMES = ["prompt", "prompt_given", "prefix", "prefix_given", "verify"]


def _make(B, dev, name):
    """The call's tensors and the call, which takes a stream."""
    def f(*shape, dtype=torch.bfloat16):
        return FakeTensor(torch.zeros(*shape, dtype=dtype), dev)

    def i(n):
        return f(n, dtype=torch.int32)

    def r(*shape):
        return f(*shape, dtype=torch.float32)
    if name == "verify":
        t = dict(p=r(5, 50), q=r(3, 50), drafts=i(3), off=i(3), u_accept=r(3), u_draw=r(2), status=i(1))
        return list(t.values()), lambda s: B.verify_drafts(**t, stream=s)
    if name.startswith("prompt"):
        fn, t = B.attn_prompt, dict(q=f(6, 4, 32), k=f(9, 2, 32), v=f(9, 2, 32), q_off=i(3), kv_off=i(3), status=i(1))
    else:
        fn, t = B.attn_prefix, dict(q=f(6, 4, 32), cache=f(20, 2, 64), row_off=i(3), prefix=i(8), prefix_off=i(3),
                                    tail=i(9), tail_off=i(7), status=i(1))
    if name.endswith("given"):
        t.update(out=f(6, 4, 32), scratch=f(4000, dtype=torch.uint8))
    return list(t.values()), lambda s: fn(**t, stream=s)


@pytest.mark.parametrize("name", NAMES)
def test_tensors_are_recorded_on_a_given_stream(world, name):
    """Memory freed by the caller behind the call must not be given out again while it is read."""
    B, lib, _ = world
    tensors, call = _make(B, 0, name)
    stream = FakeStream()
    call(stream)
    assert [t.recorded for t in tensors] == [[stream]] * len(tensors)
    assert lib.calls[-1][2][-1] == FakeStream.cuda_stream


@pytest.mark.parametrize("name", NAMES)
def test_current_stream_needs_no_record(world, name):
    B, lib, _ = world
    tensors, call = _make(B, 0, name)
    call(None)
    assert all(not t.recorded for t in tensors)
    assert lib.calls[-1][2][-1] == 5


@pytest.mark.parametrize("name", ["prompt", "prefix"])
@pytest.mark.parametrize("stream", [None, FakeStream()])
def test_scratch_is_sized_for_the_tensors_device(world, name, stream):
    """The bytes depend on the device's processors: they are asked for with the tensors' device current,
    as the launch is made, and the current device is left as it was."""
    B, lib, cuda = world
    _, call = _make(B, 1, name)
    call(stream)
    assert [(n, d) for n, d, _ in lib.calls] == [(f"lt_attn_{name}_scratch_bytes", 1), (f"lt_attn_{name}", 1)]
    assert lib.calls[-1][2][-3] == 1001 and cuda["current"] == 0
