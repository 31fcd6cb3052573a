"""The expert-layer and gradient calls take tensors of one device and run on it, whichever device
is current.  Without a GPU: the tensors are fakes (no memory), and so is the library."""
import contextlib
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import table_embedding_bag_gb300 as tbe
from table_embedding_bag_gb300 import experts

FP8 = torch.float8_e4m3fn


class FakeLibrary:
    """Notes on which device each call is made, and its stream."""

    def __init__(self):
        self.current, self.calls = 0, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.current, args[-1]))
            return 0
        return call


class FakeStream:
    cuda_stream = 77

    def __init__(self, device_index):
        self.device_index = device_index


@pytest.fixture
def lib(monkeypatch):
    fake = FakeLibrary()

    @contextlib.contextmanager
    def on_device(device):
        before, fake.current = fake.current, device
        yield
        fake.current = before

    monkeypatch.setattr(experts, "_lib_", fake)
    monkeypatch.setattr(experts, "_current_device", lambda: fake.current)
    monkeypatch.setattr(experts, "_on_device", on_device)
    monkeypatch.setattr(experts, "_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(experts, "_empty", lambda stream, shape, dtype, like: torch.empty(
        shape, dtype=dtype, device=like.device))
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")  # a fake tensor's address
        yield fake


def make(device, swap=None):
    """Every tensor of the calls below on `device`, but the one called `swap` on the other."""
    shapes = dict(ids=((6, 2), torch.int32), offsets=(4, torch.int32), source=(12, torch.int32),
                  position=((6, 2), torch.int32), x=((6, 32), torch.float32),
                  rows=((12, 32), torch.float32), weights=((6, 2), torch.float32),
                  q=((12, 32), FP8), scale=((12, 1), torch.float32), w=((3, 16, 32), torch.float32),
                  w8=((3, 16, 32), FP8), w_scale=((3, 1, 1), torch.float32),
                  out=((12, 16), torch.bfloat16), status=(1, torch.int32),
                  norm=((), torch.float32), ws=(16384, torch.uint8))
    return {k: torch.empty(shape, dtype=dtype, device=f"cuda:{1 - device if k == swap else device}")
            for k, (shape, dtype) in shapes.items()}


# each call, and the tensors it is given
CALLS = {
    "sort": (lambda t, s=None: tbe.tbe_expert_sort(
        t["ids"], 3, t["offsets"], t["source"], t["position"], stream=s),
        "ids offsets source position"),
    "dispatch": (lambda t, s=None: tbe.tbe_expert_dispatch(
        t["x"], t["offsets"], t["position"], t["rows"], stream=s), "x offsets position rows"),
    "dispatch_fp8": (lambda t, s=None: tbe.tbe_expert_dispatch_fp8(
        t["x"], t["offsets"], t["position"], t["q"], t["scale"], stream=s),
        "x offsets position q scale"),
    "quantize_rows": (lambda t, s=None: tbe.tbe_quantize_rows(
        t["rows"], t["q"], t["scale"], stream=s), "rows q scale"),
    "quantize_weights": (lambda t, s=None: tbe.tbe_quantize_weights(
        t["w"], t["w8"], t["w_scale"], stream=s), "w w8 w_scale"),
    "combine": (lambda t, s=None: tbe.tbe_expert_combine(
        t["rows"], t["position"], t["weights"], t["x"], stream=s), "rows position weights x"),
    "dispatch_backward": (lambda t, s=None: tbe.tbe_expert_dispatch_backward(
        t["rows"], t["position"], t["x"], stream=s), "rows position x"),
    "combine_backward": (lambda t, s=None: tbe.tbe_expert_combine_backward(
        t["x"], t["rows"], t["offsets"], t["position"], t["weights"], stream=s),
        "x rows offsets position weights"),
    "product": (lambda t, s=None: tbe.tbe_expert_product(
        t["q"], t["scale"], t["w8"], t["w_scale"], t["offsets"], t["out"], status=t["status"],
        stream=s), "q scale w8 w_scale offsets out status"),
    "norm": (lambda t, s=None: tbe.tbe_grad_norm(
        [t["x"], t["rows"]], t["norm"], t["ws"], stream=s), "x rows norm ws"),
    "clip": (lambda t, s=None: tbe.tbe_grad_clip(
        [t["x"], t["rows"]], 1.0, [t["x"], t["rows"]], t["norm"], t["ws"], stream=s),
        "x rows norm ws"),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("device", [0, 1])
def test_the_tensors_device_is_current_during_the_call(lib, name, device):
    call, _ = CALLS[name]
    call(make(device))
    assert [c[1:] for c in lib.calls] == [(device, 1000 + device)]
    assert lib.current == 0
    call(make(device), FakeStream(device))
    assert lib.calls[-1][1:] == (device, 77)


@pytest.mark.parametrize("name,swap", [(n, t) for n, (_, ts) in CALLS.items() for t in ts.split()])
def test_a_tensor_of_another_device_is_refused(lib, name, swap):
    call, _ = CALLS[name]
    for device in (0, 1):
        with pytest.raises(ValueError, match="device"):
            call(make(device, swap))
    assert not lib.calls


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(lib, name):
    call, _ = CALLS[name]
    with pytest.raises(ValueError, match="stream"):
        call(make(0), FakeStream(1))
    assert not lib.calls


def test_clipped_gradients_on_another_device_are_refused(lib):
    a, b = make(0), make(1)
    with pytest.raises(ValueError, match="device"):
        tbe.tbe_grad_clip([a["x"], b["x"]], 1.0)  # two devices in one list
    with pytest.raises(ValueError, match="device"):
        tbe.tbe_grad_clip([a["x"]], 1.0, out=[b["x"]])
    assert not lib.calls
