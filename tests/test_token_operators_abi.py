"""Token embedding, norm and routing without a GPU: the library exports what the
headers declare, bad arguments and shared memory are refused before anything is launched, and
the binding's calls run on their tensors' device."""
import contextlib
import ctypes
import os
import re
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import table_embedding_bag_gb300 as tbe
from table_embedding_bag_gb300 import experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F16, I32, I64, BF16, F32 = 1, 2, 3, 4, 5
A, B, C, D, E, W = (i << 28 for i in range(1, 7))  # never dereferenced by the host-side checks
BIG = 1 << 27


@pytest.fixture(scope="module")
def lib():
    tbe.build()
    return tbe.configure(ctypes.CDLL(tbe.lib_path))


def source(header):
    return open(os.path.join(ROOT, "include", header)).read()


@pytest.mark.parametrize("header", ["tbe_embed.h", "tbe_norm.h", "tbe_experts.h"])
def test_declared_functions_are_exported_and_bound(lib, header):
    src = re.sub(r"/\*.*?\*/", "", source(header), flags=re.S)
    names = sorted(set(re.findall(r"\b(tbe_[a-z0-9_]+)\s*\(", src)))
    assert names
    for name in names:
        assert hasattr(lib, name), name
        assert getattr(lib, name).argtypes is not None, name


def test_binding_constants_match_the_headers():
    for header, name in (("tbe_norm.h", "TBE_MAX_NORM_WIDTH"), ("tbe_experts.h", "TBE_MAX_CHOSEN")):
        assert getattr(tbe, name) == int(re.search(rf"#define {name} (\d+)", source(header)).group(1))
    enum = dict(re.findall(r"TBE_SCORE_(\w+) = (\d+)", source("tbe_experts.h")))
    assert {k.upper(): str(v) for k, v in experts._SCORE.items()} == enum


EMBED = dict(table=A, dt=F16, rows=100, width=32, ts=32, ids=B, it=I32, tokens=8, scale=1.0, out=C,
             os=32)
BACK = dict(grad=A, dt=BF16, tokens=2000, width=32, gs=32, ids=B, it=I64, rows=100, scale=1.0, acc=0,
            out=C, ot=BF16, os=32, ws=W, n=BIG)
NORM = dict(x=A, res=B, w=C, dt=F16, wt=F32, rows=8, width=256, xs=256, rs=256, eps=1e-6, h=D,
            hs=256, y=E, ys=256)
NORM8 = dict(x=A, res=B, w=C, dt=F16, wt=F16, rows=8, width=256, xs=256, rs=256, eps=1e-6, h=D,
             hs=256, q=E, qs=256, scale=W)
NBACK = dict(gy=A, h=B, w=C, gh=D, dt=F32, wt=F32, rows=8, width=256, gys=256, hs=256, ghs=256,
             eps=1e-6, gx=E, gxs=256, gw=W, ws=W + BIG, n=BIG)
ROUTE = dict(l=A, dt=F32, tokens=8, e=64, ls=64, bias=B, score=1, k=4, groups=8, top=4, best=2,
             renorm=1, scale=1.0, ids=C, it=I32, w=D)
RBACK = dict(gw=A, l=B, dt=BF16, tokens=8, e=64, ls=64, ids=C, it=I64, k=4, score=2, renorm=1,
             scale=1.0, out=D, os=64)
NAN, INF = float("nan"), float("inf")

REFUSED = [
    ("tbe_embed", EMBED, tbe.TBE_EINVAL, [
        dict(rows=-1), dict(width=-1), dict(tokens=-1), dict(ts=31), dict(os=31), dict(table=None),
        dict(ids=None), dict(out=None), dict(table=A + 1), dict(ids=B + 2), dict(ids=B + 4, it=I64),
        dict(scale=NAN), dict(scale=INF), dict(out=A), dict(out=A + 64 * 99), dict(out=B),
        dict(ids=C + 64), dict(ts=1 << 60)]),
    ("tbe_embed", EMBED, tbe.TBE_EUNSUPPORTED, [
        dict(dt=0), dict(dt=I32), dict(it=F32), dict(rows=(1 << 31) - 1), dict(tokens=1 << 31),
        dict(width=(1 << 20) + 1)]),
    ("tbe_embed_backward", BACK, tbe.TBE_EINVAL, [
        dict(tokens=-1), dict(rows=-1), dict(width=-1), dict(gs=31), dict(os=31), dict(grad=None),
        dict(ids=None), dict(out=None), dict(grad=A + 1), dict(ids=B + 4), dict(out=C + 1),
        dict(scale=NAN), dict(out=A), dict(out=B), dict(ws=C), dict(ws=C - 16), dict(ws=A),
        dict(ids=W + 64), dict(out=W + 1024)]),
    ("tbe_embed_backward", BACK, tbe.TBE_EUNSUPPORTED, [
        dict(dt=9), dict(ot=F16), dict(it=BF16), dict(tokens=1 << 31), dict(rows=1 << 31),
        dict(width=1 << 21)]),
    ("tbe_embed_backward", BACK, tbe.TBE_EWORKSPACE, [
        dict(ws=None), dict(ws=W + 8), dict(n=100)]),
    ("tbe_rms_norm", NORM, tbe.TBE_EINVAL, [
        dict(rows=-1), dict(width=0), dict(x=None), dict(y=None), dict(xs=255), dict(rs=255),
        dict(hs=255), dict(ys=255), dict(x=A + 1), dict(res=B + 1), dict(h=D + 1), dict(y=E + 1),
        dict(w=C + 2), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(res=None),  # h without one
        dict(h=A), dict(h=B), dict(y=A), dict(y=B), dict(y=D), dict(y=C), dict(h=C - 512)]),
    ("tbe_rms_norm", NORM, tbe.TBE_EUNSUPPORTED, [
        dict(dt=0), dict(wt=BF16), dict(rows=1 << 31), dict(width=16385)]),
    ("tbe_rms_norm_fp8", NORM8, tbe.TBE_EINVAL, [
        dict(q=None), dict(scale=None), dict(scale=W + 2), dict(qs=255), dict(q=A), dict(q=D),
        dict(scale=E), dict(scale=A), dict(scale=D + 8)]),
    ("tbe_rms_norm_backward", NBACK, tbe.TBE_EINVAL, [
        dict(gy=None), dict(h=None), dict(gx=None), dict(rows=-1), dict(width=0), dict(gys=255),
        dict(hs=255), dict(ghs=255), dict(gxs=255), dict(gx=E + 2), dict(gw=W + 2), dict(eps=NAN),
        dict(gx=A), dict(gx=B), dict(gx=D), dict(gx=C), dict(gw=C), dict(gw=E), dict(gw=A),
        dict(ws=E), dict(ws=A), dict(ws=W)]),
    ("tbe_rms_norm_backward", NBACK, tbe.TBE_EUNSUPPORTED, [
        dict(dt=3), dict(wt=F16), dict(width=1 << 20)]),
    ("tbe_rms_norm_backward", NBACK, tbe.TBE_EWORKSPACE, [
        dict(ws=None), dict(ws=W + BIG + 8), dict(n=8 * 256 * 4 - 1)]),
    ("tbe_expert_route", ROUTE, tbe.TBE_EINVAL, [
        dict(tokens=-1), dict(e=0), dict(k=0), dict(l=None), dict(ids=None), dict(w=None),
        dict(ls=63), dict(l=A + 2), dict(bias=B + 2), dict(ids=C + 2), dict(ids=C + 4, it=I64),
        dict(w=D + 1), dict(score=0), dict(score=3), dict(groups=0), dict(groups=7), dict(top=0),
        dict(top=9), dict(best=0), dict(best=3), dict(top=1, k=9), dict(scale=NAN), dict(ids=A),
        dict(w=A), dict(w=B), dict(ids=B), dict(w=C)]),
    ("tbe_expert_route", ROUTE, tbe.TBE_EUNSUPPORTED, [
        dict(dt=0), dict(it=F32), dict(e=1025), dict(k=32), dict(tokens=1 << 30),
        dict(groups=64, top=64)]),
    ("tbe_expert_route_backward", RBACK, tbe.TBE_EINVAL, [
        dict(tokens=-1), dict(gw=None), dict(l=None), dict(ids=None), dict(out=None), dict(ls=63),
        dict(os=63), dict(gw=A + 2), dict(ids=C + 4), dict(out=D + 1), dict(score=9),
        dict(scale=INF), dict(out=A), dict(out=B), dict(out=C)]),
    ("tbe_expert_route_backward", RBACK, tbe.TBE_EUNSUPPORTED, [
        dict(dt=2), dict(it=1), dict(e=1025), dict(k=32)]),
]


@pytest.mark.parametrize("call,base,code,change", [
    (call, base, code, change) for call, base, code, changes in REFUSED for change in changes])
def test_bad_arguments_refused_before_any_launch(lib, call, base, code, change):
    before = lib.tbe_kernel_launches()
    assert getattr(lib, call)(*dict(base, **change).values(), None) == code
    assert lib.tbe_kernel_launches() == before


def test_empty_problems_launch_nothing(lib):
    before = lib.tbe_kernel_launches()
    for call, base, change in [
            ("tbe_embed", EMBED, dict(tokens=0)), ("tbe_embed", EMBED, dict(width=0)),
            ("tbe_embed_backward", BACK, dict(rows=0)), ("tbe_embed_backward", BACK, dict(width=0)),
            ("tbe_embed_backward", BACK, dict(tokens=0, acc=1, ws=None, n=0)),
            ("tbe_rms_norm", NORM, dict(rows=0)), ("tbe_rms_norm_fp8", NORM8, dict(rows=0)),
            ("tbe_rms_norm_backward", NBACK, dict(rows=0, gw=None, ws=None, n=0)),
            ("tbe_expert_route", ROUTE, dict(tokens=0)),
            ("tbe_expert_route_backward", RBACK, dict(tokens=0))]:
        assert getattr(lib, call)(*dict(base, **change).values(), None) == tbe.TBE_OK
    assert lib.tbe_kernel_launches() == before


def test_workspace_sizes(lib):
    assert tbe.tbe_embed_workspace_size(0, 10, 16) == 0
    assert tbe.tbe_embed_workspace_size(100, 1000, 4096) == 0
    for n in (2000, 98304, 98305, 1 << 24, (1 << 31) - 2000):
        # the sorted tokens twice, and two parts for each piece of 8 to 64 of them
        pieces = min(n // 8 + 1, max(4864, n // 64 + 1))
        got = tbe.tbe_embed_workspace_size(n, 1000, 4096)
        assert 16 * n < got <= 16 * n + 4096 + (5 << 20) + pieces * 2 * 4096 * 4
    assert tbe.tbe_rms_norm_workspace_size(0, 128) == 0
    assert tbe.tbe_rms_norm_workspace_size(10, 1000) == 40_000
    assert tbe.tbe_rms_norm_workspace_size(1 << 30, 16384) <= 128 << 20
    for call, sizes in ((tbe.tbe_embed_workspace_size, (-1, 1, 1)),
                        (tbe.tbe_embed_workspace_size, (1, 1, 1 << 30)),
                        (tbe.tbe_rms_norm_workspace_size, (1, 0)),
                        (tbe.tbe_rms_norm_workspace_size, (1, 16385))):
        with pytest.raises(tbe.TBEError):
            call(*sizes)


def test_binding_refuses_what_the_kernels_cannot_read():
    x, ids = torch.zeros(4, 16), torch.zeros(4, dtype=torch.int64)
    for error, call in [
            (ValueError, lambda: tbe.tbe_embed(x, ids)),                  # not on the GPU
            (TypeError, lambda: tbe.tbe_embed(x.double(), ids)),
            (ValueError, lambda: tbe.tbe_embed_backward(x, ids, 10)),
            (ValueError, lambda: tbe.tbe_rms_norm(x)),
            (ValueError, lambda: tbe.tbe_rms_norm(x.view(-1))),
            (TypeError, lambda: tbe.tbe_rms_norm_fp8(x.int())),
            (ValueError, lambda: tbe.tbe_rms_norm_backward(x, x)),
            (ValueError, lambda: tbe.tbe_expert_route(x, 2)),
            (ValueError, lambda: tbe.tbe_expert_route_backward(x[:, :2], x, ids.view(4, 1)))]:
        with pytest.raises(error):
            call()


# ------------------------------------------------------------ devices and shapes, on fakes

class FakeLibrary:
    """Notes on which device each call is made, and its stream."""

    def __init__(self):
        self.current, self.calls = 0, []

    def __getattr__(self, name):
        def call(*args):
            if not name.endswith("workspace_size"):
                self.calls.append((name, self.current, args[-1]))
            return 0
        return call


class FakeStream:
    cuda_stream = 77

    def __init__(self, device_index):
        self.device_index = device_index


@pytest.fixture
def fake(monkeypatch):
    lib = FakeLibrary()

    @contextlib.contextmanager
    def on_device(device):
        before, lib.current = lib.current, device
        yield
        lib.current = before

    monkeypatch.setattr(experts, "_lib_", lib)
    monkeypatch.setattr(experts, "_sizes", {})
    monkeypatch.setattr(experts, "_current_device", lambda: lib.current)
    monkeypatch.setattr(experts, "_on_device", on_device)
    monkeypatch.setattr(experts, "_raw_stream", lambda device: 1000 + device)
    empty = lambda stream, shape, dtype, like: torch.empty(shape, dtype=dtype, device=like.device)
    for module in (experts, tbe._embed, tbe._norm):
        monkeypatch.setattr(module, "_empty", empty)
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")  # a fake tensor's address
        yield lib


def make(device, swap=None):
    shapes = dict(table=((20, 32), torch.float32), ids=(6, torch.int64), x=((6, 32), torch.float32),
                  y=((6, 32), torch.float32), z=((6, 32), torch.float32),
                  out=((6, 32), torch.float32), grad=((20, 32), torch.float32),
                  weight=(32, torch.float32), gw=(32, torch.float32), ws=(1 << 20, torch.uint8),
                  q=((6, 32), torch.float8_e4m3fn), scale=((6, 1), torch.float32),
                  bias=(32, torch.float32), chosen=((6, 2), torch.int32),
                  cw=((6, 2), torch.float32))
    return {k: torch.empty(shape, dtype=dtype, device=f"cuda:{1 - device if k == swap else device}")
            for k, (shape, dtype) in shapes.items()}


CALLS = {
    "embed": (lambda t, s=None: tbe.tbe_embed(t["table"], t["ids"], 1.0, t["out"], stream=s),
              "table ids out"),
    "embed_backward": (lambda t, s=None: tbe.tbe_embed_backward(
        t["x"], t["ids"], 20, out=t["grad"], ws=t["ws"], stream=s), "x ids grad ws"),
    "rms_norm": (lambda t, s=None: tbe.tbe_rms_norm(
        t["x"], t["weight"], t["y"], out=t["out"], h=t["z"], stream=s), "x weight y out z"),
    "rms_norm_fp8": (lambda t, s=None: tbe.tbe_rms_norm_fp8(
        t["x"], t["weight"], t["y"], out=t["q"], scale=t["scale"], h=t["z"], stream=s),
        "x weight y q scale z"),
    "rms_norm_backward": (lambda t, s=None: tbe.tbe_rms_norm_backward(
        t["x"], t["y"], t["weight"], t["z"], grad_x=t["out"], grad_weight=t["gw"], ws=t["ws"],
        stream=s), "x y weight z out gw ws"),
    "route": (lambda t, s=None: tbe.tbe_expert_route(
        t["x"], 2, bias=t["bias"], ids=t["chosen"], weights=t["cw"], stream=s), "x bias chosen cw"),
    "route_backward": (lambda t, s=None: tbe.tbe_expert_route_backward(
        t["cw"], t["x"], t["chosen"], out=t["out"], stream=s), "cw x chosen out"),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("device", [0, 1])
def test_the_tensors_device_is_current_during_the_call(fake, name, device):
    call, _ = CALLS[name]
    call(make(device))
    assert [c[1:] for c in fake.calls] == [(device, 1000 + device)]
    assert fake.current == 0
    call(make(device), FakeStream(device))
    assert fake.calls[-1][1:] == (device, 77)


@pytest.mark.parametrize("name,swap", [(n, t) for n, (_, ts) in CALLS.items() for t in ts.split()])
def test_a_tensor_of_another_device_is_refused(fake, name, swap):
    call, _ = CALLS[name]
    for device in (0, 1):
        with pytest.raises(ValueError, match="device"):
            call(make(device, swap))
    assert not fake.calls


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(fake, name):
    call, _ = CALLS[name]
    with pytest.raises(ValueError, match="stream"):
        call(make(0), FakeStream(1))
    assert not fake.calls


@pytest.mark.parametrize("error,call", [
    (TypeError, lambda t: tbe.tbe_embed(t["table"], t["x"])),
    (ValueError, lambda t: tbe.tbe_embed(t["table"], torch.empty(6, 2, dtype=torch.int64,
                                                                 device="cuda:0")[:, 0])),
    (ValueError, lambda t: tbe.tbe_embed(t["table"], t["ids"], out=t["table"])),
    (ValueError, lambda t: tbe.tbe_embed(t["table"].T, t["ids"])),
    (ValueError, lambda t: tbe.tbe_embed_backward(t["x"][:5], t["ids"], 20)),
    (ValueError, lambda t: tbe.tbe_embed_backward(t["x"], t["ids"], -1)),
    (ValueError, lambda t: tbe.tbe_embed_backward(t["x"], t["ids"], 20, accumulate=True)),
    (ValueError, lambda t: tbe.tbe_embed_backward(t["x"], t["ids"], 21, out=t["grad"])),
    (TypeError, lambda t: tbe.tbe_embed_backward(t["x"], t["ids"], 20, out_dtype=torch.float16)),
    (TypeError, lambda t: tbe.tbe_embed_backward(t["x"], t["ids"], 20, out=t["grad"],
                                                 out_dtype=torch.float16)),
    (ValueError, lambda t: tbe.tbe_embed_backward(t["x"], t["ids"], 20, ws=t["x"])),
    (ValueError, lambda t: tbe.tbe_rms_norm(t["x"], h=t["z"])),
    (ValueError, lambda t: tbe.tbe_rms_norm(t["x"], t["weight"][:31])),
    (TypeError, lambda t: tbe.tbe_rms_norm(t["x"], t["weight"].half())),
    (TypeError, lambda t: tbe.tbe_rms_norm(t["x"], residual=t["y"].half())),
    (ValueError, lambda t: tbe.tbe_rms_norm(t["x"], residual=t["y"][:5])),
    (TypeError, lambda t: tbe.tbe_rms_norm_fp8(t["x"], out=t["y"])),
    (ValueError, lambda t: tbe.tbe_rms_norm_fp8(t["x"], scale=t["cw"])),
    (ValueError, lambda t: tbe.tbe_rms_norm_backward(t["x"], t["table"])),
    (ValueError, lambda t: tbe.tbe_rms_norm_backward(t["x"], t["y"], grad_weight=t["gw"],
                                                     need_weight=False)),
    (TypeError, lambda t: tbe.tbe_rms_norm_backward(t["x"], t["y"], grad_weight=t["gw"].half())),
    (ValueError, lambda t: tbe.tbe_expert_route(t["x"], 0)),
    (ValueError, lambda t: tbe.tbe_expert_route(t["x"], 32)),
    (ValueError, lambda t: tbe.tbe_expert_route(t["x"], 2, groups=5)),
    (ValueError, lambda t: tbe.tbe_expert_route(t["x"], 9, groups=4, top_groups=1)),
    (ValueError, lambda t: tbe.tbe_expert_route(t["x"], 2, groups=4, top_groups=5)),
    (ValueError, lambda t: tbe.tbe_expert_route(t["x"], 2, group_best=3)),
    (ValueError, lambda t: tbe.tbe_expert_route(t["x"], 2, score="tanh")),
    (TypeError, lambda t: tbe.tbe_expert_route(t["x"], 2, bias=t["bias"].half())),
    (ValueError, lambda t: tbe.tbe_expert_route(t["x"], 3, ids=t["chosen"])),
    (TypeError, lambda t: tbe.tbe_expert_route(t["x"], 2, ids=t["cw"])),
    (ValueError, lambda t: tbe.tbe_expert_route_backward(t["cw"], t["x"], t["chosen"][:, :1])),
    (TypeError, lambda t: tbe.tbe_expert_route_backward(t["cw"], t["x"], t["cw"])),
    (TypeError, lambda t: tbe.tbe_expert_route_backward(t["cw"].half(), t["x"], t["chosen"])),
])
def test_the_binding_refuses_wrong_types_and_shapes(fake, error, call):
    with pytest.raises(error):
        call(make(0))
    assert not fake.calls


def test_outputs_that_are_not_given(fake):
    t = make(0)
    assert tbe.tbe_embed(t["table"], t["ids"].view(2, 3)).shape == (2, 3, 32)
    assert tbe.tbe_embed_backward(t["x"].view(2, 3, 32), t["ids"].view(2, 3), 20).shape == (20, 32)
    assert tbe.tbe_rms_norm(t["x"]).shape == (6, 32)
    y, h = tbe.tbe_rms_norm(t["x"], residual=t["y"])
    assert y.shape == h.shape == (6, 32)
    q, scale, h = tbe.tbe_rms_norm_fp8(t["x"], residual=t["y"])
    assert q.dtype == torch.float8_e4m3fn and scale.shape == (6, 1) and h.shape == (6, 32)
    gx, gw = tbe.tbe_rms_norm_backward(t["x"], t["y"])
    assert gx.shape == (6, 32) and gw.shape == (32,) and gw.dtype == torch.float32
    assert tbe.tbe_rms_norm_backward(t["x"], t["y"], need_weight=False)[1] is None
    ids, w = tbe.tbe_expert_route(t["x"], 5)
    assert ids.shape == w.shape == (6, 5) and ids.dtype == torch.int32
    assert tbe.tbe_expert_route_backward(w, t["x"], ids).shape == (6, 32)
