"""The expert-layer and gradient-norm entry points without a GPU: the library
exports what include/tbe_experts.h and include/tbe_grads.h declare, and bad
arguments are refused before anything is launched."""
import ctypes
import os
import re

import pytest
import torch

import table_embedding_bag_gb300 as tbe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x1000  # never dereferenced by the host-side checks
F16, I32, I64, BF16, F32 = 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    tbe.build()
    return tbe.configure(ctypes.CDLL(tbe.lib_path))


def declared(header):
    src = open(os.path.join(ROOT, "include", header)).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(tbe_[a-z0-9_]+)\s*\(", src)))


def test_declared_functions_are_exported(lib):
    names = declared("tbe_experts.h") + declared("tbe_grads.h")
    assert {"tbe_expert_sort", "tbe_expert_product", "tbe_grad_clip"} <= set(names)
    for name in names:
        assert hasattr(lib, name), name


def test_binding_constants_match_the_headers():
    src = open(os.path.join(ROOT, "include", "tbe_experts.h")).read()
    src += open(os.path.join(ROOT, "include", "tbe_grads.h")).read()
    for name in ("TBE_MAX_EXPERTS", "TBE_SCALE_BLOCK", "TBE_GRAD_WORKSPACE_BYTES"):
        value = re.search(rf"#define {name} (\d+)", src).group(1)
        assert getattr(tbe, name) == int(value)


SORT = dict(ids=FAKE, dt=I32, tokens=8, k=2, e=4, offsets=FAKE, source=FAKE, position=FAKE)
DISPATCH = dict(x=FAKE, dt=F16, tokens=8, k=2, width=32, xs=32, offsets=FAKE, e=4, position=FAKE,
                rows=FAKE, rs=32)
FP8 = dict(x=FAKE, dt=F16, tokens=8, k=2, width=32, xs=32, offsets=FAKE, e=4, position=FAKE,
           q=FAKE, qs=32, scale=FAKE)
COMBINE = dict(y=FAKE, dt=F16, tokens=8, k=2, width=32, ys=32, position=FAKE, w=FAKE, out=FAKE,
               os=32)
BACK = dict(go=FAKE, y=FAKE, dt=F16, tokens=8, k=2, width=32, gs=32, ys=32, offsets=FAKE, e=4,
            position=FAKE, w=FAKE, gy=FAKE, gys=32, gw=FAKE)
QW = dict(w=FAKE, dt=F16, e=2, n=8, k=16, q=FAKE, scale=FAKE)
PRODUCT = dict(a=FAKE, as_=32, sa=FAKE, w=FAKE, sw=FAKE, offsets=FAKE, rows=8, n=16, k=32, e=2,
               out=FAKE, dt=BF16, os=16, status=None)


@pytest.mark.parametrize("call,base,change,code", [
    ("tbe_expert_sort", SORT, dict(tokens=-1), tbe.TBE_EINVAL),
    ("tbe_expert_sort", SORT, dict(k=0), tbe.TBE_EINVAL),
    ("tbe_expert_sort", SORT, dict(e=0), tbe.TBE_EINVAL),
    ("tbe_expert_sort", SORT, dict(ids=None), tbe.TBE_EINVAL),
    ("tbe_expert_sort", SORT, dict(offsets=None), tbe.TBE_EINVAL),
    ("tbe_expert_sort", SORT, dict(position=FAKE + 2), tbe.TBE_EINVAL),
    ("tbe_expert_sort", SORT, dict(ids=FAKE + 4, dt=I64), tbe.TBE_EINVAL),
    ("tbe_expert_sort", SORT, dict(dt=F32), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_sort", SORT, dict(e=1025), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_sort", SORT, dict(tokens=1 << 30, k=2), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_dispatch", DISPATCH, dict(tokens=-1), tbe.TBE_EINVAL),
    ("tbe_expert_dispatch", DISPATCH, dict(xs=31), tbe.TBE_EINVAL),
    ("tbe_expert_dispatch", DISPATCH, dict(rs=31), tbe.TBE_EINVAL),
    ("tbe_expert_dispatch", DISPATCH, dict(x=FAKE + 1), tbe.TBE_EINVAL),
    ("tbe_expert_dispatch", DISPATCH, dict(position=None), tbe.TBE_EINVAL),
    ("tbe_expert_dispatch", DISPATCH, dict(dt=I32), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_dispatch", DISPATCH, dict(tokens=1 << 31, k=1), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_dispatch_fp8", FP8, dict(qs=31), tbe.TBE_EINVAL),
    ("tbe_expert_dispatch_fp8", FP8, dict(scale=None), tbe.TBE_EINVAL),
    ("tbe_expert_dispatch_fp8", FP8, dict(position=None), tbe.TBE_EINVAL),  # k is not 1
    ("tbe_expert_dispatch_fp8", FP8, dict(dt=9), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_combine", COMBINE, dict(k=0), tbe.TBE_EINVAL),
    ("tbe_expert_combine", COMBINE, dict(w=FAKE + 2), tbe.TBE_EINVAL),
    ("tbe_expert_combine", COMBINE, dict(out=None), tbe.TBE_EINVAL),
    ("tbe_expert_combine", COMBINE, dict(dt=0), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_combine_backward", BACK, dict(go=None), tbe.TBE_EINVAL),
    ("tbe_expert_combine_backward", BACK, dict(gys=8), tbe.TBE_EINVAL),
    ("tbe_expert_combine_backward", BACK, dict(y=None), tbe.TBE_EINVAL),
    ("tbe_quantize_weights", QW, dict(e=-1), tbe.TBE_EINVAL),
    ("tbe_quantize_weights", QW, dict(w=None), tbe.TBE_EINVAL),
    ("tbe_quantize_weights", QW, dict(dt=3), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_product", PRODUCT, dict(rows=-1), tbe.TBE_EINVAL),
    ("tbe_expert_product", PRODUCT, dict(k=0), tbe.TBE_EINVAL),
    ("tbe_expert_product", PRODUCT, dict(offsets=None), tbe.TBE_EINVAL),  # two experts
    ("tbe_expert_product", PRODUCT, dict(os=15), tbe.TBE_EINVAL),
    ("tbe_expert_product", PRODUCT, dict(as_=16), tbe.TBE_EINVAL),
    ("tbe_expert_product", PRODUCT, dict(k=24), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_product", PRODUCT, dict(as_=40), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_product", PRODUCT, dict(a=FAKE + 8), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_product", PRODUCT, dict(w=FAKE + 8), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_product", PRODUCT, dict(dt=2), tbe.TBE_EUNSUPPORTED),
    ("tbe_expert_product", PRODUCT, dict(e=2000), tbe.TBE_EUNSUPPORTED),
])
def test_bad_arguments_refused_before_any_launch(lib, call, base, change, code):
    before = lib.tbe_kernel_launches()
    args = dict(base, **change)
    assert getattr(lib, call)(*args.values(), None) == code
    assert lib.tbe_kernel_launches() == before


def test_empty_problems_launch_nothing(lib):
    before = lib.tbe_kernel_launches()
    for call, base, change in [
            ("tbe_expert_dispatch", DISPATCH, dict(tokens=0)),
            ("tbe_expert_dispatch", DISPATCH, dict(width=0)),
            ("tbe_expert_dispatch_fp8", FP8, dict(tokens=0)),
            ("tbe_expert_combine", COMBINE, dict(tokens=0)),
            ("tbe_expert_combine_backward", BACK, dict(tokens=0)),
            ("tbe_quantize_weights", QW, dict(e=0)),
            ("tbe_expert_product", PRODUCT, dict(rows=0)),
            ("tbe_expert_product", PRODUCT, dict(n=0))]:
        assert getattr(lib, call)(*dict(base, **change).values(), None) == tbe.TBE_OK
    assert lib.tbe_kernel_launches() == before


@pytest.mark.parametrize("entry,kw,code", [
    (dict(), dict(count=-1), tbe.TBE_EINVAL),
    (dict(), dict(norm=None), tbe.TBE_EINVAL),
    (dict(), dict(norm=FAKE + 1), tbe.TBE_EINVAL),
    (dict(), dict(max_norm=-1.0), tbe.TBE_EINVAL),
    (dict(), dict(max_norm=float("nan")), tbe.TBE_EINVAL),
    (dict(numel=-1), dict(), tbe.TBE_EINVAL),
    (dict(grad=None), dict(), tbe.TBE_EINVAL),
    (dict(grad=FAKE + 2), dict(), tbe.TBE_EINVAL),
    (dict(out=None), dict(), tbe.TBE_EINVAL),
    (dict(dtype=2), dict(), tbe.TBE_EUNSUPPORTED),
    (dict(numel=(1 << 40) + 1), dict(), tbe.TBE_EUNSUPPORTED),
    (dict(), dict(ws=None), tbe.TBE_EWORKSPACE),
    (dict(), dict(ws=FAKE + 8), tbe.TBE_EWORKSPACE),
    (dict(), dict(ws_bytes=100), tbe.TBE_EWORKSPACE),
])
def test_bad_gradient_lists_refused(lib, entry, kw, code):
    from table_embedding_bag_gb300.grads import tbe_grad_tensor
    e = dict(dict(grad=FAKE, out=FAKE, numel=10, dtype=F32, reserved=0), **entry)
    a = dict(dict(count=1, max_norm=1.0, norm=FAKE, ws=FAKE, ws_bytes=1 << 14), **kw)
    table = (tbe_grad_tensor * 1)(tuple(e.values()))
    before = lib.tbe_kernel_launches()
    assert lib.tbe_grad_clip(table, a["count"], a["max_norm"], a["norm"], a["ws"], a["ws_bytes"],
                             None) == code
    if "max_norm" not in kw and "out" not in entry:
        assert lib.tbe_grad_norm(table, a["count"], a["norm"], a["ws"], a["ws_bytes"],
                                 None) == code
    assert lib.tbe_kernel_launches() == before


def test_binding_refuses_what_the_kernels_cannot_read():
    ids = torch.zeros(4, 2, dtype=torch.int32)
    x = torch.zeros(4, 16)
    off, pos = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.int32)
    q, w8 = torch.zeros(4, 16).to(torch.float8_e4m3fn), torch.zeros(2, 8, 16).to(torch.float8_e4m3fn)
    for error, call in [
            (TypeError, lambda: tbe.tbe_expert_sort(ids.float(), 4)),
            (ValueError, lambda: tbe.tbe_expert_sort(ids.view(-1), 4)),
            (ValueError, lambda: tbe.tbe_expert_sort(ids, 4)),           # not on the GPU
            (ValueError, lambda: tbe.tbe_expert_dispatch(x, off, pos)),
            (ValueError, lambda: tbe.tbe_expert_combine(x, pos)),
            (TypeError, lambda: tbe.tbe_quantize_rows(x.double())),
            (ValueError, lambda: tbe.tbe_quantize_rows(x)),
            (ValueError, lambda: tbe.tbe_quantize_weights(x)),
            (TypeError, lambda: tbe.tbe_expert_product(x, None, w8, None)),
            (ValueError, lambda: tbe.tbe_expert_product(q, None, w8, None)),
            (ValueError, lambda: tbe.tbe_grad_norm([])),
            (ValueError, lambda: tbe.tbe_grad_clip([], 1.0)),
            (ValueError, lambda: tbe.tbe_grad_norm([x])),
            (TypeError, lambda: tbe.tbe_grad_norm([ids])),
            (ValueError, lambda: tbe.tbe_grad_clip([x], 1.0, out=[]))]:
        with pytest.raises(error):
            call()
