"""Refusals of the paged-cache serving entry points, on the host: bad
arguments are answered before anything touches a device, so no GPU is needed.
A handle needs a device to be built; these calls take a block of host memory
laid out like one (head size, device)."""
import ctypes

import pytest

import quantized_attention_smoothing_b200 as sage
from quantized_attention_smoothing_b200 import build as sage_build

P = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module")
def L():
    sage_build.build()
    return sage.lib()


class _Handle(ctypes.Structure):
    _fields_ = [("D", ctypes.c_int), ("device", ctypes.c_int), ("host", ctypes.c_void_p)]


def handle(D=128):
    return ctypes.byref(_Handle(D, 0, None))


def view(cls, size, ptr=0x20000, stride=None):
    v = cls()
    v.ptr = ptr
    s = stride or (size[1] * size[2] * size[3], size[2] * size[3], size[3], 1)
    for i in range(4):
        v.size[i], v.stride[i] = size[i], s[i]
    return v


def ptr(a):
    return ctypes.c_void_p(a)


PLAN = dict(cached=ptr(0x1000), new=ptr(0x2000), prefix=ptr(0x3000), pp=2, free=ptr(0x4000), count=ptr(0x5000), B=4,
            max_pages=8, page=64, num_pages=100, max_tokens=32, table=ptr(0x6000), ctx=ptr(0x7000),
            count_out=ptr(0x8000), offsets=ptr(0x9000), slots=ptr(0xa000))


@pytest.mark.parametrize("change,status", [
    (dict(cached=None), "INVALID_ARG"), (dict(new=None), "INVALID_ARG"), (dict(free=None), "INVALID_ARG"),
    (dict(count=None), "INVALID_ARG"), (dict(table=None), "INVALID_ARG"), (dict(ctx=None), "INVALID_ARG"),
    (dict(count_out=None), "INVALID_ARG"), (dict(offsets=None), "INVALID_ARG"), (dict(slots=None), "INVALID_ARG"),
    (dict(prefix=None), "INVALID_ARG"), (dict(pp=-1), "INVALID_ARG"), (dict(pp=9), "INVALID_ARG"),
    (dict(B=0), "INVALID_ARG"), (dict(max_pages=0), "INVALID_ARG"), (dict(num_pages=0), "INVALID_ARG"),
    (dict(max_tokens=-1), "INVALID_ARG"), (dict(page=0), "INVALID_ARG"), (dict(page=48), "UNSUPPORTED"),
    (dict(page=256), "UNSUPPORTED"), (dict(B=8193), "UNSUPPORTED"), (dict(max_pages=1 << 25, pp=0), "UNSUPPORTED"),
    (dict(num_pages=1 << 25), "UNSUPPORTED"), (dict(ctx=ptr(0x2000)), "INVALID_ARG"),
    (dict(offsets=ptr(0x1000)), "INVALID_ARG"), (dict(slots=ptr(0xa002)), "ALIGNMENT"),
    (dict(table=ptr(0x6001)), "ALIGNMENT"),
])
def test_plan_refuses(L, change, status):
    a = {**PLAN, **change}
    st = L.sage_page_plan(a["cached"], a["new"], a["prefix"], a["pp"], a["free"], a["count"], a["B"], a["max_pages"],
                          a["page"], a["num_pages"], a["max_tokens"], a["table"], a["ctx"], a["count_out"],
                          a["offsets"], a["slots"], None)
    assert sage.status_string(st) == "SAGE_ERR_" + status


APPEND = dict(h=128, k=(1, 5, 2, 128), v=(1, 5, 2, 128), kp=0x20000, mean=ptr(0x100), slots=P, kc=P, vc=P, ks=P, vs=P,
              page=64, pages=10, flags=0)


@pytest.mark.parametrize("change,status", [
    (dict(h=None), "INVALID_ARG"), (dict(kp=0), "INVALID_ARG"), (dict(slots=None), "INVALID_ARG"),
    (dict(kc=None), "INVALID_ARG"), (dict(vc=None), "INVALID_ARG"), (dict(ks=None), "INVALID_ARG"),
    (dict(vs=None), "INVALID_ARG"), (dict(v=(1, 4, 2, 128)), "INVALID_ARG"), (dict(h=64), "INVALID_ARG"),
    (dict(k=(2, 5, 2, 128), v=(2, 5, 2, 128)), "INVALID_ARG"), (dict(pages=0), "INVALID_ARG"),
    (dict(page=0), "INVALID_ARG"), (dict(page=24), "UNSUPPORTED"), (dict(flags=4), "INVALID_ARG"),
    (dict(flags=2), "UNSUPPORTED"), (dict(pages=1 << 26), "UNSUPPORTED"),
    (dict(k=(1, 1 << 30, 2, 128), v=(1, 1 << 30, 2, 128)), "UNSUPPORTED"), (dict(kc=ptr(0x1008)), "ALIGNMENT"),
    (dict(mean=ptr(0x104)), "ALIGNMENT"), (dict(slots=ptr(0x1002)), "ALIGNMENT"), (dict(ks=ptr(0x1001)), "ALIGNMENT"),
])
def test_append_refuses(L, change, status):
    a = {**APPEND, **change}
    h = handle(a["h"]) if a["h"] else None
    st = L.sage_kv_append(h, view(sage.CView4, a["k"], a["kp"]), view(sage.CView4, a["v"]), a["mean"], a["slots"],
                          a["kc"], a["vc"], a["ks"], a["vs"], a["page"], a["pages"], a["flags"], None)
    assert sage.status_string(st) == "SAGE_ERR_" + status


def test_append_mxfp4_refuses(L):
    k = view(sage.CView4, (1, 5, 2, 128))
    k64 = view(sage.CView4, (1, 5, 2, 64))

    def call(h, k, ksf, vsf):
        return sage.status_string(L.sage_kv_append_mxfp4(h, k, k, None, P, P, P, ksf, vsf, 64, 10, None))
    assert call(None, k, P, P) == "SAGE_ERR_INVALID_ARG"
    assert call(handle(), k, None, P) == "SAGE_ERR_INVALID_ARG"
    assert call(handle(64), k64, P, P) == "SAGE_ERR_UNSUPPORTED"
    assert call(handle(), k, ptr(0x1008), P) == "SAGE_ERR_ALIGNMENT"


SHARED = dict(h=128, q=(2, 4, 16, 128), out=(2, 4, 16, 128), kc=P, vc=P, ks=P, vs=P, prefix=P, pages_p=8, length=P,
              table=P, ctx=P, B=2, T=4, H=16, Hk=1, D=128, page=128, mp=16, pages=100, window=4096, scale=0.1, flags=0,
              ws=P, wsb=1 << 30)


def call_shared(L, a, mx=False):
    h = handle(a["h"]) if a["h"] else None
    args = [h, view(sage.CView4, a["q"]), a["kc"], a["vc"], a["ks"], a["vs"], a["prefix"], a["pages_p"], a["length"],
            a["table"], a["ctx"], a["B"], a["T"], a["H"], a["Hk"], a["D"], a["page"], a["mp"], a["pages"],
            a["window"], a["scale"]] + ([] if mx else [a["flags"]]) + \
           [view(sage.View4, a["out"]), a["ws"], a["wsb"], None]
    return sage.status_string((L.sage_attn_decode_shared_mxfp4 if mx else L.sage_attn_decode_shared)(*args))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("change,status", [
    (dict(h=None), "INVALID_ARG"), (dict(kc=None), "INVALID_ARG"), (dict(vs=None), "INVALID_ARG"),
    (dict(table=None), "INVALID_ARG"), (dict(ctx=None), "INVALID_ARG"), (dict(B=3), "INVALID_ARG"),
    (dict(out=(2, 4, 16, 64)), "INVALID_ARG"), (dict(window=0), "INVALID_ARG"), (dict(scale=float("nan")), "INVALID_ARG"),
    (dict(h=64), "INVALID_ARG"), (dict(Hk=3), "UNSUPPORTED"), (dict(page=48), "UNSUPPORTED"),
    (dict(ws=None), "WORKSPACE"), (dict(wsb=64), "WORKSPACE"), (dict(ws=ptr(0x10008)), "ALIGNMENT"),
])
def test_shared_refuses(L, change, status, mx):
    assert call_shared(L, {**SHARED, **change}, mx) == "SAGE_ERR_" + status


def test_shared_flags_refused(L):
    assert call_shared(L, {**SHARED, "flags": 8}) == "SAGE_ERR_INVALID_ARG"


def test_shared_workspace_is_host_only(L):
    assert L.sage_attn_decode_shared_workspace(0, 1, 16, 1, 128) == 0
    assert L.sage_attn_decode_shared_workspace(2, 1, 16, 3, 128) == 0
    assert L.sage_attn_decode_shared_workspace(2, 1, 16, 1, 128) > 0
