"""What the Python binding itself does for the paged-cache entry points, with
the library replaced by one that accepts every call: no GPU is needed."""
import contextlib
import types

import pytest
import torch

import quantized_attention_smoothing_b200 as sage


class _Accepts:
    """A library whose entry points all return SAGE_OK and keep their arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("_workspace") else sage.SAGE_OK
        return entry


@pytest.fixture
def lib(monkeypatch):
    L = _Accepts()
    monkeypatch.setattr(sage, "lib", lambda: L)
    return L


HANDLE = types.SimpleNamespace(handle=None, device=-1, head_dim=128)      # (CPU tensors: device -1)


def attend_args(B=2, T=1, H=8, Hk=2, D=128, page=16, mx=False):
    Dc = D // 2 if mx else D
    cache = [torch.zeros((9, Hk, page, Dc), dtype=torch.uint8) for _ in range(2)]
    scale = [torch.zeros((9, Hk, page, D // 32), dtype=torch.uint8) if mx else torch.zeros((9, Hk, page)) for _ in range(2)]
    q = torch.zeros((B, T, H, D), dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)
    return dict(q=q, k_cache=cache[0], v_cache=cache[1], scales=scale, prefix=i32(3), length=i32(1), table=i32(B, 5),
                ctx=i32(B), page=page, pages=9, out=torch.zeros_like(q))


def attend(name, a, **kw):
    if "shared" in name:
        getattr(sage, name)(HANDLE, a["q"], a["k_cache"], a["v_cache"], *a["scales"], a["prefix"], a["length"], a["table"],
                            a["ctx"], a["page"], a["pages"], 1000, 0.1, a["out"], **kw)
    else:
        getattr(sage, name)(HANDLE, a["q"], a["k_cache"], a["v_cache"], *a["scales"], a["table"], a["ctx"], a["page"],
                            a["pages"], 1000, 0.1, a["out"], **kw)


ATTEND = ["sage_attn_decode", "sage_attn_decode_mxfp4", "sage_attn_decode_shared", "sage_attn_decode_shared_mxfp4"]


@pytest.mark.parametrize("name", ATTEND)
@pytest.mark.parametrize("stream", ["current", "other", "raw"])
def test_own_workspace_belongs_to_the_calls_stream(lib, monkeypatch, name, stream):
    """A workspace that the binding makes is released when the call returns;
    only memory of the stream that the kernels run on is then reused behind them."""
    made, current = [], ["the current stream"]
    empty = torch.empty

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()

    def recorded(*args, **kw):
        made.append(current[-1])
        return empty(*args, **kw)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda p, device=None: "stream %d" % p)
    monkeypatch.setattr(sage, "_stream", lambda s: 0)
    a = attend_args(mx="mxfp4" in name)
    other = types.SimpleNamespace(cuda_stream=77)
    monkeypatch.setattr(torch, "empty", recorded)
    attend(name, a, stream={"current": None, "other": other, "raw": 99}[stream])
    assert made == [{"current": "the current stream", "other": other, "raw": "stream 99"}[stream]]
    made.clear()
    attend(name, a, ws=torch.zeros(4096, dtype=torch.uint8), stream=other)
    assert not made                                       # a caller's workspace is used as it is
