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
            if name == "sage_status_string":
                return b"refused"
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


# ---- tensors that do not hold what the call's sizes say

def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


@pytest.fixture
def on_cpu(lib, monkeypatch):
    """The calls take CPU tensors (device -1) and the null stream."""
    monkeypatch.setattr(sage, "_stream", lambda s: 0)
    monkeypatch.setattr(sage, "_device", lambda: -1, raising=False)
    return lib


class Elsewhere(torch.Tensor):
    """A tensor of device 1, by its own word."""
    __torch_function__ = torch._C._disabled_torch_function_impl

    def get_device(self):
        return 1


def wrong(t, how):
    """A tensor like t that a call of t's sizes must not take."""
    if how == "type":
        return t.to(torch.int64 if t.dtype == torch.int32 else torch.float64 if t.dtype == torch.float32 else torch.float16)
    if how == "short":
        return t.reshape(-1)[:-1] if t.dim() == 1 else t[:-1]
    if how == "strided":
        return torch.zeros(t.shape + (2,), dtype=t.dtype)[..., 0]
    if how == "expanded":
        return t.reshape(-1)[:1].expand(t.numel()).view(t.shape) if t.dim() == 1 else t[:1].expand(t.shape)
    return t.as_subclass(Elsewhere)


PLAN_ARGS = dict(cached_lens=(4,), new_lens=(4,), free_list=(30,), free_count=(1,), page_table=(4, 6), ctx_lens=(4,),
                 free_count_out=(1,), token_offsets=(5,), slot_map=(9,), prefix_table=(2,))


def plan(a):
    sage.sage_page_plan(a["cached_lens"], a["new_lens"], a["free_list"], a["free_count"], 16, a["page_table"], a["ctx_lens"],
                        a["free_count_out"], a["token_offsets"], a["slot_map"], prefix_table=a["prefix_table"])


HOW = ["type", "device", "short", "strided", "expanded"]


def cases(names, unless):
    """Every (name, how) but those that are not the binding's to refuse: a name's
    own length may be the call's, a single element has no layout, views any."""
    return [(n, how) for n in names for how in HOW if how not in unless.get(n, ())]


SHORT, LAYOUT = ("short",), ("short", "strided", "expanded")


@pytest.mark.parametrize("name,how", cases(PLAN_ARGS, dict(free_list=SHORT, slot_map=SHORT, prefix_table=SHORT,
                                                           page_table=SHORT, free_count=LAYOUT, free_count_out=LAYOUT)))
def test_plan_binding_refuses(on_cpu, name, how):
    a = {n: i32(*s) for n, s in PLAN_ARGS.items()}
    plan(a)
    n = len(on_cpu.calls)
    with pytest.raises(ValueError, match=name):
        plan({**a, name: wrong(a[name], how)})
    assert len(on_cpu.calls) == n


def test_plan_binding_leaves_out_what_it_may(on_cpu):
    a = {n: i32(*s) for n, s in PLAN_ARGS.items()}
    plan({**a, "slot_map": None, "prefix_table": None})
    plan({**a, "token_offsets": i32(6), "slot_map": i32(0)})
    with pytest.raises(sage.SageError):
        plan({**a, "new_lens": None})
    assert [c[0] for c in on_cpu.calls if "plan" in c[0]] == ["sage_page_plan"] * 2


def append_tensors(mx, tensor=False, N=5, Hk=2, D=128, page=16, pages=3):
    Dc = D // 2 if mx else D
    a = dict(k=torch.zeros((N, Hk, D), dtype=torch.bfloat16), v=torch.zeros((N, Hk, D), dtype=torch.bfloat16), slot_map=i32(N))
    a.update({n: torch.zeros((pages, Hk, page, Dc), dtype=torch.uint8) for n in ("k_cache", "v_cache")})
    a.update({n: torch.zeros((pages, Hk, page, D // 32), dtype=torch.uint8) if mx else
              torch.zeros(1) if tensor else torch.zeros((pages, Hk, page)) for n in ("k scales", "v scales")})
    return dict(a, k_mean=torch.zeros((Hk, D)))


def append(mx, a, tensor=False):
    f = sage.sage_kv_append_mxfp4 if mx else sage.sage_kv_append
    f(HANDLE, a["k"], a["v"], a["slot_map"], a["k_cache"], a["v_cache"], a["k scales"], a["v scales"], k_mean=a["k_mean"],
      **({} if mx else dict(kv_flags=1 if tensor else 0)))


@pytest.mark.parametrize("name,how", cases(["k", "v", "slot_map", "k_cache", "v_cache", "k scales", "v scales", "k_mean"],
                                           dict(k=LAYOUT, v=LAYOUT, k_cache=SHORT)))
@pytest.mark.parametrize("mx", [False, True])
def test_append_binding_refuses(on_cpu, mx, name, how):
    a = append_tensors(mx)
    append(mx, a)
    n = len(on_cpu.calls)
    with pytest.raises(ValueError, match=name):
        append(mx, {**a, name: wrong(a[name], how)})
    assert len(on_cpu.calls) == n


@pytest.mark.parametrize("mx", [False, True])
def test_append_binding_refuses_a_cache_of_other_heads(on_cpu, mx):
    a = append_tensors(mx)
    for Hk, D in ((1, 128), (3, 128), (2, 64)):
        b = append_tensors(mx, Hk=Hk, D=D)
        with pytest.raises(ValueError, match="k_cache"):
            append(mx, {**a, "k_cache": b["k_cache"], "v_cache": b["v_cache"]})
    with pytest.raises(ValueError):
        append(mx, {**a, "k": a["k"][0]})
    with pytest.raises(sage.SageError):
        append(mx, {**a, "k scales": None})
    assert not [c for c in on_cpu.calls if "append" in c[0]]


def test_append_binding_takes_what_it_may(on_cpu):
    a = append_tensors(False, tensor=True)
    append(False, {**a, "k_mean": None}, tensor=True)
    append(False, {**a, "slot_map": i32(99)}, tensor=True)
    append(False, {**a, "k_cache": a["k_cache"].view(torch.float8_e4m3fn)}, tensor=True)
    append(False, {**a, "k": a["k"][:0], "v": a["v"][:0], "slot_map": None}, tensor=True)
    b = append_tensors(True)
    append(True, {**b, "k scales": b["k scales"].view(torch.float8_e8m0fnu)})
    assert len([c for c in on_cpu.calls if "append" in c[0]]) == 5
    with pytest.raises(ValueError, match="k scales"):
        append(False, a)                                  # one scale in all, without its flag


SHARED_NAMES = {"q": "q", "out": "out", "k_cache": "k_cache", "v_cache": "v_cache", "prefix": "prefix_table",
                "length": "prefix_len", "table": "page_table", "ctx": "ctx_lens", 0: "k scales", 1: "v scales", "ws": "ws"}


@pytest.mark.parametrize("key,how", cases(SHARED_NAMES, dict(q=LAYOUT, out=LAYOUT, prefix=SHORT, length=LAYOUT,
                                                             ws=("type",) + LAYOUT)))
@pytest.mark.parametrize("mx", [False, True])
def test_shared_binding_refuses(on_cpu, mx, key, how):
    name = "sage_attn_decode_shared" + ("_mxfp4" if mx else "")
    a = dict(attend_args(mx=mx), ws=torch.zeros(4096, dtype=torch.uint8))
    attend(name, a, ws=a["ws"])
    n = len(on_cpu.calls)
    b = dict(a, scales=list(a["scales"]))
    if key in (0, 1):
        b["scales"][key] = wrong(b["scales"][key], how)
    else:
        b[key] = wrong(b[key], how)
    with pytest.raises(ValueError, match=SHARED_NAMES[key]):
        attend(name, b, ws=b["ws"])
    assert len(on_cpu.calls) == n


@pytest.mark.parametrize("mx", [False, True])
def test_shared_binding_compares_the_call_with_the_caches(on_cpu, mx):
    name = "sage_attn_decode_shared" + ("_mxfp4" if mx else "")
    a, ws = attend_args(mx=mx), torch.zeros(4096, dtype=torch.uint8)
    for change in (dict(pages=10), dict(page=32), dict(table=i32(1, 5)), dict(length=None)):
        with pytest.raises((ValueError, sage.SageError)):
            attend(name, {**a, **change}, ws=ws)
    assert not [c for c in on_cpu.calls if not c[0].endswith("workspace")]
    attend(name, {**a, "pages": 4}, ws=ws)                # fewer pages than there are
    attend(name, {**a, "scales": [torch.zeros(1), torch.zeros(1)]}, ws=ws, kv_flags=1) if not mx else None
