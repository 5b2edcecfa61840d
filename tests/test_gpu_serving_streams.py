"""GPU tests of the decode entry points on another stream than the current one,
with the workspace that the binding makes."""
import pytest
import torch

import quantized_attention_smoothing_b200 as sage
import serving_helpers as sh

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handle():
    from quantized_attention_smoothing_b200 import build
    build.build()
    return sage.Hadamard(128)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("fmt", ["token", "mxfp4"])
def test_own_workspace_on_a_side_stream(handle, fmt, shared, raw):
    """While the call waits on its stream, the current stream takes as much
    memory as the workspace has: it stays what the current stream wrote, and
    the call's result is the one of a workspace of the caller's."""
    B, T, H, Hk, page, ctx = 4, 2, 16, 1, 64, [900, 600, 777, 1000]
    d = sh.make_shared(B, T, H, Hk, 128, page, 512 if shared else 0, ctx, seed=6, fmt=fmt)
    t = {n: d[n].cuda() for n in ("q", "kc", "vc", "ks", "vs", "prefix", "length", "ctx")}
    t["table"] = torch.where(d["table"] > 1 << 20, 0, d["table"]).cuda()
    name = "sage_attn_decode" + ("_shared" if shared else "") + ("_mxfp4" if fmt == "mxfp4" else "")
    n = sage.sage_attn_decode_shared_workspace(B, T, H, Hk, 128) if shared else \
        sage.sage_attn_decode_workspace(B, T, H, Hk, 128, 9999)
    assert n > 0

    def call(out, ws, stream):
        between = (t["prefix"], t["length"]) if shared else ()
        getattr(sage, name)(handle, t["q"], t["kc"], t["vc"], t["ks"], t["vs"], *between, t["table"], t["ctx"], page,
                            d["pages"], 9999, 0.09, out, ws=ws, stream=stream)
    want, out = torch.empty_like(t["q"]), torch.zeros_like(t["q"])
    call(want, torch.empty((n,), dtype=torch.uint8, device="cuda"), None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)                     # some 25 ms
    call(out, None, side.cuda_stream if raw else side)
    mine = [torch.zeros((n,), dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert not any(x.any() for x in mine)
    assert torch.equal(out, want) and sage.sage_device_error(side) == sage.SAGE_OK


def test_own_workspace_in_a_captured_call(handle):
    """Captured without a workspace of the caller's: the graph keeps its own."""
    d = sh.make_shared(5, 1, 16, 1, 128, 64, 500, [700, 600, 510, 0, 900], seed=8)
    t = {n: d[n].cuda() for n in ("q", "kc", "vc", "ks", "vs", "prefix", "length", "ctx", "table")}

    def call(out, stream=None):
        sage.sage_attn_decode_shared(handle, t["q"], t["kc"], t["vc"], t["ks"], t["vs"], t["prefix"], t["length"],
                                     t["table"], t["ctx"], 64, d["pages"], 9999, 0.09, out, stream=stream)
    want, outs = torch.empty_like(t["q"]), [torch.empty_like(t["q"]) for _ in range(2)]
    call(want)
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        for o in outs:
            call(o, s)
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        junk = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        del junk
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want)
