"""GPU tests of sage_attn_decode_shared with logits far from zero, where the
16-bit weights depend on which maximum they are held against, at the bound of
the roundings that each cache format has."""
import math

import numpy as np
import pytest
import torch

import quantized_attention_smoothing_b200 as sage
import serving_bounds as sb
import serving_helpers as sh
from gpu_helpers import workloads_f32, bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handles():
    from quantized_attention_smoothing_b200 import build
    build.build()
    return {64: sage.Hadamard(64), 128: sage.Hadamard(128)}


def run(h, d, page, window, scale):
    t = {n: d[n].cuda() for n in ("q", "kc", "vc", "ks", "vs", "prefix", "length", "table", "ctx")}
    out = torch.full(d["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    a = [h, t["q"], t["kc"], t["vc"], t["ks"], t["vs"], t["prefix"], t["length"], t["table"], t["ctx"], page,
         d["pages"], window, scale, out]
    if d["fmt"] == "mxfp4":
        sage.sage_attn_decode_shared_mxfp4(*a)
    else:
        sage.sage_attn_decode_shared(*a, kv_flags=(1 if d["fmt"].startswith("tensor") else 0) |
                                     (2 if d["fmt"].endswith("vt") else 0))
    assert sage.sage_device_error() == sage.SAGE_OK
    return out


def worst_error(out, d, window, scale):
    ref, tol, mean = sb.bound_shared(d, window, scale)
    g = workloads_f32(bits(out.contiguous())).astype(np.float64)
    assert np.isfinite(g).all()
    return np.max(np.abs(g - ref) / tol), mean


# who attends: prefix CTAs of 256 and of 128 rows, 17 to 64 rows behind a long
# prefix, own keys of sequences of many rows, and the kernel for few rows
PATHS = {
    "rows256": dict(B=10, T=1, H=16, Hk=1, prefix=1000, ctx=[1000 + 21 * i for i in range(10)]),
    "rows96": dict(B=6, T=2, H=8, Hk=1, prefix=900, ctx=[902, 1500, 903, 0, 700, 940]),
    "few rows, long prefix": dict(B=1, T=4, H=128, Hk=8, prefix=8100, ctx=[8140]),
    "own keys": dict(B=16, T=4, H=16, Hk=1, prefix=200, ctx=[204 + 113 * i for i in range(16)]),
    "few rows": dict(B=2, T=1, H=16, Hk=2, prefix=500, ctx=[700, 501]),
}


@pytest.mark.parametrize("offset", [-10, -14, -20, -30, -45, -70, 40])
@pytest.mark.parametrize("fmt,D", [("token", 128), ("tensor", 64), ("token_vt", 64), ("tensor_vt", 128), ("mxfp4", 128)])
@pytest.mark.parametrize("path", list(PATHS))
def test_shared_logits_far_from_zero(handles, path, fmt, D, offset):
    p = PATHS[path]
    d = sb.offset_logits(p["B"], p["T"], p["H"], p["Hk"], D, 128 if fmt.endswith("vt") else 64, p["prefix"], p["ctx"],
                         seed=3, fmt=fmt, offset=offset)
    page, scale = 128 if fmt.endswith("vt") else 64, 1.0 / math.sqrt(D)
    worst, mean = worst_error(run(handles[D], d, page, 10 ** 6, scale), d, 10 ** 6, scale)
    print("mean logit %.1f, worst error %.3f of the bound" % (mean, worst))
    assert abs(mean - offset) < 0.15 * abs(offset) + 1 and worst <= 1.0


@pytest.mark.parametrize("path,window", [("rows256", 700), ("rows96", 333), ("own keys", 500)])
def test_shared_window_leaves_the_high_logits_out(handles, path, window):
    """The first tokens take most of the weight until a window leaves them
    behind; the other logits lie 30 below."""
    p, D = PATHS[path], 128
    d = sb.offset_logits(p["B"], p["T"], p["H"], p["Hk"], D, 64, p["prefix"], p["ctx"], seed=5, fmt="token", offset=-25,
                         spread=2.0)
    d["kc"][d["prefix"][0], :, :4] ^= 0x80                  # the first keys turned round: logits of about +25
    scale = 1.0 / math.sqrt(D)
    for w in (window, 10 ** 6):
        worst, _ = worst_error(run(handles[D], d, 64, w, scale), d, w, scale)
        print("window %d: worst error %.3f of the bound" % (w, worst))
        assert worst <= 1.0


@pytest.mark.parametrize("spread", [1.0, 4.0])
@pytest.mark.parametrize("fmt,D", [("token", 64), ("token", 128), ("tensor", 128), ("token_vt", 128), ("tensor_vt", 64),
                                   ("mxfp4", 128)])
@pytest.mark.parametrize("path", list(PATHS))
def test_shared_within_the_roundings_of_its_format(handles, path, fmt, D, spread):
    """Three fp16 roundings over an FP8 cache, not the bf16 one that
    serving_helpers.ref_shared allows every format."""
    p, page = PATHS[path], 128
    d = sb.offset_logits(p["B"], p["T"], p["H"], p["Hk"], D, page, p["prefix"], p["ctx"], seed=11, fmt=fmt, offset=0.0,
                         spread=spread)
    scale = 1.0 / math.sqrt(D)
    worst, _ = worst_error(run(handles[D], d, page, 10 ** 6, scale), d, 10 ** 6, scale)
    print("worst error %.3f of the bound" % worst)
    assert worst <= 1.0


@pytest.mark.parametrize("fmt", ["token", "mxfp4"])
@pytest.mark.parametrize("path", ["few rows", "rows96", "rows256"])
def test_shared_queries_near_the_smallest_number(handles, path, fmt):
    """Query rows whose largest rotated element is so small that 448 divided by
    it is not a finite fp32, with elements of zero beside it: logits of zero,
    the mean of the values that the row sees."""
    p, D, page = PATHS[path], 128, 64
    d = sh.make_shared(p["B"], p["T"], p["H"], p["Hk"], D, page, p["prefix"], p["ctx"], seed=2, fmt=fmt)
    rows = d["q"].view(-1, D)
    rows[::3] = 0
    rows[::3, :2] = 2.0 ** -126                          # rotated: 2^-125 and 0, alternating
    rows[3, :2] = 2.0 ** -133                            # (bf16's own subnormal numbers)
    out = run(handles[D], d, page, 10 ** 6, D ** -0.5)
    d["q"].view(-1, D)[::3] = 0
    assert worst_error(out, d, 10 ** 6, D ** -0.5)[0] <= 1.0
