"""Query rows so small that 448 divided by their largest rotated element is not
a finite fp32: the quotient is the largest finite number instead, in the oracle
and in the decode kernels, and an element of zero has the code of zero."""
import numpy as np
import pytest
import torch

import oracle
import quantized_attention_smoothing_b200 as sage
import serving_helpers as sh
import workloads


def small_rows(q):
    rows = q.view(-1, q.shape[-1])
    rows[::2] = 0
    rows[::2, :2] = 2.0 ** -126                          # rotated: 2^-125 and 0, alternating
    rows[2, :2] = 2.0 ** -133                            # (bf16's own subnormal numbers)
    return q


def test_oracle_codes_of_small_rows():
    q = small_rows(torch.ones((1, 2, 4, 128), dtype=torch.bfloat16))
    codes, scales = oracle.decode_quant_q(workloads.bits_u16(q))
    x = oracle.e4m3_decode(codes).reshape(-1, 128)
    assert np.isfinite(x).all() and (x[::2, 1::2] == 0).all() and (x[::2, ::2] > 0).all()
    # 2^-125 times 2^128, and 2^-132 times it, rounded to e4m3
    assert (x[0, ::2] == 8.0).all() and (x[2, ::2] == 2.0 ** -4).all()
    assert (x[1, 1:] == 0).all() and x[1, 0] == 448


@pytest.mark.gpu
@pytest.mark.parametrize("D,fmt", [(128, "token"), (64, "tensor"), (128, "mxfp4")])
def test_decode_of_small_rows(D, fmt):
    """Codes and scales as the oracle's, and outputs that are the mean of the
    values (the logits are below 2^-100) within the bf16 weights and output."""
    h, page = sage.Hadamard(D), 64
    d = sh.make_shared(3, 2, 8, 2, D, page, 0, [400, 130, 2], seed=4, fmt=fmt)
    small_rows(d["q"])
    t = {n: d[n].cuda() for n in ("q", "kc", "vc", "ks", "vs", "ctx")}
    table = torch.where(d["table"] > 1 << 20, 0, d["table"]).cuda()
    out = torch.empty_like(t["q"])
    q8 = torch.empty(t["q"].shape, dtype=torch.uint8, device="cuda")
    qs = torch.empty(t["q"].shape[:3], dtype=torch.float32, device="cuda")
    a = [h, t["q"], t["kc"], t["vc"], t["ks"], t["vs"], table, t["ctx"], page, d["pages"], 9999, D ** -0.5, out]
    if fmt == "mxfp4":
        sage.sage_attn_decode_mxfp4(*a, q8_out=q8, q_scale_out=qs)
    else:
        sage.sage_attn_decode(*a, q8_out=q8, q_scale_out=qs, kv_flags=1 if fmt == "tensor" else 0)
    assert sage.sage_device_error() == sage.SAGE_OK
    codes, scales = oracle.decode_quant_q(workloads.bits_u16(d["q"]))
    assert np.array_equal(q8.cpu().numpy(), codes) and np.array_equal(qs.cpu().numpy(), scales)
    ref, tol = sh.ref_shared(d, 9999, D ** -0.5)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all()
