"""GPU tests of sage_page_plan at the ends of its ranges."""
import pytest
import torch

import quantized_attention_smoothing_b200 as sage

pytestmark = pytest.mark.gpu


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("count", [1, 0])
def test_plan_longest_slot_map(count):
    """2^31 - 1 slots (8.6 GB), of a step that is served and of one that is
    refused for want of a page: -1 in every slot without a token, and nothing
    written around the map."""
    from quantized_attention_smoothing_b200 import build
    build.build()
    n, pad = 2 ** 31 - 1, 1024
    buf = torch.full((n + 2 * pad,), -9, dtype=torch.int32, device="cuda")
    slots = buf[pad:pad + n]
    free, table, ctx, out, off = i32(5, 6, 7), i32(3, -4).view(1, 2), i32(-9), i32(-9), i32(-9, -9)
    sage.sage_page_plan(i32(16), i32(2), free, i32(count), 16, table, ctx, out, off, slots)
    st = sage.sage_device_error_where()[:2]
    assert (buf[:pad] == -9).all() and (buf[pad + n:] == -9).all()
    if count:
        assert st[0] == sage.SAGE_OK
        assert slots[:2].tolist() == [80, 81] and table.tolist() == [[3, 5]] and (ctx.item(), out.item()) == (18, 0)
        slots[:2] = -1
    else:
        assert st == (sage.SAGE_ERR_INVALID_ARG, sage.SAGE_KERNEL_PLAN)
        assert table.tolist() == [[3, -4]] and (ctx.item(), out.item()) == (16, 0) and off.tolist() == [0, 0]
    assert slots.max().item() == slots.min().item() == -1
