"""GPU tests of the quantised cache write on elements that are not finite: the
row that holds one (its block, over an MXFP4 cache) is what the header says, and
every other row holds the bits that it has without it."""
import math

import pytest
import torch

import quantized_attention_smoothing_b200 as sage

pytestmark = pytest.mark.gpu

N, HK, D, PAGE, PAGES = 40, 2, 128, 32, 3
BAD = {3: math.inf, 9: -math.inf, 20: math.nan}          # token -> element 37 of head 1


@pytest.fixture(scope="module")
def handle():
    from quantized_attention_smoothing_b200 import build
    build.build()
    return sage.Hadamard(D)


def inputs():
    g = torch.Generator().manual_seed(4)
    clean = torch.randn((2, N, HK, D), generator=g).to(torch.bfloat16)
    bad = clean.clone()
    for n, x in BAD.items():
        bad[:, n, 1, 37] = x
    slots = torch.randperm(PAGE * PAGES, generator=g)[:N].int()
    return clean.cuda(), bad.cuda(), slots


def rows(cache, slots):
    """[N, Hk, ...] of a cache [pages, Hk, page, ...]."""
    s = slots.long()
    return cache.cpu()[s // PAGE, :, s % PAGE]


def test_mxfp4_blocks_with_elements_not_finite(handle):
    clean, bad, slots = inputs()
    got = []
    for kv in (clean, bad):
        c = [torch.zeros((PAGES, HK, PAGE, D // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
        s = [torch.zeros((PAGES, HK, PAGE, D // 32), dtype=torch.uint8, device="cuda") for _ in range(2)]
        sage.sage_kv_append_mxfp4(handle, kv[0], kv[1], slots.cuda(), *c, *s)
        got.append([rows(x, slots) for x in (*c, *s)])
    assert sage.sage_device_error() == sage.SAGE_OK
    (ck, cv, sk, sv), (bk, bv, tk, tv) = got
    assert (tk <= 252).all() and (tv <= 252).all()       # E at most 125
    other = torch.tensor([n for n in range(N) if n not in BAD])
    for a, b in ((ck, bk), (cv, bv), (sk, tk), (sv, tv)):
        assert torch.equal(a[other], b[other]) and torch.equal(a[:, 0], b[:, 0])
    nib = torch.stack((bv & 15, bv >> 4), -1).flatten(-2)
    blocks = [i for i in range(4) if i != 1]             # element 37 is in block 1
    for n, x in BAD.items():
        assert torch.equal(sv[n, 1, blocks], tv[n, 1, blocks])
        assert torch.equal(cv[n, 1].view(4, 16)[blocks], bv[n, 1].view(4, 16)[blocks])
        if math.isinf(x):
            assert tv[n, 1, 1] == 252 and nib[n, 1, 37] == (7 if x > 0 else 15)
            rest = nib[n, 1, 32:64][torch.arange(32) != 5]
            assert ((rest & 7) == 0).all()               # nothing beside 2^125
        else:
            keep = [i for i in range(32, 64) if i != 37]
            clean_nib = torch.stack((cv & 15, cv >> 4), -1).flatten(-2)
            if sv[n, 1, 1] == tv[n, 1, 1]:               # (element 37 was not the block's largest)
                assert torch.equal(nib[n, 1, keep], clean_nib[n, 1, keep])


@pytest.mark.parametrize("tensor", [False, True])
def test_fp8_rows_with_elements_not_finite(handle, tensor):
    clean, bad, slots = inputs()
    got = []
    for kv in (clean, bad):
        c = [torch.zeros((PAGES, HK, PAGE, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
        s = [torch.full((1,), 0.1, device="cuda") for _ in range(2)] if tensor else \
            [torch.zeros((PAGES, HK, PAGE), device="cuda") for _ in range(2)]
        sage.sage_kv_append(handle, kv[0], kv[1], slots.cuda(), *c, *s, kv_flags=1 if tensor else 0)
        got.append([rows(x, slots) for x in c] + ([] if tensor else [rows(x, slots) for x in s]))
    assert sage.sage_device_error() == sage.SAGE_OK
    other = torch.tensor([n for n in range(N) if n not in BAD])
    for a, b in zip(*got):
        assert torch.equal(a[other], b[other]) and torch.equal(a[:, 0], b[:, 0])
    vc = got[1][1]
    for n, x in BAD.items():
        code = int(vc[n, 1, 37])
        if math.isnan(x):
            assert (code & 127) == 127
        elif tensor:
            assert code == (126 if x > 0 else 254)       # saturated
        else:
            assert (code & 127) == 127 and got[1][3][n, 1] == math.inf
