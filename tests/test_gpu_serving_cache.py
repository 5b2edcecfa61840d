"""GPU test of what a serving loop leaves in the cache: codes and scales of K
and of V, token by token, and nothing else."""
import math

import numpy as np
import pytest
import torch

import oracle
import quantized_attention_smoothing_b200 as sage
import serving_helpers as sh
import workloads

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


@pytest.mark.parametrize("fmt,D,page,Hk", [("token", 128, 32, 2), ("token", 64, 16, 3), ("tensor", 128, 64, 1),
                                           ("token_vt", 64, 128, 2), ("tensor_vt", 128, 128, 1), ("mxfp4", 128, 32, 3)])
def test_cache_after_a_serving_loop(fmt, D, page, Hk):
    """Requests join behind a prefix, grow, end and give pages to others. Every
    byte of the caches and scales is what the reference writes at the slots of
    the reference's plan (a signed zero stands for zero), and the initial fill
    everywhere else."""
    from quantized_attention_smoothing_b200 import build
    build.build()
    h, B, mp, pages, room = sage.Hadamard(D), 6, 12, 60, 4 * page + 90
    mx, tensor, vt = fmt == "mxfp4", fmt.startswith("tensor"), fmt.endswith("vt")
    rng, g = np.random.default_rng(page), torch.Generator().manual_seed(page + D)
    mean = torch.randn((Hk, D), generator=g)
    shape = (pages, Hk, page, D // 2 if mx else D)
    want = {n: np.full(shape, 0x55, np.uint8) for n in ("k", "v")}
    if tensor:
        scale = {"k": np.full(1, 5 * math.sqrt(D) / 448, np.float32), "v": np.full(1, 5 / 448, np.float32)}
    else:
        scale = {n: np.full((pages, Hk, page, D // 32) if mx else (pages, Hk, page), 77,
                            np.uint8 if mx else np.float32) for n in "kv"}
    gpu = {n: torch.from_numpy(want[n].swapaxes(2, 3).copy() if n == "v" and vt else want[n].copy()).cuda() for n in "kv"}
    gpu_s = {n: torch.from_numpy(scale[n].copy()).cuda() for n in "kv"}
    perm = rng.permutation(pages)
    prefix, free, count = perm[:2], np.concatenate((perm[2:], perm[:2])), pages - 2
    table, cached = np.zeros((B, mp), np.int64), np.zeros(B, np.int64)
    d = dict(table=dev(table), free=dev(free), count=dev([count]), cached=dev(cached), off=dev(np.zeros(B + 1)),
             slots=dev(np.zeros(room)), prefix=dev(prefix))

    def write(slots, slots_gpu, n):
        kv = torch.randn((n, 2 * Hk, D), generator=g).to(torch.bfloat16)
        a = (h, kv.cuda()[:, :Hk], kv.cuda()[:, Hk:], slots_gpu, gpu["k"], gpu["v"], gpu_s["k"], gpu_s["v"])
        if mx:
            sage.sage_kv_append_mxfp4(*a, k_mean=mean.cuda())
        else:
            sage.sage_kv_append(*a, k_mean=mean.cuda(), kv_flags=(1 if tensor else 0) | (2 if vt else 0))
        ok = slots >= 0
        pg, off = slots[ok] // page, slots[ok] % page
        bits = workloads.bits_u16(kv)
        for name, x in (("k", sh.rotated(bits[:, :Hk], mean.numpy())), ("v", oracle.bf16_to_f32(bits[:, Hk:]))):
            x = x[ok].astype(np.float32)
            codes, s = sh.ref_append_mx(x) if mx else sh.ref_append_fp8(x, float(scale[name][0]) if tensor else None)
            want[name][pg, :, off] = codes
            if not tensor:
                scale[name][pg, :, off] = s
    first = (prefix[:, None] * page + np.arange(page)[None]).ravel()
    write(first, dev(first), 2 * page)
    for new in ([70, 3, 0, 2, 2 * page + 1, 2], [2, 2, 0, 2, 2, 2], [2, -1, 5, -1, 2, 2], [2, 2, 2, 0, -1, 3], [2] * 6):
        table, free, cached, count, _, slots = sh.ref_plan(cached, np.array(new), free, count, page, table, room, prefix)
        sage.sage_page_plan(d["cached"], dev(new), d["free"], d["count"], page, d["table"], d["cached"], d["count"],
                            d["off"], d["slots"], prefix_table=d["prefix"])
        write(slots, d["slots"], room)
        assert np.array_equal(d["slots"].cpu().numpy(), slots)
    assert sage.sage_device_error() == sage.SAGE_OK
    for n in "kv":
        have = gpu[n].cpu().numpy()
        have = have.swapaxes(2, 3) if n == "v" and vt else have
        halves = [(have & 15, want[n] & 15, 7), (have >> 4, want[n] >> 4, 7)] if mx else [(have, want[n], 127)]
        for a, b, magnitude in halves:
            assert not ((a != b) & ~(((a & magnitude) == 0) & ((b & magnitude) == 0))).any(), n
        assert np.array_equal(gpu_s[n].cpu().numpy(), scale[n]), n
