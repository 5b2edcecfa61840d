"""GPU tests of the paged-cache serving operators (sage_page_plan,
sage_kv_append, sage_attn_decode_shared and their MXFP4 forms) against plain
references, and of the three together as a serving loop uses them."""
import math

import numpy as np
import pytest
import torch

import oracle
import quantized_attention_smoothing_b200 as sage
import workloads
import serving_helpers as sh
from gpu_helpers import workloads_f32, bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def handles():
    from quantized_attention_smoothing_b200 import build
    build.build()
    return {64: sage.Hadamard(64), 128: sage.Hadamard(128)}


def dev(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


# ------------------------------------------------------------------- plan

def plan_inputs(B, page, max_pages, pp, seed, spare=3, mode="mixed"):
    rng = np.random.default_rng(seed)
    cap, P = max_pages * page, pp * page
    kind = rng.integers(0, 6, B) if mode == "mixed" else np.full(B, 1)
    cached, new = np.zeros(B, np.int64), np.zeros(B, np.int64)
    for b in range(B):
        if kind[b] == 0:                                 # joins
            new[b] = rng.integers(1, cap - P + 1) if cap > P else 0
            continue
        cached[b] = rng.integers(max(P, 1), cap + 1)
        new[b] = -1 if kind[b] == 2 else 0 if kind[b] == 3 else min(cap - cached[b], rng.integers(1, 5))
    if mode == "mixed" and B > 1:
        cached[B - 1], new[B - 1] = 0, 0                 # an empty row
    held = -(-cached // page)
    own = int(np.maximum(held - pp, 0).sum())
    start = np.where((cached == 0) & (new > 0), P, cached)
    need = int(np.where(new < 0, 0, -(-(start + new) // page) - -(-start // page)).sum())
    gone = int(np.where(new < 0, np.maximum(held - pp, 0), 0).sum())
    count = max(0, need - gone) + spare
    total = own + pp + count + gone
    perm = rng.permutation(total)
    table = rng.integers(0, 1 << 20, (B, max_pages))
    o = 0
    prefix = perm[own:own + pp]
    for b in range(B):
        if cached[b]:
            table[b, :pp] = prefix
            table[b, pp:held[b]] = perm[o:o + max(0, held[b] - pp)]
            o += max(0, held[b] - pp)
    free = np.full(total, -7)
    free[:count] = perm[own + pp:own + pp + count]
    return cached, new, table, prefix, free, count


def run_plan(cached, new, table, prefix, free, count, page, max_tokens, in_place=False, stream=None):
    c, n, t, f = dev(cached), dev(new), dev(table), dev(free)
    cnt = dev([count])
    B = len(cached)
    ctx, cnt2 = (c, cnt) if in_place else (torch.full_like(c, -9), torch.full_like(cnt, -9))
    off = torch.full((B + 1,), -9, dtype=torch.int32, device="cuda")
    slots = torch.full((max_tokens + 3,), -9, dtype=torch.int32, device="cuda")
    sage.sage_page_plan(c, n, f, cnt, page, t, ctx, cnt2, off, slots[:max_tokens],
                        prefix_table=dev(prefix) if len(prefix) else None, stream=stream)
    torch.cuda.synchronize()
    assert (slots[max_tokens:] == -9).all()
    return [x.cpu().numpy() for x in (t, f, ctx, cnt2, off, slots[:max_tokens])]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,max_pages,pp,mode,room", [
    (1, 16, 1, 0, "step", 0), (1, 128, 4, 2, "mixed", 5), (3, 16, 9, 0, "mixed", 1), (33, 32, 40, 7, "mixed", 0),
    (100, 64, 17, 17, "mixed", 9), (777, 16, 12, 3, "mixed", 100), (1500, 16, 5, 0, "mixed", 3),
    (2500, 32, 6, 1, "step", 0), (8192, 16, 3, 1, "mixed", 0), (40, 128, 60, 2, "mixed", 70001),
    (6, 16, 2000, 0, "mixed", 2),
])
def test_plan_matches_the_loop(handles, B, page, max_pages, pp, mode, room, in_place):
    cached, new, table, prefix, free, count = plan_inputs(B, page, max_pages, pp, B + page + pp, mode=mode)
    max_tokens = int(np.maximum(new, 0).sum()) + room
    ref = sh.ref_plan(cached, new, free, count, page, table, max_tokens, prefix)
    assert ref is not None
    got = run_plan(cached, new, table, prefix, free, count, page, max_tokens, in_place)
    for name, g, r in zip(("table", "free", "ctx", "count", "offsets", "slots"), got, ref):
        assert np.array_equal(g.ravel(), np.asarray(r).ravel()), name
    assert sage.sage_device_error() == sage.SAGE_OK


@pytest.mark.parametrize("what", ["pages", "slots", "length", "negative", "inside prefix", "count", "overflow"])
def test_plan_refuses_the_whole_step(handles, what):
    """A step that cannot be served changes nothing and is reported."""
    page, pp = 32, 2
    cached, new, table, prefix, free, count = plan_inputs(50, page, 20, pp, 5, spare=0)
    max_tokens = int(np.maximum(new, 0).sum())
    if what == "pages":
        count -= 1
    elif what == "slots":
        max_tokens -= 1
    elif what == "length":
        cached[7], new[7] = 20 * page, 1
    elif what == "negative":
        cached[7] = -3
    elif what == "inside prefix":
        cached[7] = pp * page - 1
    elif what == "count":
        count = len(free) + 1
    else:
        cached[7], new[7] = 20 * page, 2 ** 31 - 1
    assert sh.ref_plan(cached, new, free, count, page, table, max_tokens, prefix) is None
    got = run_plan(cached, new, table, prefix, free, count, page, max_tokens)
    assert np.array_equal(got[0], table) and np.array_equal(got[1], free) and np.array_equal(got[2], cached)
    assert got[3][0] == count and not got[4].any() and (got[5] == -1).all()
    assert sage.sage_device_error_where()[:2] == (sage.SAGE_ERR_INVALID_ARG, sage.SAGE_KERNEL_PLAN)
    assert sage.sage_device_error() == sage.SAGE_OK


def test_plan_captured_step_replays_in_place(handles):
    """A captured step run many times in place: lengths grow, pages move."""
    page, B, mp = 16, 5, 40
    cached, count = dev([1, 16, 17, 0, 300]), dev([150])
    new = dev([1, 2, 3, 1, 4])
    rng = np.random.default_rng(0)
    table0 = rng.permutation(1000)[:B * mp].reshape(B, mp)
    free0 = 2000 + rng.permutation(200)
    table, free = dev(table0), dev(free0)
    off, slots = dev(np.zeros(B + 1)), dev(np.zeros(16))
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        sage.sage_page_plan(cached, new, free, count, page, table, cached, count, off, slots, stream=s)
    r_c, r_t, r_f, r_n = np.array([1, 16, 17, 0, 300]), table0, free0, 150
    for step in range(30):
        g.replay()
        torch.cuda.synchronize()
        r_t, r_f, r_c, r_n, r_o, r_s = sh.ref_plan(r_c, np.array([1, 2, 3, 1, 4]), r_f, r_n, page, r_t, 16)
        assert np.array_equal(cached.cpu().numpy(), r_c) and np.array_equal(table.cpu().numpy(), r_t), step
        assert count.item() == r_n and np.array_equal(slots.cpu().numpy(), r_s), step


# ------------------------------------------------------------------- append

def append_inputs(N, Hk, D, page, seed, layout="slices", skip=0.1):
    g = torch.Generator().manual_seed(seed)
    kv = torch.randn((N, 2 * Hk, D), generator=g)
    kv[:, :Hk] += 2.0 * torch.randn((Hk, D), generator=g)
    if N > 2:
        kv[1] = 0.0                                       # a row of zeros
        kv[2, :, ::3] *= 1e-30
    kv = kv.to(torch.bfloat16)
    if layout == "odd":                                   # neither unit stride nor aligned
        buf = torch.zeros((N, 2 * Hk, D, 2), dtype=torch.bfloat16)
        buf[..., 1] = kv
        kv = buf.cuda()[..., 1]
    elif layout == "token-last":
        kv = kv.permute(1, 2, 0).contiguous().cuda().permute(2, 0, 1)
    else:
        kv = kv.cuda()
    pages = -(-N // page) + 3
    slots = torch.randperm(pages * page, generator=g)[:N].int()
    slots[torch.rand(N, generator=g) < skip] = -1
    mean = (2.0 * torch.randn((Hk, D), generator=g)).float()
    return kv[:, :Hk], kv[:, Hk:], slots, mean, pages


@pytest.mark.parametrize("N,Hk,D,page,flags,layout,with_mean", [
    (1, 1, 128, 128, 0, "slices", True), (7, 2, 128, 16, 0, "slices", True), (300, 3, 128, 64, 0, "odd", True),
    (129, 1, 64, 32, 0, "slices", False), (1000, 8, 64, 128, 0, "token-last", True),
    (50, 2, 128, 128, 2, "slices", True), (333, 4, 64, 128, 3, "slices", True), (65, 2, 64, 16, 1, "odd", False),
    (2000, 5, 128, 32, 1, "slices", True),
])
def test_append_fp8_bit_exact(handles, N, Hk, D, page, flags, layout, with_mean):
    k, v, slots, mean, pages = append_inputs(N, Hk, D, page, N + D + flags, layout)
    m = mean.numpy() if with_mean else None
    g = torch.Generator().manual_seed(1)
    kc = torch.randint(0, 256, (pages, Hk, page, D), generator=g).to(torch.uint8)
    vc = torch.randint(0, 256, (pages, Hk, D, page) if flags & 2 else (pages, Hk, page, D), generator=g).to(torch.uint8)
    if flags & 1:
        ks, vs = torch.tensor([4.0 * math.sqrt(D) / 448]), torch.tensor([2.5 / 448])
    else:
        ks, vs = (torch.rand((pages, Hk, page), generator=g) for _ in range(2))
    kg, vg, ksg, vsg = kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda()
    sage.sage_kv_append(handles[D], k, v, slots.cuda(), kg, vg, ksg, vsg, k_mean=mean.cuda() if with_mean else None,
                        kv_flags=flags)
    assert sage.sage_device_error() == sage.SAGE_OK
    kb, vb = workloads.bits_u16(k.cpu().contiguous()), workloads.bits_u16(v.cpu().contiguous())
    ok = slots.numpy() >= 0
    pg, off = slots.numpy()[ok] // page, slots.numpy()[ok] % page
    for x, cache, scale, got, got_s, vt in ((sh.rotated(kb, m), kc, ks, kg, ksg, False),
                                            (oracle.bf16_to_f32(vb), vc, vs, vg, vsg, bool(flags & 2))):
        codes, sc = sh.ref_append_fp8(x[ok].astype(np.float32), float(scale[0]) if flags & 1 else None)
        want, want_s = cache.numpy().copy(), scale.numpy().copy()
        if vt:
            want[pg, :, :, off] = codes
        else:
            want[pg, :, off] = codes
        if sc is not None:
            want_s[pg, :, off] = sc
        have = got.cpu().numpy()
        # -0 and +0 stand for one value; everything else bit for bit
        bad = (have != want) & ~(((have & 127) == 0) & ((want & 127) == 0))
        assert not bad.any(), "%d codes differ" % bad.sum()
        assert np.array_equal(got_s.cpu().numpy().view(np.uint32), want_s.view(np.uint32))


@pytest.mark.parametrize("N,Hk,page,layout", [(1, 1, 16, "slices"), (77, 2, 128, "slices"), (130, 3, 32, "odd"),
                                              (1024, 2, 64, "token-last")])
def test_append_mxfp4_bit_exact(handles, N, Hk, page, layout):
    D = 128
    k, v, slots, mean, pages = append_inputs(N, Hk, D, page, N, layout)
    g = torch.Generator().manual_seed(2)
    c0 = torch.randint(0, 256, (2, pages, Hk, page, D // 2), generator=g).to(torch.uint8)
    s0 = torch.randint(0, 256, (2, pages, Hk, page, D // 32), generator=g).to(torch.uint8)
    c, s = c0.cuda(), s0.cuda()
    sage.sage_kv_append_mxfp4(handles[D], k, v, slots.cuda(), c[0], c[1], s[0], s[1], k_mean=mean.cuda())
    assert sage.sage_device_error() == sage.SAGE_OK
    ok = slots.numpy() >= 0
    pg, off = slots.numpy()[ok] // page, slots.numpy()[ok] % page
    kb, vb = workloads.bits_u16(k.cpu().contiguous()), workloads.bits_u16(v.cpu().contiguous())
    for i, x in enumerate((sh.rotated(kb, mean.numpy()), oracle.bf16_to_f32(vb))):
        codes, sf = sh.ref_append_mx(x[ok].astype(np.float32))
        want, want_s = c0[i].numpy().copy(), s0[i].numpy().copy()
        want[pg, :, off], want_s[pg, :, off] = codes, sf
        have = c[i].cpu().numpy()
        assert np.array_equal(s[i].cpu().numpy(), want_s)
        for shift in (0, 4):
            a, b = (have >> shift) & 15, (want >> shift) & 15
            assert not ((a != b) & ~((a & 7 == 0) & (b & 7 == 0))).any()


def test_append_values_against_64_bits(handles):
    """What the cache stands for is within half an e4m3 step of the rotated
    key (2^-4 of the value; 2^-10 of the row's scale below the normal range),
    plus the fp32 rounding of seven sums and two scalings."""
    N, Hk, D, page = 500, 2, 128, 64
    k, v, slots, mean, pages = append_inputs(N, Hk, D, page, 3, skip=0.0)
    kc, vc = (torch.zeros((pages, Hk, page, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, Hk, page), device="cuda") for _ in range(2))
    sage.sage_kv_append(handles[D], k, v, slots.cuda(), kc, vc, ks, vs, k_mean=mean.cuda())
    pg, off = slots.numpy() // page, slots.numpy() % page
    H = oracle.hadamard(D).astype(np.float64)
    for x, c, s in (((k.cpu().double().numpy() - mean.numpy().astype(np.float64)) @ H, kc, ks),
                    (v.cpu().double().numpy(), vc, vs)):
        sc = s.cpu().numpy()[pg, :, off].astype(np.float64)[..., None]
        got = oracle.e4m3_decode(c.cpu().numpy()[pg, :, off]) * sc
        amax = np.abs(x).max(-1, keepdims=True)
        tol = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * sc) + 2.0 ** -19 * amax
        assert (np.abs(got - x) <= tol).all(), np.max(np.abs(got - x) / np.maximum(tol, 1e-300))


def test_append_bad_slot_is_skipped_and_reported(handles):
    N, Hk, D, page = 9, 2, 128, 32
    k, v, slots, mean, pages = append_inputs(N, Hk, D, page, 8, skip=0.0)
    slots[4], slots[6] = pages * page, -5
    buf = [torch.zeros((pages, Hk, page, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros((pages, Hk, page), device="cuda") for _ in range(2)]
    sage.sage_kv_append(handles[D], k, v, slots.cuda(), *buf, *sc)
    assert sage.sage_device_error_where()[:2] == (sage.SAGE_ERR_INVALID_ARG, sage.SAGE_KERNEL_APPEND)
    assert sage.sage_device_error() == sage.SAGE_OK
    written = (sc[0] > 0).sum().item()
    assert written == (N - 2 - 1) * Hk                   # row 1 is zeros: scale 0


def test_append_of_nothing(handles):
    e = torch.empty((0, 2, 128), dtype=torch.bfloat16, device="cuda")
    c = torch.zeros((2, 2, 16, 128), dtype=torch.uint8, device="cuda")
    s = torch.zeros((2, 2, 16), device="cuda")
    sage.sage_kv_append(handles[128], e, e, torch.empty(0, dtype=torch.int32, device="cuda"), c, c.clone(), s, s.clone())
    sage.sage_kv_append_mxfp4(handles[128], e, e, torch.empty(0, dtype=torch.int32, device="cuda"), c, c.clone(),
                              c.clone(), c.clone())
    assert sage.sage_device_error() == sage.SAGE_OK


# --------------------------------------------------------- shared attention

def run_shared(h, d, page, window, scale, q=None, out=None, ws=None, stream=None, prefix_len=None):
    q = d["q"].cuda() if q is None else q
    out = torch.full(d["q"].shape, float("nan"), dtype=torch.bfloat16, device="cuda") if out is None else out
    length = d["length"].cuda() if prefix_len is None else prefix_len
    a = [h, q, d["kc"].cuda(), d["vc"].cuda(), d["ks"].cuda(), d["vs"].cuda(), d["prefix"].cuda(), length,
         d["table"].cuda(), d["ctx"].cuda(), page, d["pages"], window, scale, out]
    if d["fmt"] == "mxfp4":
        sage.sage_attn_decode_shared_mxfp4(*a, ws=ws, stream=stream)
    else:
        flags = (1 if d["fmt"].startswith("tensor") else 0) | (2 if d["fmt"].endswith("vt") else 0)
        sage.sage_attn_decode_shared(*a, ws=ws, stream=stream, kv_flags=flags)
    return out


def check_shared(out, d, window, scale):
    ref, tol = sh.ref_shared(d, window, scale)
    g = workloads_f32(bits(out.contiguous())).astype(np.float64)
    worst = np.max(np.abs(g - ref) / tol)
    print("worst error %.3f of the tolerance" % worst)
    assert worst <= 1.0
    return g, ref


@pytest.mark.parametrize("B,T,H,Hk,D,page,prefix,ctx,window,fmt", [
    # one token in all, one key behind a prefix, a prefix alone
    (1, 1, 4, 1, 128, 16, 0, [1], 10, "token"),
    (1, 1, 8, 1, 128, 16, 16, [17], 100, "token"),
    (2, 1, 8, 2, 128, 32, 64, [64, 65], 1000, "token"),
    # the prefix ends inside a tile and inside a page; empty and short rows
    (5, 1, 16, 2, 128, 64, 777, [778, 0, 1000, 777, 3], 5000, "token"),
    (4, 3, 8, 1, 128, 16, 200, [203, 200, 201, 900], 5000, "token"),
    # windows shorter than the sequence: some rows see none of the prefix
    (4, 4, 16, 1, 128, 128, 512, [516, 640, 1100, 2000], 300, "token"),
    (3, 2, 4, 1, 64, 32, 300, [302, 310, 700], 1, "token"),
    # many rows (several row tiles), odd numbers of them; long prefixes
    (37, 1, 16, 1, 128, 128, 1500, list(range(1501, 1501 + 37 * 9, 9)), 9999, "token"),
    (9, 4, 12, 3, 128, 64, 2500, [2500 + 7 * i for i in range(1, 10)], 9999, "token"),
    (70, 1, 2, 1, 64, 16, 400, [400 + i for i in range(70)], 9999, "token"),
    (3, 4, 16, 1, 128, 128, 9000, [9004, 9300, 9100], 99999, "token"),
    # one scale for the cache, transposed V, both
    (6, 2, 16, 2, 128, 64, 640, [700, 650, 642, 645, 1000, 0], 9999, "tensor"),
    (6, 2, 16, 2, 64, 128, 640, [700, 650, 642, 645, 1000, 0], 9999, "tensor_vt"),
    (5, 1, 16, 1, 128, 128, 900, [1000, 950, 942, 945, 1400], 9999, "token_vt"),
    # the MXFP4 cache
    (5, 1, 16, 1, 128, 128, 900, [1000, 950, 942, 945, 1400], 9999, "mxfp4"),
    (4, 4, 8, 2, 128, 16, 333, [337, 0, 350, 1000], 200, "mxfp4"),
    (20, 2, 16, 1, 128, 32, 1024, [1026 + 3 * i for i in range(20)], 9999, "mxfp4"),
])
def test_shared_shapes(handles, B, T, H, Hk, D, page, prefix, ctx, window, fmt):
    d = sh.make_shared(B, T, H, Hk, D, page, prefix, ctx, seed=B + prefix + D, fmt=fmt)
    scale = 1.0 / math.sqrt(D)
    out = run_shared(handles[D], d, page, window, scale)
    torch.cuda.synchronize()
    assert sage.sage_device_error() == sage.SAGE_OK
    g, _ = check_shared(out, d, window, scale)
    for b in range(B):
        if ctx[b] == 0:
            assert not g[b].any()


def test_shared_peaked_logits(handles):
    """Logits with a spread of several units: the running maxima move, weights
    differ by orders of magnitude, single keys dominate rows."""
    d = sh.make_shared(7, 2, 16, 1, 128, 128, 3000, [3002 + 50 * i for i in range(7)], seed=4, k_std=60.0)
    out = run_shared(handles[128], d, 128, 9999, 1.0 / math.sqrt(128))
    check_shared(out, d, 9999, 1.0 / math.sqrt(128))


def test_shared_views_and_reused_workspace(handles):
    """Strided queries and output, a workspace with another call's leftovers."""
    B, T, H, D, page = 6, 2, 8, 128, 64
    d = sh.make_shared(B, T, H, 2, D, page, 500, [510, 600, 502, 0, 777, 640], seed=9)
    plain = run_shared(handles[D], d, page, 9999, 0.08)
    buf = torch.zeros((B, H, T, D + 8), dtype=torch.bfloat16)
    buf[..., :D] = d["q"].permute(0, 2, 1, 3)
    qg = buf.cuda().permute(0, 2, 1, 3)[..., :D]
    og = torch.full((B, H, T, D + 8), 7.0, dtype=torch.bfloat16, device="cuda").permute(0, 2, 1, 3)
    ws = torch.full((sage.sage_attn_decode_shared_workspace(B, T, H, 2, D),), 255, dtype=torch.uint8, device="cuda")
    run_shared(handles[D], d, page, 9999, 0.08, q=qg, out=og[..., :D], ws=ws)
    assert torch.equal(plain, og[..., :D]) and (og[..., D:] == 7.0).all()
    odd = torch.empty((B, T, H, 2 * D), dtype=torch.bfloat16, device="cuda")[..., ::2]      # no unit stride
    odd.copy_(d["q"])
    assert torch.equal(plain, run_shared(handles[D], d, page, 9999, 0.08, q=odd, ws=ws))
    check_shared(plain, d, 9999, 0.08)


def test_shared_equals_plain_decode_without_a_prefix(handles):
    """L = 0 is sage_attn_decode: the same result within the two kernels' roundings."""
    d = sh.make_shared(4, 2, 16, 2, 128, 64, 0, [100, 700, 257, 3], seed=12)
    d["table"] = torch.where(d["table"] > 1 << 20, 0, d["table"])
    out = run_shared(handles[128], d, 64, 9999, 0.1)
    ref = torch.empty_like(out)
    sage.sage_attn_decode(handles[128], d["q"].cuda(), d["kc"].cuda(), d["vc"].cuda(), d["ks"].cuda(), d["vs"].cuda(),
                          d["table"].cuda(), d["ctx"].cuda(), 64, d["pages"], 9999, 0.1, ref)
    _, tol = sh.ref_shared(d, 9999, 0.1)
    assert (np.abs((out.double() - ref.double()).cpu().numpy()) <= 2 * tol).all()


def test_shared_graph_follows_the_lengths(handles):
    """prefix_len and ctx_lens are read on the device: a captured call replayed
    with other lengths gives the other result."""
    d = sh.make_shared(5, 1, 16, 1, 128, 32, 640, [700, 641, 800, 650, 0], seed=21)
    h = handles[128]
    t = {n: d[n].cuda() for n in ("q", "kc", "vc", "ks", "vs", "prefix", "length", "ctx")}
    table = torch.where(d["table"] > 1 << 20, d["prefix"][:1], d["table"])
    full = table.clone()
    full[:, :20] = d["prefix"][None]                      # every entry of the rows is real here
    t["table"] = full.cuda()
    out = torch.empty(d["q"].shape, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty((sage.sage_attn_decode_shared_workspace(5, 1, 16, 1, 128),), dtype=torch.uint8, device="cuda")

    def call(stream=None):
        sage.sage_attn_decode_shared(h, t["q"], t["kc"], t["vc"], t["ks"], t["vs"], t["prefix"], t["length"], t["table"],
                                     t["ctx"], 32, d["pages"], 9999, 0.09, out, ws, stream=stream)
    call()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        call(s)
    d["table"] = full
    for length, ctx in ((640, [700, 641, 800, 650, 0]), (100, [700, 641, 800, 650, 0]), (0, [30, 600, 1, 650, 7]),
                        (640, [640, 0, 650, 1, 800])):
        t["length"].fill_(length)
        t["ctx"].copy_(torch.tensor(ctx, dtype=torch.int32))
        d["length"], d["ctx"] = torch.tensor([length]), torch.tensor(ctx, dtype=torch.int32)
        out.fill_(float("nan"))
        g.replay()
        check_shared(out, d, 9999, 0.09)


@pytest.mark.parametrize("B,T,H,Hk,D,page,prefix,ctx,fmt", [
    (3, 2, 16, 1, 128, 64, 500, [502, 700, 650], "token"), (3, 1, 16, 2, 64, 16, 77, [78, 0, 90], "token"),
    (9, 4, 16, 1, 128, 32, 500, [504 + 31 * i for i in range(9)], "token"),
    (5, 4, 16, 1, 64, 128, 300, [304 + 31 * i for i in range(5)], "token_vt"),
    (9, 2, 16, 1, 128, 128, 300, [302 + 31 * i for i in range(9)], "tensor_vt"),
    (2, 1, 16, 1, 128, 128, 300, [302, 1], "token_vt"),
    (9, 2, 16, 1, 128, 16, 300, [302 + 31 * i for i in range(9)], "mxfp4"),
])
def test_shared_slots_without_a_key_may_hold_anything(handles, B, T, H, Hk, D, page, prefix, ctx, fmt):
    """NaN codes and NaN or infinite scales behind a sequence's end, behind the
    prefix's end, before a sequence's first own token, and in unused pages (page
    0 among them) change nothing."""
    d = sh.make_shared(B, T, H, Hk, D, page, prefix, ctx, seed=77, fmt=fmt)
    # page 0 unused: its tokens move to a page of their own
    spare = d["pages"]
    for n in ("kc", "vc") + (() if fmt.startswith("tensor") else ("ks", "vs")):
        d[n] = torch.cat((d[n], d[n][:1]))
    d["pages"] += 1
    d["prefix"] = torch.where(d["prefix"] == 0, spare, d["prefix"]).int()
    d["table"] = torch.where(d["table"] == 0, spare, d["table"]).int()
    used = np.zeros((d["pages"], page), bool)
    for j in range(prefix):
        used[d["prefix"][j // page], j % page] = True
    for b in range(B):
        for j in range(prefix, ctx[b]):
            used[d["table"][b, j // page], j % page] = True
    dead = torch.from_numpy(~used)
    for n in ("k", "v"):
        c = d[n + "c"]
        if n == "v" and fmt.endswith("vt"):
            c = c.transpose(2, 3)
        c.copy_(torch.where(dead[:, None, :, None], torch.tensor(127 if n == "k" else 255, dtype=torch.uint8), c))
        if fmt == "mxfp4":
            d[n + "s"] = torch.where(dead[:, None, :, None], torch.tensor(255, dtype=torch.uint8), d[n + "s"])
        elif not fmt.startswith("tensor"):
            d[n + "s"] = torch.where(dead[:, None, :], float("nan") if n == "k" else float("inf"), d[n + "s"])
    out = run_shared(handles[D], d, page, 9999, 1.0 / math.sqrt(D))
    torch.cuda.synchronize()
    assert sage.sage_device_error() == sage.SAGE_OK
    check_shared(out, d, 9999, 1.0 / math.sqrt(D))


def test_shared_reports_bad_pages_and_lengths(handles):
    d = sh.make_shared(3, 1, 16, 1, 128, 64, 500, [600, 700, 650], seed=2)
    bad = dict(d, prefix=d["prefix"].clone())
    bad["prefix"][3] = d["pages"] + 5
    out = run_shared(handles[128], bad, 64, 9999, 0.09)
    assert sage.sage_device_error() == sage.SAGE_ERR_INVALID_ARG
    assert torch.isfinite(out).all()
    bad = dict(d, table=d["table"].clone())
    bad["table"][1, 9] = -1
    out = run_shared(handles[128], bad, 64, 9999, 0.09)
    assert sage.sage_device_error() == sage.SAGE_ERR_INVALID_ARG
    assert torch.isfinite(out).all()
    for n in (-1, 8 * 64 + 1):
        out = run_shared(handles[128], d, 64, 9999, 0.09, prefix_len=dev([n]))
        assert sage.sage_device_error() == sage.SAGE_ERR_INVALID_ARG
    assert sage.sage_device_error() == sage.SAGE_OK


@pytest.mark.parametrize("B,T,H,Hk,D,page,prefix,lo,hi,window,fmt,poison", [
    (16, 4, 16, 1, 128, 128, 500, 4, 2100, 10 ** 6, "token", True), (16, 4, 16, 1, 128, 16, 300, 4, 1500, 900, "token", True),
    (12, 3, 24, 2, 64, 32, 77, 3, 1300, 10 ** 6, "tensor", True), (12, 4, 32, 2, 64, 128, 130, 1, 1300, 700, "token_vt", True),
    (16, 4, 16, 1, 128, 128, 257, 4, 1800, 10 ** 6, "tensor_vt", True), (14, 3, 12, 1, 128, 64, 129, 0, 1500, 10 ** 6, "mxfp4", False),
    (16, 4, 16, 1, 128, 16, 40, 4, 1500, 400, "mxfp4", False),
])
def test_shared_many_rows_and_long_own_keys(handles, B, T, H, Hk, D, page, prefix, lo, hi, window, fmt, poison):
    """36 to 64 rows a sequence and hundreds to thousands of own keys each, of
    very different lengths; NaN codes wherever no key is."""
    rng = np.random.default_rng(B + prefix + hi)
    ctx = [int(prefix + rng.integers(lo, hi)) for _ in range(B)]
    ctx[0], ctx[1], ctx[2], ctx[3] = prefix + hi, prefix + 1, prefix, 0
    d = sh.make_shared(B, T, H, Hk, D, page, prefix, ctx, seed=B + hi, fmt=fmt)
    if poison:
        used = np.zeros((d["pages"], page), bool)
        for b in range(B):
            for j in range(ctx[b]):
                used[d["prefix"][j // page] if j < prefix else d["table"][b, j // page], j % page] = True
        dead = torch.from_numpy(~used)
        for n in ("k", "v"):
            c = d[n + "c"].transpose(2, 3) if n == "v" and fmt.endswith("vt") else d[n + "c"]
            c.copy_(torch.where(dead[:, None, :, None], torch.tensor(127, dtype=torch.uint8), c))
            if not fmt.startswith("tensor"):
                d[n + "s"] = torch.where(dead[:, None, :], float("nan"), d[n + "s"])
    out = run_shared(handles[D], d, page, window, 1.0 / math.sqrt(D))
    torch.cuda.synchronize()
    assert sage.sage_device_error() == sage.SAGE_OK
    check_shared(out, d, window, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("B,T,H,Hk,D,page,prefix,fmt", [
    (4, 1, 128, 8, 64, 16, 7990, "token"), (1, 4, 128, 8, 128, 128, 8100, "tensor_vt"), (3, 2, 80, 8, 128, 32, 8077, "mxfp4"),
    (17, 1, 8, 8, 128, 64, 8000, "token"),
])
def test_shared_few_rows_behind_a_long_prefix(handles, B, T, H, Hk, D, page, prefix, fmt):
    """17 to 64 rows a head and many key tiles a split, where either kernel may
    take the prefix; one sequence ends inside it."""
    ctx = [prefix + 5 + 40 * b for b in range(B)]
    ctx[-1] = prefix // 2 if B > 1 else ctx[-1]
    d = sh.make_shared(B, T, H, Hk, D, page, prefix, ctx, seed=B + H, fmt=fmt)
    for window in (10 ** 6, 3000):
        out = run_shared(handles[D], d, page, window, 1.0 / math.sqrt(D))
        torch.cuda.synchronize()
        assert sage.sage_device_error() == sage.SAGE_OK
        check_shared(out, d, window, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("seed", range(32))
def test_shared_random_shapes(handles, seed):
    """Sizes drawn over what the interface takes: row counts on both sides of
    64, 128 and 256, every page size, 1 to 64 rows a sequence, prefixes that end
    anywhere, windows, rows that see nothing."""
    rng = np.random.default_rng(1000 + seed)
    fmt = ["token", "tensor", "mxfp4", "token_vt", "tensor_vt"][seed % 5]
    D = 128 if fmt == "mxfp4" or seed % 3 else 64
    page = 128 if fmt.endswith("vt") else int(rng.choice([16, 32, 64, 128]))
    G, T, Hk = int(rng.integers(1, 17)), int(rng.integers(1, 5)), int(rng.integers(1, 4))
    B = int(max(1, min(40, rng.choice([60, 120, 250, 500]) // (G * T))))
    prefix = int(rng.choice([0, 1, rng.integers(1, 900), rng.integers(1, 2000)]))
    most = max(2, min(600, 30000 // (B * T)))
    ctx = [int(prefix + rng.integers(0, most)) if rng.random() < 0.85 else int(rng.integers(0, prefix + 1)) for _ in range(B)]
    window = int(rng.choice([10 ** 6, 2 ** 31 - 1, rng.integers(1, prefix + most + 1)]))
    d = sh.make_shared(B, T, G * Hk, Hk, D, page, prefix, ctx, seed=seed, fmt=fmt)
    out = run_shared(handles[D], d, page, window, 1.0 / math.sqrt(D))
    torch.cuda.synchronize()
    assert sage.sage_device_error() == sage.SAGE_OK
    check_shared(out, d, window, 1.0 / math.sqrt(D))


@pytest.mark.parametrize("B,prefix,ctx", [(5, 700, [702, 900, 760, 1300, 701]), (1, 300, [900])])
def test_shared_value_scales_far_apart(handles, B, prefix, ctx):
    """Value scales that differ by 2^12 inside a tile, and whole runs of keys
    2^10 larger than those before them (the exponent they are held against
    moves). fp16 keeps 2^-25 of the largest scale, 2^-13 of the smallest one's
    unit, so the bf16-step tolerance holds as it is."""
    d = sh.make_shared(B, 2, 16, 1, 128, 64, prefix, ctx, seed=31)
    g = torch.Generator().manual_seed(6)
    f = torch.exp2(torch.randint(-6, 7, d["vs"].shape, generator=g).float())
    order = {int(pg): i for i, pg in enumerate(d["prefix"].tolist())}
    for pg in range(d["pages"]):
        f[pg] *= 2.0 ** (5 if order.get(pg, pg) % 7 > 3 else -5)
    d["vs"] = d["vs"] * f
    out = run_shared(handles[128], d, 64, 9999, 0.09)
    check_shared(out, d, 9999, 0.09)


@pytest.mark.parametrize("B,T,H,prefix,ctx,fmt", [
    (9, 1, 16, 700, [700 + 30 * b for b in range(9)], "token"), (1, 2, 8, 300, [700], "token"),
    (16, 4, 16, 130, [130 + 100 * b for b in range(16)], "token"), (9, 1, 16, 700, [700 + 30 * b for b in range(9)], "token_vt"),
])
def test_shared_tokens_of_zeros(handles, B, T, H, prefix, ctx, fmt):
    """Keys and values of zeros (scale 0, as the cache write leaves them): whole
    first tiles of them, then single ones; and queries of zeros."""
    d = sh.make_shared(B, T, H, 1, 128, 128, prefix, ctx, seed=B + T, fmt=fmt)
    first = [int(d["prefix"][0]), int(d["prefix"][1])] + [int(x) for x in d["table"][:, prefix // 128] if x < 1 << 20]
    for n in ("ks", "vs"):
        d[n][first] = 0.0
        d[n][:, :, 5::17] = 0.0
    d["q"][0, 0, 1] = 0
    out = run_shared(handles[128], d, 128, 9999, 0.09)
    check_shared(out, d, 9999, 0.09)
    d["vs"].zero_()
    assert not run_shared(handles[128], d, 128, 9999, 0.09).any()


def test_shared_and_append_far_into_a_large_cache(handles):
    """Caches of over 2^32 bytes: pages at their far end give the same bits as
    the same pages in a small cache, for reading and for writing."""
    Hk, D, page, pages = 8, 128, 128, 36000
    for B, T in ((2, 1), (9, 2)):
        d = sh.make_shared(B, T, 32, Hk, D, page, 300, [300 + 40 * (i + 1) for i in range(B)], seed=B)
        small = run_shared(handles[D], d, page, 9999, 0.09)
        far = {n: torch.zeros((pages,) + tuple(d[n].shape[1:]), dtype=d[n].dtype, device="cuda")
               for n in ("kc", "vc", "ks", "vs")}
        n = d["pages"]
        for k in far:
            far[k][pages - n:] = d[k].cuda().flip(0)
        big = dict(d, pages=pages, prefix=pages - 1 - d["prefix"],
                   table=torch.where(d["table"] > 1 << 20, d["table"], pages - 1 - d["table"]))
        out = torch.empty_like(small)
        sage.sage_attn_decode_shared(handles[D], big["q"].cuda(), far["kc"], far["vc"], far["ks"], far["vs"],
                                     big["prefix"].cuda(), big["length"].cuda(), big["table"].cuda(), big["ctx"].cuda(),
                                     page, pages, 9999, 0.09, out)
        assert sage.sage_device_error() == sage.SAGE_OK
        assert torch.equal(out, small)
    k, v, slots, mean, few = append_inputs(200, Hk, D, page, 5)
    near = [torch.zeros((few, Hk, page, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    near_s = [torch.zeros((few, Hk, page), device="cuda") for _ in range(2)]
    sage.sage_kv_append(handles[D], k, v, slots.cuda(), *near, *near_s, k_mean=mean.cuda())
    for t in far.values():
        t[pages - few:] = 0
    moved = torch.where(slots >= 0, slots + (pages - few) * page, slots).int()
    sage.sage_kv_append(handles[D], k, v, moved.cuda(), far["kc"], far["vc"], far["ks"], far["vs"], k_mean=mean.cuda())
    assert sage.sage_device_error() == sage.SAGE_OK
    for a, b in zip(near + near_s, (far["kc"], far["vc"], far["ks"], far["vs"])):
        assert torch.equal(a, b[pages - few:])


@pytest.mark.parametrize("B,T", [(2, 1), (20, 2)])
def test_shared_two_at_once(handles, B, T):
    """Two calls on two streams at once, each with its workspace, and two
    captured graphs replayed at once: the results of one after the other. A
    call's result does not depend on the run."""
    ds = [sh.make_shared(B, T, 16, 1, 128, 64, 1500, [1500 + 30 * (i + 1) for i in range(B)], seed=s) for s in (1, 2)]
    h = handles[128]
    want = [run_shared(h, d, 64, 9999, 0.09) for d in ds]
    gpu = [{n: d[n].cuda() for n in ("q", "kc", "vc", "ks", "vs", "prefix", "length", "table", "ctx")} for d in ds]
    ws = [torch.empty((sage.sage_attn_decode_shared_workspace(B, T, 16, 1, 128),), dtype=torch.uint8, device="cuda")
          for _ in ds]
    outs = [torch.zeros_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in ds]

    def call(i):
        t = gpu[i]
        sage.sage_attn_decode_shared(h, t["q"], t["kc"], t["vc"], t["ks"], t["vs"], t["prefix"], t["length"], t["table"],
                                     t["ctx"], 64, ds[i]["pages"], 9999, 0.09, outs[i], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            call(i)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    graphs = [torch.cuda.CUDAGraph() for _ in ds]
    for i in range(2):
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            for _ in range(10):
                call(i)
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for i in range(2):
        with torch.cuda.stream(streams[i]):
            graphs[i].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert sage.sage_device_error() == sage.SAGE_OK


# ------------------------------------------------------------- all together

@pytest.mark.parametrize("fmt,page,Hk,side", [("token", 32, 2, False), ("tensor_vt", 128, 1, True),
                                              ("mxfp4", 64, 2, False)])
def test_serving_loop(handles, fmt, page, Hk, side):
    """A shared prompt enters the cache, requests join behind it, grow, end and
    join again; every step plans, appends and attends, and each step's attention
    is that of the keys and values the test keeps for itself (in the cache's
    format), on the current stream or on another one."""
    D, G, B, T = 128, 4, 6, 2
    H, P, mp, pages = G * Hk, 4 * page, 12, 60
    h = handles[D]
    g = torch.Generator().manual_seed(page)
    mean = torch.randn((Hk, D), generator=g).cuda()
    mx, tensor, vt = fmt == "mxfp4", fmt.startswith("tensor"), fmt.endswith("vt")
    shape = (pages, Hk, page, D // 2 if mx else D)
    kc = torch.zeros(shape, dtype=torch.uint8, device="cuda")
    vc = torch.zeros((pages, Hk, D, page) if vt else shape, dtype=torch.uint8, device="cuda")
    if mx:
        ks, vs = (torch.zeros((pages, Hk, page, D // 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    elif tensor:
        ks, vs = torch.full((1,), 5 * math.sqrt(D) / 448, device="cuda"), torch.full((1,), 5 / 448, device="cuda")
    else:
        ks, vs = (torch.zeros((pages, Hk, page), device="cuda") for _ in range(2))
    flags = (1 if tensor else 0) | (2 if vt else 0)
    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()

    def append(k, v, slots):
        if mx:
            sage.sage_kv_append_mxfp4(h, k, v, slots, kc, vc, ks, vs, k_mean=mean, stream=stream)
        else:
            sage.sage_kv_append(h, k, v, slots, kc, vc, ks, vs, k_mean=mean, kv_flags=flags, stream=stream)

    def tokens(n):
        return (torch.randn((n, Hk, D), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    perm = torch.randperm(pages, generator=g).int()
    prefix, free = perm[:4].cuda(), torch.cat((perm[4:], perm[:4])).cuda()
    cached, count = dev(np.zeros(B)), dev([pages - 4])
    table = dev(np.zeros((B, mp)))
    off, slots = dev(np.zeros(B + 1)), dev(np.zeros(600))
    length = dev([P])
    ws = torch.empty((sage.sage_attn_decode_shared_workspace(B, T, H, Hk, D),), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    pk, pv = tokens(P)
    pslots = (prefix[:, None] * page + torch.arange(page, device="cuda")[None]).reshape(-1).int()
    stream.wait_stream(torch.cuda.current_stream())
    append(pk, pv, pslots)
    lens = [0] * B
    for step, new in enumerate(([70, 3, 0, 2, 200, 2], [2, 2, 0, 2, 2, 2], [2, -1, 5, -1, 2, 2], [2, 2, 2, 0, -1, 3],
                                [2, 2, 2, 2, 2, 2])):
        n_new = sum(max(x, 0) for x in new)
        k, v = tokens(600)                                # a padded batch: slots behind the last token are -1
        q = torch.randn((B, T, H, D), generator=g).to(torch.bfloat16).cuda()
        out = torch.empty_like(q)
        nd = dev(new)
        stream.wait_stream(torch.cuda.current_stream())
        sage.sage_page_plan(cached, nd, free, count, page, table, cached, count, off, slots, prefix_table=prefix,
                            stream=stream)
        append(k, v, slots)
        a = [h, q, kc, vc, ks, vs, prefix, length, table, cached, page, pages, 10 ** 6, 0.09, out]
        if mx:
            sage.sage_attn_decode_shared_mxfp4(*a, ws=ws, stream=stream)
        else:
            sage.sage_attn_decode_shared(*a, ws=ws, stream=stream, kv_flags=flags)
        torch.cuda.synchronize()
        assert sage.sage_device_error(stream) == sage.SAGE_OK
        for b in range(B):
            lens[b] = 0 if new[b] < 0 else (P if lens[b] == 0 and new[b] > 0 else lens[b]) + new[b]
        assert cached.cpu().tolist() == lens and off[B].item() == n_new
        live = sorted(table[b, e].item() for b in range(B) for e in range(4, -(-lens[b] // page)))
        rest = free[:count.item()].cpu().tolist()
        assert sorted(live + rest + prefix.cpu().tolist()) == list(range(pages))        # no page lost or shared
        d = dict(q=q.cpu(), kc=kc.cpu(), vc=vc.cpu(), ks=ks.cpu(), vs=vs.cpu(), fmt=fmt, prefix=prefix.cpu(),
                 table=table.cpu(), ctx=cached.cpu(), length=length.cpu())
        check_shared(out, d, 10 ** 6, 0.09)
    # the cache itself holds what was appended: the last step's tokens
    s = slots[:n_new].cpu().numpy()
    x = sh.rotated(workloads.bits_u16(k[:n_new].cpu()), mean.cpu().numpy())
    if mx:
        want = sh.ref_append_mx(x)[0]
    else:
        want = sh.ref_append_fp8(x, float(ks[0]) if tensor else None)[0]
    have = kc.cpu().numpy()[s // page, :, s % page]
    if mx:
        assert np.mean(have != want) < 1e-3               # signed zeros
    else:
        assert not ((have != want) & ((have & 127) != 0)).any()


@pytest.mark.parametrize("B,T,G,fmt", [(40, 1, 16, "token"), (3, 2, 4, "token"), (9, 3, 16, "mxfp4")])
def test_serving_steps_without_waiting(handles, B, T, G, fmt):
    """Steps issued back to back, where a kernel may start before the one before
    it has ended: every step's output is the one that the same steps give with
    the GPU waited for after every call."""
    D, Hk, page, P, mp, steps = 128, 2, 32, 70, 16, 40
    h, H, mx = handles[D], G * Hk, fmt == "mxfp4"
    pages = B * mp + 8
    g = torch.Generator().manual_seed(3)
    mean = torch.randn((Hk, D), generator=g).cuda()
    kv = [torch.randn((max(B * T, P), 2 * Hk, D), generator=g).to(torch.bfloat16).cuda() for _ in range(steps + 1)]
    q = [torch.randn((B, T, H, D), generator=g).to(torch.bfloat16).cuda() for _ in range(steps)]
    perm = torch.randperm(pages, generator=g).int()
    new = torch.full((B,), T, dtype=torch.int32).cuda()
    length = dev([2 * page])

    def run(wait):
        shape = (pages, Hk, page, D // 2 if mx else D)
        kc, vc = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros((pages, Hk, page) + ((D // 32,) if mx else ()), dtype=torch.uint8 if mx else torch.float32,
                              device="cuda") for _ in range(2))
        prefix, free = perm[:2].cuda(), torch.cat((perm[2:], perm[:2])).cuda()
        cached, count = dev(np.zeros(B)), dev([pages - 2])
        table, off, slots = dev(np.zeros((B, mp))), dev(np.zeros(B + 1)), dev(np.zeros(B * T))
        ws = torch.empty((sage.sage_attn_decode_shared_workspace(B, T, H, Hk, D),), dtype=torch.uint8, device="cuda")
        outs = [torch.zeros_like(x) for x in q]
        fill = (prefix[:, None] * page + torch.arange(page, device="cuda")[None]).reshape(-1).int()
        append = sage.sage_kv_append_mxfp4 if mx else sage.sage_kv_append
        attend = sage.sage_attn_decode_shared_mxfp4 if mx else sage.sage_attn_decode_shared
        x = kv[steps][:2 * page]
        append(h, x[:, :Hk], x[:, Hk:], fill, kc, vc, ks, vs, k_mean=mean)
        torch.cuda.synchronize()
        for i in range(steps):
            x = kv[i][:B * T]
            sage.sage_page_plan(cached, new, free, count, page, table, cached, count, off, slots, prefix_table=prefix)
            if wait:
                torch.cuda.synchronize()
            append(h, x[:, :Hk], x[:, Hk:], slots, kc, vc, ks, vs, k_mean=mean)
            if wait:
                torch.cuda.synchronize()
            attend(h, q[i], kc, vc, ks, vs, prefix, length, table, cached, page, pages, 10 ** 6, 0.09, outs[i], ws)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert sage.sage_device_error() == sage.SAGE_OK
        return outs
    want, got = run(True), run(False)
    assert all(torch.isfinite(x).all() for x in want)
    for i in range(steps):
        assert torch.equal(want[i], got[i]), i
