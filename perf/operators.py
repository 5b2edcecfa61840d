"""Cases and plain forms of the paged-cache serving operators.

Three operators, used together in a serving step over the paged KV cache:

``plan``    sage_page_plan: from the lengths of a batch's requests, the pages
            they take from and give back to a free list, their block tables
            and the slot of every new token.
``append``  sage_kv_append / sage_kv_append_mxfp4: the new tokens' K (smoothed
            by a fixed per-head mean, rotated) and V, quantised to the cache's
            format and written into their slots.
``shared``  sage_attn_decode_shared / sage_attn_decode_shared_mxfp4: decode
            attention of a batch whose sequences begin with the same prefix,
            the prefix's keys and values read once for all of them.

``run`` computes a case in its plain form (elementary torch operations), or
with ``own`` set through the library. Everything it needs beyond torch is in
this file; the library is imported only where ``own`` is true.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
NEG_INF = float("-inf")


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a 32-sequence batch: one token each, pages of 128
        dict(name="plan_step_b32", op="plan", B=32, page=128, max_pages=257, mode="step", T=1, prefix_pages=0),
        # a step of a large serving batch behind a shared prompt of 2048 tokens, some requests ending, some joining
        dict(name="plan_mixed_b1000", op="plan", B=1000, page=32, max_pages=1024, mode="mixed", T=4, prefix_pages=64),
        # a batch of prompts entering the cache, pages of 16: the longest slot map
        dict(name="plan_prompts_b61", op="plan", B=61, page=16, max_pages=2048, mode="prompt", T=1, prefix_pages=0),
        # the tokens of one decode step: 16 sequences of 4 query tokens, one KV head (latency)
        dict(name="append_step_n64", op="append", N=64, Hk=1, D=128, page=128, fmt="token", pad=0),
        # a prompt of 32760 tokens with 8 KV heads, per-token scales: the largest write
        dict(name="append_prompt_n32760", op="append", N=32760, Hk=8, D=128, page=64, fmt="token", pad=8),
        # head size 64, one scale for the cache, V kept transposed (pages of 128)
        dict(name="append_tensor_vt_n4099", op="append", N=4099, Hk=4, D=64, page=128, fmt="tensor_vt", pad=0),
        # the same over an MXFP4 cache
        dict(name="append_mxfp4_n8192", op="append", N=8192, Hk=2, D=128, page=32, fmt="mxfp4", pad=0),
        # few sequences behind a prompt of 2000 tokens that ends inside a 128-key tile (latency)
        dict(name="shared_b3_l2000", op="shared", B=3, T=1, H=16, Hk=2, D=128, page=16, prefix=2000, lo=1, hi=100, window=0, fmt="token", pad=0),
        # 16 sequences, 4 query tokens, window 4096, behind a shared prompt of 4096
        dict(name="shared_window_b16", op="shared", B=16, T=4, H=16, Hk=1, D=128, page=128, prefix=4096, lo=4, hi=4096, window=4096, fmt="token", pad=0),
        # head size 64, 8 KV heads, one scale for the cache, a padded batch
        dict(name="shared_d64_b48_l8192", op="shared", B=48, T=2, H=32, Hk=8, D=64, page=64, prefix=8192, lo=2, hi=700, window=0, fmt="tensor", pad=5),
        # the MXFP4 cache: 32 sequences, one query token, prompt of 16384
        dict(name="shared_mxfp4_b32_l16384", op="shared", B=32, T=1, H=16, Hk=1, D=128, page=128, prefix=16384, lo=1, hi=1024, window=0, fmt="mxfp4", pad=0),
        # batch 256 behind a prompt of 32768 tokens: the largest
        dict(name="shared_b256_l32768", op="shared", B=256, T=1, H=16, Hk=1, D=128, page=128, prefix=32768, lo=1, hi=512, window=0, fmt="token", pad=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "shared", "shared"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 1200)
        mode = rng.choice(["step", "mixed", "prompt"])
        most = {"step": 1 << 20, "mixed": 1 << 20, "prompt": 61 * 2048 * 16}[mode]   # entries, or tokens
        cap = max(2, min(2048, most // (B * (page if mode == "prompt" else 1))))
        max_pages = _log(rng, 2, cap)
        return dict(op=op, B=B, page=page, max_pages=max_pages, mode=mode, T=rng.randint(1, 4),
                    prefix_pages=rng.choice([0, rng.randint(0, max_pages // 2)]))
    if op == "append":
        fmt = rng.choice(["token", "tensor", "token_vt", "tensor_vt", "mxfp4"])
        Hk = rng.choice([1, 2, 3, 4, 8])
        D = 128 if fmt == "mxfp4" else rng.choice([64, 128])
        most = 32760 * 8 * 128 // (4 if fmt == "mxfp4" else 1)
        N = _log(rng, 1, most // (Hk * D) if most // (Hk * D) < 60000 else 60000)
        return dict(op=op, N=N, Hk=Hk, D=D, page=128 if fmt.endswith("vt") else page, fmt=fmt,
                    pad=rng.choice([0, rng.randint(0, N // 8)]))
    fmt = rng.choice(["token", "token", "tensor", "tensor_vt", "mxfp4"])
    if fmt.endswith("vt"):
        page = 128
    D = 128 if fmt == "mxfp4" else rng.choice([64, 128])
    T, G, Hk = rng.choice([1, 1, 2, 3, 4]), rng.choice([1, 4, 8, 12, 16]), rng.choice([1, 1, 2, 3, 8])
    B = _log(rng, 1, max(1, 4096 // (T * G * Hk)))
    prefix = _log(rng, 1, 32768)
    hi = _log(rng, T, max(T, min(4096, 131072 // (B * Hk))))
    window = rng.choice([0, 0, 0, rng.randint(1, prefix + hi)])
    return dict(op=op, B=B, T=T, H=G * Hk, Hk=Hk, D=D, page=page, prefix=prefix, lo=min(T, hi), hi=hi,
                window=window, fmt=fmt, pad=rng.choice([0, 0, B // 4]))


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randint(g, lo, hi, n):
    """n whole numbers in [lo, hi], int64."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda")


def prepare(case, seed):
    s = {"plan": _prepare_plan, "append": _prepare_append, "shared": _prepare_shared}[case["op"]](case, _gen(seed))
    s["case"] = case
    if own:
        import quantized_attention_smoothing_b200 as sage
        s["sage"] = sage
        if "D" in case:
            s["h"] = sage.Hadamard(case["D"])
        if case["op"] == "shared":
            n = sage.sage_attn_decode_shared_workspace(case["B"], case["T"], case["H"], case["Hk"], case["D"])
            s["ws"] = torch.empty((n,), dtype=torch.uint8, device="cuda")
    return s


def _prepare_plan(c, g):
    B, page, mp, pp = c["B"], c["page"], c["max_pages"], c["prefix_pages"]
    P, cap = pp * page, mp * page
    room = cap - P
    if c["mode"] == "prompt":                       # every request enters with its prompt
        cached = torch.zeros(B, dtype=torch.int64, device="cuda")
        new = _randint(g, 1, room, B)
    else:
        new = _randint(g, 1, min(c["T"], room), B)
        cached = P + (torch.rand(B, generator=g, device="cuda") * (room - new)).long()
        if c["mode"] == "mixed":                    # one in eight ends, joins with a prompt, or waits
            kind = _randint(g, 0, 23, B)
            new = torch.where(kind == 0, -1, new)
            cached = torch.where(kind == 1, 0, cached)
            new = torch.where(kind == 1, 1 + (new * 37) % min(512, room), new)
            new = torch.where(kind == 2, 0, new)
        if not pp:
            cached = torch.where(cached == 0, (new < 0).long(), cached)
    held = (cached + page - 1) // page
    mine = torch.arange(mp, device="cuda")[None] < held[:, None]
    mine[:, :pp] = False                            # pages of its own, behind the prefix
    total = pp + 2 * B * mp                         # the cache's pages: held, shared or free
    perm = torch.randperm(total, generator=g, device="cuda").int()
    table = torch.zeros((B, mp), dtype=torch.int32, device="cuda")
    n = int(mine.sum())
    table[mine] = perm[:n]
    prefix = perm[n:n + pp].clone()
    table[:, :pp] = torch.where((cached > 0)[:, None], prefix[None], 0)
    free = torch.zeros(total, dtype=torch.int32, device="cuda")
    free[:total - n - pp] = perm[n + pp:]
    return dict(cached=cached.int(), new=new.int(), table=table, prefix=prefix, free=free,
                count=torch.tensor([total - n - pp], dtype=torch.int32, device="cuda"),
                ctx=torch.zeros(B, dtype=torch.int32, device="cuda"),
                count_out=torch.zeros(1, dtype=torch.int32, device="cuda"),
                offsets=torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
                slots=torch.zeros(_slot_room(c), dtype=torch.int32, device="cuda"))


def _slot_room(c):
    """The slot map's length: a program keeps one that its largest step fits."""
    if c["mode"] == "prompt":
        return c["B"] * (c["max_pages"] - c["prefix_pages"]) * c["page"]
    return c["B"] * c["T"] if c["mode"] == "step" else 16 * c["B"] + 1200


def _mx_draw(g, shape, lo, hi):
    """Random E2M1 codes, two a byte, and e8m0 scales of 2^lo .. 2^hi."""
    codes = torch.randint(0, 256, shape[:-1] + (shape[-1] // 2,), generator=g, device="cuda").to(torch.uint8)
    sf = torch.randint(127 + lo, 128 + hi, shape[:-1] + (shape[-1] // 32,), generator=g, device="cuda").to(torch.uint8)
    return codes, sf


def _prepare_append(c, g):
    N, Hk, D, page, fmt = c["N"], c["Hk"], c["D"], c["page"], c["fmt"]
    # the projection's output: [N, heads, D] slices of one row of K and V heads
    kv = torch.randn((N, 2 * Hk, D), generator=g, device="cuda")
    bias = 2.0 * torch.randn((Hk, D), generator=g, device="cuda")
    kv[:, :Hk] += bias
    kv = kv.to(torch.bfloat16)
    pages = (N + page - 1) // page + 5
    order = torch.randperm(pages, generator=g, device="cuda")
    at = 3 + torch.arange(N, device="cuda")         # a context that goes on at its fourth token
    slots = (order[at // page] * page + at % page).int()
    if c["pad"]:
        slots[N - c["pad"]:] = -1                   # a padded batch
    s = dict(k=kv[:, :Hk], v=kv[:, Hk:], mean=(bias + 0.1 * torch.randn((Hk, D), generator=g, device="cuda")),
             slots=slots)
    if fmt == "mxfp4":
        s["kc"], s["ksf"] = _mx_draw(g, (pages, Hk, page, D), -2, 1)
        s["vc"], s["vsf"] = _mx_draw(g, (pages, Hk, page, D), -2, 1)
        return s
    for n in ("kc", "vc"):
        s[n] = torch.randint(0, 120, (pages, Hk, page, D), generator=g, device="cuda").to(torch.uint8)
    if fmt.endswith("vt"):
        s["vc"] = s["vc"].transpose(2, 3).contiguous()
    if fmt.startswith("tensor"):                    # calibrated: the largest values saturate now and then
        s["ks"] = torch.full((1,), 4.5 * math.sqrt(D) / E4M3_MAX, device="cuda")
        s["vs"] = torch.full((1,), 4.5 / E4M3_MAX, device="cuda")
    else:
        s["ks"] = torch.rand((pages, Hk, page), generator=g, device="cuda") + 0.01
        s["vs"] = torch.rand((pages, Hk, page), generator=g, device="cuda") + 0.01
    return s


def _fp8_draw(g, shape, std, tensor):
    """Codes and scales of N(0, std^2) rows as e4m3, one scale a token or one in all."""
    x = std * torch.randn(shape, generator=g, device="cuda")
    a = x.abs().amax() if tensor else x.abs().amax(dim=-1)
    scale = a / E4M3_MAX
    codes = (x / (scale if tensor else scale[..., None])).clamp(-E4M3_MAX, E4M3_MAX)
    return codes.to(torch.float8_e4m3fn).view(torch.uint8), scale.reshape(1) if tensor else scale


def _prepare_shared(c, g):
    B, T, H, Hk, D, page, L = (c[n] for n in ("B", "T", "H", "Hk", "D", "page", "prefix"))
    ctx = L + _randint(g, c["lo"], c["hi"], B)
    if c["pad"]:
        ctx[B - c["pad"]:] = 0                      # a padded batch: these rows see nothing
    lp, whole = (L + page - 1) // page, L // page   # a prefix may end inside a page of its own copy
    mp = (L + c["hi"] + page - 1) // page
    need = ((ctx + page - 1) // page - whole).clamp(min=0)
    base = lp + torch.cumsum(need, 0) - need
    total = lp + int(need.sum())
    perm = torch.randperm(total, generator=g, device="cuda").int()
    e = torch.arange(mp, device="cuda")[None]
    table = perm[(base[:, None] + e - whole).clamp(0, total - 1)]
    table = torch.where(e < whole, perm[e.clamp(max=lp - 1)], table)
    table = torch.where(e < ((ctx + page - 1) // page)[:, None], table, 0).contiguous()
    s = dict(prefix=perm[:lp].clone(), table=table, ctx=ctx.int(), pages=total,
             length=torch.tensor([L], dtype=torch.int32, device="cuda"),
             window=c["window"] or L + c["hi"] + 1, scale=1.0 / math.sqrt(D),
             q=torch.randn((B, T, H, D), generator=g, device="cuda").to(torch.bfloat16),
             out=torch.empty((B, T, H, D), dtype=torch.bfloat16, device="cuda"))
    shape = (total, Hk, page, D)
    # keys as the rotation leaves them: sqrt(D) times the head's own spread
    if c["fmt"] == "mxfp4":
        s["kc"], s["ksf"] = _mx_draw(g, shape, 0, 3)
        s["vc"], s["vsf"] = _mx_draw(g, shape, -3, 0)
    else:
        tensor = c["fmt"].startswith("tensor")
        s["kc"], s["ks"] = _fp8_draw(g, shape, math.sqrt(D), tensor)
        s["vc"], s["vs"] = _fp8_draw(g, shape, 1.0, tensor)
        if c["fmt"].endswith("vt"):
            s["vc"] = s["vc"].transpose(2, 3).contiguous()
    return s


# ------------------------------------------------------------- plain forms

def _butterfly(x):
    """x H along the last dimension, H the Sylvester matrix: stages of sums
    and differences, each rounded to 32 bits as the format's definition says."""
    D, h = x.shape[-1], 1
    while h < D:
        y = x.reshape(x.shape[:-1] + (D // (2 * h), 2, h))
        x = torch.stack((y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]), dim=-2).reshape(x.shape)
        h *= 2
    return x


def _e4m3_rows(x):
    """(codes as float8, scale) of each row: scale max|x| / 448."""
    a = x.abs().amax(dim=-1)
    r = torch.where(a > 0, E4M3_MAX / a, 0.0)
    return (x * r[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), a / E4M3_MAX


def _e2m1_rows(x):
    """(packed E2M1 codes, e8m0 bytes) of rows in blocks of 32."""
    b = x.reshape(x.shape[:-1] + (x.shape[-1] // 32, 32))
    a = b.abs().amax(dim=-1)
    E = torch.where(a > 0, torch.frexp(a)[1] - 3, -127).clamp(-127, 125)
    m = torch.ldexp(b.abs(), -E[..., None])
    code = ((m > 0.25).int() + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
            + 8 * (b < 0)).reshape(x.shape)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), (E + 127).to(torch.uint8)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mx_bf16(codes, sf):
    """The values that an MXFP4 cache stands for, bf16 (exact)."""
    v = torch.tensor(_E2M1, device=codes.device)
    v = torch.cat((v, -v)).to(torch.bfloat16)
    pairs = torch.stack((v.repeat(16), v.repeat_interleave(16)), dim=-1).view(torch.int32).reshape(-1)
    x = pairs[codes.int()].view(torch.bfloat16)
    e = (sf.short() << 7).view(torch.bfloat16)      # 2^(sf - 127)
    return (x.reshape(e.shape + (32,)) * e[..., None]).reshape(x.shape)


def _plain_plan(s):
    c = s["case"]
    page, pp, mp, B = c["page"], c["prefix_pages"], c["max_pages"], c["B"]
    cached, new, table, free = s["cached"].long(), s["new"].long(), s["table"], s["free"]
    fc = s["count"].long()
    ended, joins = new < 0, (cached == 0) & (new > 0)
    start = torch.where(joins, pp * page, cached)
    add = new.clamp(min=0)
    ctx = torch.where(ended, 0, start + add)
    held = (start + page - 1) // page
    need = torch.where(ended, 0, (ctx + page - 1) // page - held)
    gone = torch.where(ended, (held - pp).clamp(min=0), 0)
    need_to, gone_to, token_to = torch.cumsum(need, 0), torch.cumsum(gone, 0), torch.cumsum(add, 0)
    na, nf = need_to[-1:], gone_to[-1:]
    e = torch.arange(mp, device=table.device)[None]
    # the pages given back go on top of the list, and the new ones come off its top
    gives = ended[:, None] & (e >= pp) & (e < held[:, None])
    nowhere = free.numel()
    stack = torch.cat((free, free[:1]))
    put = torch.where(gives, fc + (gone_to - gone)[:, None] + e - pp, nowhere)
    stack.scatter_(0, put.reshape(-1), table.reshape(-1))
    k = (need_to - need)[:, None] + e - held[:, None]
    takes = (e >= held[:, None]) & (e < (held + need)[:, None])
    got = stack[(fc + nf - 1 - k).clamp(0, nowhere - 1)]
    table = torch.where(takes, got, torch.where(joins[:, None] & (e < pp), _padded(s["prefix"], mp)[None], table))
    at = torch.arange(nowhere, device=free.device)
    free = torch.where((at >= fc) & (at < fc + nf - na), stack[:-1], free)
    t = torch.arange(s["slots"].numel(), device=table.device)
    b = torch.searchsorted(token_to, t, right=True).clamp(max=B - 1)
    pos = start[b] + t - (token_to - add)[b]
    slots = table[b, (pos // page).clamp(max=mp - 1)].long() * page + pos % page
    slots = torch.where(t < token_to[-1:], slots, -1)
    offsets = torch.cat((torch.zeros_like(fc), token_to))
    s["table"].copy_(table)
    s["free"].copy_(free)
    return [s["table"], s["free"], ctx.int(), (fc + nf - na).int(), offsets.int(), slots.int()]


def _padded(x, n):
    return torch.cat((x, torch.zeros(n - x.numel(), dtype=x.dtype, device=x.device)))


def _plain_append(s):
    c = s["case"]
    page, fmt = c["page"], c["fmt"]
    slot = s["slots"].long()
    # a token without a slot writes what the first one that has a slot writes
    i = torch.where(slot >= 0, torch.arange(c["N"], device=slot.device), torch.argmax((slot >= 0).int()))
    slot = slot[i]
    pg, off, hh = (slot // page)[:, None], (slot % page)[:, None], torch.arange(c["Hk"], device=slot.device)[None]
    xk, xv = _butterfly(s["k"].float() - s["mean"]), s["v"].float()
    if fmt == "mxfp4":
        for n, x in (("k", xk), ("v", xv)):
            codes, sf = _e2m1_rows(x)
            s[n + "c"][pg, hh, off] = codes[i]
            s[n + "sf"][pg, hh, off] = sf[i]
        return _append_outputs(s)
    if fmt.startswith("tensor"):
        ck, cv = ((x * (1.0 / t)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
                  for x, t in ((xk, s["ks"]), (xv, s["vs"])))
    else:
        (ck, sk), (cv, sv) = _e4m3_rows(xk), _e4m3_rows(xv)
        s["ks"][pg, hh, off], s["vs"][pg, hh, off] = sk[i], sv[i]
    s["kc"][pg, hh, off] = ck.view(torch.uint8)[i]
    if fmt.endswith("vt"):
        s["vc"].transpose(2, 3)[pg, hh, off] = cv.view(torch.uint8)[i]
    else:
        s["vc"][pg, hh, off] = cv.view(torch.uint8)[i]
    return _append_outputs(s)


def _append_outputs(s):
    if s["case"]["fmt"] == "mxfp4":
        return [_mx_bf16(s["kc"], s["ksf"]), _mx_bf16(s["vc"], s["vsf"])]
    return [s["kc"].view(torch.float8_e4m3fn), s["vc"].view(torch.float8_e4m3fn), s["ks"], s["vs"]]


def _cache_rows(s, name, pages):
    """The cache's values in 32 bits, scales applied, of `pages` [...]: [..., Hk, page, D]."""
    c, codes = s["case"], s[name + "c"][pages]
    if c["fmt"] == "mxfp4":
        return _mx_bf16(codes, s[name + "sf"][pages]).float()
    x = codes.view(torch.float8_e4m3fn).float()
    if name == "v" and c["fmt"].endswith("vt"):
        x = x.transpose(-1, -2)
    scale = s[name + "s"]
    return x * (scale if c["fmt"].startswith("tensor") else scale[pages][..., None])


def _plain_shared(s):
    c = s["case"]
    B, T, H, Hk, D, page, L = (c[n] for n in ("B", "T", "H", "Hk", "D", "page", "prefix"))
    G = H // Hk
    codes, sq = _e4m3_rows(_butterfly(s["q"].float()))
    q = codes.float() * (sq * (s["scale"] / D))[..., None]
    q = q.reshape(B, T, Hk, G, D).permute(2, 0, 1, 3, 4)                      # [Hk, B, T, G, D]
    pos = s["ctx"].long()[:, None] - T + torch.arange(T, device=q.device)[None]   # [B, T]
    # the prefix's keys once for the rows of every sequence
    kp, vp = (_cache_rows(s, n, s["prefix"].long()).permute(1, 0, 2, 3).reshape(Hk, -1, D)[:, :L] for n in "kv")
    sp = (q.reshape(Hk, -1, D) @ kp.transpose(1, 2)).reshape(Hk, B, T, G, L)
    # each sequence's own keys, those of [L, ctx)
    first = L // page
    own_pages = s["table"][:, first:].long()
    ko, vo = (_cache_rows(s, n, own_pages).permute(2, 0, 1, 3, 4).reshape(Hk, B, -1, D) for n in "kv")
    so = torch.einsum("hbtgd,hbkd->hbtgk", q, ko)
    j = torch.arange(L, device=q.device)
    jo = first * page + torch.arange(so.shape[-1], device=q.device)

    def seen(j):
        return (j <= pos[..., None]) & (j > pos[..., None] - s["window"])     # [B, T, keys]
    sp = sp.masked_fill_(~seen(j)[:, :, None], NEG_INF)
    so = so.masked_fill_(~(seen(jo) & (jo >= L))[:, :, None], NEG_INF)
    m = torch.maximum(sp.amax(-1), so.amax(-1))[..., None]
    m = torch.where(m == NEG_INF, 0.0, m)
    sp, so = sp.sub_(m).exp_(), so.sub_(m).exp_()
    den = sp.sum(-1) + so.sum(-1)
    # slots behind a sequence's end may hold anything: they weigh nothing
    o = (sp.reshape(Hk, -1, L) @ vp).reshape(Hk, B, T, G, D) + torch.einsum("hbtgk,hbkd->hbtgd", so, vo)
    o = torch.where(den[..., None] > 0, o / den[..., None], 0.0)
    s["out"].copy_(o.permute(1, 2, 0, 3, 4).reshape(B, T, H, D))
    return s["out"]


# ----------------------------------------------------------------- one pass

def run(s):
    if own:
        return _own(s)
    return {"plan": _plain_plan, "append": _plain_append, "shared": _plain_shared}[s["case"]["op"]](s)


def _own(s):
    sage, c = s["sage"], s["case"]
    if c["op"] == "plan":
        sage.sage_page_plan(s["cached"], s["new"], s["free"], s["count"], c["page"], s["table"], s["ctx"],
                            s["count_out"], s["offsets"], s["slots"],
                            prefix_table=s["prefix"] if c["prefix_pages"] else None)
        return [s["table"], s["free"], s["ctx"], s["count_out"], s["offsets"], s["slots"]]
    if c["op"] == "append":
        if c["fmt"] == "mxfp4":
            sage.sage_kv_append_mxfp4(s["h"], s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ksf"], s["vsf"],
                                      k_mean=s["mean"])
        else:
            sage.sage_kv_append(s["h"], s["k"], s["v"], s["slots"], s["kc"], s["vc"], s["ks"], s["vs"],
                                k_mean=s["mean"], kv_flags=_flags(sage, c))
        return _append_outputs(s)
    if c["fmt"] == "mxfp4":
        sage.sage_attn_decode_shared_mxfp4(s["h"], s["q"], s["kc"], s["vc"], s["ksf"], s["vsf"], s["prefix"],
                                           s["length"], s["table"], s["ctx"], c["page"], s["pages"], s["window"],
                                           s["scale"], s["out"], s["ws"])
    else:
        sage.sage_attn_decode_shared(s["h"], s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["prefix"], s["length"],
                                     s["table"], s["ctx"], c["page"], s["pages"], s["window"], s["scale"], s["out"],
                                     s["ws"], kv_flags=_flags(sage, c))
    return s["out"]


def _flags(sage, c):
    return ((sage.SAGE_KV_PER_TENSOR_SCALES if c["fmt"].startswith("tensor") else 0)
            | (sage.SAGE_KV_V_TRANSPOSED if c["fmt"].endswith("vt") else 0))


# -------------------------------------------------------------------- work

_CACHE_BYTES = {"token": (1.0, 4), "token_vt": (1.0, 4), "tensor": (1.0, 0), "tensor_vt": (1.0, 0),
                "mxfp4": (0.5 + 1.0 / 32, 0)}       # bytes a value, bytes a token and head


def work(c):
    if c["op"] == "plan":
        B, page, mp, pp = c["B"], c["page"], c["max_pages"], c["prefix_pages"]
        room = (mp - pp) * page
        tokens = _slot_room(c)
        pages = B * room / 2 / page if c["mode"] == "prompt" else B * (0.2 + 0.5 * mp / 24 * (c["mode"] == "mixed"))
        return dict(bytes=4 * (4 * B + tokens + 2 * pages), flops=0)
    per, tok = _CACHE_BYTES[c["fmt"]]
    if c["op"] == "append":
        n = (c["N"] - c["pad"]) * c["Hk"]
        return dict(bytes=2 * n * (2 * c["D"] + per * c["D"] + tok) + 4 * c["N"] + 4 * c["Hk"] * c["D"],
                    flops=n * c["D"] * (math.log2(c["D"]) + 6))
    live, W = c["B"] - c["pad"], c["window"] or 1 << 40
    mean = (c["lo"] + c["hi"]) / 2
    mine = min(mean, W)
    pref = max(0.0, min(c["prefix"], W - mean)) if W < c["prefix"] + mean else c["prefix"]
    reach = c["prefix"] if live and W >= c["prefix"] + c["lo"] else max(0.0, min(c["prefix"], W - c["lo"]))
    keys = c["Hk"] * (reach + live * mine)
    rows = live * c["T"] * c["H"]
    return dict(bytes=2 * keys * (per * c["D"] + tok) + 4 * c["B"] * c["T"] * c["H"] * c["D"],
                flops=4.0 * rows * c["D"] * (pref + mine))


# ------------------------------------------------- the definition in 64 bits

def _sylvester(D):
    i = torch.arange(D, device="cuda")
    bits = i[:, None] & i[None]
    odd = torch.zeros_like(bits)
    for n in range(7):
        odd ^= (bits >> n) & 1
    return 1.0 - 2.0 * odd.double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None                                 # whole numbers
    return _exact_append(case, s) if case["op"] == "append" else _exact_shared(case, s)


def _exact_fp4(x):
    """Each block of 32 rounded to E2M1 times 2^floor(log2 of its largest / 4)."""
    b = x.unflatten(-1, (-1, 32))
    unit = torch.exp2(torch.floor(torch.log2(b.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100))) - 2)
    m = (b / unit).abs().clamp(max=6.0)
    step = torch.exp2(torch.floor(torch.log2(m.clamp(min=1.0))) - 1)
    return (torch.sign(b) * torch.round(m / step) * step * unit).flatten(-2)


def _mx_values(codes, sf):
    n = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).long()
    mag, e = (n & 1).double(), (n >> 1) & 3
    v = torch.where(e > 0, (1 + mag / 2) * torch.exp2(e.double() - 1), mag / 2)
    return torch.where(n >= 8, -v, v) * torch.exp2(sf.double() - 127).repeat_interleave(32, dim=-1)


def _exact_append(c, s):
    page, fmt = c["page"], c["fmt"]
    ok = s["slots"] >= 0
    slot = s["slots"][ok].long()
    pg, off = slot // page, slot % page
    xk = (s["k"][ok].double() - s["mean"].double()) @ _sylvester(c["D"])
    xv = s["v"][ok].double()
    outs = []
    if fmt == "mxfp4":
        for n, x in (("k", xk), ("v", xv)):
            y = _mx_values(s[n + "c"], s[n + "sf"])
            y[pg, :, off] = _exact_fp4(x)
            outs.append(y)
        return outs
    scales = []
    for n, x in (("k", xk), ("v", xv)):
        y = s[n + "c"].view(torch.float8_e4m3fn).double()
        t = s[n + "s"].double()
        if fmt.startswith("tensor"):
            z = (x / t).clamp(-E4M3_MAX, E4M3_MAX)
        else:
            t[pg, :, off] = x.abs().amax(-1) / E4M3_MAX
            z = x * (E4M3_MAX / x.abs().amax(-1, keepdim=True))
        if n == "v" and fmt.endswith("vt"):
            y.transpose(2, 3)[pg, :, off] = z
        else:
            y[pg, :, off] = z
        outs.append(y)
        scales.append(t)
    return outs + scales


def _exact_shared(c, s):
    B, T, H, Hk, D, page = (c[n] for n in ("B", "T", "H", "Hk", "D", "page"))
    if c["fmt"] == "mxfp4":
        K, V = _mx_values(s["kc"], s["ksf"]), _mx_values(s["vc"], s["vsf"])
    else:
        K, V = s["kc"].view(torch.float8_e4m3fn).double(), s["vc"].view(torch.float8_e4m3fn).double()
        if c["fmt"].endswith("vt"):
            V = V.transpose(2, 3)
        if c["fmt"].startswith("tensor"):
            K, V = K * s["ks"].double(), V * s["vs"].double()
        else:
            K, V = K * s["ks"].double()[..., None], V * s["vs"].double()[..., None]
    x = s["q"].double() @ _sylvester(D)
    a = x.abs().amax(-1, keepdim=True)
    q = (x * (E4M3_MAX / a)).float().to(torch.float8_e4m3fn).double() * (a / E4M3_MAX)   # the query is held in 8 bits
    out = torch.zeros((B, T, H, D), dtype=torch.float64, device="cuda")
    ctxs = s["ctx"].tolist()
    for b in range(B):
        ctx = ctxs[b]
        lo = max(0, ctx - T + 1 - s["window"])
        n = ctx - lo
        if n <= 0:
            continue
        j = torch.arange(lo, ctx, device="cuda")
        # the prefix's tokens by the prefix's table, the others by the sequence's own
        pref = s["prefix"][(j // page).clamp(max=s["prefix"].numel() - 1)]
        pg = torch.where(j < c["prefix"], pref, s["table"][b][j // page]).long()
        k, v = K[pg, :, j % page].transpose(0, 1), V[pg, :, j % page].transpose(0, 1)    # [Hk, n, D]
        pos = ctx - T + torch.arange(T, device="cuda")
        hid = (j[None] > pos[:, None]) | (j[None] <= pos[:, None] - s["window"])         # [T, n]
        z = torch.einsum("thgd,hnd->htgn", q[b].reshape(T, Hk, H // Hk, D), k) * (s["scale"] / D)
        p = torch.softmax(z.masked_fill(hid[None, :, None], NEG_INF), dim=-1)
        p = torch.nan_to_num(p, nan=0.0)
        out[b] = torch.einsum("htgn,hnd->thgd", p, v).reshape(T, H, D)
    return out
