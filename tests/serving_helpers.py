"""Plain references of the paged-cache serving operators: the page plan as a
loop over the requests, the quantised cache write in fp32 steps (bit for bit)
and in 64 bits, and the attention of a batch that shares a prefix in 64
bits with the error that the kernels' roundings can make."""
import numpy as np
import torch

import oracle
import workloads


# ------------------------------------------------------------------- plan

def ref_plan(cached, new, free, count, page, table, max_tokens, prefix=()):
    """(page_table, free_list, ctx, count, offsets, slots), or None where the
    step is refused. Works on copies of numpy int arrays, request by request."""
    table, free = table.copy(), free.copy()
    B, max_pages = table.shape
    pp = len(prefix)
    cap = max_pages * page
    if not 0 <= count <= len(free):
        return None
    start, ctx = np.zeros(B, np.int64), np.zeros(B, np.int64)
    for b in range(B):
        have, add = int(cached[b]), int(new[b])
        start[b] = pp * page if have == 0 and add > 0 else have
        ctx[b] = 0 if add < 0 else start[b] + add
        if have < 0 or 0 < have < pp * page or start[b] > cap or ctx[b] > cap:
            return None
    stack = [int(x) for x in free[:count]]
    held = -(-start // page)
    for b in range(B):
        if new[b] < 0:
            stack += [int(x) for x in table[b, pp:held[b]]]
    need = [0 if new[b] < 0 else int(-(-ctx[b] // page) - held[b]) for b in range(B)]
    tokens = int(np.maximum(new, 0).sum())
    if sum(need) > len(stack) or len(stack) > len(free) or tokens > max_tokens:
        return None
    slots, offsets = np.full(max_tokens, -1, np.int64), np.zeros(B + 1, np.int64)
    t = 0
    for b in range(B):
        if cached[b] == 0 and new[b] > 0:
            table[b, :pp] = prefix
        for e in range(int(held[b]), int(held[b]) + need[b]):
            table[b, e] = stack.pop()
        offsets[b] = t
        for pos in range(int(start[b]), int(ctx[b])):
            slots[t] = int(table[b, pos // page]) * page + pos % page
            t += 1
    offsets[B] = t
    free[count:len(stack)] = stack[count:]
    return table, free, ctx, len(stack), offsets, slots


# ------------------------------------------------------------------- append

def rotated(k_bits, mean):
    """butterfly(K - mean) in fp32, the kernels' operations. k_bits uint16 [N, Hk, D]."""
    x = oracle.bf16_to_f32(k_bits).astype(np.float32)
    if mean is not None:
        x = x - mean.astype(np.float32)[None]
    return oracle.fwht_f32(x)


_E4M3 = np.array(sorted({v for v in oracle.e4m3_decode(np.arange(127, dtype=np.uint8))}))


def e4m3_codes(x):
    """e4m3 codes of fp32 values: nearest, ties to the even code, saturating.
    The positive values in code order are increasing, so the code is an index."""
    a = np.minimum(np.abs(x.astype(np.float64)), 448.0)
    hi = np.clip(np.searchsorted(_E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _E4M3[lo], _E4M3[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def ref_append_fp8(x, scale=None):
    """Codes and scales of rows x fp32 [..., D]: one scale a row, or the given one."""
    if scale is not None:
        return e4m3_codes(x * (np.float32(1.0) / np.float32(scale))), None
    a = np.abs(x).max(-1)
    with np.errstate(divide="ignore"):
        r = np.where(a > 0, np.float32(448.0) / a, np.float32(0)).astype(np.float32)
    codes = e4m3_codes(x * r[..., None])
    codes[a == 0] &= 128
    return codes, (a / np.float32(448.0)).astype(np.float32)


def ref_append_mx(x):
    """(packed E2M1 codes, e8m0 bytes) of rows x fp32 [..., D]."""
    b = x.reshape(x.shape[:-1] + (-1, 32)).astype(np.float64)
    a = np.abs(b).max(-1)
    with np.errstate(divide="ignore"):
        E = np.where(a >= 2.0 ** -126, np.floor(np.log2(np.maximum(a, 2.0 ** -126))) - 2, -127)
    E = np.clip(E, -127, 125)
    m = np.minimum(np.abs(b) * 2.0 ** -E[..., None], 6.0)
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
    hi = np.clip(np.searchsorted(grid, m), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dl, dh = m - grid[lo], grid[hi] - m
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = (code + 8 * np.signbit(b)).reshape(x.shape)
    code[np.repeat(a == 0, 32, axis=-1).reshape(x.shape)] = 0
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), (E + 127).astype(np.uint8)


# --------------------------------------------------------- shared attention

def make_shared(B, T, H, Hk, D, page, prefix, ctx, seed, fmt="token", k_std=None):
    """A batch behind a prefix of `prefix` tokens: ctx[b] tokens in all (0: an
    empty row). CPU tensors; every sequence's own pages start at the page that
    holds token `prefix`, the unread entries of its table are poisoned."""
    g = torch.Generator().manual_seed(seed)
    lp, whole = -(-prefix // page), prefix // page
    need = [max(0, -(-c // page) - whole) for c in ctx]
    total = lp + sum(need) + 2
    perm = torch.randperm(total, generator=g).int()
    mp = max([1] + [-(-c // page) for c in ctx])
    table = torch.full((B, mp), 1 << 30, dtype=torch.int32)
    o = lp
    for b in range(B):
        table[b, whole:whole + need[b]] = perm[o:o + need[b]]
        o += need[b]
    d = dict(prefix=perm[:max(lp, 1)].clone(), table=table, ctx=torch.tensor(ctx, dtype=torch.int32), pages=total,
             length=torch.tensor([prefix], dtype=torch.int32), fmt=fmt,
             q=torch.randn((B, T, H, D), generator=g).to(torch.bfloat16))
    shape = (total, Hk, page, D)
    if fmt == "mxfp4":
        for n, lo in (("k", -1), ("v", -3)):
            d[n + "c"] = torch.randint(0, 256, shape[:-1] + (D // 2,), generator=g).to(torch.uint8)
            d[n + "s"] = torch.randint(127 + lo, 131 + lo, shape[:-1] + (D // 32,), generator=g).to(torch.uint8)
        return d
    for n, std in (("k", D ** 0.5 if k_std is None else k_std), ("v", 1.0)):
        x = std * torch.randn(shape, generator=g)
        a = x.abs().amax() if fmt.startswith("tensor") else x.abs().amax(-1)
        d[n + "s"] = (a / 448.0).reshape(1) if fmt.startswith("tensor") else a / 448.0
        d[n + "c"] = (x / (d[n + "s"] if fmt.startswith("tensor") else d[n + "s"][..., None])) \
            .clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    if fmt.endswith("vt"):
        d["vc"] = d["vc"].transpose(2, 3).contiguous()
    return d


def cache_values(d, n):
    """fp64 values [pages, Hk, page, D] of a cache."""
    c, s = d[n + "c"].numpy(), d[n + "s"].numpy()
    if d["fmt"] == "mxfp4":
        x = np.stack((oracle.e2m1_decode(c & 15), oracle.e2m1_decode(c >> 4)), -1).reshape(c.shape[:-1] + (-1,))
        return x * np.repeat(2.0 ** (s.astype(np.float64) - 127), 32, axis=-1)
    x = oracle.e4m3_decode(c)
    if n == "v" and d["fmt"].endswith("vt"):
        x = x.swapaxes(2, 3)
    return x * (float(s[0]) if d["fmt"].startswith("tensor") else s.astype(np.float64)[..., None])


def ref_shared(d, window, scale):
    """(out, tol) fp64 [B, T, H, D]. The kernels hold S, the softmax statistics
    and O in fp32 and round twice: every product of a weight and a value (to
    bf16, at most half a step, 2^-8 of it; or in fp16 the weight, the value's
    scale and the scaled value, 3 times 2^-11) and the output (2^-8). Logits are
    fp32 sums of 128 exact products: an error of 2^-17 of sum |q k| each, and
    2^-20 for their scaling and the exponential, which moves a weight and the
    denominator by as much. So |error| <= (2^-8 + 2 e) sum p |v| + 2^-8 |y|."""
    B, T, H, D = d["q"].shape
    K, V = cache_values(d, "k"), cache_values(d, "v")
    Hk, page = K.shape[1], K.shape[2]
    G, L = H // Hk, int(d["length"][0])
    codes, qs = oracle.decode_quant_q(workloads.bits_u16(d["q"]))
    q = oracle.e4m3_decode(codes) * qs.astype(np.float64)[..., None]
    out, tol = np.zeros((B, T, H, D)), np.full((B, T, H, D), 1e-30)
    for b in range(B):
        ctx = int(d["ctx"][b])
        j = np.arange(ctx)
        if ctx == 0:
            continue
        pref = d["prefix"].numpy()[np.minimum(j // page, d["prefix"].numel() - 1)]
        pg = np.where(j < L, pref, d["table"][b].numpy()[j // page])
        for h in range(H):
            k, v = K[pg, h // G, j % page], V[pg, h // G, j % page]
            for t in range(T):
                p = ctx - T + t
                see = (j <= p) & (j > p - window)
                if not see.any():
                    continue
                x = (k[see] @ q[b, t, h]) * (scale / D)
                mag = (np.abs(k[see]) @ np.abs(q[b, t, h])) * (scale / D)
                w = np.exp(x - x.max())
                w /= w.sum()
                out[b, t, h] = w @ v[see]
                e = 2.0 ** -17 * mag.max() + 2.0 ** -20 * (np.abs(x).max() + 1)
                tol[b, t, h] = (2.0 ** -8 + 2 * e) * (w @ np.abs(v[see])) + 2.0 ** -8 * np.abs(out[b, t, h]) + 1e-30
    return out, tol
