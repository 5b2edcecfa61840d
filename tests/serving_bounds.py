"""A 64-bit reference of the shared-prefix decode with the bound that the
kernels' own roundings give, cache format by cache format."""
import numpy as np
import torch

import oracle
import serving_helpers as sh
import workloads


def offset_logits(B, T, H, Hk, D, page, prefix, ctx, seed, fmt, offset, spread=1.0):
    """serving_helpers.make_shared with logits around `offset` (natural units,
    softmax scale 1 / sqrt(D)) of a standard deviation of about `spread`: the
    queries have a common part 2 u, the keys a multiple of the rotated u."""
    d = sh.make_shared(B, T, H, Hk, D, page, prefix, ctx, seed, fmt)
    g = torch.Generator().manual_seed(seed + 1)
    u = torch.randint(0, 2, (D,), generator=g).float() * 2 - 1
    q = torch.randn((B, T, H, D), generator=g)
    d["q"] = (q + 2 * u).to(torch.bfloat16)
    # q_hat . k_hat = D (q . k); q . u is about 2 D, |q| about sqrt(5 D)
    Hu = torch.from_numpy(oracle.fwht_f32(u.numpy()[None]).astype(np.float32))[0]
    shape = (d["pages"], Hk, page, D)
    x = spread * (D / 5) ** 0.5 * torch.randn(shape, generator=g) + offset / (2 * D ** 0.5) * Hu
    if fmt == "mxfp4":
        c, s = sh.ref_append_mx(x.numpy())
        d["kc"], d["ks"] = torch.from_numpy(c), torch.from_numpy(s)
    else:
        tensor = fmt.startswith("tensor")
        a = x.abs().amax() if tensor else x.abs().amax(-1)
        d["ks"] = (a / 448.0).reshape(1) if tensor else a / 448.0
        d["kc"] = (x / (d["ks"] if tensor else d["ks"][..., None])).clamp(-448, 448) \
            .to(torch.float8_e4m3fn).view(torch.uint8)
    return d


def bound_shared(d, window, scale):
    """(out, tol, mean logit) in 64 bits; out and tol [B, T, H, D].

    With w the weights, w = exp(x - max) / their sum, the kernels round
      logits: as serving_helpers.ref_shared, e = 2^-17 of the largest sum
        |q k| and 2^-20 (max |x| + 1); a weight and the denominator move by e;
      weights: FP8 cache fp16, as are the value's scale and the scaled value
        (3 times 2^-11), MXFP4 cache bf16 (2^-8);
      fp16 has a smallest step: weights are held against a maximum that is at
        most 2^8 below the row's own and for which the row's weights add up to
        1 or more, so each is off by at most 2^-25 of the denominator; a scaled
        value, in units of at most twice the largest scale of a run of keys, by
        2^-24 of that scale, and where the scale is multiplied into the weight
        instead, each product of the two by as much times the value's code;
      sums: n / 16 steps of an fp32 accumulator and n / 4 of the denominator's,
        2^-24 each and as much for alignment: below n 2^-24 of sum w |v|;
      the output: bf16, 2^-8 of it."""
    B, T, H, D = d["q"].shape
    K, V = sh.cache_values(d, "k"), sh.cache_values(d, "v")
    Hk, page = K.shape[1], K.shape[2]
    G, L, mx = H // Hk, int(d["length"][0]), d["fmt"] == "mxfp4"
    if not mx:
        smax = float(d["vs"][torch.isfinite(d["vs"])].max())
        C = np.abs(oracle.e4m3_decode(d["vc"].numpy()))
        C = C.swapaxes(2, 3) if d["fmt"].endswith("vt") else C
    codes, qs = oracle.decode_quant_q(workloads.bits_u16(d["q"]))
    q = oracle.e4m3_decode(codes) * qs.astype(np.float64)[..., None]
    out, tol, logits = np.zeros((B, T, H, D)), np.full((B, T, H, D), 1e-30), []
    table, prefix = d["table"].numpy(), d["prefix"].numpy()
    for b in range(B):
        ctx = int(d["ctx"][b])
        j = np.arange(ctx)
        pg = np.where(j < L, prefix[np.minimum(j // page, len(prefix) - 1)], table[b][j // page]) if ctx else j
        for hk in range(Hk if ctx else 0):
            k, v = K[pg, hk, j % page], V[pg, hk, j % page]
            rows = q[b, :, hk * G:(hk + 1) * G].reshape(T * G, D)
            x = rows @ k.T * (scale / D)
            mag = (np.abs(rows) @ np.abs(k).T).max(-1) * (scale / D)
            pos = (ctx - T + np.arange(T)).repeat(G)[:, None]
            see = (j <= pos) & (j > pos - window)
            any_ = see.any(-1)
            logits.append(x[see])
            top = np.where(see, x, -np.inf).max(-1, keepdims=True)
            w = np.where(see, np.exp(np.where(see, x - np.where(any_[:, None], top, 0), 0)), 0)
            w /= np.maximum(w.sum(-1, keepdims=True), 1e-300)
            y = w @ v
            e = 2.0 ** -17 * mag + 2.0 ** -20 * (np.abs(np.where(see, x, 0)).max(-1) + 1)
            wv = w @ np.abs(v)
            rel = (2.0 ** -8 if mx else 3 * 2.0 ** -11) + 2 * e[:, None] + ctx * 2.0 ** -24
            t = rel * wv + 2.0 ** -8 * np.abs(y) + 1e-30
            if not mx:
                t = t + 2.0 ** -25 * (see @ np.abs(v)) + 2.0 ** -24 * smax * (1 + see @ C[pg, hk, j % page])
            sl = (b, slice(None), slice(hk * G, (hk + 1) * G))
            out[sl] = np.where(any_[:, None], y, 0).reshape(T, G, D)
            tol[sl] = np.where(any_[:, None], t, 1e-30).reshape(T, G, D)
    return out, tol, float(np.mean(np.concatenate(logits)))
