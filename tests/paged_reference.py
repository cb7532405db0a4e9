"""Plain 64-bit references of the rotary positions and of the paged cache's
operators, on the CPU, with bounds on what a correct kernel may be off by."""
from __future__ import annotations

import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def inv_freq(rot, theta=10000.0, scaling="none", factor=1.0, original=0.0, low=1.0, high=32.0):
    out = []
    base = theta * factor ** (rot / (rot - 2)) if scaling == "base" else theta
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f = f / factor
        if scaling == "parts":
            g = min(1.0, max(0.0, (original * f / (2 * math.pi) - low) / (high - low)))
            f = g * f + (1 - g) * f / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64)


def rope(x, positions, freq, interleaved, factor=1.0, sign=1.0):
    """x [batch, heads, n, d] of any dtype, positions [batch, n] integers.
    Returns (y, tol) in fp64; tol counts, per element, 2^-21 of m (|x_a| +
    |x_b|) for the angle (1.6 units of 2^-24), the sine (2), the factor (1)
    and the two products and their sum (2), the frequency's own rounding
    (2^-52 of the angle), and half a step of the output's type."""
    rot = 2 * freq.numel()
    xd = x.double().cpu()
    angle = sign * positions.double().cpu()[:, None, :, None] * freq
    c, s = factor * torch.cos(angle), factor * torch.sin(angle)
    y, size = xd.clone(), torch.zeros_like(xd)
    if interleaved:
        ia, ib = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    else:
        ia, ib = torch.arange(0, rot // 2), torch.arange(rot // 2, rot)
    a, b = xd[..., ia], xd[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    each = abs(factor) * (a.abs() + b.abs()) * (2.0 ** -21 + angle.abs() * 2.0 ** -51)
    size[..., ia], size[..., ib] = each, each
    tol = size + HALF_STEP[x.dtype] * (y.abs() + size)
    tol[..., rot:] = 0.0
    return y, tol


def append(k, v, kbar, new_k, new_v, cu, start, table):
    """The cache after an append: (k, v, kbar fp64, tolerance of kbar).  A mean
    of n terms is off by at most n + 1 roundings of 2^-24 of the mean of their
    sizes."""
    page = k.shape[2]
    k, v, kbar = k.clone(), v.clone(), kbar.double().clone()
    tol = torch.zeros_like(kbar)
    for s in range(len(start)):
        n = cu[s + 1] - cu[s]
        for i in range(n):
            p = start[s] + i
            k[table[s][p // page], :, p % page] = new_k[cu[s] + i]
            v[table[s][p // page], :, p % page] = new_v[cu[s] + i]
        if n == 0:
            continue
        for b in range(start[s] // page, (start[s] + n - 1) // page + 1):
            rows = min(page, start[s] + n - b * page)
            at = k[table[s][b], :, :rows].double()
            kbar[table[s][b]] = at.mean(1)
            tol[table[s][b]] = (rows + 1) * 2.0 ** -24 * at.abs().mean(1)
    return k, v, kbar, tol


def select(score, topk, own):
    """Ascending ids of the topk best of score [nb] (fp64; ties to the lower
    id, NaN as -inf), block `own` (or None) always among them."""
    s = [(-math.inf if x != x else x) for x in score.tolist()]
    order = sorted((b for b in range(len(s)) if b != own), key=lambda b: (-s[b], b))
    kept = order[:topk - (own is not None)] + ([] if own is None else [own])
    return sorted(kept)


def decode(k, v, kbar, q, table, lens, topk, token_seq=None, local=True, share=False, scale=None):
    """(out, tol, idx): fp64 attention of each token over its selected blocks.

    tol counts the output's rounding to bf16 (half a step of the value), and,
    relative to sum w |v|: P's rounding to bf16 (2^-8), the rounding of the
    scores (a dot product of d terms and the scaling, 2^-24 (d + 2) of
    sum |q||k|, at each of numerator and denominator), the exponentials and
    rescalings (2^-20), and the sums over n keys (2 n 2^-24)."""
    hkv, page, d = k.shape[1], k.shape[2], k.shape[3]
    tokens, hq = q.shape[0], q.shape[1]
    g = hq // hkv
    scale = scale or 1.0 / math.sqrt(d)
    out = torch.zeros(tokens, hq, d, dtype=torch.float64)
    tol = torch.zeros(tokens, hq, d, dtype=torch.float64)
    idx = torch.full((tokens, hkv if share else hq, topk), -1, dtype=torch.int32)
    qd = q.double().cpu()
    for t in range(tokens):
        n = int(lens[t])
        if n == 0:
            continue
        s = t if token_seq is None else int(token_seq[t])
        nb = -(-n // page)
        pages = table[s][:nb].tolist()
        own = nb - 1 if local else None
        for h in range(hkv):
            means = kbar[pages, h].double()                       # [nb, d]
            per_head = qd[t, h * g:(h + 1) * g] @ means.T
            rows = [qd[t, h * g:(h + 1) * g].sum(0) @ means.T] if share else list(per_head)
            for r, score in enumerate(rows):
                ids = select(score, topk, own) if nb > topk else list(range(nb))
                idx[t, h if share else h * g + r, :len(ids)] = torch.tensor(ids, dtype=torch.int32)
                kk = torch.cat([k[pages[b], h, :min(page, n - b * page)] for b in ids]).double()
                vv = torch.cat([v[pages[b], h, :min(page, n - b * page)] for b in ids]).double()
                for hh in (range(h * g, (h + 1) * g) if share else [h * g + r]):
                    logit = kk @ qd[t, hh] * scale
                    w = torch.softmax(logit, 0)
                    out[t, hh] = w @ vv
                    size = w @ vv.abs()
                    slip = (kk.abs() @ qd[t, hh].abs()).max() * scale * (d + 2) * 2.0 ** -24
                    rel = 2.0 ** -8 + 2 * float(slip) + 2.0 ** -20 + 2 * kk.shape[0] * 2.0 ** -24
                    tol[t, hh] = rel * size * 1.01
                    tol[t, hh] += 2.0 ** -8 * (out[t, hh].abs() + tol[t, hh])
    return out, tol, idx


def assert_within(got, ref, tol, what):
    got = got.double().cpu()
    off = (got - ref).abs()
    bad = ~(off <= tol + 1e-30)
    if bool(bad.any()):
        i = int(torch.where(bad, off / (tol + 1e-30), torch.zeros_like(off)).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; worst at {i}: "
                             f"{got.flatten()[i]:.6g} vs {ref.flatten()[i]:.6g} "
                             f"(tolerance {tol.flatten()[i]:.3g})")
