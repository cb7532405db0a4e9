"""Plain 64-bit references of the 8-bit cache and of attention over the paged
cache, on the CPU, with bounds on what a correct kernel may be off by."""
from __future__ import annotations

import math

import torch

# a weight's rounding as it enters the product with V (half a step, relative)
WEIGHT = {16: 2.0 ** -8, 8: 2.0 ** -11}


def quantise(x):
    """(codes int8, scale fp32) of rows x [..., d] bf16.  127 x / a in fp64
    lands on a half only if the exact quotient does (both have 8 bits: it is at
    least 2^-17 of itself away otherwise), and a / 127 in fp64 rounds to the
    same fp32 number as the exact one (53 >= 2 * 24 + 2 bits)."""
    x = x.double()
    a = x.abs().amax(-1)
    codes = torch.round(torch.where(a[..., None] > 0, 127 * x / a[..., None], torch.zeros_like(x)))
    scale = (a / 127).float()
    bad = ~torch.isfinite(x).all(-1)
    codes[bad] = 0
    scale[bad] = float("nan")
    return codes.to(torch.int8), scale


def values(codes, scale):
    """What codes and scales stand for, fp64."""
    return codes.double() * scale.double()[..., None]


def tree_masks(parents):
    """Words (as int64) of a tree: parents[i] < i, or -1 for a root."""
    words = []
    for i, p in enumerate(parents):
        words.append((words[p] if p >= 0 else 0) | 1 << i)
    return [w - (1 << 64) if w >> 63 else w for w in words]


def sight(start, n, words, window, sinks):
    """bool [n, start + n]: which keys each of n new tokens sees."""
    seen = torch.zeros(n, start + n, dtype=torch.bool)
    if words is None:
        place = [start + i for i in range(n)]
        kin = [list(range(i + 1)) for i in range(n)]
    else:
        kin = [[j for j in range(n) if words[i] >> j & 1] for i in range(n)]
        place = [start + sum(j != i for j in kin[i]) for i in range(n)]
    at = list(range(start)) + place
    for i in range(n):
        for j in list(range(start)) + [start + j for j in kin[i]]:
            seen[i, j] = window == 0 or at[j] > place[i] - window or at[j] < sinks
    return seen


def attention(k, v, q, table, cu, start, words=None, window=0, sinks=0, scale=None, bits=16, skipped=()):
    """(out, tol) fp64 of new tokens; k, v [pages, heads, page, d] (any dtype,
    the values themselves), words per token or None.

    tol counts the output's rounding to bf16 (half a step of the value), and,
    relative to sum w |v|: the weights' rounding (WEIGHT), the rounding of the
    scores (a dot product of d terms and the factors, 2^-24 (d + 6) of
    sum |q||k|, at each of numerator and denominator), the exponentials and
    rescalings (2^-20), and the sums over n keys (2 n 2^-24).  Weights in fp16
    below its normal range are off by 2^-29 of the largest |v|."""
    hkv, page, d = k.shape[1], k.shape[2], k.shape[3]
    hq = q.shape[1]
    g = hq // hkv
    scale = scale or 1.0 / math.sqrt(d)
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    for s in range(len(start)):
        n = cu[s + 1] - cu[s]
        if n == 0:
            continue
        end = start[s] + n
        seen = sight(start[s], n, None if words is None else words[cu[s]:cu[s + 1]], window, sinks)
        pages = table[s][:-(-end // page)]
        gone = torch.tensor([p in skipped for p in pages]).repeat_interleave(page)[:end]
        seen &= ~gone
        pages = [0 if p in skipped else p for p in pages]
        for h in range(hkv):
            kk = k[pages, h].double().reshape(-1, d)[:end]
            vv = v[pages, h].double().reshape(-1, d)[:end]
            # keys that no token sees hold anything
            alive = seen.any(0)
            kk, vv = (torch.where(alive[:, None], x, 0.0) for x in (kk, vv))
            for r in range(h * g, (h + 1) * g):
                qq = q[cu[s]:cu[s + 1], r].double()
                logit = (qq @ kk.T * scale).masked_fill(~seen, -math.inf)
                w = torch.softmax(logit, -1)
                w = torch.where(seen, w, 0.0)
                o, size = w @ vv, w @ vv.abs()
                slip = ((qq.abs() @ kk.abs().T).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
                        * scale * (d + 6) * 2.0 ** -24)
                rel = WEIGHT[bits] + 2 * slip + 2.0 ** -20 + 2 * end * 2.0 ** -24
                t = rel * size * 1.01
                if bits == 8:
                    t = t + end * 2.0 ** -29 * vv.abs().amax(0)
                out[cu[s]:cu[s + 1], r] = o
                tol[cu[s]:cu[s + 1], r] = t + 2.0 ** -8 * (o.abs() + t)
    return out, tol
