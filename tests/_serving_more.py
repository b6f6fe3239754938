"""Plain 64-bit forms of the serving calls over caches of 8 bits, with windows and shared prefixes, and their error bounds."""
from __future__ import annotations

import math

import torch

import _serving as R

D = 128
TOP = {torch.float8_e4m3fn: 448.0, torch.int8: 127.0}
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def quantise(x, kv):
    """(held values, scales) of rows, as the append's definition has them, in 64 bits up to the scale's rounding."""
    s = (x.double().abs().amax(-1) / TOP[kv]).float()
    y = x.double() / torch.where(s > 0, s, 1.0).double()[..., None]
    return (y.round() if kv == torch.int8 else y.float()).to(kv), s


def values(q, s, pages_first=True):
    """What a cache of 8 bits [N, page, Hkv, D] with scales [N, Hkv, page] stands for, in 64 bits."""
    return q.view(torch.int8).view(q.dtype).double() * s.double().transpose(1, 2)[..., None]


def make_cache(B, room, Hkv, page, kv, lens, seed, dtype=None, spread=3.0, behind=float("nan")):
    """A cache (CPU) whose first lens[b] rows of each sequence hold data; every other slot holds `behind` (in a cache of 8
    bits NaN codes and NaN scales), page numbers behind a sequence's last page are far out of range. Rows differ in size by
    up to 2^spread either way. Returns (k, v, pages, k_scale, v_scale), scales None unless of 8 bits."""
    held = kv in TOP
    k, v, pages = R.make_cache(B, room, Hkv, page, torch.float32 if held else kv, seed, fill=0.0 if held else behind)
    R.fill_prefix(k, v, pages, lens, seed + 1)
    if not held:
        return k, v, pages, None, None
    g = torch.Generator().manual_seed(seed + 2)
    out = []
    for x in (k, v):
        x = x * torch.exp2((torch.rand(*x.shape[:3], 1, generator=g) * 2 - 1) * spread)
        q, s = quantise(x, kv)
        s = s.transpose(1, 2).contiguous()
        there = torch.zeros(x.shape[0], page, dtype=torch.bool)
        for b, n in enumerate(lens):
            pg, row = R.slots(pages, page, b, torch.arange(n))
            there[pg, row] = True
        q.view(torch.int8)[~there] = 0x7F if kv == torch.float8_e4m3fn else 93
        s[(~there)[:, None].expand_as(s)] = behind
        out.append((q, s))
    return out[0][0], out[1][0], pages, out[0][1], out[1][1]


def positions(n, count, parents):
    """(position of each new row, truth values [count, count]: the new rows that each sees)."""
    see = torch.zeros(count, count, dtype=torch.bool)
    depth = []
    for i in range(count):
        up = i - 1 if parents is None else int(parents[i])
        up = up if -1 <= up < i else -1
        depth.append(0 if up < 0 else depth[up] + 1)
        if up >= 0:
            see[i] = see[up]
        see[i, i] = True
    return torch.tensor(depth) + n, see


def seen(n, count, parents, window, sinks):
    """[count, n + count] truth values: the keys that each row sees."""
    at, see = positions(n, count, parents)
    vis = torch.cat((torch.ones(count, n, dtype=torch.bool), see), 1)
    if window:
        key = torch.cat((torch.arange(n), at))
        vis &= (at[:, None] - key[None] < window) | (key < sinks)[None]
    return vis


def attention(q, k, v, pages, lens, counts, parents, window=0, sinks=0, scales=None, scale=None, room=None):
    """(o, lse, bound on |o|'s error, bound on lse's) in 64 bits; all inputs on the CPU, k and v as they lie in the cache.

    Per row the bounds count: the scores' fp32 sums of 128 products and their factors (140 roundings of 2^-24 of the terms'
    size, twice, and for q rows brought to fp16 by a power of two 2^-34 of the row's largest element), ex2's 2^-21, half a
    step of the 16-bit type that the weights are rounded to (fp16 over a cache of 8 bits, none with 32-bit rows), weights
    below fp16's range (half its smallest step, 2^-25, where the largest weight is 2^7 times at most its key's share of the
    largest V row), the sums over the keys, and half a step of the output's type."""
    B, T, H, _ = q.shape
    Hkv, page = k.shape[2], k.shape[1]
    G = H // Hkv
    sc = scale if scale else 1 / math.sqrt(D)
    o = torch.zeros(B, T, H, D, dtype=torch.float64)
    bound = torch.zeros_like(o)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64)
    lse_bound = torch.zeros(B, H, T, dtype=torch.float64)
    half = R.HALF[q.dtype]
    held = scales is not None
    weight = 0.0 if q.dtype == torch.float32 else R.HALF[torch.float16] if held else half
    kd, vd = (values(x, s) for x, s in zip((k, v), scales)) if held else (k.double(), v.double())
    for b in range(B):
        n, c = int(lens[b]), T if counts is None else int(counts[b])
        if c == 0:
            continue
        par = None if parents is None else parents[min(b, parents.shape[0] - 1)].tolist()
        vis = seen(n, c, par, window, sinks)
        kept = vis.any(0).nonzero()[:, 0]
        hide = ~vis[:, kept]
        pg, row = R.slots(pages, page, b, kept)
        m = len(kept)
        for h in range(Hkv):
            kk, vv = kd[pg, row, h], vd[pg, row, h]
            for g in range(h * G, (h + 1) * G):
                qq = q[b, :c, g].double()
                s = (qq @ kk.T * sc).masked_fill(hide, -math.inf)
                ds = (qq.abs() @ kk.abs().T * abs(sc) * 140 * 2.0 ** -23).masked_fill(hide, 0).amax(-1) + 2.0 ** -21
                if held and q.dtype == torch.bfloat16:
                    ds = ds + qq.abs().amax(-1) * kk.abs().sum(-1).amax() * abs(sc) * 2.0 ** -34
                p = torch.softmax(s, -1)
                o[b, :c, g] = p @ vv
                lse[b, g, :c] = torch.logsumexp(s, -1)
                sums = (m + 64) * 2.0 ** -24
                rel = weight + 2 * ds + 2 * sums
                size = p @ vv.abs()
                bound[b, :c, g] = rel[:, None] * size * (1 + half) + half * o[b, :c, g].abs()
                if weight == R.HALF[torch.float16]:
                    bound[b, :c, g] += m * 2.0 ** (-31 if held else -25) * vv.abs().max()
                if q.dtype == torch.float16:
                    bound[b, :c, g] += 2.0 ** -25  # the output's own smallest numbers
                lse_bound[b, g, :c] = ds + sums + 2.0 ** -22 * (1 + lse[b, g, :c].abs())
    return o, lse, bound, lse_bound
