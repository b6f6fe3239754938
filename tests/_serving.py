"""Plain 64-bit forms of the serving calls, and the error bounds that their tests hold the kernels to."""
from __future__ import annotations

import math

import torch

D = 128
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}  # half a step, relative


def tree(B, T, branch, seed):
    """Parents before children, node 0 the root."""
    g = torch.Generator().manual_seed(seed)
    par = torch.full((B, T), -1, dtype=torch.int32)
    for i in range(1, T):
        par[:, i] = torch.randint(max(0, i - branch), i, (B,), generator=g).to(torch.int32)
    return par


def make_cache(B, room, Hkv, page, dtype, seed, fill=float("nan"), spare=2):
    """k, v, pages (CPU) with every slot holding `fill`; pages in a shuffled order, entries behind a sequence's last
    page pointing far out of range."""
    g = torch.Generator().manual_seed(seed)
    need = [max(1, -(-r // page)) for r in room]
    n = sum(need) + spare
    order = torch.randperm(n, generator=g)[: sum(need)].to(torch.int32)
    pages = torch.full((B, max(need)), 1 << 30, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        pages[b, :m] = order[at: at + m]
        at += m
    k = torch.full((n, page, Hkv, D), fill, dtype=dtype)
    return k, k.clone(), pages


def slots(pages, page, b, pos):
    return pages[b].long()[pos // page], pos % page


def fill_prefix(k, v, pages, lens, seed):
    g = torch.Generator().manual_seed(seed)
    page = k.shape[1]
    for b, n in enumerate(lens):
        if n > 0:
            pg, row = slots(pages, page, b, torch.arange(n))
            k[pg, row] = torch.randn(n, k.shape[2], D, generator=g).to(k.dtype)
            v[pg, row] = torch.randn(n, k.shape[2], D, generator=g).to(v.dtype)


def rotate(x, w, ang, eps):
    """RMS norm and rotation in 64 bits; also the size of the terms of each element's sum."""
    x, w = x.double(), w.double()
    n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w
    a, b = n[..., 0::2], n[..., 1::2]
    c, s = torch.cos(ang)[:, :, None], torch.sin(ang)[:, :, None]
    y = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    size = torch.stack((a.abs() + b.abs(), a.abs() + b.abs()), -1).flatten(-2)
    return y, size


def angles(ids, axes, theta):
    parts = []
    for a, d in enumerate(axes):
        j = torch.arange(d // 2, dtype=torch.float64)
        parts.append(ids[..., a: a + 1].double() * theta ** (-2.0 * j / d))
    return torch.cat(parts, -1)


def seen(T, n, count, parents):
    """[count, n + count] truth values: the keys that each row sees."""
    see = torch.zeros(count, n + count, dtype=torch.bool)
    see[:, :n] = True
    for i in range(count):
        if parents is None:
            see[i, n: n + i + 1] = True
            continue
        j = i
        while j >= 0:
            see[i, n + j] = True
            up = int(parents[j])
            j = up if up < j else -1
    return see


def attention(q, k, v, pages, lens, counts, parents, scale=None):
    """(o, lse, bound on |o|'s error, bound on lse's) in 64 bits; all inputs on the CPU.

    The bounds count, per row: half a step of the weights' 16-bit type (none in 32 bits) on each weight, half a step of
    the output's type, the fp32 sums of 128 products (each product and partial sum off by at most 2^-23 of the terms'
    size, so that scores are off by ds), ex2's 2^-21, and the sums over the keys."""
    B, T, H, _ = q.shape
    Hkv, page, dt = k.shape[2], k.shape[1], k.dtype
    G = H // Hkv
    sc = scale if scale else 1 / math.sqrt(D)
    o = torch.zeros(B, T, H, D, dtype=torch.float64)
    bound = torch.zeros_like(o)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64)
    lse_bound = torch.zeros(B, H, T, dtype=torch.float64)
    half = HALF[dt]
    for b in range(B):
        n, c = int(lens[b]), T if counts is None else int(counts[b])
        if c == 0:
            continue
        par = None if parents is None else parents[min(b, parents.shape[0] - 1)].tolist()
        hide = ~seen(T, n, c, par)
        pg, row = slots(pages, page, b, torch.arange(n + c))
        for h in range(Hkv):
            kk, vv = k[pg, row, h].double(), v[pg, row, h].double()
            for g in range(h * G, (h + 1) * G):
                qq = q[b, :c, g].double()
                s = (qq @ kk.T * sc).masked_fill(hide, -math.inf)
                ds = (qq.abs() @ kk.abs().T * abs(sc) * 130 * 2.0 ** -23).masked_fill(hide, 0).amax(-1) + 2.0 ** -21
                p = torch.softmax(s, -1)
                o[b, :c, g] = p @ vv
                lse[b, g, :c] = torch.logsumexp(s, -1)
                sums = (n + c + 64) * 2.0 ** -24
                rel = (0.0 if dt == torch.float32 else half) + 2 * ds + 2 * sums
                size = p @ vv.abs()
                bound[b, :c, g] = rel[:, None] * size * (1 + half) + half * o[b, :c, g].abs()
                if dt == torch.float16:
                    # weights below fp16's range: off by half a step of its smallest numbers, the largest being 1
                    bound[b, :c, g] += (n + c) * 2.0 ** -25 * vv.abs().max()
                    # and the output's own smallest numbers
                    bound[b, :c, g] += 2.0 ** -25
                lse_bound[b, g, :c] = ds + sums + 2.0 ** -22 * (1 + lse[b, g, :c].abs())
    return o, lse, bound, lse_bound


def close(name, got, want, bound):
    got = got.double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{name}: infinities differ"
    bad = ~((got - want).abs() <= bound) & ~inf
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}: "
                           f"{got[bad][0].item()} for {want[bad][0].item()}, bound {bound[bad][0].item():.3e}")


def verify(target, draft, tokens, parents, u_accept, u_sample, counts=None):
    """The walk by its definition: accept, or go on with the normalised residual, in 64 bits (CPU)."""
    B, T, V = target.shape
    paths, ns, nexts = torch.full((B, T), -1, dtype=torch.int32), [], []
    for b in range(B):
        c = T if counts is None else max(0, min(int(counts[b]), T))
        if c == 0:
            ns.append(0)
            nexts.append(-1)
            continue
        par = parents[min(b, parents.shape[0] - 1)].tolist()
        tok, u = tokens[b].tolist(), u_accept[b].double().tolist()
        cur, got = 0, [0]
        p = torch.nan_to_num(target[b].double(), 0.0).clamp(0, 1)
        q = None if draft is None else torch.nan_to_num(draft[b].double(), 0.0).clamp(0, 1)
        w, total = p[0].clone(), 1.0
        gone = torch.zeros(V, dtype=torch.float64)
        for i in range(1, c):
            if par[i] != cur or not 0 <= tok[i] < V:
                continue
            x = tok[i]
            qx = 1.0 if q is None else float(q[cur, x])
            if u[i] * qx * total < float(w[x]):
                cur = i
                got.append(i)
                w, total = p[i].clone(), 1.0
                gone = torch.zeros(V, dtype=torch.float64)
            elif q is None:
                total -= float(w[x])
                w[x] = 0
            else:
                gone += total * q[cur]
                w = (p[cur] - gone).clamp(min=0)
                total = float(w.sum())
        if float(w.sum()) == 0:
            w = p[cur]
        cum = torch.cumsum(w, 0)
        if float(cum[-1]) == 0:
            nexts.append(-1)
        else:
            nexts.append(int((cum <= min(max(float(u_sample[b]), 0.0), 1 - 2.0 ** -53) * cum[-1]).sum().clamp(max=V - 1)))
        ns.append(len(got))
        paths[b, : len(got)] = torch.tensor(got, dtype=torch.int32)
    return paths, torch.tensor(ns, dtype=torch.int32), torch.tensor(nexts, dtype=tokens.dtype)
