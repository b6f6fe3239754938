"""Timing cases of the serving operators: appending to a paged K/V cache, attention over it for single tokens, prompts
and trees of drafted tokens, the verification of such trees, and the compaction of a cache.

``run`` computes them in elementary torch operations, or, where ``own`` is true, through the library's entry points.
"""
import math

import torch

own = False

D = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


def listed():
    return [
        # one decoding step of a busy server: every sequence adds one token to its cache
        dict(name="append_token_batch", op="append", dtype="bf16", src="bf16", B=64, T=1, H=32, Hkv=8, length=4000, page=16,
             axes="128"),
        # a long prompt of two samples enters the cache; q and k arrive in 32 bits, as under autocast
        dict(name="append_prompt", op="append", dtype="bf16", src="fp32", B=2, T=4608, H=24, Hkv=24, length=300, page=64,
             axes="16,56,56"),
        # one user, one token, a short context: latency
        dict(name="attend_token_short", op="attend", dtype="bf16", B=1, T=1, H=32, Hkv=8, length=777, page=16, tree=False),
        # a decoding step of a batch whose contexts have every length
        dict(name="attend_token_batch", op="attend", dtype="fp16", B=64, T=1, H=24, Hkv=8, length=8191, page=32, tree=False),
        # drafted trees of a batch, checked in one step
        dict(name="attend_tree_batch", op="attend", dtype="bf16", B=16, T=61, H=32, Hkv=8, length=16896, page=64, tree=True),
        # one drafted tree after a very long context, as many K/V heads as query heads
        dict(name="attend_tree_long", op="attend", dtype="bf16", B=1, T=24, H=24, Hkv=24, length=262143, page=128, tree=True),
        # a prompt's next chunk after what the cache already holds
        dict(name="attend_chunk", op="attend", dtype="bf16", B=1, T=2048, H=32, Hkv=8, length=16384, page=64, tree=False),
        # a small tree where everything is kept in 32 bits
        dict(name="attend_tree_fp32", op="attend", dtype="fp32", B=4, T=13, H=16, Hkv=2, length=2001, page=16, tree=True),
        # one user's chain of five drafted tokens
        dict(name="verify_chain", op="verify", dtype="fp32", B=1, T=6, V=32000, branch=1, drafted=True),
        # a batch of drafted trees over a large vocabulary
        dict(name="verify_tree_batch", op="verify", dtype="fp32", B=32, T=61, V=131072, branch=6, drafted=True),
        # the accepted path of each tree becomes the end of its sequence
        dict(name="keep_path", op="keep", dtype="bf16", B=32, T=61, N=8, Hkv=8, length=9000, page=64),
        # caches are thinned out: most rows stay and move up
        dict(name="keep_thinned", op="keep", dtype="bf16", B=4, T=32761, N=28672, Hkv=8, length=4, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "verify", "keep"])
    page = rng.choice([8, 16, 24, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "append":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        B = _log_int(rng, 1, 64)
        return dict(op=op, dtype=dtype, src=rng.choice([dtype, "fp32"]), B=B, T=_log_int(rng, 1, 8192 // B), H=H, Hkv=Hkv,
                    length=_log_int(rng, 1, 8000), page=page, axes=rng.choice(["128", "16,56,56", "32,96"]))
    if op == "attend":
        dtype = rng.choice(["bf16", "bf16", "bf16", "fp16", "fp16", "fp16", "fp32"])
        tree = rng.random() < 0.5
        B = _log_int(rng, 1, 32)
        T = _log_int(rng, 1, 128) if tree else _log_int(rng, 1, 1024)
        if dtype == "fp32":
            B, T = min(B, 8), min(T, 64)
        # the plain form's scores, B H T length in 32 bits, and its products stay below the largest listed case's
        most = min(65536, (1 << 29) // (B * H * T), (1 << 22) // (B * Hkv))
        if dtype == "fp32":
            most = min(most, (1 << 24) // (B * H * T) + 64)
        return dict(op=op, dtype=dtype, B=B, T=T, H=H, Hkv=Hkv, length=_log_int(rng, 1, max(2, most)), page=page, tree=tree)
    if op == "verify":
        B = _log_int(rng, 1, 32)
        T = _log_int(rng, 2, 61)
        return dict(op=op, dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]), B=B, T=T, V=_log_int(rng, 500, 131072),
                    branch=rng.choice([1, 2, 4, 8]), drafted=rng.random() < 0.7)
    B = _log_int(rng, 1, 32)
    T = _log_int(rng, 8, (1 << 17) // B)
    return dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), B=B, T=T, N=_log_int(rng, 1, max(1, T - T // 8)), Hkv=Hkv,
                length=_log_int(rng, 1, 4000), page=page)


# ---------------------------------------------------------------- inputs
def _spread(B, most):
    """B lengths from most/B to most: the contexts of a batch are of every length, their sum goes by the case alone."""
    return [max(1, most * (i + 1) // B) for i in range(B)]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed), torch.Generator().manual_seed(seed)


def _cache(g, gc, lens, room, Hkv, page, dtype):
    """Pages in a shuffled order, as a server's allocator leaves them; every sequence has room for `room` tokens more."""
    need = [(n + room + page - 1) // page for n in lens]
    total = sum(need)
    order = torch.randperm(total + 3, generator=gc)[:total].to(torch.int32)
    pages = torch.zeros(len(lens), max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        pages[b, :n] = order[at:at + n]
        at += n
    k = torch.empty(total + 3, page, Hkv, D, dtype=dtype, device=DEV).normal_(generator=g)
    v = torch.empty(total + 3, page, Hkv, D, dtype=dtype, device=DEV).normal_(generator=g)
    return k, v, pages.to(DEV)


def _tree(gc, B, T, branch):
    """Parents before children; the root is node 0."""
    par = torch.full((B, T), -1, dtype=torch.int32)
    for i in range(1, T):
        par[:, i] = torch.randint(max(0, i - branch), i, (B,), generator=gc).to(torch.int32)
    return par


def prepare(case, seed):
    c = dict(case)
    g, gc = _gen(seed)
    dt = DTYPES[c["dtype"]]
    op, B, T = c["op"], c["B"], c["T"]
    s = {"case": c}
    if op == "verify":
        V = c["V"]
        par = _tree(gc, B, T, c["branch"])
        logits = torch.empty(B, T, V, device=DEV).normal_(generator=g).mul_(3.0)
        s["target"] = torch.softmax(logits, -1).to(dt)
        draft = torch.softmax(logits.add_(torch.empty_like(logits).normal_(generator=g)), -1)
        del logits
        up = par.clamp(min=0).long().to(DEV)
        drawn = torch.multinomial(draft.reshape(B * T, V), T, replacement=True, generator=g).reshape(B, T, T)
        # node i's token is drawn from the draft at its parent
        s["tokens"] = drawn[torch.arange(B, device=DEV)[:, None], up, torch.arange(T, device=DEV)[None, :]].to(torch.int32)
        s["draft"] = draft.to(dt) if c["drafted"] else None
        s["parents"] = par.to(DEV)
        s["u_accept"] = torch.rand(B, T, device=DEV, generator=g)
        s["u_sample"] = torch.rand(B, device=DEV, generator=g)
        return s
    perm = torch.randperm(B, generator=gc).tolist()
    spread = _spread(B, c["length"])
    lens = [spread[i] for i in perm]
    s["lens"] = torch.tensor(lens, dtype=torch.int32).to(DEV)
    s["k"], s["v"], s["pages"] = _cache(g, gc, lens, T, c["Hkv"], c["page"], dt)
    if op == "append":
        src = DTYPES[c["src"]]
        s["axes"] = tuple(int(a) for a in c["axes"].split(","))
        s["nq"] = torch.empty(B, T, c["H"], D, dtype=src, device=DEV).normal_(generator=g)
        s["nk"] = torch.empty(B, T, c["Hkv"], D, dtype=src, device=DEV).normal_(generator=g)
        s["nv"] = torch.empty(B, T, c["Hkv"], D, dtype=dt, device=DEV).normal_(generator=g)
        s["wq"] = 1 + 0.1 * torch.empty(D, device=DEV).normal_(generator=g)
        s["wk"] = 1 + 0.1 * torch.empty(D, device=DEV).normal_(generator=g)
        first = s["lens"][:, None] + torch.arange(T, device=DEV, dtype=torch.int32)[None]
        s["ids"] = torch.stack([first // (a + 1) for a in range(len(s["axes"]))], -1).to(torch.int32).contiguous()
    elif op == "attend":
        s["q"] = torch.empty(B, T, c["H"], D, dtype=dt, device=DEV).normal_(generator=g)
        s["parents"] = _tree(gc, B, T, 8).to(DEV) if c["tree"] else None
        # of the smaller half of a batch's trees, a tenth of the nodes is not there
        s["counts"] = None
        if B > 1:
            s["counts"] = torch.tensor([T - (T // 10 if i < B // 2 else 0) for i in perm], dtype=torch.int32).to(DEV)
    else:
        N = c["N"]
        rows = torch.rand(B, T, device=DEV, generator=g).argsort(-1)[:, :N].sort(-1).values
        s["rows"] = rows.to(torch.int32).contiguous()
        s["n_rows"] = torch.tensor([N - (N // 4 if i < B // 2 else 0) for i in perm], dtype=torch.int32).to(DEV)
    return s


# ---------------------------------------------------------------- plain forms
def _slots(pages, page, pos):
    """(page, row) of the positions pos [B, n] of each sequence."""
    return torch.gather(pages.long(), 1, pos // page), pos % page


def _rotate(x, w, cos, sin):
    """RMS norm and rotation of interleaved pairs, in 32 bits."""
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)


def _angles(ids, axes, theta):
    """The angle of each token and pair, in 64 bits."""
    parts = [ids[..., a:a + 1].double() * theta ** (-2.0 * torch.arange(d // 2, device=DEV, dtype=torch.float64) / d)
             for a, d in enumerate(axes)]
    return torch.cat(parts, -1)


def _plain_append(s):
    c = s["case"]
    dt = s["k"].dtype
    ang = _angles(s["ids"], s["axes"], 1e4)[:, :, None]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    q = _rotate(s["nq"], s["wq"], cos, sin).to(dt)
    k = _rotate(s["nk"], s["wk"], cos, sin).to(dt)
    pos = s["lens"][:, None].long() + torch.arange(c["T"], device=DEV)[None]
    pg, row = _slots(s["pages"], c["page"], pos)
    s["k"][pg, row] = k
    s["v"][pg, row] = s["nv"]
    return q, s["k"], s["v"]


def _visible(s, keys, kind):
    """[B, T, keys]: the prefix, the node itself and its ancestors (or, without a tree, every token before it)."""
    c = s["case"]
    T = c["T"]
    B = s["lens"].shape[0]
    own_ = torch.eye(T, dtype=torch.bool, device=DEV).expand(B, T, T)
    if s["parents"] is None:
        seen = torch.ones(T, T, dtype=torch.bool, device=DEV).tril().expand(B, T, T)
    else:
        # ancestors by doubling: who is seen from the node as far up as reached, and the node reached
        par = s["parents"].long()
        seen = own_ | ((par[:, :, None] == torch.arange(T, device=DEV)) & (par >= 0)[:, :, None])
        for _ in range(max(1, (T - 1).bit_length())):
            seen = torch.bmm(seen.to(kind), seen.to(kind)) > 0
    node = torch.arange(keys, device=DEV)[None] - s["lens"][:, None].long()
    inside = (node >= 0) & (node < T)
    if s["counts"] is not None:
        inside = inside & (node < s["counts"][:, None])
    vis = torch.gather(seen, 2, node.clamp(0, T - 1)[:, None].expand(B, T, keys)) & inside[:, None]
    vis = vis | (node < 0)[:, None]
    if s["counts"] is not None:
        vis = vis & (torch.arange(T, device=DEV)[None] < s["counts"][:, None])[:, :, None]
    return vis


def _plain_attend(s):
    c = s["case"]
    B, T, H, Hkv = c["B"], c["T"], c["H"], c["Hkv"]
    keys = c["length"] + T
    pos = torch.arange(keys, device=DEV)[None].expand(B, keys)
    pos = torch.minimum(pos, torch.full_like(pos, s["pages"].shape[1] * c["page"] - 1))
    pg, row = _slots(s["pages"], c["page"], pos)
    k = s["k"][pg, row].float().permute(0, 2, 3, 1)                       # B Hkv D keys
    v = s["v"][pg, row].float().permute(0, 2, 1, 3)                       # B Hkv keys D
    q = s["q"].float().reshape(B, T, Hkv, H // Hkv, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * (H // Hkv), D)
    x = torch.matmul(q, k).mul_(1 / math.sqrt(D)).reshape(B, Hkv, T, H // Hkv, keys)
    del k
    x.masked_fill_(~_visible(s, keys, torch.float32)[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(torch.where(top.isinf(), torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hkv, T * (H // Hkv), keys), v).reshape(B, Hkv, T, H // Hkv, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log()).squeeze(-1)                                  # B Hkv T G
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, H, D).to(s["q"].dtype)
    return o, lse.permute(0, 1, 3, 2).reshape(B, H, T)


def _plain_verify(s):
    """Node after node, for all sequences at once, the residual weights of each sequence's present node in 64 bits."""
    p, q, par, tok = s["target"], s["draft"], s["parents"].long(), s["tokens"].long()
    B, T, V = p.shape
    at = torch.arange(B, device=DEV)
    cur = torch.zeros(B, dtype=torch.long, device=DEV)
    n = torch.ones(B, dtype=torch.long, device=DEV)
    path = torch.full((B, T + 1), -1, dtype=torch.long, device=DEV)
    path[:, 0] = 0
    w = p[:, 0].double()
    a, c = torch.zeros(B, dtype=torch.float64, device=DEV), torch.ones(B, dtype=torch.float64, device=DEV)
    for i in range(1, T):
        child = par[:, i] == cur
        x = tok[:, i]
        wx = w[at, x]
        ask = s["u_accept"][:, i].double() * c
        if q is not None:
            ask = ask * q[at, cur, x].double()
        yes = child & (ask < wx)
        no = child & ~yes
        cur = torch.where(yes, i, cur)
        path[at, torch.where(yes, n, T)] = i
        n = n + yes
        row = p[at, cur].double()
        if q is not None:
            a = torch.where(no, a + c, torch.where(yes, torch.zeros_like(a), a))
            w = (row - a[:, None] * q[at, cur].double()).clamp_(min=0)
            c = torch.where(no, w.sum(-1), torch.where(yes, torch.ones_like(c), c))
        else:
            c = torch.where(no, c - wx, torch.where(yes, torch.ones_like(c), c))
            w = torch.where(yes[:, None], row, w)
            w[at, x] = torch.where(no, torch.zeros_like(wx), w[at, x])
    total = w.sum(-1, keepdim=True)
    w = torch.where(total > 0, w, p[at, cur].double())
    total = w.sum(-1, keepdim=True)
    token = (w.cumsum(-1) <= s["u_sample"].double()[:, None] * total).sum(-1).clamp(max=V - 1)
    path = torch.where(torch.arange(T, device=DEV)[None] < n[:, None], path[:, :T], -1)
    return path.to(torch.int32), n.to(torch.int32), token.to(torch.int32)


def _plain_keep(s):
    c = s["case"]
    start, n = s["lens"].long()[:, None], s["n_rows"].long()[:, None]
    i = torch.arange(c["N"], device=DEV)[None]
    i = torch.where(i < n, i, 0)  # what is behind the last kept row repeats the first move
    src = start + torch.where(n > 0, torch.gather(s["rows"].long(), 1, i), 0)
    spg, srow = _slots(s["pages"], c["page"], src)
    dpg, drow = _slots(s["pages"], c["page"], start + i)
    s["k"][dpg, drow] = s["k"][spg, srow]
    s["v"][dpg, drow] = s["v"][spg, srow]
    return s["k"], s["v"], s["lens"] + s["n_rows"]


def _own(s):
    from qk_norm_rope_gb300 import api
    op = s["case"]["op"]
    if op == "verify":
        return api.st_tree_verify(s["target"], s["draft"], s["tokens"], s["parents"], s["u_accept"], s["u_sample"])
    cache = api.KVCache(s["k"], s["v"], s["pages"])
    if op == "append":
        q = api.st_cache_append(s["nq"], s["nk"], s["nv"], s["wq"], s["wk"], 1e-6, s["ids"], s["axes"], 1e4, cache,
                                s["lens"])
        return q, s["k"], s["v"]
    if op == "attend":
        return api.st_cache_attn(s["q"], cache, s["lens"], counts=s["counts"], parents=s["parents"])
    return s["k"], s["v"], api.st_cache_keep(cache, s["lens"], s["rows"], s["n_rows"])


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    if op == "append":
        return _plain_append(s)
    if op == "attend":
        return _plain_attend(s)
    return _plain_verify(s) if op == "verify" else _plain_keep(s)


# ---------------------------------------------------------------- what cannot be done without
def work(case):
    c = case
    e = 4 if c["dtype"] == "fp32" else 2
    B, T = c["B"], c["T"]
    if c["op"] == "verify":
        # the row that the next token is drawn from, of the target and of the draft, and each node's two probabilities
        return {"bytes": B * ((2 if c["drafted"] else 1) * (c["V"] * e + T * e) + T * 20), "flops": B * c["V"] * 4}
    if c["op"] == "append":
        es = 4 if c["src"] == "fp32" else 2
        rows = B * T * D
        return {"bytes": rows * ((c["H"] + c["Hkv"]) * (es + e) + 2 * c["Hkv"] * e), "flops": rows * (c["H"] + c["Hkv"]) * 8}
    if c["op"] == "attend":
        counts = [T - (T // 10 if i < B // 2 and B > 1 else 0) for i in range(B)]
        lens = _spread(B, c["length"])
        keys = sum(n + t for n, t in zip(lens, counts))
        pairs = sum(t * n + (t * (t + 1) // 2) for n, t in zip(lens, counts))
        return {"bytes": keys * c["Hkv"] * D * 2 * e + sum(counts) * c["H"] * (2 * D * e + 4), "flops": 4 * pairs * c["H"] * D}
    n = sum(c["N"] - (c["N"] // 4 if i < B // 2 else 0) for i in range(B))
    return {"bytes": n * (c["Hkv"] * D * e * 2 * 2 + 4), "flops": 0}


# ---------------------------------------------------------------- by the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "verify": _exact_verify, "keep": _exact_keep}[case["op"]](s)


def _exact_append(s):
    c = s["case"]
    pair = torch.cat([torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d for d in s["axes"]])
    axis = torch.cat([torch.full((d // 2,), a, device=DEV) for a, d in enumerate(s["axes"])])
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["ids"].double()[..., axis] * torch.exp(-pair * math.log(1e4)))

    def rot(x, w):
        x = x.double()
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + 1e-6) * w.double()
        return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], D // 2, 2)) * turn[:, :, None]).flatten(-2)

    k, v = s["k"].double(), s["v"].double()
    nk = rot(s["nk"], s["wk"])
    for b, n in enumerate(s["lens"].tolist()):
        pos = n + torch.arange(c["T"], device=DEV)
        pg = s["pages"][b].long()[pos // c["page"]]
        k[pg, pos % c["page"]] = nk[b]
        v[pg, pos % c["page"]] = s["nv"][b].double()
    return rot(s["nq"], s["wq"]), k, v


def _exact_attend(s):
    """Sequence by sequence and K/V head by K/V head, the tree's mask from a walk up from each node."""
    c = s["case"]
    B, T, H, Hkv, page = c["B"], c["T"], c["H"], c["Hkv"], c["page"]
    G = H // Hkv
    o = torch.zeros(B, T, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device=DEV)
    counts = [T] * B if s["counts"] is None else s["counts"].tolist()
    for b, (n, t) in enumerate(zip(s["lens"].tolist(), counts)):
        see = torch.zeros(t, n + t, dtype=torch.bool)
        see[:, :n] = True
        if s["parents"] is None:
            see[:, n:] = torch.ones(t, t).tril().bool()
        else:
            par = s["parents"][b].tolist()
            for i in range(t):
                j = i
                while j >= 0:
                    see[i, n + j] = True
                    j = par[j]
        hide = ~see.to(DEV)
        pg = s["pages"][b, :(n + t + page - 1) // page].long()
        for h in range(Hkv):
            k = s["k"][pg, :, h].reshape(-1, D)[:n + t].double()
            v = s["v"][pg, :, h].reshape(-1, D)[:n + t].double()
            for g in range(h * G, (h + 1) * G):
                x = (s["q"][b, :t, g].double() @ k.T / math.sqrt(D)).masked_fill(hide, -math.inf)
                lse[b, g, :t] = torch.logsumexp(x, -1)
                o[b, :t, g] = torch.softmax(x, -1) @ v
    return o, lse


def _exact_verify(s):
    """Each sequence by itself: accept, or go on with the normalised residual distribution."""
    p, q = s["target"], s["draft"]
    B, T, V = p.shape
    par, tok, u = s["parents"].tolist(), s["tokens"].tolist(), s["u_accept"].double().tolist()
    paths, counts, tokens = torch.full((B, T), -1, dtype=torch.int32), [], []
    for b in range(B):
        cur, i, got = 0, 0, [0]
        dist = p[b, 0].double()
        while i + 1 < T:
            i += 1
            if par[b][i] != cur:
                continue
            x = tok[b][i]
            drafted = torch.zeros(V, dtype=torch.float64, device=DEV) if q is None else q[b, cur].double()
            if q is None:
                drafted[x] = 1
            if u[b][i] * float(drafted[x]) < float(dist[x]):
                cur = i
                got.append(i)
                dist = p[b, i].double()
            elif q is None:
                left = 1 - float(dist[x])
                dist[x] = 0
                dist = dist / left if left > 0 else dist
            else:
                rest = (dist - drafted).clamp(min=0)
                total = rest.sum()
                dist = rest / total if float(total) > 0 else rest
        if float(dist.sum()) == 0:
            dist = p[b, cur].double()
        cum = torch.cumsum(dist, 0)
        tokens.append(int(torch.searchsorted(cum, s["u_sample"][b].double() * cum[-1], right=True).clamp(max=V - 1)))
        paths[b, :len(got)] = torch.tensor(got, dtype=torch.int32)
        counts.append(len(got))
    return paths, torch.tensor(counts, dtype=torch.int32), torch.tensor(tokens, dtype=torch.int32)


def _exact_keep(s):
    c = s["case"]
    k, v = s["k"].double(), s["v"].double()
    ends = []
    for b, (n, m) in enumerate(zip(s["lens"].tolist(), s["n_rows"].tolist())):
        src = n + s["rows"][b, :m].long()
        dst = n + torch.arange(m, device=DEV)
        pg = s["pages"][b].long()
        for t, old in ((k, s["k"]), (v, s["v"])):
            t[pg[dst // c["page"]], dst % c["page"]] = old[pg[src // c["page"]], src % c["page"]].double()
        ends.append(n + m)
    return k, v, torch.tensor(ends, dtype=torch.int32)
