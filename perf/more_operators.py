"""Timing cases of a second set of serving operators, over the same paged K/V cache: a cache of 8 bits (quantised as it is
written, read back, attended over), attention with a sliding window and visible first tokens, and attention for a batch
whose sequences share a long prefix.

``run`` computes them in elementary torch operations, or, where ``own`` is true, through the library's entry points.
"""
import math

import torch

own = False

D = 128
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}  # what a row's largest magnitude is held as
DEV = "cuda"


def listed():
    return [
        # one decoding step of a busy server: every sequence adds one token to a cache of 8-bit floats
        dict(name="append_token_batch", op="append", dtype="bf16", src="bf16", kv="e4m3", B=64, T=1, H=32, Hkv=8, length=4000,
             page=16, axes="128"),
        # a long prompt of two samples, q and k in 32 bits as under autocast, enters an int8 cache and is read back for
        # what goes on in 16 bits
        dict(name="append_prompt", op="append", dtype="bf16", src="fp32", kv="int8", B=2, T=4608, H=24, Hkv=24, length=300,
             page=64, axes="16,56,56"),
        # the last rows of a batch's sequences are read back
        dict(name="read_tails", op="read", dtype="fp16", kv="int8", B=32, T=61, Hkv=8, length=9000, page=16),
        # whole contexts leave a cache of 8-bit floats, to be kept or moved in 16 bits
        dict(name="read_contexts", op="read", dtype="bf16", kv="e4m3", B=4, T=16333, Hkv=8, length=16333, page=64),
        # one user, one token, a short context: latency
        dict(name="attend_token_short", op="attend", dtype="bf16", kv="e4m3", B=1, T=1, H=32, Hkv=8, length=777, page=16,
             tree=False, window=0, sinks=0, shared=0),
        # a decoding step of a batch whose contexts have every length
        dict(name="attend_token_batch", op="attend", dtype="bf16", kv="e4m3", B=64, T=1, H=32, Hkv=8, length=8191, page=16,
             tree=False, window=0, sinks=0, shared=0),
        # drafted trees of a batch over an int8 cache
        dict(name="attend_tree_batch", op="attend", dtype="fp16", kv="int8", B=16, T=61, H=32, Hkv=8, length=9000, page=64,
             tree=True, window=0, sinks=0, shared=0),
        # a decoding step of a model with a window, long after the contexts outgrew it
        dict(name="window_token_batch", op="attend", dtype="bf16", kv="bf16", B=48, T=1, H=32, Hkv=8, length=32768, page=32,
             tree=False, window=4096, sinks=4, shared=0),
        # a prompt's next chunk of such a model
        dict(name="window_chunk", op="attend", dtype="bf16", kv="bf16", B=1, T=2048, H=32, Hkv=8, length=16384, page=64,
             tree=False, window=4096, sinks=4, shared=0),
        # small trees where everything is kept in 32 bits
        dict(name="window_tree_fp32", op="attend", dtype="fp32", kv="fp32", B=4, T=13, H=16, Hkv=2, length=20001, page=16,
             tree=True, window=1000, sinks=17, shared=0),
        # many answers to one long prompt: each sequence has a short part of its own
        dict(name="shared_token_batch", op="attend", dtype="bf16", kv="bf16", B=64, T=1, H=32, Hkv=8, length=1000, page=16,
             tree=False, window=0, sinks=0, shared=16384),
        # drafted trees after a prompt that all share, over 8-bit floats
        dict(name="shared_tree_batch", op="attend", dtype="bf16", kv="e4m3", B=8, T=24, H=24, Hkv=8, length=2000, page=64,
             tree=True, window=0, sinks=0, shared=32768),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend", "attend", "attend", "attend"])
    page = rng.choice([8, 16, 24, 32, 64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    kv = rng.choice(["e4m3", "int8"])
    if op == "append":
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        B = _log_int(rng, 1, 64)
        return dict(op=op, dtype=dtype, src=rng.choice([dtype, "fp32"]), kv=kv, B=B, T=_log_int(rng, 1, 8192 // B), H=H, Hkv=Hkv,
                    length=_log_int(rng, 1, 8000), page=page, axes=rng.choice(["128", "16,56,56", "32,96"]))
    if op == "read":
        B = _log_int(rng, 1, 32)
        T = _log_int(rng, 1, 65536 // B)
        return dict(op=op, dtype=rng.choice(["bf16", "fp16", "fp32"]), kv=kv, B=B, T=T, Hkv=Hkv, length=T + _log_int(rng, 1, 4000),
                    page=page)
    kind = rng.choice(["whole", "whole", "window", "window", "shared", "shared"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp16", "fp16", "fp16", "fp32"])
    kv = kv if kind == "whole" or rng.random() < 0.4 else dtype
    tree = rng.random() < 0.4
    B = _log_int(rng, 2 if kind == "shared" else 1, 48)
    T = _log_int(rng, 1, 100) if tree else _log_int(rng, 1, 32 if kind == "shared" else 1024)
    if dtype == "fp32":
        B, T = min(B, 8), min(T, 48)
    window = _log_int(rng, 16, 8192) if kind == "window" else 0
    # the plain form's scores, B H T keys in 32 bits, and its products stay below the largest listed case's
    T = min(T, math.isqrt((1 << 27) // (B * H)))
    most = min(65536, (1 << 28) // (B * H * T), (1 << 22) // (B * Hkv))
    if dtype == "fp32":
        most = min(most, (1 << 24) // (B * H * T) + 64)
    c = dict(op=op, dtype=dtype, kv=kv, B=B, T=T, H=H, Hkv=Hkv, length=0, page=page, tree=tree, window=0, sinks=0, shared=0)
    if kind == "window":
        c["window"] = max(1, min(window, most - 64))
        c["sinks"] = rng.choice([0, 1, 4, 17, 64])
        c["length"] = _log_int(rng, 1, min(65536, (1 << 22) // (B * Hkv)))
    elif kind == "shared":
        c["shared"] = _log_int(rng, page, max(2 * page, min(32768, most)))
        c["length"] = _log_int(rng, 1, max(2, min(2000, most)))
    else:
        c["length"] = _log_int(rng, 1, max(2, most))
    return c


# ---------------------------------------------------------------- inputs
def _spread(B, most):
    """B lengths from most/B to most: the contexts of a batch are of every length, their sum goes by the case alone."""
    return [max(1, most * (i + 1) // B) for i in range(B)]


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed), torch.Generator().manual_seed(seed)


def _quantise(x, kv):
    """Rows of 8 bits and a scale each: the row's largest magnitude becomes the type's largest."""
    x = x.float()
    scale = x.abs().amax(-1) / TOP[kv]
    x = x / torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    return (x.round() if kv == "int8" else x).to(DTYPES[kv]), scale


def _fill(g, shape, dtype, kv):
    """Rows of a cache, and their scales [N, Hkv, page] where it is of 8 bits. Rows differ in size, as a model's do."""
    if kv not in TOP:
        return torch.empty(*shape, dtype=dtype, device=DEV).normal_(generator=g), None
    out = torch.empty(*shape, dtype=torch.int8, device=DEV).view(DTYPES[kv])
    scale = torch.empty(shape[0], shape[2], shape[1], device=DEV)
    step = max(1, (1 << 26) // (shape[1] * shape[2] * D))
    for i in range(0, shape[0], step):
        n = min(step, shape[0] - i)
        x = torch.empty(n, *shape[1:], device=DEV).normal_(generator=g)
        x.mul_(torch.exp2(torch.empty(n, *shape[1:3], 1, device=DEV).uniform_(-1, 1, generator=g)))
        q, s = _quantise(x, kv)
        out[i:i + n].view(torch.int8).copy_(q.view(torch.int8))
        scale[i:i + n] = s.transpose(1, 2)
    return out, scale


def _cache(g, gc, lens, room, c, shared=0):
    """Pages in a shuffled order, as a server's allocator leaves them; every sequence has room for `room` tokens more. The
    first `shared` tokens (whole pages) lie in the same pages for all."""
    page = c["page"]
    head = shared // page
    need = [(n + room + page - 1) // page - head for n in lens]
    total = head + sum(need)
    order = torch.randperm(total + 3, generator=gc)[:total].to(torch.int32)
    pages = torch.zeros(len(lens), head + max(need), dtype=torch.int32)
    pages[:, :head] = order[:head]
    at = head
    for b, n in enumerate(need):
        pages[b, head:head + n] = order[at:at + n]
        at += n
    shape = (total + 3, page, c["Hkv"], D)
    k, ks = _fill(g, shape, DTYPES[c["dtype"]], c["kv"])
    v, vs = _fill(g, shape, DTYPES[c["dtype"]], c["kv"])
    return dict(k=k, v=v, k_scale=ks, v_scale=vs, pages=pages.to(DEV))


def _tree(gc, B, T, branch):
    """Parents before children; the root is node 0."""
    par = torch.full((B, T), -1, dtype=torch.int32)
    for i in range(1, T):
        par[:, i] = torch.randint(max(0, i - branch), i, (B,), generator=gc).to(torch.int32)
    return par


def _shared(c):
    """The shared tokens of a case: whole pages."""
    return c.get("shared", 0) // c["page"] * c["page"]


def _lens(c):
    if c["op"] == "read":
        return [c["length"] - (c["length"] - c["T"]) * i // max(1, c["B"]) for i in range(c["B"])]
    return [_shared(c) + n for n in _spread(c["B"], c["length"])]


def prepare(case, seed):
    c = dict(case)
    g, gc = _gen(seed)
    dt = DTYPES[c["dtype"]]
    op, B, T = c["op"], c["B"], c["T"]
    perm = torch.randperm(B, generator=gc).tolist()
    spread = _lens(c)
    lens = [spread[i] for i in perm]
    s = _cache(g, gc, lens, 0 if op == "read" else T, c, _shared(c))
    s["case"] = c
    s["lens"] = torch.tensor(lens, dtype=torch.int32).to(DEV)
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
    elif op == "read":
        s["start"] = s["lens"] - T
        s["counts"] = torch.tensor([T - (T // 10 if i < B // 2 else 0) for i in perm], dtype=torch.int32).to(DEV)
    else:
        s["q"] = torch.empty(B, T, c["H"], D, dtype=dt, device=DEV).normal_(generator=g)
        s["parents"] = _tree(gc, B, T, 8).to(DEV) if c["tree"] else None
        # of the smaller half of a batch's sequences, a tenth of the rows is not there
        s["counts"] = None
        if B > 1:
            s["counts"] = torch.tensor([T - (T // 10 if i < B // 2 else 0) for i in perm], dtype=torch.int32).to(DEV)
        s["shared"] = torch.tensor([_shared(c)], dtype=torch.int32).to(DEV) if c["shared"] else None
    return s


# ---------------------------------------------------------------- plain forms
def _rows(s, name, pg, row):
    """Rows of the cache in 32 bits, [..., Hkv, D]."""
    x = s[name]
    if s[name + "_scale"] is None:
        return x[pg, row].float()
    x = x.view(torch.int8)[pg, row].view(x.dtype).float()
    return x * s[name + "_scale"][pg, :, row][..., None]


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


def _written(s, q, back):
    """What an append answers: q and the cache of 8-bit floats; of an int8 cache the new rows, as they are read back."""
    if back is None:
        return q, s["k"], s["v"], s["k_scale"], s["v_scale"]
    return q, back[0], back[1]


def _plain_append(s):
    c = s["case"]
    dt = s["nv"].dtype
    ang = _angles(s["ids"], s["axes"], 1e4)[:, :, None]
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    q = _rotate(s["nq"], s["wq"], cos, sin).to(dt)
    pos = s["lens"][:, None].long() + torch.arange(c["T"], device=DEV)[None]
    pg, row = _slots(s["pages"], c["page"], pos)
    for name, x in (("k", _rotate(s["nk"], s["wk"], cos, sin)), ("v", s["nv"])):
        x, scale = _quantise(x, c["kv"])
        s[name].view(torch.int8)[pg, row] = x.view(torch.int8)
        s[name + "_scale"][pg, :, row] = scale
    back = None if c["kv"] == "e4m3" else (_rows(s, "k", pg, row).to(dt), _rows(s, "v", pg, row).to(dt))
    return _written(s, q, back)


def _plain_read(s):
    c = s["case"]
    i = torch.arange(c["T"], device=DEV)[None]
    pg, row = _slots(s["pages"], c["page"], s["start"].long()[:, None] + i)
    there = (i < s["counts"][:, None])[..., None, None]
    return tuple(torch.where(there, _rows(s, n, pg, row), 0.0).to(DTYPES[c["dtype"]]) for n in "kv")


def _ancestors(s):
    """[B, T, T] truth values: the nodes that each row sees."""
    c = s["case"]
    B, T = c["B"], c["T"]
    if s["parents"] is None:
        return torch.ones(T, T, dtype=torch.bool, device=DEV).tril().expand(B, T, T)
    # by doubling: who is seen from the node as far up as reached, and the node reached
    par = s["parents"].long()
    seen = torch.eye(T, dtype=torch.bool, device=DEV) | ((par[:, :, None] == torch.arange(T, device=DEV)) & (par >= 0)[:, :, None])
    for _ in range(max(1, (T - 1).bit_length())):
        seen = torch.bmm(seen.float(), seen.float()) > 0
    return seen


def _visible(s, pos):
    """[B, T, keys]: which of the keys at the slots pos [B, keys] each row sees."""
    c = s["case"]
    T = c["T"]
    lens = s["lens"].long()[:, None]
    seen = _ancestors(s)
    depth = seen.sum(-1) - 1                                                  # B T
    node = pos - lens
    inside = (node >= 0) & (node < T)
    if s["counts"] is not None:
        inside = inside & (node < s["counts"][:, None])
    at = node.clamp(0, T - 1)
    vis = torch.gather(seen, 2, at[:, None].expand(-1, T, -1)) & inside[:, None]
    vis = vis | ((node < 0) & (pos >= 0))[:, None]
    if c["window"]:
        key = torch.where(node < 0, pos, lens + torch.gather(depth, 1, at))   # the key's position
        near = (lens + depth)[:, :, None] - key[:, None] < c["window"]
        vis = vis & (near | (key < c["sinks"])[:, None])
    if s["counts"] is not None:
        vis = vis & (torch.arange(T, device=DEV)[None] < s["counts"][:, None])[:, :, None]
    return vis


def _plain_attend(s):
    """Scores over the shared tokens, for all rows at once, beside those over each sequence's own (with a window: over the
    first tokens and what no row's window has left), one softmax over both."""
    c = s["case"]
    B, T, H, Hkv, page = c["B"], c["T"], c["H"], c["Hkv"], c["page"]
    G = H // Hkv
    lens = s["lens"].long()[:, None]
    first = _shared(c)
    if c["window"]:
        near = torch.arange(c["window"] + T, device=DEV)[None] + (lens - c["window"] + 1).clamp(min=c["sinks"])
        pos = torch.cat((torch.arange(c["sinks"], device=DEV)[None].expand(B, -1), near), 1)
        pos = torch.where(pos < lens + T, pos, -1)                            # no key there
    else:
        pos = first + torch.arange(c["length"] + T, device=DEV)[None].expand(B, -1)
        pos = torch.where(pos < lens + T, pos, -1)
    keys = pos.shape[1]
    pg, row = _slots(s["pages"], page, pos.clamp(min=0))
    q = s["q"].float().reshape(B, T, Hkv, G, D).mul(1 / math.sqrt(D))
    x = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D), _rows(s, "k", pg, row).permute(0, 2, 3, 1))
    x = x.reshape(B, Hkv, T, G, keys).masked_fill_(~_visible(s, pos)[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    if first:
        slot = torch.arange(first, device=DEV)
        pg0, row0 = s["pages"][0].long()[slot // page], slot % page
        z = torch.matmul(q.permute(2, 0, 1, 3, 4).reshape(Hkv, B * T * G, D), _rows(s, "k", pg0, row0).permute(1, 2, 0))
        z = z.reshape(Hkv, B, T, G, first).permute(1, 0, 2, 3, 4)
        if s["counts"] is not None:
            gone = (torch.arange(T, device=DEV)[None] >= s["counts"][:, None])[:, None, :, None, None]
            z = z.masked_fill_(gone, -math.inf)
        top = torch.maximum(top, z.amax(-1, keepdim=True))
    use = torch.where(top.isinf(), torch.zeros_like(top), top)
    p = x.sub_(use).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, Hkv, T * G, keys), _rows(s, "v", pg, row).permute(0, 2, 1, 3)).reshape(B, Hkv, T, G, D)
    if first:
        z = z.sub_(use).exp_()
        total = total + z.sum(-1, keepdim=True)
        z = z.permute(1, 0, 2, 3, 4).reshape(Hkv, B * T * G, first)
        z = torch.matmul(z, _rows(s, "v", pg0, row0).permute(1, 0, 2))
        o = o + z.reshape(Hkv, B, T, G, D).permute(1, 0, 2, 3, 4)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log()).squeeze(-1)                                     # B Hkv T G
    o = o.permute(0, 2, 1, 3, 4).reshape(B, T, H, D).to(s["q"].dtype)
    return o, lse.permute(0, 1, 3, 2).reshape(B, H, T)


def _own(s):
    from qk_norm_rope_gb300 import api
    c = s["case"]
    cache = api.KVCache(s["k"], s["v"], s["pages"], s["k_scale"], s["v_scale"])
    if c["op"] == "append":
        q = api.st_cache_append(s["nq"], s["nk"], s["nv"], s["wq"], s["wk"], 1e-6, s["ids"], s["axes"], 1e4, cache,
                                s["lens"])
        back = None if c["kv"] == "e4m3" else api.st_cache_read(cache, s["lens"], c["T"], dtype=s["nv"].dtype)
        return _written(s, q, back)
    if c["op"] == "read":
        return api.st_cache_read(cache, s["start"], c["T"], counts=s["counts"], dtype=DTYPES[c["dtype"]])
    return api.st_cache_attn(s["q"], cache, s["lens"], counts=s["counts"], parents=s["parents"], window=c["window"],
                             sinks=c["sinks"], shared=s["shared"])


def run(s):
    if own:
        return _own(s)
    op = s["case"]["op"]
    return _plain_append(s) if op == "append" else _plain_read(s) if op == "read" else _plain_attend(s)


# ---------------------------------------------------------------- what cannot be done without
def work(case):
    c = case
    size = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1, "int8": 1}
    e, ek = size[c["dtype"]], size[c["kv"]]
    B, T = c["B"], c["T"]
    row = D * ek + (4 if c["kv"] in TOP else 0)  # of a key or a value, with its scale
    if c["op"] == "append":
        n = B * T
        back = 0 if c["kv"] == "e4m3" else n * c["Hkv"] * 2 * D * e  # the rows that are read back have just been computed
        return {"bytes": n * ((c["H"] + c["Hkv"]) * D * size[c["src"]] + (c["Hkv"] + c["H"]) * D * e + 2 * c["Hkv"] * row) + back,
                "flops": n * D * (c["H"] * 8 + c["Hkv"] * 14)}
    counts = [T - (T // 10 if i < B // 2 and B > 1 else 0) for i in range(B)]
    if c["op"] == "read":
        n = sum(counts) if B > 1 else T
        return {"bytes": 2 * c["Hkv"] * (n * row + B * T * D * e), "flops": 2 * n * c["Hkv"] * D}
    first, keys, pairs = _shared(c), 0, 0
    for n, t in zip(_lens(c), counts):
        if c["window"] and n + t > c["sinks"] + c["window"]:
            keys += min(n + t, c["sinks"] + c["window"] + t - 1)
            pairs += t * (c["sinks"] + min(c["window"], n + t))
        else:
            keys += n + t - first
            pairs += t * n + t * (t + 1) // 2
    return {"bytes": (first + keys) * c["Hkv"] * 2 * row + sum(counts) * c["H"] * (2 * D * e + 4), "flops": 4 * pairs * c["H"] * D}


# ---------------------------------------------------------------- by the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)


def _exact_values(s, name, b, n):
    """The first n rows of sequence b, [n, Hkv, D]."""
    c = s["case"]
    pg = s["pages"][b, :(n + c["page"] - 1) // c["page"]].long()
    if s[name + "_scale"] is None:
        x = s[name][pg].double()
    else:
        x = s[name].view(torch.int8)[pg].view(s[name].dtype).double() * s[name + "_scale"][pg].double().transpose(1, 2)[..., None]
    return x.reshape(-1, c["Hkv"], D)[:n]


def _exact_append(s):
    """The cache of 8-bit floats before its rounding (the type's own); int8 rows with theirs."""
    c = s["case"]
    pair = torch.cat([torch.arange(0, d, 2, dtype=torch.float64, device=DEV) / d for d in s["axes"]])
    axis = torch.cat([torch.full((d // 2,), a, device=DEV) for a, d in enumerate(s["axes"])])
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV), s["ids"].double()[..., axis] * torch.exp(-pair * math.log(1e4)))

    def rot(x, w):
        x = x.double()
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + 1e-6) * w.double()
        return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:-1], D // 2, 2)) * turn[:, :, None]).flatten(-2)

    new = (rot(s["nk"], s["wk"]), s["nv"].double())
    scales = tuple(x.abs().amax(-1) / TOP[c["kv"]] for x in new)
    if c["kv"] == "int8":
        return (rot(s["nq"], s["wq"]),) + tuple(torch.round(x / z[..., None]) * z[..., None] for x, z in zip(new, scales))
    held = [s["k"].double(), s["v"].double()]
    sc = [s["k_scale"].double(), s["v_scale"].double()]
    for b, n in enumerate(s["lens"].tolist()):
        at = n + torch.arange(c["T"], device=DEV)
        pg, r = s["pages"][b].long()[at // c["page"]], at % c["page"]
        for i in (0, 1):
            held[i][pg, r] = new[i][b] / scales[i][b][..., None]
            sc[i][pg, :, r] = scales[i][b]
    return (rot(s["nq"], s["wq"]), held[0], held[1], sc[0], sc[1])


def _exact_read(s):
    c = s["case"]
    out = torch.zeros(2, c["B"], c["T"], c["Hkv"], D, dtype=torch.float64, device=DEV)
    for b, (a, n) in enumerate(zip(s["start"].tolist(), s["counts"].tolist())):
        for i, name in enumerate("kv"):
            out[i, b, :n] = _exact_values(s, name, b, a + n)[a:]
    return out[0], out[1]


def _exact_attend(s):
    """Sequence by sequence and K/V head by K/V head over its whole context, the mask from a walk up from each node."""
    c = s["case"]
    B, T, H, Hkv = c["B"], c["T"], c["H"], c["Hkv"]
    G = H // Hkv
    o = torch.zeros(B, T, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device=DEV)
    counts = [T] * B if s["counts"] is None else s["counts"].tolist()
    for b, (n, t) in enumerate(zip(s["lens"].tolist(), counts)):
        up = [i - 1 for i in range(t)] if s["parents"] is None else s["parents"][b].tolist()
        see = torch.zeros(t, t, dtype=torch.bool)
        deep = [0] * t
        for i in range(t):
            if up[i] >= 0:
                deep[i] = deep[up[i]] + 1
                see[i] = see[up[i]]
            see[i, i] = True
        at = torch.tensor(deep, device=DEV) + n                               # the rows' positions
        key = torch.cat((torch.arange(n, device=DEV), at))
        hide = ~torch.cat((torch.ones(t, n, dtype=torch.bool), see), 1).to(DEV)
        if c["window"]:
            hide |= (at[:, None] - key[None] >= c["window"]) & (key >= c["sinks"])[None]
        kept = (~hide).any(0).nonzero()[:, 0]                                 # keys that no row sees are left out
        hide = hide[:, kept]
        kk, vv = (_exact_values(s, name, b, n + t)[kept] for name in "kv")
        for h in range(Hkv):
            for g in range(h * G, (h + 1) * G):
                x = (s["q"][b, :t, g].double() @ kk[:, h].T / math.sqrt(D)).masked_fill(hide, -math.inf)
                lse[b, g, :t] = torch.logsumexp(x, -1)
                o[b, :t, g] = torch.softmax(x, -1) @ vv[:, h]
    return o, lse
