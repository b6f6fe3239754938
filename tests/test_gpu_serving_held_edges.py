"""Edges of the calls over 8-bit caches, on the GPU: rows beside keys that they do not see, caches without pages, of many
heads and spread over more than 2^32 places, arguments that are not there, CTAs without work, windows behind the table,
quotients near a tie."""
import math

import pytest
import torch

import _serving as R
import _serving_more as M
from test_gpu_serving_more import D, DT, HELD, attend_inputs, dev_cache, gpu, i32, rand

pytestmark = pytest.mark.gpu


def row_by_row(q, c, lens, parents, window, sinks):
    """The 64-bit results and bounds of each row over the keys that it sees and no others. Of V's rows a row's bound has the
    largest that it sees: its weights times V's scales are rounded to fp16 where the largest of them is 2^7, or down to 2^-1
    where V's scales differ by up to 2^8 among 128 keys, and the smallest numbers' half step is 2^-25: 2^-24 of the largest."""
    B, T, H, _ = q.shape
    o, lse = torch.zeros(B, T, H, D, dtype=torch.float64), torch.zeros(B, H, T, dtype=torch.float64)
    bound, lse_bound = torch.zeros_like(o), torch.zeros_like(lse)
    page = c[0].shape[1]
    for b, n in enumerate(lens):
        vis = M.seen(n, T, None if parents is None else parents[b].tolist(), window, sinks)
        for t in range(T):
            kept = vis[t].nonzero()[:, 0]
            pg, row = R.slots(c[2], page, b, kept)
            k, v = (x.view(torch.int8)[pg, row][None].view(x.dtype) for x in c[:2])
            ks, vs = (s[pg, :, row].T[None].contiguous() for s in c[3:])
            m = len(kept)
            w = M.attention(q[b:b + 1, t:t + 1], k, v, i32([[0]]), [m - 1], None, None, scales=(ks, vs))
            top = M.values(v, vs).abs().amax((0, 1, 3)).repeat_interleave(H // k.shape[2])
            o[b, t], bound[b, t] = w[0][0, 0], w[2][0, 0] + (m * 2.0 ** -24 * top)[:, None]
            lse[b, :, t], lse_bound[b, :, t] = w[1][0, :, 0], w[3][0, :, 0]
    return o, lse, bound, lse_bound


@pytest.mark.parametrize("kv", HELD)
@pytest.mark.parametrize("B,T,tree,window", [(2, 6, False, 0), (2, 6, True, 0), (1, 40, False, 0), (2, 50, True, 0),
                                             (2, 6, False, 100), (2, 48, True, 90)])
@pytest.mark.parametrize("wide", [False, True])
def test_rows_beside_much_larger_values(cuda_lib, kv, B, T, tree, window, wide):
    """V rows of 2^40 times a row's own, that it does not see (later rows, other branches, keys before its window), lie in
    its tiles of 128 keys."""
    H, Hkv, page, sinks = 8, 2, 16, 2 if window else 0
    lens = [300, 130][:B]
    q, c, par, _ = attend_inputs("bf16", kv, B, T, H, Hkv, lens, None, page, tree, 0, 0)
    scale = c[4].clone()
    for b, n in enumerate(lens):
        at = torch.arange(n + T)
        up = torch.zeros(n + T)
        up[n + T // 2:] = 1.0            # the later half of the new rows
        if window:
            up[sinks:n - window + 3] = 1.0   # keys that leave the window from the third position on
        pg, row = R.slots(c[2], page, b, at)
        scale[pg, :, row] *= torch.exp2(40 * up - 20)[:, None]
    c = (*c[:4], scale)
    d = c
    if wide:  # dealt over all CTAs instead of clusters
        pages = torch.full((B, 6000), 1 << 30, dtype=torch.int32)
        pages[:, :c[2].shape[1]] = c[2]
        d = (c[0], c[1], pages, c[3], c[4])
    o, lse = cuda_lib.st_cache_attn(q.cuda(), dev_cache(cuda_lib, d), i32(lens).cuda(), parents=gpu(par), window=window, sinks=sinks)
    cuda_lib.st_check_status()
    want = row_by_row(q, c, lens, par, window, sinks)
    R.close("o", o, want[0], want[2])
    R.close("lse", lse, want[1], want[3])


@pytest.mark.parametrize("kv", HELD)
@pytest.mark.parametrize("T", [1, 40])
def test_a_key_with_all_the_weight_and_a_small_value(cuda_lib, kv, T):
    """The key that has nearly the whole weight lies beside one of 2^44 times its V row and 2^-115 of its weight."""
    H, Hkv, page, n = 4, 2, 16, 200
    q, c, _, _ = attend_inputs("bf16", kv, 1, T, H, Hkv, [n], None, page, False, 0, 0, spread=0.0)
    q[:] = q[:, :1, :1]
    pg, row = R.slots(c[2], page, 0, torch.arange(n + T))
    c[4][pg, :, row] *= 2.0 ** -22
    x = q[0, 0, 0].float() / q.float().abs().max()
    held = ((x * M.TOP[DT[kv]]).round()).to(DT[kv]).view(torch.int8)
    for at, sign in ((70, 1.0), (90, -1.0)):
        pg, row = R.slots(c[2], page, 0, torch.tensor([at]))
        c[0].view(torch.int8)[pg, row] = held
        c[3][pg, :, row] = sign * 6.0 / M.TOP[DT[kv]]
    c[4][pg, :, row] *= 2.0 ** 44
    o, lse = cuda_lib.st_cache_attn(q.cuda(), dev_cache(cuda_lib, c), i32([n]).cuda())
    cuda_lib.st_check_status()
    pg, row = R.slots(c[2], page, 0, torch.tensor([90]))
    small = (*c[:4], c[4].clone())
    small[4][pg, :, row] = 0.0           # its own share is below 2^-40 of the result
    want = row_by_row(q, small, [n], None, 0, 0)
    R.close("o", o, want[0], want[2])
    R.close("lse", lse, want[1], want[3])


# ---------------------------------------------------------- caches without pages
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("kv", HELD)
@pytest.mark.parametrize("T,tree", [(1, False), (5, True)])
def test_a_cache_without_pages(cuda_lib, dtype, kv, T, tree):
    """Every page number is out of range: the keys read as zeros, so that O is 0 and LSE the logarithm of their number, and
    the status says so. A table of more than 64 tokens splits the keys."""
    B, H, Hkv, page, lens = 2, 4, 2, 16, [200, 70]
    k = torch.empty(0, page, Hkv, D, dtype=torch.int8, device="cuda").view(DT[kv])
    s = torch.empty(0, Hkv, page, device="cuda")
    cache = cuda_lib.KVCache(k, k.clone(), torch.zeros(B, 20, dtype=torch.int32, device="cuda"), s, s.clone())
    q, par = rand(1, B, T, H, D, dtype=DT[dtype]).cuda(), R.tree(B, T, 2, 3) if tree else None
    o = torch.full_like(q, 7.0)
    _, lse = cuda_lib.st_cache_attn(q, cache, i32(lens).cuda(), parents=gpu(par), o=o)
    with pytest.raises(cuda_lib.StError) as e:
        cuda_lib.st_check_status()
    assert e.value.status == cuda_lib.ST_ERR_INVALID_ARG
    assert bool((o == 0).all())
    for b, n in enumerate(lens):
        seen = M.seen(n, T, None if par is None else par[b].tolist(), 0, 0).sum(-1).double().log()
        # the sum of as many ones, log2 and a product with ln 2, each rounded
        R.close("lse", lse[b], seen.expand(H, T), (2.0 ** -22 * (1 + seen)).expand(H, T))
    rows = i32([[0, 2], [1, 3]]).cuda()
    new = cuda_lib.st_cache_keep(cache, i32([0, 4]).cuda(), rows, i32([2, 2]).cuda())
    assert new.tolist() == [2, 6]
    with pytest.raises(cuda_lib.StError):
        cuda_lib.st_check_status()
    back = cuda_lib.st_cache_read(cache, i32([0, 4]).cuda(), 3, dtype=DT[dtype])
    assert bool((back[0] == 0).all()) and bool((back[1] == 0).all())
    with pytest.raises(cuda_lib.StError):
        cuda_lib.st_check_status()


# ---------------------------------------------------------------- many heads
@pytest.mark.parametrize("kv", HELD)
@pytest.mark.parametrize("Hkv", [16383, 16384, 32767])
def test_keep_of_many_heads(cuda_lib, kv, Hkv):
    """As many heads as a cache may have: rows and scales move all the same."""
    g = torch.Generator(device="cuda").manual_seed(Hkv)
    page, n = 2, 3
    k, v = (torch.randint(-127, 128, (n, page, Hkv, D), generator=g, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.rand(n, Hkv, page, generator=g, device="cuda") for _ in range(2))
    cache = cuda_lib.KVCache(k.view(DT[kv]), v.view(DT[kv]), i32([[2, 0, 1]]).cuda(), ks, vs)
    flat = lambda x, rows_first: (x if rows_first else x.transpose(1, 2))[[2, 0, 1]].reshape(n * page, Hkv, -1).clone()  # noqa: E731
    want = [flat(k, True), flat(v, True), flat(ks, False), flat(vs, False)]
    for w in want:
        w[1:4] = w[[2, 4, 5]].clone()
    lens = cuda_lib.st_cache_keep(cache, i32([1]).cuda(), i32([[1, 3, 4]]).cuda(), i32([3]).cuda())
    cuda_lib.st_check_status()
    assert lens.tolist() == [4]
    for x, rows_first, w in ((k, True, want[0]), (v, True, want[1]), (ks, False, want[2]), (vs, False, want[3])):
        assert torch.equal(flat(x, rows_first), w)


# ------------------------------------------------------- arguments that are not there
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_what_a_cache_needs(cuda_lib, kv):
    """Each call refuses a cache without K, V, pages or (of 8 bits) scales, and calls without lengths or numbers of rows."""
    B, T, H, Hkv, page = 2, 3, 4, 2, 16
    q, c, _, _ = attend_inputs("bf16", kv, B, T, H, Hkv, [20, 7], None, page, False, 0, 0)
    x, k, lens = q.cuda(), rand(2, B, T, Hkv, D, dtype=torch.bfloat16).cuda(), i32([20, 7]).cuda()
    w, ids, rows = torch.ones(D).cuda(), torch.zeros(1, T, 1, dtype=torch.int32).cuda(), i32([[0], [0]]).cuda()
    one = i32([1, 1]).cuda()
    calls = {
        "append": lambda cache, n: cuda_lib.st_cache_append(x, k, k, w, w, 1e-6, ids, (128,), 1e4, cache, n),
        "attn": lambda cache, n: cuda_lib.st_cache_attn(x, cache, n),
        "read": lambda cache, n: cuda_lib.st_cache_read(cache, n, T),
        "keep": lambda cache, n: cuda_lib.st_cache_keep(cache, n, rows, one),
    }
    names = ["k", "v", "pages"] + (["k_scale", "v_scale"] if kv == "e4m3" else [])
    for name, call in calls.items():
        for gone in names:
            cache = dev_cache(cuda_lib, c)
            setattr(cache, gone, None)
            with pytest.raises(cuda_lib.StError) as e:
                call(cache, lens)
            assert e.value.status == cuda_lib.ST_ERR_INVALID_ARG, (name, gone)
        call(dev_cache(cuda_lib, c), lens)
        with pytest.raises(cuda_lib.StError) as e:
            call(dev_cache(cuda_lib, c), None)
        assert e.value.status == cuda_lib.ST_ERR_INVALID_ARG, name
    with pytest.raises(TypeError):
        cuda_lib.st_cache_read(dev_cache(cuda_lib, c), lens, None)
    cuda_lib.st_check_status()


# ------------------------------------------------------------- CTAs without work
@pytest.mark.parametrize("kv", HELD)
@pytest.mark.parametrize("kw", [dict(), dict(window=50, sinks=2), dict(shared=True)])
def test_fewer_tiles_than_ctas(cuda_lib, kv, kw):
    """Short contexts under a wide table leave CTAs without a range. What an earlier kernel left in their shared memory (words
    of 0x7fffffff: V's rows in NaN) must not become the number of a sequence."""
    x = torch.full((64 * 260, 16, 8, 2 * D), -1, dtype=torch.int8, device="cuda").view(torch.bfloat16)
    x.view(torch.int32).fill_(0x7FFFFFFF)
    pages = torch.arange(64 * 260, dtype=torch.int32, device="cuda").view(64, 260)
    q = rand(1, 64, 1, 32, D, dtype=torch.bfloat16).cuda()
    cuda_lib.st_cache_attn(q, cuda_lib.KVCache(torch.zeros_like(x), x, pages), i32([4100] * 64).cuda())
    B, lens = 3, [90, 1, 130]
    q, c, _, _ = attend_inputs("bf16", kv, B, 1, 8, 2, lens, None, 16, False, kw.get("window", 0), kw.get("sinks", 0))
    wide = torch.full((B, 6000), 1 << 30, dtype=torch.int32)
    wide[:, :c[2].shape[1]] = c[2]
    if "shared" in kw:
        kw = dict(shared=i32([0]).cuda())
    o, lse = cuda_lib.st_cache_attn(q.cuda(), dev_cache(cuda_lib, (c[0], c[1], wide, c[3], c[4])), i32(lens).cuda(), **kw)
    cuda_lib.st_check_status()
    want = M.attention(q, c[0], c[1], c[2], lens, None, None, kw.get("window", 0), kw.get("sinks", 0), (c[3], c[4]))
    R.close("o", o, want[0], want[2])
    R.close("lse", lse, want[1], want[3])


# ----------------------------------------------------------- places far apart
@pytest.mark.parametrize("far", ["k", "v", "k_scale", "v_scale"])
@pytest.mark.parametrize("dtype,kv", [("bf16", "e4m3"), ("fp16", "int8"), ("fp32", "int8")])
def test_places_beyond_32_bits(cuda_lib, far, dtype, kv):
    """Pages (16 GB of rows) or scales (2^32 of them, which takes 16-bit rows to the CUDA cores, too) that lie far apart: append,
    read, attention of single tokens, a chunk, a tree, with a window, and compaction, each as over the same cache packed."""
    B, H, Hkv, page, lens = 2, 8, 2, 16, [333, 70]
    T = 5
    c = M.make_cache(B, [n + T for n in lens], Hkv, page, DT[kv], lens, 11, behind=0.0)
    near = dev_cache(cuda_lib, c)
    wide = dev_cache(cuda_lib, c)
    x = getattr(near, far)
    item = x.element_size()
    step = -(-((1 << 34) // item // (x.shape[0] - 1)) // 16 + 1) * 16
    room = torch.empty((x.shape[0] - 1) * step + x[0].numel(), dtype=torch.int8 if item == 1 else x.dtype, device="cuda")
    y = room.as_strided(x.shape, (step, *x.stride()[1:]))
    if item == 1:
        y.copy_(x.view(torch.int8))
        y = y.view(x.dtype)
    else:
        y.copy_(x)
    setattr(wide, far, y)
    pick = lambda cache: [getattr(cache, n) for n in ("k", "v", "k_scale", "v_scale")]  # noqa: E731

    def same(a, b):
        for i, j in zip(a, b):
            i, j = (t.view(torch.int8) if t.element_size() == 1 else t for t in (i, j))
            assert torch.equal(i, j)

    q, k, v = rand(1, B, T, H, D, dtype=DT[dtype]).cuda(), *(rand(s, B, T, Hkv, D, dtype=DT[dtype]).cuda() for s in (2, 3))
    w, ids, dl = torch.ones(D).cuda(), torch.zeros(1, T, 1, dtype=torch.int32).cuda(), i32(lens).cuda()
    qr = [cuda_lib.st_cache_append(q, k, v, w, w, 1e-6, ids, (128,), 1e4, cache, dl) for cache in (near, wide)]
    same(pick(near), pick(wide))
    same(qr[:1], qr[1:])
    same(*(cuda_lib.st_cache_read(cache, dl - 60, 60 + T) for cache in (near, wide)))
    qr, host = qr[0].cpu(), [t.cpu() for t in pick(near)]
    par = R.tree(B, T, 3, 3)
    for rows, parents, window, sinks in ((1, None, 0, 0), (T, None, 0, 0), (T, par, 0, 0), (T, None, 100, 3), (T, par, 30, 0)):
        o, lse = cuda_lib.st_cache_attn(qr[:, :rows].cuda(), wide, dl, parents=gpu(parents), window=window, sinks=sinks)
        want = M.attention(qr[:, :rows], host[0], host[1], c[2], lens, None, parents, window, sinks, (host[2], host[3]))
        R.close("o", o, want[0], want[2])
        R.close("lse", lse, want[1], want[3])
    rows = i32([[0, 2, 4], [1, 3, 4]]).cuda()
    for cache in (near, wide):
        cuda_lib.st_cache_keep(cache, dl, rows, i32([3, 2]).cuda())
    same(pick(near), pick(wide))
    cuda_lib.st_check_status()


# ------------------------------------------------------- windows behind the table
@pytest.mark.parametrize("dtype,kv,page", [("bf16", "bf16", 16), ("fp16", "e4m3", 16), ("bf16", "int8", 5), ("fp32", "fp32", 16), ("fp32", "int8", 8)])
@pytest.mark.parametrize("B,sinks", [(2, 3), (2, 150), (90, 1), (90, 130)])
def test_windows_behind_the_table_leave_the_first_tokens(cuda_lib, dtype, kv, page, B, sinks):
    """Lengths beyond the page table's room: a row sees the first tokens, and nothing else is in its window."""
    q, c, _, _ = attend_inputs(dtype, kv, B, 1, 4, 2, [200] * B, None, page, False, 0, 0)
    o, lse = cuda_lib.st_cache_attn(q.cuda(), dev_cache(cuda_lib, c), i32([1 << 30] * B).cuda(), window=30, sinks=sinks)
    with pytest.raises(cuda_lib.StError):
        cuda_lib.st_check_status()
    want = M.attention(q, c[0], c[1], c[2], [sinks - 1] * B, None, None, scales=None if c[3] is None else (c[3], c[4]))
    R.close("o", o, want[0], want[2])
    R.close("lse", lse, want[1], want[3])


# ------------------------------------------------------------ quotients near a tie
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T", [3, 700])
def test_v_in_int8_is_what_elementwise_code_holds(cuda_lib, dtype, T):
    """v and its scales bit for bit as max / 127, x / scale and the rounding to nearest even in fp32: 16-bit rows have quotients
    on and next to ties, which a product with 1 / scale sends to the other side."""
    B, Hkv, page = 2, 5, 16
    v = (rand(1, B, T, Hkv, D) * torch.exp2(rand(2, B, T, Hkv, 1) * 2)).to(DT[dtype])
    v[0, 1] = 0
    v[1, :, 0] = (torch.randint(-127, 128, (T, D), generator=torch.Generator().manual_seed(4)) + 0.5).to(DT[dtype])
    v[1, :, 0, 5] = 127 * 4                              # scale 4: every eighth quotient is a tie
    v[1, :, 1] = v[1, :, 0] * 3
    v[1, :, 1, 5] = 127 * 1.5                            # some larger than the row's fifth, scales with many bits
    c = M.make_cache(B, [T] * B, Hkv, page, torch.int8, [0] * B, 3, behind=0.0)
    cache = dev_cache(cuda_lib, c)
    w, ids, k = torch.ones(D).cuda(), torch.zeros(1, T, 1, dtype=torch.int32).cuda(), rand(3, B, T, Hkv, D, dtype=DT[dtype]).cuda()
    cuda_lib.st_cache_append(k, k, v.cuda(), w, w, 1e-6, ids, (128,), 1e4, cache, i32([0] * B).cuda())
    cuda_lib.st_check_status()
    s = v.float().abs().amax(-1) / 127.0
    held = (v.float() / torch.where(s > 0, s, torch.ones_like(s))[..., None]).round().to(torch.int8)
    for b in range(B):
        pg, row = R.slots(c[2], page, b, torch.arange(T))
        assert torch.equal(cache.v_scale.cpu()[pg, :, row], s[b])
        assert torch.equal(cache.v.cpu()[pg, row], held[b])


def test_v_in_int8_of_every_size(cuda_lib):
    """fp32 rows from 2^-92 (scales near the least that is held) to 2^120, their elements as much as 2^60 apart."""
    B, T, Hkv, page = 1, 2000, 3, 16
    g = torch.Generator().manual_seed(9)
    v = rand(1, B, T, Hkv, D) * torch.exp2(-60 * torch.rand(B, T, Hkv, D, generator=g) ** 4)
    v = v * torch.exp2(torch.randint(-92, 119, (B, T, Hkv, 1), generator=g).float())
    c = M.make_cache(B, [T], Hkv, page, torch.int8, [0], 3, behind=0.0)
    cache = dev_cache(cuda_lib, c)
    w, ids, k = torch.ones(D).cuda(), torch.zeros(1, T, 1, dtype=torch.int32).cuda(), rand(3, B, T, Hkv, D).cuda()
    cuda_lib.st_cache_append(k, k, v.cuda(), w, w, 1e-6, ids, (128,), 1e4, cache, i32([0]).cuda())
    s = v.abs().amax(-1) / 127.0
    s = torch.where(s < 2.0 ** -100, torch.zeros_like(s), s)
    held = torch.where(s[..., None] > 0, v / s[..., None], torch.zeros_like(v)).round().to(torch.int8)
    pg, row = R.slots(c[2], page, 0, torch.arange(T))
    assert torch.equal(cache.v_scale.cpu()[pg, :, row], s[0])
    assert torch.equal(cache.v.cpu()[pg, row], held[0])
