"""The serving calls on the GPU against their plain 64-bit forms: cache append, cached attention (single tokens, chunks,
trees), tree verification, cache compaction, and a decoding loop made of all four."""
import math

import pytest
import torch

import _serving as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
D = 128


def rand(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32).cpu()


def dev_cache(api, k, v, pages):
    return api.KVCache(k.cuda(), v.cuda(), pages.cuda())


# ------------------------------------------------------------------ append
APPEND = [
    # dtype, q/k dtype, B, T, H, Hkv, lens, counts, page, axes
    ("bf16", "bf16", 3, 1, 8, 2, [0, 15, 16], None, 16, (128,)),
    ("fp16", "fp16", 2, 7, 3, 3, [5, 1000], [7, 3], 24, (16, 56, 56)),
    ("bf16", "fp32", 2, 9, 4, 1, [0, 33], [0, 9], 7, (32, 96)),
    ("fp16", "fp32", 1, 130, 1, 1, [70000], None, 128, (128,)),
    ("fp32", "fp32", 2, 5, 5, 5, [3, 250], None, 1, (64, 64)),
    ("fp32", "fp32", 1, 1, 1, 1, [0], None, 8, (128,)),
    ("bf16", "bf16", 5, 3, 70, 7, [2, 4, 6, 8, 10], [3, 2, 1, 0, 3], 8, (128,)),
]


@pytest.mark.parametrize("dtype,src,B,T,H,Hkv,lens,counts,page,axes", APPEND)
@pytest.mark.parametrize("form", ["ids", "ids_f32", "tables"])
def test_append(cuda_lib, dtype, src, B, T, H, Hkv, lens, counts, page, axes, form):
    dt, st = DT[dtype], DT[src]
    q, k, v = rand(1, B, T, H, D, dtype=st) * 3, rand(2, B, T, Hkv, D, dtype=st), rand(3, B, T, Hkv, D, dtype=dt)
    wq, wk = 1 + 0.2 * rand(4, D), 1 + 0.2 * rand(5, D)
    kc, vc, pages = R.make_cache(B, [n + T for n in lens], Hkv, page, dt, 6, fill=0.25)
    first = i32(lens)[:, None] + torch.arange(T, dtype=torch.int32)
    ids = torch.stack([first // (a + 1) * (1 if a == 0 else -1) for a in range(len(axes))], -1).to(torch.int32)
    ang = R.angles(ids, axes, 1e4)
    rot = ids.cuda()
    if form == "ids_f32":
        rot = ids.float().cuda()  # whole numbers up to 70130: exact
    if form == "tables":
        tab = torch.stack((torch.cos(ang), torch.cos(ang)), -1).flatten(-2).float()
        tas = torch.stack((torch.sin(ang), torch.sin(ang)), -1).flatten(-2).float()
        rot = cuda_lib.RopeTables(tab.cuda(), tas.cuda())
    cache = dev_cache(cuda_lib, kc, vc, pages)
    cnt = None if counts is None else i32(counts)
    got = cuda_lib.st_cache_append(q.cuda(), k.cuda(), v.cuda(), wq.cuda(), wk.cuda(), 1e-6, rot, axes, 1e4, cache,
                                   i32(lens).cuda(), counts=None if cnt is None else cnt.cuda())
    cuda_lib.st_check_status()
    yq, sq = R.rotate(q, wq, ang, 1e-6)
    yk, sk = R.rotate(k, wk, ang, 1e-6)
    # fp32 angle (reduced, below pi: 2^-22 of it), sincosf and rsqrt (2^-22 each), five fp32 products; then one rounding
    tol = lambda y, s: R.HALF[dt] * y.abs() + 2.0 ** -19 * s * (1 + R.HALF[dt]) + 2.0 ** -25
    want_k, want_v = kc.double(), vc.double()
    tol_k, tol_v = torch.zeros_like(want_k), torch.zeros_like(want_v)
    for b in range(B):
        c = T if counts is None else counts[b]
        yq[b, c:] = 0
        sq[b, c:] = 0
        if c:
            pg, row = R.slots(pages, page, b, lens[b] + torch.arange(c))
            want_k[pg, row], want_v[pg, row] = yk[b, :c], v[b, :c].double()
            tol_k[pg, row] = tol(yk, sk)[b, :c]
    R.close("q_rot", got, yq, tol(yq, sq))
    R.close("cache.k", cache.k, want_k, tol_k)  # everything else keeps its bits
    R.close("cache.v", cache.v, want_v, tol_v)


def test_append_strided_views_and_in_place(cuda_lib):
    """q, k, v as slices of one projection, q_rot in q's place, the cache as a view of a larger tensor."""
    B, T, H, Hkv, page, lens = 2, 6, 4, 2, 16, [3, 20]
    qkv = rand(1, B, T, H + 2 * Hkv, D, dtype=torch.bfloat16).cuda()
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    q0, k0, v0 = q.cpu(), k.cpu(), v.cpu()
    big = torch.zeros(2, 7, Hkv, page, D, dtype=torch.bfloat16, device="cuda")  # K and V in one, heads before rows
    kc, vc = big[0].transpose(1, 2), big[1].transpose(1, 2)
    pages = i32([[4, 1], [0, 6]])
    w = torch.ones(D)
    ids = (i32(lens)[:, None] + torch.arange(T, dtype=torch.int32))[..., None].contiguous()
    cache = cuda_lib.KVCache(kc, vc, pages.cuda())
    got = cuda_lib.st_cache_append(q, k, v, w.cuda(), w.cuda(), 1e-6, ids.cuda(), (128,), 1e4, cache, i32(lens).cuda(), q_rot=q)
    cuda_lib.st_check_status()
    assert got.data_ptr() == qkv.data_ptr()
    ang = R.angles(ids, (128,), 1e4)
    yq, sq = R.rotate(q0, w, ang, 1e-6)
    yk, sk = R.rotate(k0, w, ang, 1e-6)
    tol = lambda y, s: 2.0 ** -8 * y.abs() + 2.0 ** -18 * s
    R.close("q_rot", got, yq, tol(yq, sq))
    for b in range(B):
        pg, row = R.slots(pages, page, b, lens[b] + torch.arange(T))
        R.close("k", kc.cpu()[pg, row], yk[b], tol(yk, sk)[b])
        assert torch.equal(vc.cpu()[pg, row], v0[b])
    assert torch.equal(qkv[:, :, H:].cpu(), torch.cat((k0, v0), 2))


def test_append_beyond_the_pages(cuda_lib):
    """Rows beyond the page table or with a bad page number are left out, the others enter, and the status says so."""
    x = rand(1, 2, 4, 1, D, dtype=torch.bfloat16).cuda()
    w = torch.ones(D, device="cuda")
    kc = torch.zeros(3, 8, 1, D, dtype=torch.bfloat16, device="cuda")
    cache = cuda_lib.KVCache(kc, kc.clone(), i32([[0, 1], [2, 3]]).cuda())  # page 3 does not exist
    ids = torch.zeros(1, 4, 1, dtype=torch.int32, device="cuda")
    cuda_lib.st_cache_append(x, x, x, w, w, 1e-6, ids, (128,), 1e4, cache, i32([14, 6]).cuda())
    with pytest.raises(cuda_lib.StError) as e:
        cuda_lib.st_check_status()
    assert e.value.status == cuda_lib.ST_ERR_INVALID_ARG
    cuda_lib.st_check_status()  # reported once
    v = cache.v.cpu()
    assert torch.equal(v[1, 6:8], x[0, :2].cpu()) and torch.equal(v[2, 6:8], x[1, :2].cpu())
    v[1, 6:8] = 0
    v[2, 6:8] = 0
    assert not v.any()


# --------------------------------------------------------------- attention
ATTN = [
    # dtype, B, T, H, Hkv, lens, counts, page, tree
    ("bf16", 1, 1, 8, 1, [0], None, 16, False),                        # the very first token
    ("bf16", 1, 1, 1, 1, [1], None, 8, False),
    ("fp16", 3, 1, 12, 4, [127, 128, 129], None, 32, False),            # tile borders
    ("bf16", 5, 1, 32, 8, [0, 5, 640, 1023, 3000], [1, 0, 1, 1, 1], 16, False),
    ("bf16", 2, 7, 5, 1, [300, 2], [7, 4], 24, True),                   # a group of 5 heads
    ("fp16", 2, 61, 14, 2, [777, 64], [61, 50], 64, True),              # 7 heads, several row tiles
    ("bf16", 1, 256, 4, 4, [130], None, 128, True),                     # the largest tree
    ("bf16", 1, 200, 8, 2, [1000], None, 64, False),                    # a chunk after a prefix
    ("fp16", 2, 333, 3, 3, [0, 90], [333, 129], 16, False),             # a prompt from nothing
    ("bf16", 1, 33, 256, 2, [257], None, 256, True),                    # 128 heads a group
    ("bf16", 1, 3, 6, 2, [6000], None, 8, True),
    ("fp32", 1, 1, 4, 2, [700], None, 16, False),
    ("fp32", 2, 13, 16, 2, [2001, 63], [13, 11], 16, True),
    ("fp32", 1, 70, 2, 2, [5], None, 5, False),
    ("bf16", 2, 6, 8, 4, [100, 31], None, 7, True),                     # pages of 7 rows
    ("fp16", 1, 2, 2, 1, [40], None, 1, False),                         # pages of one row
    ("fp32", 5, 1, 8, 2, [0, 3000, 17, 900, 64], [1, 1, 1, 1, 0], 7, False),   # key ranges dealt by length
    ("fp32", 40, 2, 2, 1, [(37 * i * i) % 700 for i in range(40)], None, 16, True),
    ("fp16", 36, 1, 4, 1, [5 * i for i in range(36)], [i % 2 for i in range(36)], 5, False),
    ("fp32", 1, 1, 2, 2, [9000], None, 64, False),                      # as many ranges as an item may have
]


def attn_case(dtype, B, T, H, Hkv, lens, counts, page, is_tree, seed=0, one_tree=False, scale_q=1.0):
    dt = DT[dtype]
    full = [n + (T if counts is None else counts[b]) for b, n in enumerate(lens)]
    k, v, pages = R.make_cache(B, full, Hkv, page, dt, seed + 1)  # NaN wherever nothing was written
    R.fill_prefix(k, v, pages, full, seed + 2)
    q = rand(seed + 3, B, T, H, D, dtype=dt) * scale_q
    parents = R.tree(1 if one_tree else B, T, 4, seed + 4) if is_tree else None
    return q, k, v, pages, parents


@pytest.mark.parametrize("room", ["tight", "wide"])
@pytest.mark.parametrize("dtype,B,T,H,Hkv,lens,counts,page,is_tree", ATTN)
def test_attention(cuda_lib, dtype, B, T, H, Hkv, lens, counts, page, is_tree, room):
    """With page tables that fit the lengths and with ones that leave room for far more (the calls are planned by the
    room, the lengths being on the device)."""
    q, k, v, pages, parents = attn_case(dtype, B, T, H, Hkv, lens, counts, page, is_tree)
    if room == "wide":
        pages = torch.cat((pages, torch.full((B, 200000 // page), -7, dtype=torch.int32)), 1)
    cache = dev_cache(cuda_lib, k, v, pages)
    cnt = None if counts is None else i32(counts)
    cu = lambda t: None if t is None else t.cuda()
    o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda(), counts=cu(cnt), parents=cu(parents))
    cuda_lib.st_check_status()
    ro, rl, bo, bl = R.attention(q, k, v, pages, lens, counts, parents)
    R.close("o", o, ro, bo)
    R.close("lse", lse, rl, bl)
    assert torch.equal(bits(cache.k), bits(k)) and torch.equal(bits(cache.v), bits(v))


@pytest.mark.parametrize("dtype,B,T,H,Hkv,most,page,is_tree", [
    ("bf16", 40, 2, 16, 8, 900, 16, False),   # few rows a head: many short items, odd numbers of key tiles
    ("fp16", 60, 1, 5, 5, 1500, 32, False),
    ("bf16", 7, 1, 20, 5, 600, 16, False),    # clusters of four and of two
    ("fp16", 12, 3, 30, 6, 400, 64, True),
    ("bf16", 9, 70, 16, 8, 1400, 64, True),   # more than a tile of rows a head
    ("fp16", 3, 300, 6, 3, 1000, 8, False),
])
def test_attention_many_items(cuda_lib, dtype, B, T, H, Hkv, most, page, is_tree):
    """More key tiles than SMs, so that each SM works through several items, whole ones and parts."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, most, (B,), generator=g).tolist()
    counts = torch.randint(0, T + 1, (B,), generator=g).tolist()
    q, k, v, pages, parents = attn_case(dtype, B, T, H, Hkv, lens, counts, page, is_tree, seed=40)
    cache = dev_cache(cuda_lib, k, v, pages)
    o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda(), counts=i32(counts).cuda(),
                                    parents=None if parents is None else parents.cuda())
    cuda_lib.st_check_status()
    ro, rl, bo, bl = R.attention(q, k, v, pages, lens, counts, parents)
    R.close("o", o, ro, bo)
    R.close("lse", lse, rl, bl)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_attention_shared_tree_scale_and_repeat(cuda_lib, dtype):
    """One tree for the whole batch, a scale of its own, large scores (a running maximum that moves), and the same bits
    on a second run with a dirty workspace."""
    lens = [500, 3, 129]
    q, k, v, pages, parents = attn_case(dtype, 3, 9, 6, 2, lens, None, 16, True, seed=50, one_tree=True, scale_q=6.0)
    cache = dev_cache(cuda_lib, k, v, pages)
    args = (q.cuda(), cache, i32(lens).cuda())
    ws = torch.full((cuda_lib.st_cache_attn_workspace_size(q.cuda(), cache, parents.cuda()),), 0xFF, dtype=torch.uint8, device="cuda")
    o, lse = cuda_lib.st_cache_attn(*args, parents=parents.cuda(), scale=0.15, workspace=ws)
    o2, lse2 = cuda_lib.st_cache_attn(*args, parents=parents.cuda(), scale=0.15, workspace=ws)
    cuda_lib.st_check_status()
    ro, rl, bo, bl = R.attention(q, k, v, pages, lens, None, parents, scale=0.15)
    R.close("o", o, ro, bo)
    R.close("lse", lse, rl, bl)
    assert torch.equal(bits(o), bits(o2)) and torch.equal(bits(lse), bits(lse2))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_strided_views(cuda_lib, dtype):
    """q and o as BHSD views, a cache with heads before rows and K and V interleaved."""
    dt = DT[dtype]
    B, T, H, Hkv, page, lens = 2, 5, 4, 2, 16, [40, 17]
    q, k, v, pages, _ = attn_case(dtype, B, T, H, Hkv, lens, None, page, False, seed=70)
    kv = torch.stack((k, v), 1).transpose(2, 3).contiguous().cuda()  # N, 2, Hkv, page, D
    cache = cuda_lib.KVCache(kv[:, 0].transpose(1, 2), kv[:, 1].transpose(1, 2), pages.cuda())
    qv = q.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    ro, _, bo, _ = R.attention(q, k, v, pages, lens, None, None)
    turned = [t.permute(1, 2, 0, 3).contiguous().cuda().permute(2, 0, 1, 3) for t in (k, v)]  # pages innermost but D
    for c in (cache, cuda_lib.KVCache(turned[0], turned[1], pages.cuda())):
        o = torch.empty(B, H, T, D, dtype=dt, device="cuda").transpose(1, 2)
        cuda_lib.st_cache_attn(qv, c, i32(lens).cuda(), o=o)
        cuda_lib.st_check_status()
        R.close("o", o, ro, bo)


def test_attention_far_pages(cuda_lib):
    """Pages whose rows lie behind 2^32 elements (and bytes) of the cache."""
    n, page, Hkv = 2050, 2048, 8  # 2050 * 2048 * 8 * 128 > 2^32 elements
    lens, B, T, H = [300, 129], 2, 3, 8
    q, k, v, pages, _ = attn_case("bf16", B, T, H, Hkv, lens, None, page, False, seed=80)
    kc = torch.empty(n, page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    far = n - k.shape[0]
    kc[far:], vc[far:] = k.cuda(), v.cuda()
    cache = cuda_lib.KVCache(kc, vc, torch.where(pages < k.shape[0], pages + far, pages).cuda())
    o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda())
    ro, rl, bo, bl = R.attention(q, k, v, pages, lens, None, None)
    R.close("o", o, ro, bo)
    R.close("lse", lse, rl, bl)
    w = torch.ones(D, device="cuda")
    nv = rand(81, B, T, Hkv, D, dtype=torch.bfloat16)
    cuda_lib.st_cache_append(q.cuda(), nv.cuda(), nv.cuda(), w, w, 1e-6, torch.zeros(1, T, 1, dtype=torch.int32, device="cuda"),
                             (128,), 1e4, cache, i32(lens).cuda())
    cuda_lib.st_cache_keep(cache, i32(lens).cuda(), i32([[1, 2], [0, 2]]).cuda(), i32([2, 2]).cuda())
    cuda_lib.st_check_status()
    for b, src in enumerate(([1, 2], [0, 2])):
        pg, row = R.slots(pages, page, b, lens[b] + torch.arange(2))
        assert torch.equal(cache.v[(pg + far).cuda(), row.cuda()].cpu(), nv[b, src])


def test_attention_bad_lengths_pages_and_parents(cuda_lib):
    """Out-of-range values in device memory are reported and leave the other sequences alone."""
    lens = [20, 9, 30]
    q, k, v, pages, parents = attn_case("bf16", 3, 4, 4, 2, lens, None, 16, True, seed=90)
    ro, rl, bo, bl = R.attention(q, k, v, pages, lens, None, parents)

    def run(lens_, pages_, parents_, good):
        cache = dev_cache(cuda_lib, k, v, pages_)
        o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens_).cuda(), parents=parents_.cuda())
        with pytest.raises(cuda_lib.StError) as e:
            cuda_lib.st_check_status()
        assert e.value.status == cuda_lib.ST_ERR_INVALID_ARG
        for b in good:
            R.close("o", o[b], ro[b], bo[b])
            R.close("lse", lse[b], rl[b], bl[b])
        return o, lse

    run([20, -5, 30], pages, parents, [0, 2])
    run([20, 9, 1 << 30], pages, parents, [0, 1])
    bad = parents.clone()
    bad[1, 2] = 3  # a parent behind its child
    bad[2, 3] = -7
    run(lens, pages, bad, [0])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_on_a_side_stream(cuda_lib, dtype):
    lens = [900, 45]
    q, k, v, pages, parents = attn_case(dtype, 2, 6, 8, 2, lens, None, 16, True, seed=110)
    cache = dev_cache(cuda_lib, k, v, pages)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda(), parents=parents.cuda())
    s.synchronize()
    ro, rl, bo, bl = R.attention(q, k, v, pages, lens, None, parents)
    R.close("o", o, ro, bo)
    R.close("lse", lse, rl, bl)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_attention_without_room(cuda_lib, dtype):
    """A page table without columns, and a cache without pages: nothing is seen, and the status says so."""
    dt = DT[dtype]
    q = rand(1, 2, 3, 4, D, dtype=dt).cuda()
    kc = torch.zeros(2, 16, 2, D, dtype=dt, device="cuda")
    for cache in (cuda_lib.KVCache(kc, kc.clone(), torch.zeros(2, 0, dtype=torch.int32, device="cuda")),):
        o, lse = cuda_lib.st_cache_attn(q, cache, i32([0, 5]).cuda())
        with pytest.raises(cuda_lib.StError):
            cuda_lib.st_check_status()
        assert not o.any() and torch.isinf(lse).all() and (lse < 0).all()
    none = cuda_lib.KVCache(kc[:0], kc[:0].clone(), i32([[0], [1]]).cuda())
    o, lse = cuda_lib.st_cache_attn(q, none, i32([0, 5]).cuda())
    with pytest.raises(cuda_lib.StError):
        cuda_lib.st_check_status()
    assert not o.any()  # pages that do not exist read as zeros
    cuda_lib.st_check_status()


def test_two_streams_at_once(cuda_lib):
    """Calls that overlap on the GPU, each with outputs and a workspace of its own, over one cache that both read."""
    lens = [2900, 1000, 17, 640]
    q, k, v, pages, parents = attn_case("bf16", 4, 20, 16, 8, lens, None, 16, True, seed=120)
    cache = dev_cache(cuda_lib, k, v, pages)
    qd, ln, pd = q.cuda(), i32(lens).cuda(), parents.cuda()
    want, want_lse = cuda_lib.st_cache_attn(qd, cache, ln, parents=pd)
    wide = cuda_lib.KVCache(cache.k, cache.v, torch.cat((cache.pages, torch.zeros(4, 20000, dtype=torch.int32, device="cuda")), 1))
    want2, _ = cuda_lib.st_cache_attn(qd, wide, ln, parents=pd)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, cuda_lib.st_cache_attn(qd, wide if i == 1 else cache, ln, parents=pd)))
    torch.cuda.synchronize()
    cuda_lib.st_check_status()
    for i, (o, lse) in got:
        assert torch.equal(bits(o), bits(want2 if i == 1 else want))
    ro, _, bo, _ = R.attention(q, k, v, pages, lens, None, parents)
    R.close("o", want, ro, bo)
    R.close("o", want2, ro, bo)


def test_attention_rows_do_not_depend_on_the_batch(cuda_lib):
    """A sequence alone and the same one in a batch of other lengths agree within their bounds, padded rows are zero and
    untouched neighbours of strided outputs stay."""
    lens = [350, 3, 900]
    q, k, v, pages, parents = attn_case("fp16", 3, 5, 8, 2, lens, [5, 2, 4], 32, True, seed=130)
    cache = dev_cache(cuda_lib, k, v, pages)
    room = torch.full((3, 7, 10, D), 7.0, dtype=torch.float16, device="cuda")
    o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda(), counts=i32([5, 2, 4]).cuda(), parents=parents.cuda(),
                                    o=room[:, 1:6, 1:9])
    cuda_lib.st_check_status()
    ro, rl, bo, bl = R.attention(q, k, v, pages, lens, [5, 2, 4], parents)
    R.close("o", o, ro, bo)
    R.close("lse", lse, rl, bl)
    room[:, 1:6, 1:9] = 7.0
    assert (room == 7.0).all()
    for b in range(3):
        one = cuda_lib.KVCache(cache.k, cache.v, cache.pages[b:b + 1])
        ob, _ = cuda_lib.st_cache_attn(q[b:b + 1].cuda(), one, i32(lens[b:b + 1]).cuda(), counts=i32([[5, 2, 4][b]]).cuda(),
                                       parents=parents[b:b + 1].cuda())
        R.close("o", ob[0], ro[b], bo[b])


# ------------------------------------------------------------ verification
def probs(seed, *shape, sharp=2.0, dtype=torch.float32):
    return torch.softmax(rand(seed, *shape) * sharp, -1).to(dtype)


def verify_case(B, T, V, branch, drafted, dtype=torch.float32, seed=0):
    target = probs(seed + 1, B, T, V, dtype=dtype)
    draft = torch.softmax(target.float().log() + rand(seed + 2, B, T, V), -1).to(dtype)
    parents = R.tree(B, T, branch, seed + 3)
    g = torch.Generator().manual_seed(seed + 4)
    tokens = torch.zeros(B, T, dtype=torch.int32)
    for b in range(B):
        for i in range(1, T):
            tokens[b, i] = int(torch.multinomial(draft[b, max(0, int(parents[b, i]))].float(), 1, generator=g))
    ua, us = torch.rand(B, T, generator=g), torch.rand(B, generator=g)
    return target, draft if drafted else None, tokens, parents, ua, us


def run_verify(cuda_lib, target, draft, tokens, parents, ua, us, counts=None):
    cu = lambda t: None if t is None else t.cuda()
    got = cuda_lib.st_tree_verify(*(cu(t) for t in (target, draft, tokens, parents, ua, us)), counts=cu(counts))
    return tuple(t.cpu() for t in got)


VERIFY = [
    (1, 6, 32000, 1, True, "fp32"), (1, 1, 5, 1, True, "fp32"), (3, 2, 1, 1, True, "fp32"), (4, 17, 50001, 3, True, "fp32"),
    (16, 61, 999, 6, True, "fp32"), (16, 61, 999, 6, False, "fp32"), (5, 40, 20011, 8, False, "bf16"),
    (6, 30, 8191, 8, True, "bf16"), (7, 30, 4097, 4, True, "fp16"), (2, 1024, 300, 5, True, "fp32"),
    (200, 9, 130, 8, True, "fp32"), (400, 5, 70, 4, False, "fp16"),
    (310, 1, 300001, 1, False, "fp32"),  # one CTA per sequence, slices of more batches than have their sums kept
]


@pytest.mark.parametrize("B,T,V,branch,drafted,dtype", VERIFY)
def test_verify(cuda_lib, B, T, V, branch, drafted, dtype):
    case = verify_case(B, T, V, branch, drafted, DT[dtype], seed=B + T)
    got = run_verify(cuda_lib, *case)
    cuda_lib.st_check_status()
    for name, g, w in zip(("path", "n_accepted", "next_token"), got, R.verify(*case)):
        assert torch.equal(g, w), name


def test_verify_counts_int64_shared_tree_and_strides(cuda_lib):
    B, T, V = 5, 12, 777
    target, draft, tokens, parents, ua, us = verify_case(B, T, V, 3, True, seed=7)
    counts = i32([12, 0, 1, 7, 30])  # 30: cut to T
    parents = parents[:1]
    big = torch.zeros(B, T, 2, V)
    big[:, :, 0], big[:, :, 1] = target, draft
    big = big.cuda()
    tok = tokens.long()
    wide = torch.zeros(B, 2 * T, dtype=torch.int64)
    wide[:, ::2] = tok
    got = cuda_lib.st_tree_verify(big[:, :, 0], big[:, :, 1], wide.cuda()[:, ::2], parents.cuda(), ua.cuda(), us.cuda(),
                                  counts=counts.cuda())
    want = R.verify(target, draft, tok, parents, ua, us, counts)
    assert got[2].dtype == torch.int64
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), w)


def test_verify_borders(cuda_lib):
    """u q = p is no acceptance; equal distributions always accept; a zero residual falls back to p; a repeated guess is
    not accepted after its rejection; u_sample at the end takes the last token with weight."""
    V = 4
    p = torch.tensor([[0.25, 0.25, 0.5, 0.0]] * 3)[None].repeat(4, 1, 1)
    q = torch.tensor([[0.5, 0.25, 0.25, 0.0]] * 3)[None].repeat(4, 1, 1)
    tokens = i32([[0, 0, 0], [0, 2, 2], [0, 0, 1], [0, 3, 2]])
    parents = i32([[-1, 0, 1], [-1, 0, 1], [-1, 0, 0], [-1, 0, 0]])
    ua = torch.tensor([[0, 0.5, 0.1], [0, 0.999, 0.999], [0, 0.75, 0.5], [0, 0.0, 0.3]])
    us = torch.tensor([0.999, 0.75, 0.0, 0.999])
    got = run_verify(cuda_lib, p, q, tokens, parents, ua, us)
    want = R.verify(p, q, tokens, parents, ua, us)
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    assert got[1].tolist() == [1, 3, 1, 2] and got[2].tolist()[0] == 2  # 0.5 * 0.5 < 0.25 is false
    same = run_verify(cuda_lib, q, q, tokens, i32([[-1, 0, 1]]), torch.full((4, 3), 1 - 2.0 ** -24), us)
    assert same[1].tolist() == [3, 3, 3, 1]  # the last one's guess has probability 0
    # without a draft: token 2 (0.5) is rejected, guessed again, and never drawn afterwards
    for u in (0.0, 0.3, 0.49, 0.5, 0.999):
        one = run_verify(cuda_lib, p[:1], None, i32([[0, 2, 2]]), i32([[-1, 0, 0]]), torch.tensor([[0, 0.9, 0.0]]), torch.tensor([u]))
        assert one[1].tolist() == [1] and one[2].tolist() == [0 if u < 0.5 else 1]
    zero = run_verify(cuda_lib, torch.zeros(1, 1, V), None, i32([[0]]), i32([[-1]]), torch.zeros(1, 1), torch.zeros(1))
    assert zero[2].tolist() == [-1]
    lower = run_verify(cuda_lib, p[:1] / 2, q[:1], i32([[0, 0, 0]]), i32([[-1, 0, 0]]), torch.full((1, 3), 0.99), torch.tensor([0.0]))
    want = R.verify(p[:1] / 2, q[:1], i32([[0, 0, 0]]), i32([[-1, 0, 0]]), torch.full((1, 3), 0.99), torch.tensor([0.0]))
    for g, w in zip(lower, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_verify_rows_of_any_alignment(cuda_lib, dtype):
    """Rows that start on any element, and the same rows on 16 bytes: the same walk and the same token."""
    B, T, V = 3, 9, 20001
    target, draft, tokens, parents, ua, us = verify_case(B, T, V, 4, True, DT[dtype], seed=11)
    for d in (draft, None):
        want = R.verify(target, d, tokens, parents, ua, us)
        for pad in (0, 1, 2, 7):
            wide = torch.full((2, B, T, V + pad), 0.5, dtype=DT[dtype])
            wide[0, :, :, :V], wide[1, :, :, :V] = target, draft
            wide = wide.cuda()
            got = cuda_lib.st_tree_verify(wide[0, :, :, :V], None if d is None else wide[1, :, :, :V], tokens.cuda(), parents.cuda(),
                                          ua.cuda(), us.cuda())
            for g, w in zip(got, want):
                assert torch.equal(g.cpu(), w), pad
    cuda_lib.st_check_status()


def test_verify_bad_values(cuda_lib):
    target, draft, tokens, parents, ua, us = verify_case(3, 8, 50, 2, True, seed=21)
    tokens[0, 3], parents[1, 4], tokens[0, 0] = 50, 6, -9  # the root's token is not read
    target[2, 0, 5], draft[2, 0, 6] = float("nan"), -1.0
    got = run_verify(cuda_lib, target, draft, tokens, parents, ua, us)
    with pytest.raises(cuda_lib.StError) as e:
        cuda_lib.st_check_status()
    assert e.value.status == cuda_lib.ST_ERR_INVALID_ARG
    parents[1, 4] = -1  # what the bad parent amounts to
    for g, w in zip(got, R.verify(target, draft, tokens, parents, ua, us)):
        assert torch.equal(g, w)


def test_verify_keeps_the_target_distribution(cuda_lib):
    """The first token after the root is distributed as the target says, whatever the draft (both forms): of N draws each
    frequency lies within six standard deviations."""
    N, V = 60000, 6
    g = torch.Generator().manual_seed(3)
    p = torch.tensor([0.05, 0.4, 0.1, 0.25, 0.0, 0.2])
    q = torch.tensor([0.3, 0.1, 0.1, 0.1, 0.2, 0.2])
    target, draft = p.expand(N, 4, V), q.expand(N, 4, V)
    guesses = torch.multinomial(q, N * 3, replacement=True, generator=g).reshape(N, 3)
    tokens = torch.cat((torch.zeros(N, 1, dtype=torch.long), guesses), 1).to(torch.int32)
    parents = i32([[-1, 0, 0, 0]])
    ua, us = torch.rand(N, 4, generator=g), torch.rand(N, generator=g)
    for d in (draft, None):
        path, n, nxt = run_verify(cuda_lib, target.contiguous(), None if d is None else d.contiguous(), tokens, parents, ua, us)
        first = torch.where(n > 1, tokens.gather(1, path[:, 1:2].clamp(min=0).long())[:, 0], nxt)
        freq = torch.bincount(first, minlength=V).double() / N
        sd = (p.double() * (1 - p.double()) / N).sqrt()
        assert ((freq - p.double()).abs() <= 6 * sd + 1e-12).all(), (freq, p)


# -------------------------------------------------------------------- keep
KEEP = [
    # dtype, B, Hkv, page, start, N, n_rows, T
    ("bf16", 3, 2, 16, [5, 0, 31], 6, [6, 0, 3], 20),
    ("fp16", 1, 1, 8, [0], 700, [700], 1000),
    ("fp32", 2, 3, 7, [10, 3], 400, [400, 399], 900),
    ("bf16", 4, 8, 64, [1, 2, 3, 4], 2100, [2100, 2000, 64, 1], 2500),
    ("bf16", 1, 8, 32, [100], 5000, [5000], 5001),
    ("fp32", 1, 1, 16, [0], 1, [1], 1),
]


@pytest.mark.parametrize("dtype,B,Hkv,page,start,N,n_rows,T", KEEP)
def test_keep(cuda_lib, dtype, B, Hkv, page, start, N, n_rows, T):
    dt = DT[dtype]
    full = [s + T for s in start]
    k, v, pages = R.make_cache(B, full, Hkv, page, dt, 5, fill=1.0)
    R.fill_prefix(k, v, pages, full, 6)
    g = torch.Generator().manual_seed(7)
    rows = torch.rand(B, T, generator=g).argsort(-1)[:, :N].sort(-1).values.to(torch.int32)
    cache = dev_cache(cuda_lib, k, v, pages)
    lens = cuda_lib.st_cache_keep(cache, i32(start).cuda(), rows.cuda(), i32(n_rows).cuda())
    cuda_lib.st_check_status()
    wk, wv = k.clone(), v.clone()
    for b in range(B):
        n = n_rows[b]
        spg, srow = R.slots(pages, page, b, start[b] + rows[b, :n].long())
        dpg, drow = R.slots(pages, page, b, start[b] + torch.arange(n))
        wk[dpg, drow], wv[dpg, drow] = k[spg, srow], v[spg, srow]
    assert torch.equal(bits(cache.k), bits(wk)) and torch.equal(bits(cache.v), bits(wv))
    assert lens.tolist() == [s + n for s, n in zip(start, n_rows)]


def test_keep_nothing(cuda_lib):
    k, v, pages = R.make_cache(2, [32] * 2, 1, 16, torch.float16, 8, fill=3.0)
    cache = dev_cache(cuda_lib, k, v, pages)
    lens = cuda_lib.st_cache_keep(cache, i32([4, 9]).cuda(), torch.zeros(2, 0, dtype=torch.int32, device="cuda"), i32([0, 0]).cuda())
    cuda_lib.st_check_status()
    assert lens.tolist() == [4, 9] and torch.equal(bits(cache.k), bits(k)) and torch.equal(bits(cache.v), bits(v))


def test_keep_bad_rows(cuda_lib):
    """The same row twice, a falling row, a row beyond the pages, counts out of range: reported; the rest moves."""
    k, v, pages = R.make_cache(4, [32] * 4, 1, 16, torch.bfloat16, 8)
    R.fill_prefix(k, v, pages, [32] * 4, 9)
    rows = i32([[1, 1, 5], [4, 2, 6], [2, 40, 50], [0, 1, 2]])
    cache = dev_cache(cuda_lib, k, v, pages)
    lens = cuda_lib.st_cache_keep(cache, i32([0, 0, 0, 30]).cuda(), rows.cuda(), i32([3, 3, 3, 9]).cuda())
    with pytest.raises(cuda_lib.StError) as e:
        cuda_lib.st_check_status()
    assert e.value.status == cuda_lib.ST_ERR_INVALID_ARG
    assert lens.tolist() == [3, 3, 3, 32]
    wv = v.clone()
    for b, (dst, src) in enumerate((([0, 2], [1, 5]), ([0, 2], [4, 6]), ([0], [2]))):
        dpg, drow = R.slots(pages, 16, b, torch.tensor(dst))
        spg, srow = R.slots(pages, 16, b, torch.tensor(src))
        wv[dpg, drow] = v[spg, srow]
    assert torch.equal(bits(cache.v), bits(wv))


# -------------------------------------------------------- together
class Loop:
    """Speculative decoding with a fixed "model": q, k, v and the probabilities of each step are given."""

    def __init__(self, api, dtype, B, T, H, Hkv, page, lens, steps, V, seed):
        self.api, self.dt, self.page = api, DT[dtype], page
        self.lens0 = lens
        self.room = [n + T * (steps + 1) for n in lens]
        self.k, self.v, self.pages = R.make_cache(B, self.room, Hkv, page, self.dt, seed, fill=0.0)
        R.fill_prefix(self.k, self.v, self.pages, lens, seed + 1)
        self.wq, self.wk = 1 + 0.1 * rand(seed + 2, D), 1 + 0.1 * rand(seed + 3, D)
        self.steps = []
        for s in range(steps):
            z = seed + 100 * (s + 1)
            c = dict(q=rand(z, B, T, H, D, dtype=self.dt), k=rand(z + 1, B, T, Hkv, D, dtype=self.dt), v=rand(z + 2, B, T, Hkv, D, dtype=self.dt))
            target, draft, tokens, parents, ua, us = verify_case(B, T, V, 3, s % 2 == 0, seed=z + 3)
            depth = torch.zeros(B, T, dtype=torch.int32)
            for b in range(B):
                for i in range(1, T):
                    depth[b, i] = depth[b, parents[b, i]] + 1
            c.update(target=target, draft=draft, tokens=tokens, parents=parents, ua=ua, us=us, depth=depth)
            self.steps.append(c)

    def step(self, cache, lens, c):
        """One decoding step on device tensors: all four calls on the present stream."""
        api = self.api
        ids = (lens[:, None] + c["depth"])[..., None]
        q = api.st_cache_append(c["q"], c["k"], c["v"], self.wq_, self.wk_, 1e-6, ids, (128,), 1e4, cache, lens)
        o, lse = api.st_cache_attn(q, cache, lens, parents=c["parents"])
        path, n, nxt = api.st_tree_verify(c["target"], c["draft"], c["tokens"], c["parents"], c["ua"], c["us"])
        return o, lse, path, n, nxt, api.st_cache_keep(cache, lens, path, n)

    def to_dev(self):
        self.wq_, self.wk_ = self.wq.cuda(), self.wk.cuda()
        return [{n: None if t is None else t.cuda() for n, t in c.items()} for c in self.steps]


@pytest.mark.parametrize("dtype,H,Hkv,page", [("bf16", 8, 2, 16), ("fp16", 3, 1, 24), ("fp32", 4, 4, 10)])
def test_decoding_loop(cuda_lib, dtype, H, Hkv, page):
    """Three steps: what each step returns follows from the cache before it, and at the end the cache holds exactly the
    accepted rows."""
    B, T = 3, 10
    L = Loop(cuda_lib, dtype, B, T, H, Hkv, page, [0, 37, 250], 3, 40, seed=1000)
    cache = dev_cache(cuda_lib, L.k, L.v, L.pages)
    lens = i32(L.lens0).cuda()
    kept_v = [[L.v[R.slots(L.pages, page, b, torch.arange(n))] for n in [L.lens0[b]]] for b in range(B)]
    for c, d in zip(L.steps, L.to_dev()):
        before = lens.tolist()
        o, lse, path, n, nxt, new = L.step(cache, lens, d)
        cuda_lib.st_check_status()
        ids = (lens.cpu()[:, None] + c["depth"])[..., None]
        yq, _ = R.rotate(c["q"], L.wq, R.angles(ids, (128,), 1e4), 1e-6)
        for got, want in zip((path, n, nxt), R.verify(c["target"], c["draft"], c["tokens"], c["parents"], c["ua"], c["us"])):
            assert torch.equal(got.cpu(), want)
        assert new.tolist() == [x + y for x, y in zip(before, n.tolist())]
        # the attention, from a cache rebuilt with the step's rows (rounded as the append rounds them)
        k2, v2 = cache.k.cpu().clone(), cache.v.cpu().clone()
        yk, _ = R.rotate(c["k"], L.wk, R.angles(ids, (128,), 1e4), 1e-6)
        for b in range(B):
            pg, row = R.slots(L.pages, page, b, before[b] + torch.arange(T))
            k2[pg, row], v2[pg, row] = yk[b].to(L.dt), c["v"][b]
        ro, rl, bo, bl = R.attention(yq.to(L.dt), k2, v2, L.pages, before, None, c["parents"])
        # a row of q' or k' may round to the other neighbour: each element of the sum s then moves by a whole step
        slack = 2 * R.HALF[L.dt]
        smax = (yq.norm(dim=-1).amax() * yk.norm(dim=-1).amax() / math.sqrt(D)).item()
        R.close("o", o, ro, bo + 4 * slack * smax * v2.double().abs().max())
        R.close("lse", lse, rl, bl + 2 * slack * smax)
        for b in range(B):
            kept_v[b].append(c["v"][b, path[b, : n[b]].long().cpu()])
        lens = new
    for b in range(B):
        want = torch.cat(kept_v[b])
        pg, row = R.slots(L.pages, page, b, torch.arange(want.shape[0]))
        assert want.shape[0] == lens[b] and torch.equal(bits(cache.v.cpu()[pg, row]), bits(want))


def test_decoding_step_in_a_graph(cuda_lib):
    """A captured step replayed with other lengths and inputs gives what eager calls give, two graphs side by side."""
    B, T, H, Hkv, page = 3, 10, 8, 2, 16
    L = Loop(cuda_lib, "bf16", B, T, H, Hkv, page, [0, 37, 250], 3, 40, seed=3000)
    steps = L.to_dev()
    steps[1]["draft"] = steps[0]["draft"].clone()  # one form of the call for all replays
    eager_cache = dev_cache(cuda_lib, L.k, L.v, L.pages)
    lens, want = i32(L.lens0).cuda(), []
    for d in steps:
        out = L.step(eager_cache, lens, d)
        want.append([t.clone() for t in out])
        lens = out[-1]
    caches = [dev_cache(cuda_lib, L.k, L.v, L.pages) for _ in range(2)]
    graphs, ins, lns, outs = [], [], [], []
    for cache in caches:
        d = {n: t.clone() for n, t in steps[0].items()}
        ln = i32(L.lens0).cuda()
        k0, v0 = cache.k.clone(), cache.v.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            L.step(cache, ln, d)  # warm-up
        torch.cuda.current_stream().wait_stream(s)
        cache.k.copy_(k0)
        cache.v.copy_(v0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = L.step(cache, ln, d)
        graphs.append(g)
        ins.append(d)
        lns.append(ln)
        outs.append(out)
    for s, d in enumerate(steps):
        for g, i, ln, out in zip(graphs, ins, lns, outs):
            for n in i:
                i[n].copy_(d[n])
            g.replay()
        for out, ln in zip(outs, lns):
            for a, w in zip(out, want[s]):
                assert torch.equal(a, w)
            ln.copy_(out[-1])
    cuda_lib.st_check_status()
    for cache in caches:
        assert torch.equal(bits(cache.k), bits(eager_cache.k)) and torch.equal(bits(cache.v), bits(eager_cache.v))


def test_long_prompt_then_tokens_matches_the_full_attention(cuda_lib):
    """A prompt in two chunks and single tokens through the cache against the library's own causal attention over the
    whole sequence (same norm, rotation and scale)."""
    B, S, H, Hkv, page = 1, 300, 4, 2, 16
    q, k, v = (rand(s, B, S, h, D, dtype=torch.bfloat16).cuda() for s, h in ((1, H), (2, Hkv), (3, Hkv)))
    wq, wk = (1 + 0.1 * rand(4, D)).cuda(), (1 + 0.1 * rand(5, D)).cuda()
    ids = torch.arange(S, dtype=torch.int32, device="cuda")[None, :, None]
    full, lse = cuda_lib.st_rope_attn_fwd(q, k, v, wq, wk, 1e-6, ids, (128,), 1e4, causal=True)
    kc = torch.zeros(-(-S // page), page, Hkv, D, dtype=torch.bfloat16, device="cuda")
    cache = cuda_lib.KVCache(kc, kc.clone(), torch.arange(kc.shape[0], dtype=torch.int32, device="cuda")[None])
    got, got_lse, at = [], [], 0
    for n in (150, 147, 1, 1, 1):
        lens = i32([at]).cuda()
        cut = slice(at, at + n)
        qr = cuda_lib.st_cache_append(q[:, cut], k[:, cut], v[:, cut], wq, wk, 1e-6, ids[:, cut], (128,), 1e4, cache, lens)
        o, l = cuda_lib.st_cache_attn(qr, cache, lens)
        got.append(o)
        got_lse.append(l)
        at += n
    cuda_lib.st_check_status()
    from _parity import compare
    # both sides are within the bf16 parity bound of the exact result
    compare("o", torch.cat(got, 1), full.double().cpu().numpy(), atol=4e-2, rel_fro=2e-2)
    compare("lse", torch.cat(got_lse, 2), lse.double().cpu().numpy(), atol=4e-2, rel_fro=2e-2)
