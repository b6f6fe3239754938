"""Caches of 8 bits (append, read, attention, compaction), attention with a window and visible first tokens, and with a
shared prefix, on the GPU against their plain 64-bit forms; a decoding loop made of all of it."""
import math

import pytest
import torch

import _serving as R
import _serving_more as M

pytestmark = pytest.mark.gpu

DT, D = M.DT, 128
HELD = ("e4m3", "int8")


def rand(seed, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


def bits(t):
    return t.contiguous().view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu()


def gpu(x):
    return None if x is None else x.cuda()


def dev_cache(api, c):
    return api.KVCache(*(gpu(x) for x in c))


# ------------------------------------------------------------------ append
APPEND = [
    # dtype, q/k dtype, B, T, H, Hkv, lens, counts, page, axes
    ("bf16", "bf16", 3, 1, 8, 2, [0, 15, 16], None, 16, (128,)),
    ("fp16", "fp32", 2, 9, 4, 1, [0, 33], [0, 9], 7, (32, 96)),
    ("fp32", "fp32", 2, 5, 5, 5, [3, 250], None, 1, (64, 64)),
    ("bf16", "bf16", 5, 3, 70, 7, [2, 4, 6, 8, 10], [3, 2, 1, 0, 3], 8, (16, 56, 56)),
    ("fp16", "fp16", 2, 700, 3, 3, [5, 1000], [700, 300], 24, (128,)),
    ("bf16", "fp32", 2, 1300, 6, 6, [5, 1], None, 64, (128,)),
]


def held_tolerance(y, s, kv):
    """Half a step of what is held: 2^-4 of it and at least 2^-10 (e4m3), 1/2 (int8), in units of the scale. The quotient
    y / s that is rounded is a product with fl(1 / s): off by (1 + 2^-24)^2 - 1 < 2^-22.9 of itself, that is, of y, which a
    quotient near a tie adds to the half step (63.5 s + 2^-23 y is rounded to 64 s where 63 s is as near)."""
    s = s.double()[..., None]
    return (0.5 * s if kv == torch.int8 else torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s)) + 2.0 ** -22.9 * y.abs()


@pytest.mark.parametrize("dtype,src,B,T,H,Hkv,lens,counts,page,axes", APPEND)
@pytest.mark.parametrize("kv", HELD)
def test_append(cuda_lib, dtype, src, B, T, H, Hkv, lens, counts, page, axes, kv):
    dt, st, kt = DT[dtype], DT[src], DT[kv]
    q, k, v = rand(1, B, T, H, D, dtype=st) * 3, rand(2, B, T, Hkv, D, dtype=st), rand(3, B, T, Hkv, D, dtype=dt)
    v[:, 0, 0] = 0                                       # a row of zeros
    wq, wk = 1 + 0.2 * rand(4, D), 1 + 0.2 * rand(5, D)
    c = M.make_cache(B, [n + T for n in lens], Hkv, page, kt, lens, 6)
    before = [x.clone() for x in c]
    ids = (i32(lens)[:, None] + torch.arange(T, dtype=torch.int32))[..., None].expand(B, T, len(axes)).contiguous()
    cache = dev_cache(cuda_lib, c)
    cnt = None if counts is None else i32(counts)
    got = cuda_lib.st_cache_append(q.cuda(), k.cuda(), v.cuda(), wq.cuda(), wk.cuda(), 1e-6, ids.cuda(), axes, 1e4, cache,
                                   i32(lens).cuda(), counts=gpu(cnt))
    cuda_lib.st_check_status()
    assert got.dtype == dt
    ang = R.angles(ids, axes, 1e4)
    yq, sq = R.rotate(q, wq, ang, 1e-6)
    yk, sk = R.rotate(k, wk, ang, 1e-6)
    # the rows in fp32: 2^-19 of the terms (fp32 angle, sincosf, rsqrt, five products), then the rounding that is meant
    for b in range(B):
        yq[b, T if counts is None else counts[b]:] = 0
        sq[b, T if counts is None else counts[b]:] = 0
    R.close("q_rot", got, yq, R.HALF[dt] * yq.abs() + 2.0 ** -19 * sq * (1 + R.HALF[dt]) + 2.0 ** -25)
    after = [x.cpu() for x in (cache.k, cache.v, None or cache.pages, cache.k_scale, cache.v_scale)]
    same_q = torch.ones(c[0].shape[:2], dtype=torch.bool)  # slots that nothing was written to
    for i, (y, size) in enumerate(((yk, 2.0 ** -19 * sk), (v.double(), torch.zeros_like(yk)))):
        for b in range(B):
            n = T if counts is None else counts[b]
            if n == 0:
                continue
            pg, row = R.slots(c[2], page, b, lens[b] + torch.arange(n))
            same_q[pg, row] = False
            s = after[3 + i][pg, :, row]
            want = y[b, :n].abs().amax(-1) / M.TOP[kt]
            R.close("scale", s, want, size[b, :n].amax(-1) / M.TOP[kt] + 2.0 ** -23 * want)
            val = after[i].view(torch.int8)[pg, row].view(kt).double() * s.double()[..., None]
            R.close("value", val, y[b, :n], held_tolerance(y[b, :n], s, kt) * (1 + 2.0 ** -20) + size[b, :n] + 2.0 ** -40)
    for i in (0, 1):  # everything else keeps its bits
        assert torch.equal(bits(after[i])[same_q], bits(before[i])[same_q])
        assert torch.equal(bits(after[3 + i].transpose(1, 2))[same_q], bits(before[3 + i].transpose(1, 2))[same_q])


@pytest.mark.parametrize("kv", HELD)
def test_rows_that_are_not_finite_or_tiny(cuda_lib, kv):
    """A row with an infinity or NaN reads as NaN, a row below 2^-100 as zeros; their neighbours are as ever."""
    kt, T = DT[kv], 6
    v = rand(1, 1, T, 2, D)
    v[0, 1, 0, 5], v[0, 2, 1, 7] = math.inf, math.nan
    v[0, 3, 0] = 2.0 ** -96                              # scales 2^-105 and 2^-103
    v[0, 4, 1] *= 2.0 ** -60
    k = rand(2, 1, T, 2, D)
    c = M.make_cache(1, [T], 2, 8, kt, [0], 3, behind=0.0)
    cache = dev_cache(cuda_lib, c)
    w, ids = torch.ones(D).cuda(), torch.zeros(1, T, 1, dtype=torch.int32).cuda()
    start = i32([0]).cuda()
    cuda_lib.st_cache_append(k.cuda(), k.cuda(), v.cuda(), w, w, 1e-6, ids, (128,), 1e4, cache, start)
    _, got = cuda_lib.st_cache_read(cache, start, T, dtype=torch.float32)
    got = got.cpu()
    for t in range(T):
        for h in range(2):
            if (t, h) in ((1, 0), (2, 1)):
                assert got[0, t, h].isnan().all()
            elif (t, h) == (3, 0):
                assert (got[0, t, h] == 0).all()
            else:
                y = v[0, t, h].double()
                s = y.abs().amax() / M.TOP[kt]
                R.close("row", got[0, t, h], y, held_tolerance(y[None], s[None], kt)[0] * (1 + 2.0 ** -20))


def test_fp32_rows_are_divided_into_int8(cuda_lib):
    """v of fp32 is held as elementwise fp32 code holds it, bit for bit, scales too."""
    B, T, Hkv = 2, 300, 3
    v = rand(1, B, T, Hkv, D) * torch.exp2(rand(2, B, T, Hkv, 1) * 8)
    c = M.make_cache(B, [T] * B, Hkv, 16, torch.int8, [0] * B, 3, behind=0.0)
    cache = dev_cache(cuda_lib, c)
    w, ids = torch.ones(D).cuda(), torch.zeros(1, T, 1, dtype=torch.int32).cuda()
    k = rand(3, B, T, Hkv, D).cuda()
    cuda_lib.st_cache_append(k, k, v.cuda(), w, w, 1e-6, ids, (128,), 1e4, cache, i32([0] * B).cuda())
    s = v.abs().amax(-1) / 127.0
    want = (v / s[..., None]).round().to(torch.int8)
    for b in range(B):
        pg, row = R.slots(c[2], 16, b, torch.arange(T))
        assert torch.equal(cache.v.cpu()[pg, row], want[b]) and torch.equal(cache.v_scale.cpu()[pg, :, row], s[b])


def test_append_beyond_the_pages(cuda_lib):
    x = rand(1, 2, 4, 1, D, dtype=torch.bfloat16).cuda()
    w = torch.ones(D, device="cuda")
    k = torch.zeros(3, 8, 1, D, dtype=torch.int8, device="cuda")
    s = torch.full((3, 1, 8), -1.0, device="cuda")
    cache = cuda_lib.KVCache(k, k.clone(), i32([[0, 1], [2, 3]]).cuda(), s, s.clone())  # page 3 does not exist
    ids = torch.zeros(1, 4, 1, dtype=torch.int32, device="cuda")
    cuda_lib.st_cache_append(x, x, x, w, w, 1e-6, ids, (128,), 1e4, cache, i32([14, 6]).cuda())
    with pytest.raises(cuda_lib.StError) as e:
        cuda_lib.st_check_status()
    assert e.value.status == cuda_lib.ST_ERR_INVALID_ARG
    cuda_lib.st_check_status()
    written = torch.zeros(3, 8, dtype=torch.bool)
    written[1, 6:], written[2, 6:] = True, True
    for sc in (cache.k_scale, cache.v_scale):
        assert torch.equal(sc.cpu()[:, 0] > 0, written) and bool((sc.cpu()[:, 0][~written] == -1).all())
    # a negative length names no position
    cuda_lib.st_cache_append(x, x, x, w, w, 1e-6, ids, (128,), 1e4, cache, i32([-2, 0]).cuda())
    with pytest.raises(cuda_lib.StError):
        cuda_lib.st_check_status()
    assert bool((cache.k_scale.cpu()[0, 0] == -1).all())


# -------------------------------------------------------------------- read
READ = [
    # cache, out, B, T, Hkv, start, counts, page
    ("e4m3", "bf16", 3, 5, 2, [0, 7, 30], [5, 0, 3], 16),
    ("int8", "fp16", 2, 33, 8, [3, 100], None, 24),
    ("e4m3", "fp32", 1, 1, 1, [0], None, 1),
    ("int8", "bf16", 2, 19, 3, [11, 2], [19, 18], 7),
    ("e4m3", "fp16", 1, 130, 11, [900], None, 64),
    ("bf16", "bf16", 2, 21, 5, [4, 0], [7, 21], 8),
    ("fp16", "fp16", 1, 9, 1, [60], None, 16),
    ("fp32", "fp32", 2, 17, 2, [1, 40], None, 5),
]


@pytest.mark.parametrize("kv,out,B,T,Hkv,start,counts,page", READ)
@pytest.mark.parametrize("strided", [0, 1, 2])
def test_read(cuda_lib, kv, out, B, T, Hkv, start, counts, page, strided):
    kt, ot = DT[kv], DT[out]
    n = [a + T for a in start]
    c = M.make_cache(B, n, Hkv, page, kt, n, 1, spread=6.0)
    cache = dev_cache(cuda_lib, c)
    cnt = None if counts is None else i32(counts)
    outs = {}
    if strided:  # heads before rows, in one buffer, with room between
        big = torch.full((2, B, Hkv, T, 2 * D), 7.0, dtype=ot, device="cuda")
        outs = dict(k=big[0, ..., :D].transpose(1, 2), v=big[1, ..., :D].transpose(1, 2))
    if strided == 2:  # K's rows begin on 16 bytes and not on 32
        at = 16 // ot.itemsize
        outs["k"] = big[0, ..., at:at + D].transpose(1, 2)
    got = cuda_lib.st_cache_read(cache, i32(start).cuda(), T, counts=gpu(cnt), dtype=ot, **outs)
    cuda_lib.st_check_status()
    for x, s, y in zip(c[:2], c[3:], got):
        assert y.dtype == ot and y.shape == (B, T, Hkv, D)
        want = torch.zeros(B, T, Hkv, D, dtype=ot)
        for b in range(B):
            m = T if counts is None else counts[b]
            if m:
                pg, row = R.slots(c[2], page, b, start[b] + torch.arange(m))
                if s is None:
                    want[b, :m] = x[pg, row]
                else:
                    held = x.view(torch.int8)[pg, row].view(kt).float()
                    want[b, :m] = (held * s[pg, :, row][..., None]).to(ot)  # one fp32 product, one rounding
        assert torch.equal(y.cpu(), want)
    if strided == 1:
        assert bool((big[..., D:] == 7).all())
    elif strided == 2:
        assert bool((big[0, ..., :at] == 7).all()) and bool((big[0, ..., at + D:] == 7).all()) and bool((big[1, ..., D:] == 7).all())


def test_read_out_of_range(cuda_lib):
    c = M.make_cache(2, [16, 16], 2, 8, torch.int8, [16, 16], 1)
    c[2][1, 1] = 99                                      # no such page
    cache = dev_cache(cuda_lib, c)
    for start in ([10, 6], [-3, 0]):
        k, v = cuda_lib.st_cache_read(cache, i32(start).cuda(), 8)
        with pytest.raises(cuda_lib.StError):
            cuda_lib.st_check_status()
        for b in range(2):
            for t in range(8):
                pos = start[b] + t
                ok = start[b] >= 0 and pos < 16 and not (b == 1 and pos >= 8)
                assert bool((k[b, t] != 0).any()) == ok and bool((v[b, t] != 0).any()) == ok


# -------------------------------------------------------------------- keep
@pytest.mark.parametrize("kv", HELD)
@pytest.mark.parametrize("B,Hkv,page,N", [(3, 2, 16, 5), (1, 1, 7, 40), (2, 8, 64, 3000), (40, 8, 8, 9)])
def test_keep(cuda_lib, kv, B, Hkv, page, N):
    kt = DT[kv]
    g = torch.Generator().manual_seed(N)
    start = [int(x) for x in torch.randint(0, 50, (B,), generator=g)]
    room = [a + 2 * N + 3 for a in start]
    c = M.make_cache(B, room, Hkv, page, kt, room, 2)
    rows = torch.stack([torch.randperm(2 * N + 3, generator=g)[:N].sort().values for _ in range(B)]).to(torch.int32)
    rows[0, :2] = i32([0, 1])
    rows[0] = rows[0].sort().values
    if len(set(rows[0].tolist())) < N:
        rows[0] = torch.arange(N, dtype=torch.int32)
    n = i32([N if b % 3 else N - N // 4 for b in range(B)])
    cache = dev_cache(cuda_lib, c)
    lens = cuda_lib.st_cache_keep(cache, i32(start).cuda(), rows.cuda(), n.cuda())
    cuda_lib.st_check_status()
    assert torch.equal(lens.cpu(), i32(start) + n)
    want = [x.clone() for x in c]
    for b in range(B):
        m = int(n[b])
        p0, r0 = R.slots(c[2], page, b, start[b] + rows[b, :m].long())
        p1, r1 = R.slots(c[2], page, b, start[b] + torch.arange(m))
        for i in (0, 1):
            want[i].view(torch.int8)[p1, r1] = c[i].view(torch.int8)[p0, r0]
            want[3 + i][p1, :, r1] = c[3 + i][p0, :, r0]
    for x, y in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), (want[0], want[1], want[3], want[4])):
        assert torch.equal(bits(x), bits(y))


# --------------------------------------------------------------- attention
ATTEND = [
    # dtype, cache, B, T, H, Hkv, lens, counts, page, tree, window, sinks
    ("bf16", "e4m3", 1, 1, 8, 2, [0], None, 16, False, 0, 0),
    ("fp16", "int8", 1, 1, 8, 2, [300], None, 16, False, 0, 0),
    ("bf16", "e4m3", 3, 1, 32, 8, [127, 128, 500], None, 16, False, 0, 0),
    ("bf16", "int8", 2, 7, 12, 3, [5, 1000], [7, 0], 24, False, 0, 0),
    ("fp16", "e4m3", 2, 40, 8, 2, [0, 200], [40, 13], 8, False, 0, 0),
    ("bf16", "e4m3", 2, 61, 14, 2, [77, 900], [61, 50], 64, True, 0, 0),
    ("fp16", "int8", 1, 150, 4, 4, [33], None, 128, True, 0, 0),
    ("bf16", "int8", 5, 3, 7, 7, [1, 2, 3, 4, 5], None, 7, True, 0, 0),
    ("bf16", "e4m3", 2, 3, 4, 2, [300, 7], None, 1, False, 0, 0),
    ("fp32", "e4m3", 2, 5, 6, 2, [0, 333], [5, 4], 16, False, 0, 0),
    ("fp32", "int8", 2, 9, 4, 1, [100, 65], None, 5, True, 0, 0),
    ("bf16", "bf16", 2, 1, 8, 2, [700, 40], None, 16, False, 100, 0),
    ("bf16", "bf16", 1, 1, 8, 2, [2000], None, 16, False, 1, 0),
    ("fp16", "fp16", 2, 30, 6, 3, [900, 0], [30, 11], 32, False, 7, 3),
    ("bf16", "bf16", 2, 200, 4, 2, [1500, 333], None, 64, False, 256, 130),
    ("bf16", "bf16", 1, 300, 8, 8, [0], None, 16, False, 50, 4),
    ("fp16", "fp16", 3, 40, 8, 2, [513, 1027, 3], [40, 7, 39], 8, True, 20, 1),
    ("bf16", "bf16", 2, 61, 16, 4, [1200, 130], None, 128, True, 4, 0),
    ("bf16", "bf16", 2, 20, 4, 4, [400, 90], None, 12, True, 33, 5),      # CUDA cores
    ("fp32", "fp32", 2, 13, 8, 2, [1700, 60], [13, 12], 16, True, 100, 17),
    ("fp32", "fp32", 2, 70, 4, 4, [300, 5], None, 3, False, 64, 2),
    ("fp32", "fp32", 9, 1, 2, 1, [2100, 1, 0, 64, 65, 500, 1000, 15, 16], None, 16, False, 130, 16),
    ("bf16", "e4m3", 2, 1, 16, 2, [3000, 50], None, 32, False, 333, 4),
    ("fp16", "e4m3", 2, 33, 8, 2, [1000, 129], [33, 30], 16, True, 12, 2),
    ("bf16", "int8", 1, 260, 8, 4, [700], None, 64, False, 128, 128),
    ("fp32", "int8", 3, 4, 4, 2, [600, 31, 0], None, 16, False, 40, 1),
    ("fp16", "int8", 12, 1, 4, 1, list(range(0, 1200, 100)), None, 40, False, 0, 0),
    ("bf16", "e4m3", 30, 2, 8, 8, list(range(10, 640, 21)), None, 16, False, 64, 4),
    ("bf16", "bf16", 2, 4, 128, 1, [300, 1], None, 16, False, 1 << 30, 0),
    ("bf16", "e4m3", 1, 129, 128, 1, [10], None, 8, False, 0, 0),
    # whole tiles of 128 rows and several short sequences for each CTA: every stage is used again and again
    ("bf16", "int8", 60, 32, 16, 4, [(37 * i) % 500 for i in range(60)], None, 64, True, 0, 0),
    ("fp16", "e4m3", 60, 32, 16, 4, [(37 * i) % 400 for i in range(60)], None, 16, False, 0, 0),
    ("fp16", "int8", 50, 70, 8, 4, [(53 * i) % 300 for i in range(50)], None, 32, False, 90, 9),
    # many tiles of one sequence for each CTA: few rows, one query tile, two
    ("bf16", "e4m3", 3, 1, 16, 8, [60000, 33333, 50001], None, 16, False, 0, 0),
    ("fp16", "int8", 2, 12, 16, 4, [70000, 60003], None, 48, False, 0, 0),
    ("bf16", "int8", 1, 100, 16, 8, [50000], None, 64, False, 0, 0),
    ("fp16", "e4m3", 1, 70, 16, 8, [60000], None, 64, True, 30000, 200),
]


def attend_inputs(dtype, kv, B, T, H, Hkv, lens, counts, page, tree, window, sinks, spread=2.0):
    dt, kt = DT[dtype], DT[kv]
    rows = [n + (T if counts is None else counts[b]) for b, n in enumerate(lens)]
    c = M.make_cache(B, [n + T for n in lens], Hkv, page, kt, rows, 11, spread=spread)
    q = rand(1, B, T, H, D, dtype=dt) * 2
    par = R.tree(B, T, 5, 3) if tree else None
    if window:  # pages that no row's window reaches, nor the first tokens lie in, are gone
        for b, n in enumerate(lens):
            for j in range(c[2].shape[1]):
                if j * page >= sinks and (j + 1) * page <= n - window + 1:
                    c[2][b, j] = -5
    return q, c, par, None if counts is None else i32(counts)


@pytest.mark.parametrize("case", ATTEND, ids=lambda c: "-".join(str(x) for x in c if not isinstance(x, list)))
def test_attention(cuda_lib, case):
    dtype, kv, B, T, H, Hkv, lens, counts, page, tree, window, sinks = case
    q, c, par, cnt = attend_inputs(*case)
    # rows of q behind the counts may hold anything
    if cnt is not None:
        for b in range(B):
            q[b, int(cnt[b]):] = math.nan
    cache = dev_cache(cuda_lib, c)
    o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda(), counts=gpu(cnt), parents=gpu(par), window=window, sinks=sinks)
    cuda_lib.st_check_status()
    assert o.dtype == q.dtype
    scales = None if c[3] is None else (c[3], c[4])
    want = M.attention(q, c[0], c[1], c[2], lens, cnt, par, window, sinks, scales)
    R.close("o", o, want[0], want[2])
    R.close("lse", lse, want[1], want[3])
    for _ in range(4):
        again = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda(), counts=gpu(cnt), parents=gpu(par), window=window, sinks=sinks)
        assert torch.equal(bits(again[0]), bits(o)) and torch.equal(bits(again[1]), bits(lse))


@pytest.mark.parametrize("dtype,kv", [("bf16", "bf16"), ("fp16", "e4m3"), ("bf16", "int8"), ("fp32", "fp32")])
@pytest.mark.parametrize("B,T,tree", [(3, 1, False), (2, 9, True), (2, 140, False)])
def test_wide_tables(cuda_lib, dtype, kv, B, T, tree):
    """A page table with room for far more than the contexts: keys dealt out over all CTAs instead of clusters."""
    for window, sinks in ((0, 0), (77, 3)):
        lens = [800, 1, 260][:B]
        q, c, par, _ = attend_inputs(dtype, kv, B, T, 8, 2, lens, None, 16, tree, window, sinks)
        wide = torch.full((B, 6000), 1 << 30, dtype=torch.int32)
        wide[:, :c[2].shape[1]] = c[2]
        cache = dev_cache(cuda_lib, (c[0], c[1], wide, c[3], c[4]))
        o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda(), parents=gpu(par), window=window, sinks=sinks)
        cuda_lib.st_check_status()
        want = M.attention(q, c[0], c[1], c[2], lens, None, par, window, sinks, None if c[3] is None else (c[3], c[4]))
        R.close("o", o, want[0], want[2])
        R.close("lse", lse, want[1], want[3])


@pytest.mark.parametrize("window,sinks", [(64, 0), (200, 5)])
@pytest.mark.parametrize("dtype,kv,page", [("bf16", "bf16", 16), ("bf16", "e4m3", 32), ("fp32", "fp32", 16), ("fp16", "int8", 5)])
def test_keys_outside_the_window_hold_anything(cuda_lib, dtype, kv, page, window, sinks):
    """NaN in rows (and scales) that no row sees, in pages that are there and at a window's edge in the middle of one."""
    B, T, lens = 2, 3, [611, 900]
    q, c, par, _ = attend_inputs(dtype, kv, B, T, 4, 2, lens, None, page, False, window, sinks)
    want = M.attention(q, c[0], c[1], c[2], lens, None, None, window, sinks, None if c[3] is None else (c[3], c[4]))
    for b, n in enumerate(lens):
        gone = torch.arange(sinks, n - window + 1)
        gone = gone[c[2][b].long()[gone // page] >= 0]
        pg, row = R.slots(c[2], page, b, gone)
        for i in (0, 1):
            if c[3] is None:
                c[i][pg, row] = math.nan
            else:
                c[i].view(torch.int8)[pg, row] = 127
                c[3 + i][pg, :, row] = math.nan
    o, lse = cuda_lib.st_cache_attn(q.cuda(), dev_cache(cuda_lib, c), i32(lens).cuda(), window=window, sinks=sinks)
    cuda_lib.st_check_status()
    R.close("o", o, want[0], want[2])
    R.close("lse", lse, want[1], want[3])


def test_window_without_effect_is_no_window(cuda_lib):
    for dtype, kv in (("bf16", "bf16"), ("fp16", "e4m3"), ("fp32", "fp32")):
        q, c, par, _ = attend_inputs(dtype, kv, 2, 5, 8, 2, [300, 41], None, 16, True, 0, 0)
        cache, lens = dev_cache(cuda_lib, c), i32([300, 41]).cuda()
        a = cuda_lib.st_cache_attn(q.cuda(), cache, lens, parents=par.cuda())
        b = cuda_lib.st_cache_attn(q.cuda(), cache, lens, parents=par.cuda(), sinks=7)
        assert torch.equal(bits(a[0]), bits(b[0]))
        want = M.attention(q, c[0], c[1], c[2], [300, 41], None, par, 0, 0, None if c[3] is None else (c[3], c[4]))
        for w in (306, (1 << 31) - 1):
            o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, lens, parents=par.cuda(), window=w, sinks=(1 << 31) - 1)
            R.close("o", o, want[0], want[2])
            R.close("lse", lse, want[1], want[3])


@pytest.mark.parametrize("dtype,kv,page", [("bf16", "bf16", 16), ("fp16", "e4m3", 16), ("bf16", "int8", 7), ("fp32", "fp32", 16)])
@pytest.mark.parametrize("window", [0, 50])
def test_lengths_out_of_range(cuda_lib, dtype, kv, page, window):
    """A negative length counts as 0, keys beyond the table are left out, and the status says so."""
    q, c, _, _ = attend_inputs(dtype, kv, 2, 4, 4, 2, [0, 90], None, page, False, 0, 0)
    cache = dev_cache(cuda_lib, c)
    scales = None if c[3] is None else (c[3], c[4])
    o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32([-4, 90]).cuda(), window=window, sinks=2)
    with pytest.raises(cuda_lib.StError) as e:
        cuda_lib.st_check_status()
    assert e.value.status == cuda_lib.ST_ERR_INVALID_ARG
    want = M.attention(q, c[0], c[1], c[2], [0, 90], None, None, window, 2, scales)
    R.close("o", o, want[0], want[2])
    R.close("lse", lse, want[1], want[3])
    far = (1 << 31) - 1
    o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32([0, far]).cuda(), window=max(window, 1), sinks=0)
    with pytest.raises(cuda_lib.StError):
        cuda_lib.st_check_status()
    assert bool((o[1] == 0).all()) and bool((lse[1] == -math.inf).all())  # no key of these windows is in the table


@pytest.mark.parametrize("dtype,kv,T", [("bf16", "bf16", 1), ("fp16", "fp16", 70), ("bf16", "e4m3", 1), ("fp16", "int8", 40)])
def test_windows_behind_the_table_of_many_sequences(cuda_lib, dtype, kv, T):
    """More items than SMs: rows whose window has no key of the table are zeros all the same."""
    B, far = 90, 1 << 30
    lens = [(b * 37) % 200 for b in range(B)]
    q, c, _, _ = attend_inputs(dtype, kv, B, T, 4, 2, lens, None, 16, False, 0, 0)
    some = [0, 41, 89]
    lens_far = [far if b in some else n for b, n in enumerate(lens)]
    scales = None if c[3] is None else (c[3], c[4])
    cache = dev_cache(cuda_lib, c)
    need = cuda_lib.st_cache_attn_workspace_size(q.cuda(), cache, window=30)
    o, lse = torch.full_like(q, 7.0).cuda(), torch.full((B, 4, T), 7.0).cuda()
    cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens_far).cuda(), window=30, o=o, lse=lse, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    with pytest.raises(cuda_lib.StError):
        cuda_lib.st_check_status()
    assert bool((o[some] == 0).all()) and bool((lse[some] == -math.inf).all())
    want = M.attention(q, c[0], c[1], c[2], lens, None, None, 30, 0, scales)
    rest = [b for b in range(B) if b not in some]
    R.close("o", o[rest], want[0][rest], want[2][rest])
    R.close("lse", lse[rest], want[1][rest], want[3][rest])


# ------------------------------------------------------------ shared prefix
SHARED = [
    # dtype, cache, B, T, H, Hkv, shared, own lengths, counts, page, tree
    ("bf16", "bf16", 3, 1, 8, 2, 256, [0, 5, 300], None, 16, False),
    ("bf16", "bf16", 2, 1, 32, 8, 640, [1, 129], None, 128, False),
    ("fp16", "fp16", 5, 7, 6, 3, 1000, [10, 0, 40, 1, 90], [7, 3, 0, 1, 7], 8, False),
    ("bf16", "bf16", 4, 30, 16, 2, 512, [3, 100, 128, 260], None, 64, True),
    ("fp16", "fp16", 2, 70, 8, 2, 384, [40, 7], [70, 61], 16, True),
    ("bf16", "e4m3", 3, 1, 8, 2, 512, [0, 5, 300], None, 16, False),
    ("fp16", "int8", 6, 9, 12, 3, 400, [10, 0, 40, 1, 90, 2], [9, 9, 9, 0, 1, 2], 16, True),
    ("bf16", "e4m3", 2, 100, 8, 4, 256, [50, 400], None, 32, False),
    ("bf16", "bf16", 200, 1, 4, 1, 256, [i % 37 for i in range(200)], None, 16, False),
    ("fp32", "fp32", 3, 4, 4, 2, 200, [10, 0, 33], None, 16, False),
    ("fp16", "fp16", 2, 3, 4, 2, 90, [10, 0], None, 6, False),
    ("bf16", "bf16", 2, 3, 4, 2, 96, [10, 0], None, 16, False),
    ("bf16", "int8", 70, 5, 8, 2, 1024, [i for i in range(70)], None, 64, True),
]


def shared_inputs(dtype, kv, B, T, H, Hkv, shared, own, counts, page, tree):
    """Sequences of shared + own[b] tokens, whose first shared // page pages are the first one's."""
    dt, kt = DT[dtype], DT[kv]
    lens = [shared + n for n in own]
    rows = [n + (T if counts is None else counts[b]) for b, n in enumerate(lens)]
    c = M.make_cache(B, [n + T for n in lens], Hkv, page, kt, rows, 21)
    c[2][:, :shared // page] = c[2][0, :shared // page]
    q = rand(1, B, T, H, D, dtype=dt) * 2
    return q, c, lens, R.tree(B, T, 5, 3) if tree else None, None if counts is None else i32(counts), shared // page * page


@pytest.mark.parametrize("case", SHARED, ids=lambda c: "-".join(str(x) for x in c if not isinstance(x, list)))
def test_shared_prefix(cuda_lib, case):
    q, c, lens, par, cnt, shared = shared_inputs(*case)
    cache = dev_cache(cuda_lib, c)
    if cnt is not None and int(cnt[0]) > 0 and c[2].shape[0] > 2:  # a sequence without rows says nothing
        empty = (cnt == 0).nonzero()
        if len(empty):
            cache.pages[int(empty[0])] = 1 << 30
    want = M.attention(q, c[0], c[1], c[2], lens, cnt, par, scales=None if c[3] is None else (c[3], c[4]))
    for n in (shared, shared // 2 + 1, 0, -3, 1 << 30):
        if n > shared and min(x for b, x in enumerate(lens) if cnt is None or cnt[b] > 0) >= (shared // 128 + 1) * 128:
            continue  # more than is shared would be taken at its word
        o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda(), counts=gpu(cnt), parents=gpu(par), shared=i32([n]).cuda())
        cuda_lib.st_check_status()
        R.close(f"o, {n} shared", o, want[0], want[2])
        R.close(f"lse, {n} shared", lse, want[1], want[3])
        again = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda(), counts=gpu(cnt), parents=gpu(par), shared=i32([n]).cuda())
        assert torch.equal(bits(again[0]), bits(o)) and torch.equal(bits(again[1]), bits(lse))


def test_shared_prefix_is_read_from_the_first_sequence_with_rows(cuda_lib):
    """Sequence 0 has no rows and a page table that points nowhere."""
    q, c, lens, _, _, shared = shared_inputs("bf16", "bf16", 3, 2, 8, 2, 512, [9, 70, 0], None, 16, False)
    want = M.attention(q, c[0], c[1], c[2], lens, i32([0, 2, 2]), None)
    pages = c[2].clone()
    pages[0] = -1
    cache = cuda_lib.KVCache(c[0].cuda(), c[1].cuda(), pages.cuda())
    for start in (lens, [0] + lens[1:], [-1] + lens[1:]):
        o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32(start).cuda(), counts=i32([0, 2, 2]).cuda(), shared=i32([shared]).cuda())
        if start[0] >= 0:
            cuda_lib.st_check_status()
        R.close("o", o, want[0], want[2])
        R.close("lse", lse, want[1], want[3])
    with pytest.raises(cuda_lib.StError):
        cuda_lib.st_check_status()
    none = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda(), counts=i32([0, 0, 0]).cuda(), shared=i32([shared]).cuda())
    cuda_lib.st_check_status()
    assert bool((none[0] == 0).all()) and bool((none[1] == -math.inf).all())


def test_shared_prefix_with_a_window(cuda_lib):
    q, c, lens, _, _, shared = shared_inputs("bf16", "e4m3", 3, 2, 8, 2, 512, [9, 70, 0], None, 16, False)
    cache = dev_cache(cuda_lib, c)
    a = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda(), window=40, sinks=3, shared=i32([shared]).cuda())
    want = M.attention(q, c[0], c[1], c[2], lens, None, None, 40, 3, (c[3], c[4]))
    R.close("o", a[0], want[0], want[2])


# ------------------------------------------------- numbers that go wrong easily
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("kv", HELD)
def test_scales_of_every_size(cuda_lib, dtype, kv):
    """V rows from 2^-24 to 2^24 times as large as others, rows of zeros, and q rows of very different sizes."""
    B, T, H, Hkv, lens = 1, 8, 4, 2, [700]
    q, c, _, _ = attend_inputs(dtype, kv, B, T, H, Hkv, lens, None, 16, False, 0, 0)
    g = torch.Generator().manual_seed(5)
    c[4][:] = c[4] * torch.exp2(torch.randint(-24, 24 if dtype == "bf16" else 1, c[4].shape, generator=g))
    pg, row = R.slots(c[2], 16, 0, torch.arange(3, 700, 5))
    c[1].view(torch.int8)[pg, row] = 0
    c[4][pg, :, row] = 0.0
    if dtype == "bf16":  # (fp16 holds no such numbers)
        q = (q.float() * torch.exp2(torch.arange(-30, 2, 4).float())[None, :, None, None]).to(q.dtype)
    o, lse = cuda_lib.st_cache_attn(q.cuda(), dev_cache(cuda_lib, c), i32(lens).cuda())
    want = M.attention(q, c[0], c[1], c[2], lens, None, None, scales=(c[3], c[4]))
    R.close("o", o, want[0], want[2])
    R.close("lse", lse, want[1], want[3])


@pytest.mark.parametrize("kv", HELD)
@pytest.mark.parametrize("T", [1, 20, 80])
def test_scales_at_the_ends_of_their_range(cuda_lib, kv, T):
    """Tiles of V rows near 2^-48 before, between and behind others near 2^48: none is lost from the sums."""
    B, H, Hkv, lens = 2, 4, 2, [700, 640]
    q, c, _, _ = attend_inputs("bf16", kv, B, T, H, Hkv, lens, None, 16, False, 0, 0)
    for b, n in enumerate(lens):
        at = torch.arange(n + T)
        pg, row = R.slots(c[2], 16, b, at)
        c[4][pg, :, row] *= torch.exp2(torch.where((at // 128) % 2 == b, -48.0, 48.0))[:, None]
    o, lse = cuda_lib.st_cache_attn(q.cuda(), dev_cache(cuda_lib, c), i32(lens).cuda())
    want = M.attention(q, c[0], c[1], c[2], lens, None, None, scales=(c[3], c[4]))
    R.close("o", o, want[0], want[2])
    R.close("lse", lse, want[1], want[3])


@pytest.mark.parametrize("kv", HELD)
def test_one_key_far_ahead(cuda_lib, kv):
    """One key whose weight is all but the whole, with a V row 2^-12 of the others': these must not come through."""
    kt, n = DT[kv], 500
    q, c, _, _ = attend_inputs("fp16", kv, 1, 1, 2, 1, [n], None, 16, False, 0, 0, spread=0.0)
    pg, row = R.slots(c[2], 16, 0, torch.tensor([123]))
    top = M.TOP[kt]
    held = (q[0, 0, 0].float() / q[0, 0, 0].float().abs().max() * top).round()
    c[0].view(torch.int8)[pg, row] = held.to(kt).view(torch.int8)
    c[3][pg, :, row] = 40.0 / top
    c[4][pg, :, row] *= 2.0 ** -12
    o, lse = cuda_lib.st_cache_attn(q.cuda(), dev_cache(cuda_lib, c), i32([n]).cuda())
    want = M.attention(q, c[0], c[1], c[2], [n], None, None, scales=(c[3], c[4]))
    R.close("o", o, want[0], want[2])
    R.close("lse", lse, want[1], want[3])


@pytest.mark.parametrize("dtype,kv", [("bf16", "e4m3"), ("fp16", "int8"), ("fp32", "e4m3")])
def test_a_row_that_is_seen_and_not_finite(cuda_lib, dtype, kv):
    """NaN in a key's scale reaches the rows that see it and no others."""
    q, c, _, _ = attend_inputs(dtype, kv, 2, 4, 4, 2, [200, 77], None, 16, False, 0, 0)
    pg, row = R.slots(c[2], 16, 0, torch.tensor([202]))   # sequence 0's third new row
    c[3][pg, 1, row] = math.nan
    o, lse = cuda_lib.st_cache_attn(q.cuda(), dev_cache(cuda_lib, c), i32([200, 77]).cuda())
    want = torch.zeros(2, 4, 4, dtype=torch.bool)
    want[0, 2:, 2:] = True
    assert torch.equal(o.isnan().all(-1).cpu(), want) and torch.equal(o.isnan().any(-1).cpu(), want)
    assert torch.equal(lse.isnan().cpu(), want.transpose(1, 2))


# --------------------------------------------------------- strides, streams, graphs
def test_strided_scales_and_rows(cuda_lib):
    """Scales as slices of one buffer at any 4-byte offset, caches as slices of larger ones, q and o strided."""
    for kv in HELD:
        q, c, _, _ = attend_inputs("bf16", kv, 2, 3, 8, 2, [300, 45], None, 16, False, 0, 0)
        n = c[0].shape[0]
        sc = torch.full((n, 2, 2, 21), math.nan, device="cuda")
        sc[:, 0, :, 3:19], sc[:, 1, :, 3:19] = c[3].cuda(), c[4].cuda()
        big = torch.zeros(2, n, 2, 16, 256, dtype=torch.int8, device="cuda")
        for i in (0, 1):
            big[i, ..., :D] = c[i].view(torch.int8).cuda().transpose(1, 2)
        kc, vc = (big[i, ..., :D].transpose(1, 2).view(DT[kv]) for i in (0, 1))
        cache = cuda_lib.KVCache(kc, vc, c[2].cuda(), sc[:, 0, :, 3:19], sc[:, 1, :, 3:19])
        qq = torch.zeros(2, 3, 8, 3 * D, dtype=torch.bfloat16, device="cuda")
        qq[..., D:2 * D] = q.cuda()
        o = torch.full((2, 8, 3, D), 3.0, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
        got, lse = cuda_lib.st_cache_attn(qq[..., D:2 * D], cache, i32([300, 45]).cuda(), o=o)
        assert got.data_ptr() == o.data_ptr()
        want = M.attention(q, c[0], c[1], c[2], [300, 45], None, None, scales=(c[3], c[4]))
        R.close("o", got, want[0], want[2])
        R.close("lse", lse, want[1], want[3])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_streams_and_graphs(cuda_lib, kv):
    """A captured step (append, three attentions, read, keep) on a side stream replays with other lengths and a other
    shared prefix; two graphs take turns on one workspace."""
    B, T, H, Hkv, page = 3, 2, 8, 2, 16
    shared = 256
    q, c, lens, _, _, _ = shared_inputs("bf16", kv, B, T, H, Hkv, shared, [40, 3, 200], None, page, False)
    cache = dev_cache(cuda_lib, c)
    scales = lambda: None if cache.k_scale is None else (cache.k_scale.cpu(), cache.v_scale.cpu())
    dl, ds = i32(lens).cuda(), i32([shared]).cuda()
    x, kk, vv = (rand(s, B, T, h, D, dtype=torch.bfloat16).cuda() for s, h in ((5, H), (6, Hkv), (7, Hkv)))
    w = torch.ones(D, device="cuda")
    ids = torch.zeros(1, T, 1, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(cuda_lib.st_cache_attn_workspace_size(q.cuda(), cache, shared=ds),
                         cuda_lib.st_cache_attn_workspace_size(q.cuda(), cache, window=64)), dtype=torch.uint8, device="cuda")

    def step(**kw):
        qr = cuda_lib.st_cache_append(x, kk, vv, w, w, 1e-6, ids, (128,), 1e4, cache, dl)
        return qr, cuda_lib.st_cache_attn(qr, cache, dl, workspace=ws, **kw)

    step(shared=ds), step(window=64, sinks=2)  # loads the kernels
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs = []
    for kw in (dict(shared=ds), dict(window=64, sinks=2)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            out = step(**kw)
            back = cuda_lib.st_cache_read(cache, dl, T)
        graphs.append((g, out, back, kw))
    for now, sh in ((lens, shared), ([n - 2 for n in lens], 128), (lens, 0)):
        dl.copy_(i32(now))
        ds.fill_(sh)
        for g, (qr, (o, lse)), back, kw in graphs:
            o.fill_(9.0)
            g.replay()
            torch.cuda.synchronize()
            cuda_lib.st_check_status()
            want = M.attention(qr.cpu(), cache.k.cpu(), cache.v.cpu(), c[2], now, None, None, kw.get("window", 0),
                               kw.get("sinks", 0), scales())
            R.close("o", o, want[0], want[2])
            R.close("lse", lse, want[1], want[3])
            assert bool(back[1].isfinite().all())


def test_decoding_loop(cuda_lib):
    """Trees of drafted tokens over an 8-bit cache with a window: append, attention, verification, compaction, each call
    held to its own bound, for some steps; at the end the rows are read back and are what the appends held."""
    B, T, H, Hkv, page, V = 2, 6, 8, 2, 16, 50
    kt = torch.float8_e4m3fn
    lens = [20, 75]
    c = M.make_cache(B, [n + 60 for n in lens], Hkv, page, kt, lens, 3)
    cache, dl = dev_cache(cuda_lib, c), i32(lens).cuda()
    w = torch.ones(D, device="cuda")
    path = None
    for s in range(5):
        g = torch.Generator().manual_seed(s)
        par = R.tree(B, T, 3, s)
        x, k, v = (torch.randn(B, T, h, D, generator=g).to(torch.bfloat16) for h in (H, Hkv, Hkv))
        depth = torch.stack([M.positions(0, T, par[b].tolist())[0] for b in range(B)])
        ids = (dl.cpu()[:, None] + depth).to(torch.int32)[..., None].contiguous()
        now = dl.cpu().tolist()
        qr = cuda_lib.st_cache_append(x.cuda(), k.cuda(), v.cuda(), w, w, 1e-6, ids.cuda(), (128,), 1e4, cache, dl)
        o, lse = cuda_lib.st_cache_attn(qr, cache, dl, parents=par.cuda(), window=30, sinks=2)
        want = M.attention(qr.cpu(), cache.k.cpu(), cache.v.cpu(), c[2], now, None, par, 30, 2,
                           (cache.k_scale.cpu(), cache.v_scale.cpu()))
        R.close("o", o, want[0], want[2])
        R.close("lse", lse, want[1], want[3])
        p = torch.softmax(2 * torch.randn(B, T, V, generator=g), -1)
        tok = torch.randint(0, V, (B, T), generator=g).to(torch.int32)
        ua, us = torch.rand(B, T, generator=g) * 0.02, torch.rand(B, generator=g)
        path, n, nxt = cuda_lib.st_tree_verify(p.cuda(), None, tok.cuda(), par.cuda(), ua.cuda(), us.cuda())
        before = [y.cpu() for y in cuda_lib.st_cache_read(cache, dl, T, dtype=torch.float32)]
        new = cuda_lib.st_cache_keep(cache, dl, path, n)
        after = [y.cpu() for y in cuda_lib.st_cache_read(cache, dl, T, counts=n, dtype=torch.float32)]
        for b in range(B):
            m = int(n[b])
            assert m >= 1 and int(new[b]) == now[b] + m
            for y, z in zip(before, after):
                assert torch.equal(z[b, :m], y[b, path[b, :m].long().cpu()]) and bool((z[b, m:] == 0).all())
        dl = new
    cuda_lib.st_check_status()


def test_gradients_are_not_carried(cuda_lib):
    q, c, _, _ = attend_inputs("bf16", "e4m3", 1, 1, 4, 2, [30], None, 16, False, 0, 0)
    cache = dev_cache(cuda_lib, c)
    q = q.cuda().requires_grad_()
    o, lse = cuda_lib.st_cache_attn(q, cache, i32([30]).cuda(), window=8)
    k, v = cuda_lib.st_cache_read(cache, i32([0]).cuda(), 4)
    assert not (o.requires_grad or lse.requires_grad or k.requires_grad or v.requires_grad)
