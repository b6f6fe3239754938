"""Serving calls on the GPU at the edges of what they allow: values in device memory out of their range, statuses, and
inputs that ask for more bits than ordinary ones."""
import pytest
import torch

import _serving as R
from test_gpu_serving import D, DT, Loop, attn_case, bits, dev_cache, i32, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_append_negative_length_writes_nothing(cuda_lib, dtype):
    """No row of a sequence of negative length enters the cache, not even those whose lens[b] + t is a position; the
    other sequences' rows do, q comes back for all, and the status says so."""
    B, T, H, Hkv, page = 3, 6, 4, 2, 8
    lens = [-1, 5, -4]
    q, k, v = (rand(s, B, T, h, D, dtype=DT[dtype]) for s, h in ((1, H), (2, Hkv), (3, Hkv)))
    kc, vc, pages = R.make_cache(B, [T, 5 + T, T], Hkv, page, DT[dtype], 4, fill=0.5)
    cache = dev_cache(cuda_lib, kc, vc, pages)
    w = torch.ones(D)
    ids = torch.arange(T, dtype=torch.int32)[None, :, None].contiguous()
    got = cuda_lib.st_cache_append(q.cuda(), k.cuda(), v.cuda(), w.cuda(), w.cuda(), 1e-6, ids.cuda(), (128,), 1e4, cache,
                                   i32(lens).cuda())
    with pytest.raises(cuda_lib.StError) as e:
        cuda_lib.st_check_status()
    assert e.value.status == cuda_lib.ST_ERR_INVALID_ARG
    ang = R.angles(ids, (128,), 1e4)
    yq, sq = R.rotate(q, w, ang, 1e-6)
    yk, sk = R.rotate(k, w, ang, 1e-6)
    # as the append's other tests: one rounding; angle, sincosf, rsqrt and five fp32 products below 2^-19 of the terms
    tol = lambda y, s: R.HALF[DT[dtype]] * y.abs() + 2.0 ** -19 * s * (1 + R.HALF[DT[dtype]]) + 2.0 ** -25
    R.close("q_rot", got, yq, tol(yq, sq))
    pg, row = R.slots(pages, page, 1, 5 + torch.arange(T))
    R.close("k", cache.k.cpu()[pg, row], yk[1], tol(yk, sk)[1])
    assert torch.equal(cache.v.cpu()[pg, row], v[1])
    k2, v2 = cache.k.cpu(), cache.v.cpu()
    k2[pg, row], v2[pg, row] = kc[pg, row], vc[pg, row]
    assert torch.equal(bits(k2), bits(kc)) and torch.equal(bits(v2), bits(vc))


def test_status_reports_a_timeout_and_then_the_index(cuda_lib):
    """A bounded wait that ran out does not hide a value out of range met in between: one check reports each."""
    kc = torch.zeros(2, 8, 1, D, dtype=torch.bfloat16, device="cuda")
    cache = cuda_lib.KVCache(kc, kc.clone(), i32([[0, 1]]).cuda())
    cuda_lib.st_check_status()
    cuda_lib.st_cache_keep(cache, i32([0]).cuda(), i32([[2, 1]]).cuda(), i32([2]).cuda())  # the second row does not ascend
    cuda_lib.st_selftest_wait_timeout(2_000_000)
    for want in (cuda_lib.ST_ERR_TIMEOUT, cuda_lib.ST_ERR_INVALID_ARG):
        with pytest.raises(cuda_lib.StError) as e:
            cuda_lib.st_check_status()
        assert e.value.status == want
    cuda_lib.st_check_status()


def test_timing_reports_the_serving_kernels(cuda_lib):
    """The Python reader has every kind; the C struct's reader has the first nine and drops the others."""
    import ctypes
    kc = torch.zeros(2, 8, 1, D, dtype=torch.bfloat16, device="cuda")
    cache = cuda_lib.KVCache(kc, kc.clone(), i32([[0, 1]]).cuda())
    keep = lambda: cuda_lib.st_cache_keep(cache, i32([0]).cuda(), i32([[1, 2]]).cuda(), i32([2]).cuda())
    keep()
    cuda_lib.st_timing_enable(True)
    try:
        cuda_lib.st_timing_read()
        keep()
        got = cuda_lib.st_timing_read()
        assert got["cache_keep"][0] == 1 and got["cache_keep"][1] > 0 and sum(n for n, _ in got.values()) == 1
        keep()
        t = cuda_lib.st_kernel_times()
        assert cuda_lib.lib().st_timing_read(ctypes.byref(t)) == cuda_lib.ST_OK and list(t.launches) == [0] * 9
        assert sum(n for n, _ in cuda_lib.st_timing_read().values()) == 0
    finally:
        cuda_lib.st_timing_enable(False)


def test_attention_refusals_keep_their_status_in_python(cuda_lib):
    """What the C call refuses has the same status through Python, with the caller's workspace and without one."""
    E = cuda_lib
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")
    lens = z(1, dtype=torch.int32)
    cache = E.KVCache(z(2, 16, 2, D), z(2, 16, 2, D), z(1, 2, dtype=torch.int32))
    par = lambda t: z(1, t, dtype=torch.int32)
    cases = [
        (E.ST_ERR_UNSUPPORTED, "256", z(1, 257, 2, D), cache, par(257)),
        (E.ST_ERR_UNSUPPORTED, "D=128", z(1, 1, 2, 64), cache, None),
        (E.ST_ERR_UNSUPPORTED, "query heads", z(1, 1, 258, D), cache, None),
        (E.ST_ERR_DTYPE, "q_rot", z(1, 1, 2, D, dtype=torch.float16), cache, None),
        (E.ST_ERR_DTYPE, "parents", z(1, 3, 2, D), cache, par(3).long()),
        (E.ST_ERR_SHAPE, "divide", z(1, 1, 3, D), cache, None),
        (E.ST_ERR_SHAPE, "parents", z(1, 3, 2, D), cache, par(4)),
        (E.ST_ERR_ALIGN, "unit stride", z(1, 1, 2, 2 * D)[..., ::2], cache, None),
        (E.ST_ERR_ALIGN, "expanded", z(1, 1, 2, D), E.KVCache(cache.k[:1].expand(2, -1, -1, -1), cache.v, cache.pages), None),
    ]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for status, text, q, c, parents in cases:
        for w in (None, ws):
            with pytest.raises(E.StError, match=text) as e:
                E.st_cache_attn(q, c, lens, parents=parents, workspace=w)
            assert e.value.status == status, (text, w is None, e.value.status)
        with pytest.raises(E.StError, match=text) as e:
            E.st_cache_attn_workspace_size(q, c, parents)
        assert e.value.status == status, (text, e.value.status)


def test_fp16_attention_keeps_a_long_tail(cuda_lib):
    """One key far ahead of 41000 others: together they still weigh what they should. Sequences share their pages, so
    that each has a CTA or two of its own for its whole length."""
    n, B, page = 41000, 160, 40
    g = torch.Generator().manual_seed(5)
    k = torch.zeros(n // page + 1, page, 1, D, dtype=torch.float16)
    v = (1 + 0.25 * torch.rand(n // page + 1, page, 1, D, generator=g)).to(torch.float16)
    k[0, 0, 0, 0] = 1
    v[0, 0] = 0
    ahead = torch.tensor([22.0, 24.0, 25.0, 25.5, 26.0, 28.0, 31.0, 33.0])  # in bits, exact in fp16
    q = torch.zeros(B, 1, 1, D, dtype=torch.float16)
    q[:, 0, 0, 0] = ahead.repeat(B // 8).half()
    pages = torch.arange(n // page + 1, dtype=torch.int32).expand(B, -1).contiguous()
    cache = dev_cache(cuda_lib, k, v, pages)
    ln2 = 0.6931471805599453
    o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, torch.full((B,), n - 1, dtype=torch.int32).cuda(), scale=ln2)
    cuda_lib.st_check_status()
    vv = v.reshape(-1, D)[:n].double()
    w = 2.0 ** -ahead.double()[:, None]
    total = 1 + w * (n - 1)
    want = (w * vv.sum(0) / total).repeat(B // 8, 1)[:, None, None]
    # of the sum's terms: half a step of a weight, the scores' fp32 rounding (33 bits: 2^-18 together with ex2), the sums;
    # weights below fp16's range, 2^-25 where the largest is 2^7; the output's half step
    size = want.abs()
    bound = size * (2.0 ** -11 + 2 * 2.0 ** -18 + 2 * (n + 64) * 2.0 ** -24) + n * 2.0 ** -32 * vv.max() + 2.0 ** -11 * size + 2.0 ** -25
    R.close("o", o, want, bound)
    want_lse = (ahead.double() * ln2 + total[:, 0].log()).repeat(B // 8)[:, None, None]
    R.close("lse", lse, want_lse, 2.0 ** -18 + (n + 64) * 2.0 ** -24 + 2.0 ** -22 * (1 + want_lse.abs()))


@pytest.mark.parametrize("dtype,H,Hkv,page", [("bf16", 8, 2, 16), ("fp16", 3, 1, 24), ("fp32", 4, 4, 10), ("bf16", 6, 2, 7), ("fp16", 32, 8, 8)])
def test_decoding_loop_step_by_step(cuda_lib, dtype, H, Hkv, page):
    """A decoding loop in which every call is held to its own bound: q' and the new rows of the cache to one rounding of
    the exact ones, and the attention to the 64-bit form on the very q' and cache that it was given."""
    B, T = 3, 10
    L = Loop(cuda_lib, dtype, B, T, H, Hkv, page, [0, 37, 250], 3, 40, seed=2000)
    cache = dev_cache(cuda_lib, L.k, L.v, L.pages)
    lens = i32(L.lens0).cuda()
    half = R.HALF[L.dt]
    tol = lambda y, s: half * y.abs() + 2.0 ** -19 * s * (1 + half) + 2.0 ** -25  # as the append's own tests
    for c, d in zip(L.steps, L.to_dev()):
        before = lens.tolist()
        k0, v0 = cache.k.cpu(), cache.v.cpu()
        ids = (lens[:, None] + d["depth"])[..., None]
        q = cuda_lib.st_cache_append(d["q"], d["k"], d["v"], L.wq_, L.wk_, 1e-6, ids, (128,), 1e4, cache, lens)
        k1, v1 = cache.k.cpu(), cache.v.cpu()
        o, lse = cuda_lib.st_cache_attn(q, cache, lens, parents=d["parents"])
        path, n, nxt = cuda_lib.st_tree_verify(d["target"], d["draft"], d["tokens"], d["parents"], d["ua"], d["us"])
        new = cuda_lib.st_cache_keep(cache, lens, path, n)
        cuda_lib.st_check_status()

        ang = R.angles(ids.cpu(), (128,), 1e4)
        yq, sq = R.rotate(c["q"], L.wq, ang, 1e-6)
        yk, sk = R.rotate(c["k"], L.wk, ang, 1e-6)
        R.close("q_rot", q, yq, tol(yq, sq))
        want_k, tol_k, want_v = k0.double(), torch.zeros(k0.shape, dtype=torch.float64), v0.clone()
        for b in range(B):
            pg, row = R.slots(L.pages, page, b, before[b] + torch.arange(T))
            want_k[pg, row], tol_k[pg, row], want_v[pg, row] = yk[b], tol(yk, sk)[b], c["v"][b]
        R.close("cache.k", k1, want_k, tol_k)
        assert torch.equal(bits(v1), bits(want_v))
        ro, rl, bo, bl = R.attention(q.cpu(), k1, v1, L.pages, before, None, c["parents"])
        R.close("o", o, ro, bo)
        R.close("lse", lse, rl, bl)
        for got, want in zip((path, n, nxt), R.verify(c["target"], c["draft"], c["tokens"], c["parents"], c["ua"], c["us"])):
            assert torch.equal(got.cpu(), want)
        for b in range(B):  # the accepted rows moved, everything else kept its bits
            keep = path[b, : n[b]].long().cpu()
            spg, srow = R.slots(L.pages, page, b, before[b] + keep)
            dpg, drow = R.slots(L.pages, page, b, before[b] + torch.arange(keep.numel()))
            moved_k, moved_v = k1[spg, srow].clone(), v1[spg, srow].clone()
            k1[dpg, drow], v1[dpg, drow] = moved_k, moved_v
        assert torch.equal(bits(cache.k), bits(k1)) and torch.equal(bits(cache.v), bits(v1))
        assert new.tolist() == [x + y for x, y in zip(before, n.tolist())]
        lens = new


def near_case(B, T, V, near, dtype, seed):
    """Trees whose root's children are guesses that the draft overrates: all are rejected, and what is left of the row is
    as small as target and draft are close."""
    g = torch.Generator().manual_seed(seed)
    target = torch.softmax(torch.randn(B, T, V, generator=g) * 2, -1)
    draft = target * (1 + near * torch.randn(B, T, V, generator=g)).clamp(min=0.05)
    draft = draft / draft.sum(-1, keepdim=True)
    target, draft = target.to(dtype), draft.to(dtype)
    tokens = torch.zeros(B, T, dtype=torch.int32)
    for b in range(B):
        over = (draft[b, 0].double() * (1 - 2.0 ** -24) > target[b, 0].double()).nonzero()[:, 0]
        tokens[b, 1:] = over[torch.randperm(over.numel(), generator=g)[: T - 1]].to(torch.int32)
    parents = torch.zeros(B, T, dtype=torch.int32)
    parents[:, 0] = -1
    ua = torch.full((B, T), 1 - 2.0 ** -24)
    return target, draft, tokens, parents, ua, (torch.arange(B) + 0.5) / B


@pytest.mark.parametrize("near,dtype", [(0.3, "fp32"), (1e-2, "fp32"), (1e-4, "fp32"), (1e-6, "fp32"), (1e-2, "bf16"), (2e-3, "fp16")])
@pytest.mark.parametrize("B,T,V", [(24, 2, 131072), (24, 5, 20001), (320, 3, 701)])
def test_verify_draft_close_to_the_target(cuda_lib, near, dtype, B, T, V):
    """One to four rejections, and the draw from a residual of 2^-3 to 2^-21: the same token as in 64 bits. (A running sum
    of 2^17 weights is off by about 2^-30 of such a total at most, and a draw among 2^17 borders within that of one hardly
    ever; these inputs have none.)"""
    case = near_case(B, T, V, near, DT[dtype], seed=T)
    want = R.verify(*case)
    assert want[1].tolist() == [1] * B  # all guesses are rejected
    got = cuda_lib.st_tree_verify(*(t.cuda() for t in case))
    cuda_lib.st_check_status()
    for name, x, w in zip(("path", "n_accepted", "next_token"), got, want):
        assert torch.equal(x.cpu(), w), (name, (x.cpu() != w).sum().item())


def test_verify_residual_of_tiny_weights(cuda_lib):
    """All that is left are tokens far below 2^-44: the next token is one of them, in proportion, not one of the target's
    likely ones. With a draft, and without one after the only likely token's rejection."""
    V, B = 5000, 64
    target = torch.zeros(B, 3, V)
    target[:, :, 7], target[:, :, 9] = 0.5, 0.5
    tiny = torch.arange(100, 140)
    target[:, :, tiny] = 2.0 ** -60 * torch.arange(1, 41)
    draft = target.clone()
    draft[:, :, tiny] = 0
    draft[:, :, 9] = 0.5 + 2.0 ** -20
    us = (torch.arange(B) + 0.5) / B
    case = (target, draft, i32([[0, 9, 9]] * B), i32([[-1, 0, 0]]), torch.full((B, 3), 1 - 2.0 ** -24), us)
    weight = torch.arange(1, 41).double()
    want = 100 + (weight.cumsum(0)[None] <= us.double()[:, None] * weight.sum()).sum(-1)
    path, n, nxt = (t.cpu() for t in cuda_lib.st_tree_verify(*(t.cuda() for t in case)))
    assert n.tolist() == [1] * B and nxt.tolist() == want.tolist()
    for first in (0.999, 1 - 2.0 ** -24):  # every weight counts, the largest is removed
        alone = target.clone()
        alone[:, :, 7], alone[:, :, 9] = first, 0
        path, n, nxt = (t.cpu() for t in cuda_lib.st_tree_verify(alone.cuda(), None, i32([[0, 7, 7]] * B).cuda(), i32([[-1, 0, 0]]).cuda(),
                                                                 case[4].cuda(), us.cuda()))
        assert n.tolist() == [1] * B and nxt.tolist() == want.tolist()
    # subnormal numbers, and a draft that is the target's very self but for them
    sub = target.clone()
    sub[:, :, tiny] = 2.0 ** -149 * torch.arange(1, 41)
    path, n, nxt = (t.cpu() for t in cuda_lib.st_tree_verify(sub.cuda(), draft.cuda(), *(t.cuda() for t in case[2:])))
    assert n.tolist() == [1] * B and nxt.tolist() == want.tolist()


@pytest.mark.parametrize("near,dtype", [(1e-3, "fp32"), (1e-6, "fp32"), (2e-2, "bf16")])
@pytest.mark.parametrize("B,V", [(48, 3001), (320, 257)])
def test_verify_walk_behind_a_small_residual(cuda_lib, near, dtype, B, V):
    """Trees whose nodes have a child that is rejected, one that what is left accepts or not, and children of their own:
    the walk goes on behind residuals of any size."""
    T = 24
    target, draft, tokens, _, _, us = near_case(B, T, V, near, DT[dtype], seed=31)
    g = torch.Generator().manual_seed(32)
    parents = R.tree(B, T, 5, 33)
    ua = torch.rand(B, T, generator=g)
    for b in range(B):
        first = {}
        for i in range(1, T):
            par = int(parents[b, i])
            more = draft[b, par].double() > target[b, par].double()
            if par not in first:  # overrated, and asked for with the largest u: rejected
                more = draft[b, par].double() * (1 - 2.0 ** -24) > target[b, par].double()
                ua[b, i] = 1 - 2.0 ** -24
            elif i % 3:
                more = ~more
            first.setdefault(par, i)
            pick = more.nonzero()[:, 0]
            tokens[b, i] = int(pick[torch.randint(pick.numel(), (1,), generator=g)])
    case = (target, draft, tokens, parents, ua, us)
    want = R.verify(*case)
    assert int(want[1].max()) > 1  # some walks go on
    got = cuda_lib.st_tree_verify(*(t.cuda() for t in case))
    cuda_lib.st_check_status()
    for name, x, w in zip(("path", "n_accepted", "next_token"), got, want):
        assert torch.equal(x.cpu(), w), (name, (x.cpu() != w).sum().item())


def test_verify_greedy_with_nothing_left(cuda_lib):
    """Target and draft both sure of one token: a guess of another one, tried first, is rejected and leaves nothing; then
    the sure token is not accepted either, and the next one is the target's."""
    B, V = 9, 40000
    one = torch.zeros(B, 3, V)
    one[:, :, 31234] = 1.0
    for order in ([0, 5, 31234], [0, 31234, 5]):
        case = (one, one, i32([order] * B), i32([[-1, 0, 0]]), torch.full((B, 3), 0.5), torch.full((B,), 0.25))
        got = [t.cpu() for t in cuda_lib.st_tree_verify(*(t.cuda() for t in case))]
        for x, w in zip(got, R.verify(*case)):
            assert torch.equal(x, w)
        assert got[1].tolist() == [1 if order[1] == 5 else 2] * B and got[2].tolist() == [31234] * B


def test_verify_every_token_removed(cuda_lib):
    """Without a draft, rows that sum to less than 1: both of their tokens are guessed and rejected, which leaves nothing,
    and the next token is the target's. And rows of far more than 1 (scores instead of probabilities), whose draft is the
    same: some token of them."""
    V, B = 20000, 8
    p = torch.zeros(B, 3, V)
    p[:, :, 70], p[:, :, 15000] = 0.3, 0.3
    us = (torch.arange(B) + 0.5) / B
    case = (p, None, i32([[0, 70, 15000]] * B), i32([[-1, 0, 0]]), torch.full((B, 3), 0.9), us)
    got = [t.cpu() for t in cuda_lib.st_tree_verify(*(None if t is None else t.cuda() for t in case))]
    for x, w in zip(got, R.verify(*case)):
        assert torch.equal(x, w)
    assert got[2].tolist() == [70] * 4 + [15000] * 4
    V = 150000
    ones = torch.ones(B, 2, V)
    ones[:, :, 0] = 0
    case = (ones, ones, i32([[0, 0]] * B), i32([[-1, 0]]), torch.full((B, 2), 0.5), us)
    got = [t.cpu() for t in cuda_lib.st_tree_verify(*(t.cuda() for t in case))]
    for x, w in zip(got, R.verify(*case)):
        assert torch.equal(x, w)


@pytest.mark.parametrize("dtype,page,T,is_tree", [("bf16", 16, 1, False), ("fp16", 64, 61, True), ("fp32", 16, 5, True), ("bf16", 7, 3, False)])
def test_narrowed_page_table(cuda_lib, dtype, page, T, is_tree):
    """A view of a wide page table's first columns, in all three calls that read one: what the table itself gives, within
    the bound (the two may be planned in different forms), and the same writes."""
    B, H, Hkv, lens = 3, 8, 2, [777, 5, 300]
    full = [n + T for n in lens]
    q, k, v, pages, parents = attn_case(dtype, B, T, H, Hkv, lens, None, page, is_tree, seed=60)
    wide = torch.cat((pages, torch.full((B, 150000 // page), -5, dtype=torch.int32)), 1).cuda()
    bound = -(-max(full) // page)
    ro, rl, bo, bl = R.attention(q, k, v, pages, lens, None, parents)
    w, ids = torch.ones(D, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")[None, :, None].contiguous()
    new = rand(61, B, T, Hkv, D, dtype=DT[dtype]).cuda()
    after = []
    for table in (wide, wide[:, :bound]):
        cache = cuda_lib.KVCache(k.cuda(), v.cuda(), table)
        o, lse = cuda_lib.st_cache_attn(q.cuda(), cache, i32(lens).cuda(), parents=None if parents is None else parents.cuda())
        R.close("o", o, ro, bo)
        R.close("lse", lse, rl, bl)
        qr = cuda_lib.st_cache_append(q.cuda(), new, new, w, w, 1e-6, ids, (128,), 1e4, cache, i32(lens).cuda())
        got = cuda_lib.st_cache_keep(cache, i32([0, 0, 0]).cuda(), i32([[1, 4]] * B).cuda(), i32([2, 2, 0]).cuda())
        cuda_lib.st_check_status()
        after.append([bits(t) for t in (qr, cache.k, cache.v, got)])
    assert all(torch.equal(x, y) for x, y in zip(*after))
