"""CPU checks of the serving calls' host side: sizes, and every refusal with its status, before anything is launched."""
import ctypes
import re

import pytest
import torch

from qk_norm_rope_gb300 import api
from test_abi import FAKE, T


def P(t):
    return None if t is None else ctypes.pointer(t)


class Serve:
    """Valid arguments of all four calls on fake device pointers; tests perturb one field."""

    def __init__(self, B=2, T_=5, H=8, Hkv=2, page=16, max_pages=4, n_pages=9, dt=api.ST_BF16, V=100):
        self.q, self.k, self.v = T([B, T_, H, 128], dt), T([B, T_, Hkv, 128], dt), T([B, T_, Hkv, 128], dt)
        self.wq, self.wk = T([128], api.ST_F32), T([128], api.ST_F32)
        self.ids, self.axes, self.theta, self.eps, self.tabs, self.ids_k = T([1, T_, 1], api.ST_I32), [128], 1e4, 1e-6, None, None
        self.ck, self.cv = T([n_pages, page, Hkv, 128], dt), T([n_pages, page, Hkv, 128], dt)
        self.pages = T([B, max_pages], api.ST_I32)
        self.lens, self.counts = T([B], api.ST_I32), None
        self.q_rot = T([B, T_, H, 128], dt)
        self.parents = None
        self.o, self.lse = T([B, T_, H, 128], dt, data=FAKE + (1 << 30)), T([B, H, T_], api.ST_F32)
        self.scale, self.ws, self.ws_bytes = 0.0, FAKE, 1 << 40
        self.target, self.draft = T([B, T_, V], api.ST_F32), T([B, T_, V], api.ST_F32)
        self.tokens, self.vpar = T([B, T_], api.ST_I32), T([B, T_], api.ST_I32)
        self.ua, self.us = T([B, T_], api.ST_F32), T([B], api.ST_F32)
        self.path, self.n_acc, self.nxt = T([B, T_], api.ST_I32), T([B], api.ST_I32), T([B], api.ST_I32)
        self.start, self.rows, self.n_rows = T([B], api.ST_I32), T([B, 3], api.ST_I32), T([B], api.ST_I32)
        self.new_lens = T([B], api.ST_I32, data=FAKE + 4096)

    def cache(self):
        c = api.st_kv_cache()
        c.k, c.v, c.pages = (ctypes.pointer(t) if t is not None else None for t in (self.ck, self.cv, self.pages))
        return ctypes.byref(c)

    def append(self):
        r = api.st_rope()
        if self.tabs is not None:
            r.cos, r.sin = (P(t) for t in self.tabs)
        if self.ids is not None:
            r.ids = P(self.ids)
        if self.ids_k is not None:
            r.ids_k = P(self.ids_k)
        r.n_axes, r.theta = len(self.axes), self.theta
        for a, d in enumerate(self.axes):
            r.axes_dim[a] = d
        return api.lib().st_cache_append(P(self.q), P(self.k), P(self.v), P(self.wq), P(self.wk), self.eps, ctypes.byref(r),
                                         self.cache(), P(self.lens), P(self.counts), P(self.q_rot), None)

    def size(self):
        return api.lib().st_cache_attn_workspace_size(P(self.q_rot), self.cache(), P(self.parents))

    def attn(self):
        return api.lib().st_cache_attn(P(self.q_rot), self.cache(), P(self.lens), P(self.counts), P(self.parents), self.scale,
                                       P(self.o), P(self.lse), ctypes.c_void_p(self.ws), self.ws_bytes, None)

    def verify(self):
        return api.lib().st_tree_verify(P(self.target), P(self.draft), P(self.tokens), P(self.vpar), P(self.counts), P(self.ua),
                                        P(self.us), P(self.path), P(self.n_acc), P(self.nxt), None)

    def keep(self):
        return api.lib().st_cache_keep(self.cache(), P(self.start), P(self.rows), P(self.n_rows), P(self.new_lens), None)


def refused(status, want, pattern=None):
    msg = api.lib().st_last_error().decode()
    assert status == want, (api.STATUS_NAMES[status], msg)
    if pattern:
        assert re.search(pattern, msg), msg


CALLS = ("append", "attn", "verify", "keep")


def check(call, want, pattern=None, sizes=None, **fields):
    s = Serve(**(sizes or {}))
    for n, x in fields.items():
        assert hasattr(s, n), n
        setattr(s, n, x)
    refused(getattr(s, call)(), want, pattern)


@pytest.mark.parametrize("call", CALLS)
def test_valid_call_without_gpu_reports_cuda_error(call):
    if torch.cuda.is_available():
        pytest.skip("only meaningful without a GPU")
    check(call, api.ST_ERR_CUDA)
    check(call, api.ST_ERR_CUDA, sizes=dict(dt=api.ST_F16))
    check(call, api.ST_ERR_CUDA, sizes=dict(dt=api.ST_F32))
    check(call, api.ST_ERR_CUDA, sizes=dict(page=7))


def test_empty_calls_are_fine():
    for sizes in (dict(B=0), dict(T_=0)):
        s = Serve(**sizes)
        assert s.append() == api.ST_OK, api.lib().st_last_error()
        assert s.attn() == api.ST_OK, api.lib().st_last_error()
    assert Serve(B=0).verify() == api.ST_OK
    assert Serve(B=0).keep() == api.ST_OK


@pytest.mark.parametrize("call", ("append", "attn", "keep"))
def test_cache_refusals(call):
    E = api
    check(call, E.ST_ERR_INVALID_ARG, "cache", ck=None)
    check(call, E.ST_ERR_INVALID_ARG, "cache", pages=None)
    check(call, E.ST_ERR_SHAPE, "4-D", ck=T([9, 16, 256]))
    check(call, E.ST_ERR_UNSUPPORTED, "D=128", ck=T([9, 16, 2, 64]))
    check(call, E.ST_ERR_SHAPE, "cache.v", cv=T([9, 16, 1, 128]))
    check(call, E.ST_ERR_DTYPE, "cache.v", cv=T([9, 16, 2, 128], E.ST_F16))
    check(call, E.ST_ERR_DTYPE, "cache.k", ck=T([9, 16, 2, 128], E.ST_I32))
    check(call, E.ST_ERR_ALIGN, "unit stride", ck=T([9, 16, 2, 128], strides=[4096, 256, 1, 2]))
    check(call, E.ST_ERR_ALIGN, "aligned", cv=T([9, 16, 2, 128], data=FAKE + 8))
    check(call, E.ST_ERR_ALIGN, "multiple of 16", cv=T([9, 16, 2, 128], strides=[4100, 256, 128, 1]))
    check(call, E.ST_ERR_ALIGN, "expanded", ck=T([9, 16, 2, 128], strides=[4096, 256, 0, 1]))
    check(call, E.ST_ERR_ALIGN, "expanded", cv=T([9, 16, 2, 128], strides=[0, 256, 128, 1]))
    check(call, E.ST_ERR_DTYPE, "pages", pages=T([2, 4], E.ST_I64))
    check(call, E.ST_ERR_ALIGN, "pages", pages=T([2, 4], E.ST_I32, strides=[8, 2]))
    check(call, E.ST_ERR_SHAPE, "pages", pages=T([2, 4, 1], E.ST_I32))
    check(call, E.ST_ERR_SHAPE, "2\\^30", pages=T([2, (1 << 26) + 1], E.ST_I32))
    check(call, E.ST_ERR_SHAPE, "page", ck=T([9, 0, 2, 128]), cv=T([9, 0, 2, 128]))
    check(call, E.ST_ERR_SHAPE, None, pages=T([3, 4], E.ST_I32))  # another batch size


def test_append_refusals():
    E, c = api, "append"
    check(c, E.ST_ERR_INVALID_ARG, "q is NULL", q=None)
    check(c, E.ST_ERR_UNSUPPORTED, "D=128", q=T([2, 5, 8, 64]))
    check(c, E.ST_ERR_SHAPE, "divide", sizes=dict(H=7))
    check(c, E.ST_ERR_SHAPE, "k has shape", k=T([2, 5, 1, 128]))
    check(c, E.ST_ERR_SHAPE, "v has shape", v=T([2, 4, 2, 128]))
    check(c, E.ST_ERR_DTYPE, "same dtype", q=T([2, 5, 8, 128], E.ST_F32))
    check(c, E.ST_ERR_DTYPE, "q has", q=T([2, 5, 8, 128], E.ST_F16))
    check(c, E.ST_ERR_DTYPE, "v has", v=T([2, 5, 2, 128], E.ST_F32))
    check(c, E.ST_ERR_SHAPE, "q_norm_w", wq=T([64], E.ST_F32))
    check(c, E.ST_ERR_DTYPE, "k_norm_w", wk=T([128]))
    check(c, E.ST_ERR_INVALID_ARG, "eps", eps=-1.0)
    check(c, E.ST_ERR_INVALID_ARG, "axes", axes=[64, 32])
    check(c, E.ST_ERR_INVALID_ARG, "theta", theta=0.0)
    check(c, E.ST_ERR_SHAPE, "ids", ids=T([1, 4, 1], E.ST_I32))
    check(c, E.ST_ERR_INVALID_ARG, "ids", ids=None)
    check(c, E.ST_ERR_INVALID_ARG, "share one rotation", ids_k=T([1, 5, 1], E.ST_I32))
    check(c, E.ST_ERR_INVALID_ARG, "not both", tabs=(T([5, 128]), T([5, 128])))
    check(c, E.ST_ERR_SHAPE, "cos/sin", ids=None, tabs=(T([4, 128]), T([4, 128])))
    check(c, E.ST_ERR_INVALID_ARG, "lens is NULL", lens=None)
    check(c, E.ST_ERR_SHAPE, "lens", lens=T([3], E.ST_I32))
    check(c, E.ST_ERR_DTYPE, "lens", lens=T([2], E.ST_I64))
    check(c, E.ST_ERR_ALIGN, "lens", lens=T([2], E.ST_I32, strides=[2]))
    check(c, E.ST_ERR_SHAPE, "counts", counts=T([1], E.ST_I32))
    check(c, E.ST_ERR_SHAPE, "q_rot", q_rot=T([2, 5, 4, 128]))
    check(c, E.ST_ERR_DTYPE, "q_rot", q_rot=T([2, 5, 8, 128], E.ST_F32))
    if not torch.cuda.is_available():
        for cache_type in (E.ST_BF16, E.ST_F16):  # fp32 q and k for a 16-bit cache
            check(c, E.ST_ERR_CUDA, sizes=dict(dt=cache_type), q=T([2, 5, 8, 128], E.ST_F32), k=T([2, 5, 2, 128], E.ST_F32))


def test_attn_refusals():
    E, c = api, "attn"
    check(c, E.ST_ERR_INVALID_ARG, "q_rot is NULL", q_rot=None)
    check(c, E.ST_ERR_DTYPE, "q_rot", q_rot=T([2, 5, 8, 128], E.ST_F16))
    check(c, E.ST_ERR_SHAPE, "divide", sizes=dict(H=7))
    check(c, E.ST_ERR_UNSUPPORTED, "128", sizes=dict(H=258, Hkv=2))
    check(c, E.ST_ERR_SHAPE, "parents", parents=T([3, 5], E.ST_I32))
    check(c, E.ST_ERR_DTYPE, "parents", parents=T([2, 5], E.ST_I64))
    check(c, E.ST_ERR_ALIGN, "parents", parents=T([2, 5], E.ST_I32, strides=[10, 2]))
    check(c, E.ST_ERR_UNSUPPORTED, "256", sizes=dict(T_=257), parents=T([2, 257], E.ST_I32))
    check(c, E.ST_ERR_INVALID_ARG, "scale", scale=float("inf"))
    check(c, E.ST_ERR_SHAPE, "o has shape", o=T([2, 4, 8, 128]))
    check(c, E.ST_ERR_INVALID_ARG, "must not be q_rot", o=T([2, 5, 8, 128]))
    check(c, E.ST_ERR_DTYPE, "o has", o=T([2, 5, 8, 128], E.ST_F32))
    check(c, E.ST_ERR_SHAPE, "lse", lse=T([2, 5, 8], E.ST_F32))
    check(c, E.ST_ERR_DTYPE, "lse", lse=T([2, 8, 5]))
    check(c, E.ST_ERR_ALIGN, "contiguous", lse=T([2, 8, 5], E.ST_F32, strides=[40, 1, 8]))
    check(c, E.ST_ERR_WORKSPACE, "smaller", ws_bytes=Serve().size() - 1)
    check(c, E.ST_ERR_WORKSPACE, "NULL", ws=0)
    check(c, E.ST_ERR_ALIGN, "256-byte", ws=FAKE + 128)
    check(c, E.ST_ERR_SHAPE, "lens", lens=T([3], E.ST_I32))


def test_attn_workspace_size():
    assert Serve().size() >= 256 and Serve(T_=0).size() >= 256
    s = Serve()
    s.q_rot = T([2, 5, 8, 64])
    assert s.size() == 0 and "D=128" in api.lib().st_last_error().decode()


def test_verify_refusals():
    E, c = api, "verify"
    check(c, E.ST_ERR_INVALID_ARG, "target_probs is NULL", target=None)
    check(c, E.ST_ERR_SHAPE, "draft_probs", draft=T([2, 5, 99], E.ST_F32))
    check(c, E.ST_ERR_DTYPE, "same dtype", draft=T([2, 5, 100], E.ST_BF16))
    check(c, E.ST_ERR_DTYPE, "target_probs", target=T([2, 5, 100], E.ST_I32))
    check(c, E.ST_ERR_ALIGN, "unit stride", target=T([2, 5, 100], E.ST_F32, strides=[1000, 200, 2]))
    check(c, E.ST_ERR_ALIGN, "aligned", target=T([2, 5, 100], E.ST_F32, data=FAKE + 2))
    check(c, E.ST_ERR_UNSUPPORTED, "1024", sizes=dict(T_=1025))
    check(c, E.ST_ERR_SHAPE, "root", sizes=dict(T_=0))
    check(c, E.ST_ERR_DTYPE, "tokens", tokens=T([2, 5], E.ST_F32))
    check(c, E.ST_ERR_SHAPE, "tokens", tokens=T([2, 4], E.ST_I32))
    check(c, E.ST_ERR_SHAPE, "parents", vpar=T([2, 4], E.ST_I32))
    check(c, E.ST_ERR_DTYPE, "u_accept", ua=T([2, 5], E.ST_BF16))
    check(c, E.ST_ERR_ALIGN, "u_accept", ua=T([2, 5], E.ST_F32, strides=[6, 1]))
    check(c, E.ST_ERR_SHAPE, "u_sample", us=T([2, 1], E.ST_F32))
    check(c, E.ST_ERR_ALIGN, "path", path=T([2, 5], E.ST_I32, strides=[6, 1]))
    check(c, E.ST_ERR_DTYPE, "n_accepted", n_acc=T([2], E.ST_I64))
    check(c, E.ST_ERR_DTYPE, "next_token", nxt=T([2], E.ST_I64))
    check(c, E.ST_ERR_SHAPE, "counts", counts=T([3], E.ST_I32))


def test_keep_refusals():
    E, c = api, "keep"
    check(c, E.ST_ERR_SHAPE, "rows", rows=None)
    check(c, E.ST_ERR_SHAPE, "rows", rows=T([3, 3], E.ST_I32))
    check(c, E.ST_ERR_DTYPE, "rows", rows=T([2, 3], E.ST_I64))
    check(c, E.ST_ERR_ALIGN, "rows", rows=T([2, 3], E.ST_I32, strides=[1, 2]))
    check(c, E.ST_ERR_SHAPE, "start", start=T([1], E.ST_I32))
    check(c, E.ST_ERR_DTYPE, "n_rows", n_rows=T([2], E.ST_F32))
    check(c, E.ST_ERR_INVALID_ARG, "overlap", new_lens=T([2], E.ST_I32, data=FAKE + 4))


def test_python_layer_refuses_cpu_tensors():
    z = torch.zeros(1, dtype=torch.int32)
    cache = api.KVCache(torch.zeros(1, 16, 1, 128), torch.zeros(1, 16, 1, 128), z[None])
    x = torch.zeros(1, 1, 1, 128)
    with pytest.raises(api.StError):
        api.st_cache_append(x, x, x, torch.ones(128), torch.ones(128), 1e-6, torch.zeros(1, 1, 1, dtype=torch.int32), (128,), 1e4,
                            cache, z)
    with pytest.raises(api.StError):
        api.st_cache_attn(x, cache, z)
    with pytest.raises(api.StError):
        api.st_tree_verify(torch.ones(1, 1, 4), None, z[None], z[None], torch.zeros(1, 1), torch.zeros(1))
    with pytest.raises(api.StError):
        api.st_cache_keep(cache, z, z[None], z)
