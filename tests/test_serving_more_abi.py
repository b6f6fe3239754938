"""CPU checks of caches of 8 bits, windows and shared prefixes: sizes, and every refusal with its status, before anything is
launched."""
import ctypes

import pytest
import torch

from qk_norm_rope_gb300 import api
from test_abi import FAKE, T
from test_serving_abi import P, Serve, refused


class Held(Serve):
    """Valid arguments over a cache of 8 bits on fake device pointers; tests perturb one field."""

    def __init__(self, kv=api.ST_E4M3, **sizes):
        super().__init__(**sizes)
        shape = list(self.ck.shape[:4]) if isinstance(self.ck.shape, list) else [self.ck.shape[i] for i in range(4)]
        n, page, hkv, d = shape
        if kv is not None:
            self.ck, self.cv = T([n, page, hkv, d], kv), T([n, page, hkv, d], kv)
        self.ks, self.vs = (T([n, hkv, page], api.ST_F32), T([n, hkv, page], api.ST_F32)) if kv is not None else (None, None)
        self.scales_given = kv is not None
        self.window, self.sinks, self.shared = 0, 0, None
        B = self.q.shape[0]
        self.rk, self.rv = T([B, 3, hkv, d], api.ST_BF16), T([B, 3, hkv, d], api.ST_BF16)

    def scales(self):
        if not self.scales_given:
            return None
        s = api.st_kv_scales()
        s.k, s.v = (ctypes.pointer(t) if t is not None else None for t in (self.ks, self.vs))
        return ctypes.byref(s)

    def opts(self):
        o = api.st_cache_attn_opts()
        if self.scales_given:
            self._s = api.st_kv_scales()
            self._s.k, self._s.v = (ctypes.pointer(t) if t is not None else None for t in (self.ks, self.vs))
            o.scales = ctypes.pointer(self._s)
        o.window, o.sinks = self.window, self.sinks
        if self.shared is not None:
            o.shared = ctypes.pointer(self.shared)
        return ctypes.byref(o)

    def append(self):
        r = api.st_rope()
        r.ids, r.n_axes, r.theta = P(self.ids), 1, 1e4
        r.axes_dim[0] = 128
        return api.lib().st_cache_append_held(P(self.q), P(self.k), P(self.v), P(self.wq), P(self.wk), 1e-6, ctypes.byref(r),
                                              self.cache(), self.scales(), P(self.lens), P(self.counts), P(self.q_rot), None)

    def size(self):
        return api.lib().st_cache_attn_opt_workspace_size(P(self.q_rot), self.cache(), self.opts(), P(self.parents))

    def attn(self):
        return api.lib().st_cache_attn_opt(P(self.q_rot), self.cache(), self.opts(), P(self.lens), P(self.counts),
                                           P(self.parents), 0.0, P(self.o), P(self.lse), ctypes.c_void_p(self.ws), self.ws_bytes, None)

    def keep(self):
        return api.lib().st_cache_keep_held(self.cache(), self.scales(), P(self.start), P(self.rows), P(self.n_rows),
                                            P(self.new_lens), None)

    def read(self):
        return api.lib().st_cache_read(self.cache(), self.scales(), P(self.start), P(self.counts), P(self.rk), P(self.rv), None)


CALLS = ("append", "attn", "keep", "read")


def check(call, want, pattern=None, sizes=None, **fields):
    s = Held(**(sizes or {}))
    for n, x in fields.items():
        assert hasattr(s, n), n
        setattr(s, n, x)
    refused(getattr(s, call)(), want, pattern)


@pytest.mark.parametrize("call", CALLS)
def test_valid_call_without_gpu_reports_cuda_error(call):
    if torch.cuda.is_available():
        pytest.skip("only meaningful without a GPU")
    for kv in (api.ST_E4M3, api.ST_I8):
        for dt in (api.ST_BF16, api.ST_F16, api.ST_F32):
            check(call, api.ST_ERR_CUDA, sizes=dict(kv=kv, dt=dt))
        check(call, api.ST_ERR_CUDA, sizes=dict(kv=kv, page=7))
    check(call, api.ST_ERR_CUDA, sizes=dict(kv=None))  # without scales: the 16-bit cache
    check("attn", api.ST_ERR_CUDA, sizes=dict(kv=None), window=5, sinks=2, shared=T([1], api.ST_I32))


@pytest.mark.parametrize("call", CALLS)
def test_scales(call):
    E = api
    check(call, E.ST_ERR_DTYPE, "cache.k", scales_given=False)  # 8 bits without scales
    check(call, E.ST_ERR_INVALID_ARG, "k_scale is NULL", ks=None)
    check(call, E.ST_ERR_INVALID_ARG, "v_scale is NULL", vs=None)
    check(call, E.ST_ERR_SHAPE, "k_scale", ks=T([9, 16, 2], E.ST_F32))
    check(call, E.ST_ERR_SHAPE, "v_scale", vs=T([9, 2, 16, 1], E.ST_F32))
    check(call, E.ST_ERR_DTYPE, "k_scale", ks=T([9, 2, 16], E.ST_F16))
    check(call, E.ST_ERR_ALIGN, "unit stride", vs=T([9, 2, 16], E.ST_F32, strides=[32, 1, 2]))
    check(call, E.ST_ERR_ALIGN, "aligned", ks=T([9, 2, 16], E.ST_F32, data=FAKE + 2))
    check(call, E.ST_ERR_ALIGN, "expanded", ks=T([9, 2, 16], E.ST_F32, strides=[32, 0, 1]))
    check(call, E.ST_ERR_INVALID_ARG, "8 bits", ck=T([9, 16, 2, 128]), cv=T([9, 16, 2, 128]))  # scales for a 16-bit cache
    check(call, E.ST_ERR_DTYPE, "cache.v", cv=T([9, 16, 2, 128], E.ST_I8))
    check(call, E.ST_ERR_ALIGN, "multiple of 16", ck=T([9, 16, 2, 128], E.ST_E4M3, strides=[4104, 256, 128, 1]))


def test_types_of_rows():
    E = api
    check("append", E.ST_ERR_DTYPE, "v has", v=T([2, 5, 2, 128], E.ST_E4M3))
    check("append", E.ST_ERR_DTYPE, "q_rot", q_rot=T([2, 5, 8, 128], E.ST_F16))
    check("append", E.ST_ERR_DTYPE, "q has", q=T([2, 5, 8, 128], E.ST_F16))
    check("append", E.ST_ERR_DTYPE, "same dtype", q=T([2, 5, 8, 128], E.ST_F32))
    check("attn", E.ST_ERR_DTYPE, "q_rot", q_rot=T([2, 5, 8, 128], E.ST_I8))
    check("attn", E.ST_ERR_DTYPE, "o has", o=T([2, 5, 8, 128], E.ST_F16, data=FAKE + (1 << 30)))
    check("read", E.ST_ERR_DTYPE, "k has", rk=T([2, 3, 2, 128], E.ST_I8))
    check("read", E.ST_ERR_DTYPE, "v has", rv=T([2, 3, 2, 128], E.ST_F32))
    check("read", E.ST_ERR_DTYPE, "k has", sizes=dict(kv=None), rk=T([2, 3, 2, 128], E.ST_F32), rv=T([2, 3, 2, 128], E.ST_F32))


def test_read_refusals():
    E = api
    check("read", E.ST_ERR_INVALID_ARG, "k is NULL", rk=None)
    check("read", E.ST_ERR_INVALID_ARG, "v is NULL", rv=None)
    check("read", E.ST_ERR_SHAPE, "k has shape", rk=T([3, 3, 2, 128]))
    check("read", E.ST_ERR_SHAPE, "v has shape", rv=T([2, 4, 2, 128]))
    check("read", E.ST_ERR_SHAPE, "4-D", rk=T([2, 3, 256]))
    check("read", E.ST_ERR_ALIGN, "expanded", rk=T([2, 3, 2, 128], strides=[0, 256, 128, 1]))
    check("read", E.ST_ERR_ALIGN, "expanded", rv=T([2, 3, 2, 128], strides=[768, 0, 128, 1]))
    check("read", E.ST_ERR_SHAPE, "start", start=T([3], E.ST_I32))
    check("read", E.ST_ERR_DTYPE, "start", start=T([2], E.ST_I64))
    check("read", E.ST_ERR_SHAPE, "counts", counts=T([1], E.ST_I32))
    check("read", E.ST_ERR_SHAPE, "too many", rk=T([2, (1 << 29) + 1, 2, 128]), rv=T([2, (1 << 29) + 1, 2, 128]))
    s = Held()
    s.rk = s.rv = T([2, 0, 2, 128])
    assert s.read() == E.ST_OK
    assert Held(B=0).read() == E.ST_OK


def test_options():
    E = api
    check("attn", E.ST_ERR_INVALID_ARG, "window", window=-1)
    check("attn", E.ST_ERR_INVALID_ARG, "sinks", sinks=-1)
    check("attn", E.ST_ERR_SHAPE, "shared", shared=T([2], E.ST_I32))
    check("attn", E.ST_ERR_DTYPE, "shared", shared=T([1], E.ST_I64))
    check("attn", E.ST_ERR_INVALID_ARG, "shared data", shared=T([1], E.ST_I32, data=None))
    check("attn", E.ST_ERR_WORKSPACE, "smaller", ws_bytes=255)


def test_workspace_sizes():
    for kv in (None, api.ST_E4M3, api.ST_I8):
        for dt in (api.ST_BF16, api.ST_F32):
            for fields in (dict(), dict(window=7), dict(shared=T([1], api.ST_I32))):
                s = Held(kv=kv, dt=dt, max_pages=4000)
                for n, x in fields.items():
                    setattr(s, n, x)
                n = s.size()
                assert n >= 256, (kv, dt, api.lib().st_last_error())
                s.ws_bytes = n - 1
                refused(s.attn(), api.ST_ERR_WORKSPACE)
    # without options the size is that of the plain call
    s = Held(kv=None, max_pages=4000)
    assert s.size() == Serve(max_pages=4000).size() > 0


def test_the_plain_calls_take_no_cache_of_8_bits():
    s = Held()
    for call in ("append", "attn", "keep"):
        refused(getattr(Serve, call)(s), api.ST_ERR_DTYPE, "cache.k")
    assert Serve.size(s) == 0
