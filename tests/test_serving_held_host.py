"""CPU checks of the Python layer over caches with and without scales."""
import types

import pytest
import torch

from qk_norm_rope_gb300 import api


def inputs():
    q = torch.zeros(2, 1, 4, 128, dtype=torch.bfloat16)
    k = torch.zeros(5, 16, 2, 128, dtype=torch.bfloat16)
    return q, k, k.clone(), torch.zeros(2, 2, dtype=torch.int32)


def bare(k, v, pages):
    """A user's own cache, with what a cache of 16 or 32 bits has."""
    return types.SimpleNamespace(k=k, v=v, pages=pages)


class Own(api.KVCache):
    def __init__(self, k, v, pages):
        self.k, self.v, self.pages = k, v, pages


@pytest.mark.parametrize("make", [bare, Own])
def test_caches_that_know_no_scales(make):
    q, k, v, pages = inputs()
    want = api.st_cache_attn_workspace_size(q, api.KVCache(k, v, pages))
    assert api.st_cache_attn_workspace_size(q, make(k, v, pages)) == want > 0
    x, lens, w = torch.zeros(2, 1, 2, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32), torch.ones(128)
    ids = torch.zeros(1, 1, 1, dtype=torch.int32)
    tables = api.RopeTables(torch.ones(1, 128), torch.zeros(1, 128))
    cache = make(k, v, pages)
    for call in (lambda: api.st_cache_append(q, x, x, w, w, 1e-6, ids, (128,), 1e4, cache, lens),
                 lambda: api.st_cache_append(q, x, x, w, w, 1e-6, tables, None, None, cache, lens),
                 lambda: api.st_cache_attn(q, cache, lens), lambda: api.st_cache_read(cache, lens, 1),
                 lambda: api.st_cache_keep(cache, lens, lens[:, None], lens)):
        with pytest.raises(api.StError, match="CUDA device"):  # as far as a call comes with tensors on the CPU
            call()


@pytest.mark.parametrize("gone", ["k", "v", "pages", "k_scale", "v_scale"])
def test_the_size_of_a_workspace_wants_a_whole_cache(gone):
    q, k, v, pages = inputs()
    s = torch.zeros(5, 2, 16)
    held = api.KVCache(k.to(torch.int8), v.to(torch.int8), pages, s, s)
    assert api.st_cache_attn_workspace_size(q, held) > 0
    for cache in (held, api.KVCache(k, v, pages)):
        if getattr(cache, gone) is None:
            continue
        setattr(cache, gone, None)
        with pytest.raises(api.StError) as e:
            api.st_cache_attn_workspace_size(q, cache)
        assert e.value.status == api.ST_ERR_INVALID_ARG
