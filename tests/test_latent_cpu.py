"""Argument checks of the latent calls, on made-up addresses (nothing is launched)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from query_aware_sparse_quest_gb300 import binding, build

SV_OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A = 0x10000
host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up device addresses")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.raw_library()


def cache(fmt=2, latent=A, rope=A, scale=None, pages=10, heads=1, page=16, dim=512):
    return binding.sv_cache(latent, rope, None, pages, heads, page, dim, fmt, scale, None)


BAD_CACHES = [
    (cache(latent=None), INVALID), (cache(rope=None), INVALID), (cache(fmt=0), UNSUPPORTED), (cache(fmt=7), UNSUPPORTED),
    (cache(pages=0), INVALID), (cache(pages=1 << 27), UNSUPPORTED), (cache(heads=2), UNSUPPORTED),
    (cache(page=32), UNSUPPORTED), (cache(dim=128), UNSUPPORTED), (cache(latent=A + 8), INVALID), (cache(rope=A + 2), INVALID),
    (cache(fmt=3), INVALID), (cache(fmt=3, scale=A + 4), INVALID),
]


def append(lib, c, latent=A, ls=576, rope=A, rs=576, slots=A, n=4):
    return lib.sv_latent_append(ctypes.byref(c), latent, ls, rope, rs, slots, n, None)


def gather(lib, c, table=A, lens=A, batch=2, pages=8, starts=A, first=None, rows=9, latent=A, ls=512, rope=A, rs=64):
    return lib.sv_latent_gather(ctypes.byref(c), table, lens, batch, pages, starts, first, rows, latent, ls, rope, rs, None)


def attention(lib, c, q=A, heads=16, starts=None, total=2, table=A, lens=A, batch=2, pages=8, scale=0.07, out=A, lse=A, ws=A,
              size=1 << 40):
    return lib.sv_latent_attention(ctypes.byref(c), q, heads, starts, total, table, lens, batch, pages, scale, out, lse, ws, size, None)


def expanded(lib, q=A, heads=4, qs=A, total=5, k=A, ks=1024, kh=256, rope=A, rs=64, v=A, vs=1024, vh=256, kvs=A, kv=9, batch=2,
             causal=1, scale=0.07, out=A, lse=A, ws=A, size=1 << 40):
    return lib.sv_expanded_attention(q, heads, qs, total, k, ks, kh, rope, rs, v, vs, vh, kvs, kv, batch, causal, scale, out, lse,
                                     ws, size, None)


@host_only
@pytest.mark.parametrize("c,status", BAD_CACHES)
def test_caches_that_are_none(lib, c, status):
    assert append(lib, c) == status and gather(lib, c) == status and attention(lib, c) == status


@host_only
def test_other_calls_refuse_latents(lib):
    c = ctypes.byref(cache())
    assert lib.sv_quest_update_meta(c, A, A, A, 4, None) == UNSUPPORTED
    assert lib.sv_window_attention(c, A, 16, None, 2, A, A, 2, 8, 0, 0, 0.1, A, A, A, 1 << 40, None) == UNSUPPORTED
    assert lib.sv_sparse_decode(c, A, 16, A, A, 2, 8, None, None, 0, 0.1, A, A, A, 1 << 40, None) == UNSUPPORTED
    assert lib.sv_prefix_decode(c, A, 16, A, A, 2, 8, A, A, 1, 0.1, A, A, A, 1 << 40, None) == UNSUPPORTED


@host_only
def test_page_calls_take_latents(lib):
    caches = (binding.sv_cache * 2)(cache(), cache(fmt=3, scale=A))
    assert lib.sv_pages_copy(caches, 2, A, A, 0, None) == SV_OK
    caches = (binding.sv_cache * 2)(cache(), cache(pages=11))
    assert lib.sv_pages_copy(caches, 2, A, A, 0, None) == INVALID
    caches = (binding.sv_cache * 2)(cache(), cache(fmt=3))
    assert lib.sv_pages_copy(caches, 2, A, A, 0, None) == INVALID


@host_only
def test_append(lib):
    c = cache()
    assert append(lib, c, n=0, latent=None, rope=None, slots=None) == SV_OK
    for bad in (dict(n=-1), dict(latent=None), dict(rope=None), dict(slots=None), dict(latent=A + 8), dict(rope=A + 8),
                dict(ls=511), dict(ls=0), dict(ls=580), dict(rs=56), dict(rs=68), dict(rs=-64)):
        assert append(lib, c, **bad) == INVALID, bad
    assert append(lib, c, n=1 << 31) == UNSUPPORTED


@host_only
def test_gather(lib):
    c = cache()
    assert gather(lib, c, rows=0, latent=None, rope=None) == SV_OK
    for bad in (dict(rows=-1), dict(table=None), dict(lens=None), dict(starts=None), dict(batch=0), dict(pages=0),
                dict(latent=None), dict(rope=A + 8), dict(ls=500), dict(rs=32)):
        assert gather(lib, c, **bad) == INVALID, bad
    for bad in (dict(batch=65536), dict(pages=1 << 26), dict(rows=1 << 31)):
        assert gather(lib, c, **bad) == UNSUPPORTED, bad


@host_only
def test_attention(lib):
    c = cache()
    assert attention(lib, c, starts=A, total=0, q=None, out=None, lse=None) == SV_OK
    for bad in (dict(heads=0), dict(batch=0), dict(total=-1), dict(q=None), dict(table=None), dict(lens=None), dict(pages=0),
                dict(q=A + 8), dict(out=None), dict(lse=None), dict(out=A + 8), dict(scale=0.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(total=3), dict(ws=A + 8)):
        assert attention(lib, c, **bad) == INVALID, bad
    for bad in (dict(heads=129), dict(batch=65536, total=65536), dict(pages=1 << 26), dict(starts=A, total=(1 << 24) + 1),
                dict(starts=A, total=1 << 24, heads=128)):
        assert attention(lib, c, **bad) == UNSUPPORTED, bad
    need = binding.sv_latent_attention_workspace_size(2, 16, 2)
    assert need > 0
    for bad in (dict(ws=None), dict(size=need - 1)):
        assert attention(lib, c, **bad) == WORKSPACE, bad
    for sizes in ((0, 16, 2), (2, 0, 2), (2, 129, 2), (2, 16, -1), (65536, 1, 65536), (2, 128, 1 << 24)):
        assert binding.sv_latent_attention_workspace_size(*sizes) == 0


@host_only
def test_expanded(lib):
    assert expanded(lib, total=0, q=None, out=None, lse=None) == SV_OK
    for bad in (dict(heads=0), dict(batch=0), dict(total=-1), dict(kv=-1), dict(q=None), dict(qs=None), dict(kvs=None), dict(k=None),
                dict(v=None), dict(rope=None), dict(out=None), dict(lse=None), dict(q=A + 8), dict(k=A + 8), dict(v=A + 2),
                dict(rope=A + 4), dict(out=A + 16), dict(ks=1020), dict(ks=120), dict(kh=0), dict(kh=100), dict(vs=64), dict(vh=-128),
                dict(rs=56), dict(rs=1 << 36), dict(scale=0.0), dict(scale=float("nan")), dict(ws=A + 8)):
        assert expanded(lib, **bad) == INVALID, bad
    for bad in (dict(heads=65536), dict(batch=65536), dict(total=(1 << 24) + 1), dict(total=1 << 24, heads=128), dict(kv=(1 << 30) + 1)):
        assert expanded(lib, **bad) == UNSUPPORTED, bad
    need = binding.sv_expanded_attention_workspace_size(2, 4, 5)
    assert need > 0
    for bad in (dict(ws=None), dict(size=need - 1)):
        assert expanded(lib, **bad) == WORKSPACE, bad
    for sizes in ((0, 4, 5), (2, 0, 5), (2, 4, -1), (2, 65536, 5), (2, 128, 1 << 24)):
        assert binding.sv_expanded_attention_workspace_size(*sizes) == 0


def test_binding_refuses_what_the_calls_cannot_check(lib):
    t = torch.zeros
    with pytest.raises(ValueError):
        binding.LatentCache(t((3, 16, 128), dtype=torch.bfloat16), t((3, 16, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        binding.LatentCache(t((3, 16, 512), dtype=torch.bfloat16), t((4, 16, 64), dtype=torch.bfloat16))
    with pytest.raises((ValueError, TypeError)):
        binding.LatentCache(t((3, 16, 512)), t((3, 16, 64)))


def test_page_calls_take_a_latent_cache_by_itself():
    c = binding.LatentCache.__new__(binding.LatentCache)
    c.latent, c.c = torch.zeros((3, 16, 512), dtype=torch.bfloat16), cache(pages=3)
    assert binding._cache_list(c).caches == (c,)
    assert binding._cache_list(c).num_phys_pages == 3
    assert binding._cache_list((c, c)).caches == (c, c)
