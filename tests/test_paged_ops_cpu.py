"""Host-side argument checks of the window, prefix and page calls: refused
before any launch (no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from query_aware_sparse_quest_gb300 import binding, build
from test_library_cpu import (FAKE, SV_ERR_INVALID_ARG, SV_ERR_UNSUPPORTED, SV_ERR_WORKSPACE, SV_OK, _fake_cache,
                              host_only)

ODD = ctypes.c_void_p(0x20008)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.raw_library()


def test_workspace_sizes(lib):
    f = binding.sv_window_attention_workspace_size
    assert f(8, 32, 4, 8) > 0 and f(8, 32, 4, 4096) > f(8, 32, 4, 8)
    assert f(1, 32, 4, 1 << 20) < f(1, 32, 4, 4096) + (8 << 20)     # partials do not grow with the problem
    for bad in ((0, 32, 4, 8), (8, 30, 4, 8), (8, 0, 4, 8), (8, 32, 0, 8), (8, 72, 8, 8), (8, 32, 4, -1), (65536, 32, 4, 8)):
        assert f(*bad) == 0
    g = binding.sv_prefix_decode_workspace_size
    assert g(32, 32, 4, 1) >= 2 * 32 * 32 * 520
    for bad in ((0, 32, 4, 1), (8, 32, 4, 0), (8, 30, 4, 1), (8, 72, 8, 1)):
        assert g(*bad) == 0
    h = binding.sv_pages_workspace_size
    assert h(16384, 64, 100) >= 4 * (3 * 16384 + 128 + 300)
    for bad in ((0, 1, 1), (1 << 27, 1, 1), (10, 0, 1), (10, 1, -1), (10, 1, 65536)):
        assert h(*bad) == 0


@host_only
def test_window_attention_refuses(lib):
    def call(cache=_fake_cache(), q=FAKE, hq=32, qs=FAKE, total=100, pt=FAKE, sl=FAKE, batch=8, pages=100, window=64, sink=4,
             scale=0.088, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 30):
        return lib.sv_window_attention(ctypes.byref(cache), q, hq, qs, total, pt, sl, batch, pages, window, sink, scale, out,
                                       lse, ws, ws_bytes, None)
    for name in ("q", "pt", "sl", "out", "lse"):
        assert call(**{name: None}) == SV_ERR_INVALID_ARG, name
    for name in ("q", "out", "ws"):
        assert call(**{name: ODD}) == SV_ERR_INVALID_ARG, name
    assert call(out=ctypes.c_void_p(0x20010)) == SV_ERR_INVALID_ARG   # 32-byte aligned
    assert call(window=-1) == SV_ERR_INVALID_ARG
    assert call(sink=-1) == SV_ERR_INVALID_ARG
    assert call(total=-1) == SV_ERR_INVALID_ARG
    assert call(qs=None, total=9) == SV_ERR_INVALID_ARG            # one token a request without q_start
    assert call(batch=0) == SV_ERR_INVALID_ARG
    assert call(pages=0) == SV_ERR_INVALID_ARG
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == SV_ERR_INVALID_ARG
    assert call(hq=30) == SV_ERR_INVALID_ARG
    assert call(cache=_fake_cache(hkv=1), hq=16) == SV_ERR_UNSUPPORTED
    assert call(cache=_fake_cache(page_size=32)) == SV_ERR_UNSUPPORTED
    assert call(cache=_fake_cache(head_dim=64)) == SV_ERR_UNSUPPORTED
    assert call(cache=_fake_cache(null=True)) == SV_ERR_INVALID_ARG
    assert call(batch=65536) == SV_ERR_UNSUPPORTED
    assert call(pages=1 << 26) == SV_ERR_UNSUPPORTED
    assert call(total=(1 << 24) + 1, ws_bytes=1 << 40) == SV_ERR_UNSUPPORTED
    assert call(ws=None) == SV_ERR_WORKSPACE
    assert call(ws_bytes=binding.sv_window_attention_workspace_size(8, 32, 4, 100) - 1) == SV_ERR_WORKSPACE
    assert call(total=0) == SV_OK                                   # nothing to do, nothing launched
    assert call(total=0, q=None, out=None, lse=None, ws=None) == SV_OK   # empty tensors have no address
    assert call(total=0, hq=30) == SV_ERR_INVALID_ARG


@host_only
def test_prefix_decode_refuses(lib):
    def call(cache=_fake_cache(), q=FAKE, hq=32, pt=FAKE, sl=FAKE, batch=8, pages=100, gs=FAKE, sp=FAKE, groups=2,
             scale=0.088, out=FAKE, lse=FAKE, ws=FAKE, ws_bytes=1 << 30):
        return lib.sv_prefix_decode(ctypes.byref(cache), q, hq, pt, sl, batch, pages, gs, sp, groups, scale, out, lse, ws,
                                    ws_bytes, None)
    for name in ("q", "pt", "sl", "gs", "sp", "out", "lse"):
        assert call(**{name: None}) == SV_ERR_INVALID_ARG, name
    for name in ("q", "out", "ws"):
        assert call(**{name: ODD}) == SV_ERR_INVALID_ARG, name
    assert call(groups=0) == SV_ERR_INVALID_ARG
    assert call(groups=65536) == SV_ERR_UNSUPPORTED
    assert call(scale=0.0) == SV_ERR_INVALID_ARG
    assert call(hq=33) == SV_ERR_INVALID_ARG
    assert call(ws=None) == SV_ERR_WORKSPACE
    assert call(ws_bytes=binding.sv_prefix_decode_workspace_size(8, 32, 4, 2) - 1) == SV_ERR_WORKSPACE


def _caches(n, **kw):
    return (binding.sv_cache * n)(*[_fake_cache(**kw) for _ in range(n)])


@host_only
def test_page_calls_refuse(lib):
    ws = binding.sv_pages_workspace_size(10, 5, 3)

    def copy(caches=_caches(2), k=2, src=FAKE, dst=FAKE, n=3):
        return lib.sv_pages_copy(caches, k, src, dst, n, None)

    def fork(caches=_caches(2), k=2, pt=FAKE, sl=FAKE, rows=5, pages=8, rc=FAKE, p=FAKE, c=FAKE, n=3, w=FAKE, b=ws):
        return lib.sv_pages_fork(caches, k, pt, sl, rows, pages, rc, p, c, n, w, b, None)

    def reserve(pt=FAKE, sl=FAKE, rows=5, pages=8, rc=FAKE, pool=10, r=FAKE, add=FAKE, n=3, slots=FAKE, m=9, w=FAKE, b=ws):
        return lib.sv_pages_reserve(pt, sl, rows, pages, rc, pool, r, add, n, slots, m, w, b, None)

    def free(pt=FAKE, sl=FAKE, rows=5, pages=8, rc=FAKE, pool=10, r=FAKE, first=None, end=None, n=3):
        return lib.sv_pages_free(pt, sl, rows, pages, rc, pool, r, first, end, n, None)

    def compact(caches=_caches(2), k=2, pt=FAKE, sl=FAKE, rows=5, pages=8, rc=FAKE, po=FAKE, ro=FAKE, live=FAKE, w=FAKE, b=ws):
        return lib.sv_pages_compact(caches, k, pt, sl, rows, pages, rc, po, ro, live, w, b, None)

    mixed = (binding.sv_cache * 2)(_fake_cache(pages=10), _fake_cache(pages=11))
    for call in (copy, fork, compact):
        assert call(caches=None) == SV_ERR_INVALID_ARG
        assert call(k=0) == SV_ERR_INVALID_ARG
        assert call(caches=_caches(129), k=129) == SV_ERR_UNSUPPORTED
        assert call(caches=mixed) == SV_ERR_INVALID_ARG                 # one page table: one pool size
        assert call(caches=_caches(2, head_dim=64)) == SV_ERR_UNSUPPORTED
        assert call(caches=_caches(2, pages=1 << 27)) == SV_ERR_UNSUPPORTED
    for call in (fork, reserve, free, compact):
        for name in ("pt", "sl", "rc"):
            assert call(**{name: None}) == SV_ERR_INVALID_ARG
        assert call(rows=0) == SV_ERR_INVALID_ARG
        assert call(pages=0) == SV_ERR_INVALID_ARG
        assert call(pages=1 << 26) == SV_ERR_UNSUPPORTED
    for call in (reserve, free):
        assert call(pool=0) == SV_ERR_INVALID_ARG
        assert call(pool=1 << 27) == SV_ERR_UNSUPPORTED
        assert call(r=None) == SV_ERR_INVALID_ARG
    for call in (copy, fork, reserve, free):
        assert call(n=-1) == SV_ERR_INVALID_ARG
        assert call(n=0) == SV_OK
    for call in (fork, reserve, free):
        assert call(n=65536) == SV_ERR_UNSUPPORTED
    for call in (fork, reserve, compact):
        assert call(w=None) == SV_ERR_WORKSPACE
        assert call(w=ODD) == SV_ERR_INVALID_ARG
        assert call(b=100) == SV_ERR_WORKSPACE
    assert copy(src=None) == copy(dst=None) == fork(p=None) == fork(c=None) == SV_ERR_INVALID_ARG
    assert reserve(add=None) == reserve(slots=None) == reserve(m=-1) == SV_ERR_INVALID_ARG
    assert free(first=FAKE) == free(end=FAKE) == SV_ERR_INVALID_ARG      # both or neither
    assert compact(po=None) == compact(ro=None) == compact(live=None) == SV_ERR_INVALID_ARG


def test_bindings_check_shapes():
    cpu = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="children"):
        binding.sv_pages_fork(_List(), cpu, cpu, cpu, cpu, torch.zeros(3, dtype=torch.int32), cpu)
    with pytest.raises(ValueError, match="add_tokens"):
        binding.sv_pages_reserve(cpu, cpu, cpu, cpu, torch.zeros(5, dtype=torch.int32), cpu, cpu)
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    table = torch.zeros(2, 9, dtype=torch.int32)
    with pytest.raises(ValueError, match="seq_lens"):
        binding.sv_window_attention(None, q, table, cpu, 0, 0, q, q, q)
    with pytest.raises(ValueError, match="group_start"):
        binding.sv_prefix_decode(None, q, table, torch.zeros(2, dtype=torch.int32), cpu, cpu, q, q, q)
    with pytest.raises(ValueError, match="at least one"):
        binding.CacheList([])
    with pytest.raises(ValueError, match="channels"):
        binding.sv_window_attention(None, q[..., :64], table, torch.zeros(2, dtype=torch.int32), 0, 0, q, q, q)


class _List(binding.CacheList):
    def __init__(self):
        pass
