"""Host-side checks of the window, prefix and page calls that need no GPU: arguments added and sizes not taken."""
from __future__ import annotations

import ctypes

import pytest
import torch

from query_aware_sparse_quest_gb300 import binding, build
from test_library_cpu import FAKE, SV_ERR_INVALID_ARG, SV_ERR_WORKSPACE, _fake_cache, host_only
from test_paged_ops_cpu import ODD, _List


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.raw_library()


@host_only
def test_compaction_with_a_map_refuses_what_the_one_without_does(lib):
    ws = binding.sv_pages_workspace_size(10, 5, 0)
    caches = (binding.sv_cache * 2)(_fake_cache(pages=10), _fake_cache(pages=10))

    def call(caches=caches, k=2, pt=FAKE, rows=5, po=FAKE, ro=FAKE, live=FAKE, page_map=FAKE, w=FAKE, b=ws):
        return lib.sv_pages_compact_ex(caches, k, pt, FAKE, rows, 8, FAKE, po, ro, live, page_map, w, b, None)
    for bad in ("caches", "pt", "po", "ro", "live"):
        assert call(**{bad: None}) == SV_ERR_INVALID_ARG
    assert call(rows=0) == call(k=0) == call(w=ODD) == SV_ERR_INVALID_ARG
    assert call(w=None) == call(b=ws - 1) == call(page_map=None, b=ws - 1) == SV_ERR_WORKSPACE


def test_binding_checks_the_map():
    cpu = torch.zeros(4, dtype=torch.int32)
    table = torch.zeros(4, 2, dtype=torch.int32)
    caches = _List()
    caches.c = (binding.sv_cache * 1)(_fake_cache(pages=4))
    with pytest.raises(ValueError, match="page_map"):
        binding.sv_pages_compact(caches, table, cpu, cpu, table, cpu, torch.zeros(1, dtype=torch.int32), cpu,
                                 page_map=torch.zeros(5, dtype=torch.int32))


def test_workspace_sizes_of_what_is_not_taken_are_zero(lib):
    f, g = binding.sv_window_attention_workspace_size, binding.sv_prefix_decode_workspace_size
    assert f(1, 32, 4, 1 << 24) > 0 and f(1, 32, 4, (1 << 24) + 1) == 0
    assert f(65535, 1 << 15, 1 << 15, 1) > 0 and f(65535, 1 << 16, 1 << 16, 1) == 0
    assert g(8, 32, 4, 65535) > 0 and g(8, 32, 4, 65536) == 0
    assert g(65535, 1 << 16, 1 << 16, 1) == 0


def test_caches_of_a_list_are_on_one_device():
    """The calls look at the first one's device only."""
    class On:
        def __init__(self, device):
            self.k_pool, self.c = self, _fake_cache()
            self.get_device = lambda: device
    assert len(binding.CacheList([On(1), On(1)]).caches) == 2
    with pytest.raises(ValueError, match="one device"):
        binding.CacheList([On(0), On(0), On(1)])
