"""Results while another stream fills the load and store units: reads of a ring's slot stay in front of its next copy."""
from __future__ import annotations

import pytest
import torch

from attend_ref import DIM, PagedCase
from query_aware_sparse_quest_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


def repeats(call):
    """The same bits alone and beside transposed copies, whose stores take a sector each."""
    noise = torch.randn((4096, 4096), device=DEV)
    sink, side = torch.empty_like(noise), torch.cuda.Stream()
    first = call()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(side):
            for _ in range(4):
                sink.copy_(noise.t())
        got = [call() for _ in range(10)]
        torch.cuda.synchronize()
        assert all(torch.equal(first, x) for x in got)
    assert binding.sv_get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("size", [1, 16, 90])
def test_window_attention_repeats_exactly_beside_scattered_stores(size, fp8):
    case = PagedCase([1500 + 37 * i for i in range(24)], 2, fp8=fp8)
    rows, cache, table = 24 * size, case.cache(), case.table.to(DEV)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    lens, starts = ints(case.lens), None if size == 1 else ints([size * b for b in range(25)])
    q = torch.randn((rows, 16, DIM), device=DEV).bfloat16()
    ws = torch.empty(binding.sv_window_attention_workspace_size(24, 16, 2, rows), dtype=torch.uint8, device=DEV)

    def call():
        out, lse = torch.empty_like(q), torch.empty((rows, 16), device=DEV)
        binding.sv_window_attention(cache, q, table, lens, 1000, 5, out, lse, ws, q_start=starts)
        return torch.cat([out.float().flatten(), lse.flatten()])
    repeats(call)


@pytest.mark.parametrize("per_q_head", [0, 1])
def test_scores_repeat_exactly_beside_scattered_stores(per_q_head):
    B, Hkv, group, pages = 4, 4, 8, 3000
    g = torch.Generator(device=DEV).manual_seed(1)
    meta = torch.randn((B * pages, Hkv, 2, 128), generator=g, device=DEV).bfloat16()
    pool = torch.zeros((B * pages, Hkv, 16, 128), dtype=torch.bfloat16, device=DEV)
    cache = binding.Cache(pool, pool, meta)
    table = torch.randperm(B * pages, generator=g, device=DEV).int().view(B, pages).contiguous()
    lens = torch.full((B,), pages * 16, dtype=torch.int32, device=DEV)
    q = torch.randn((B, Hkv * group, 128), generator=g, device=DEV).bfloat16()
    rows = Hkv * (group if per_q_head else 1)
    idx = torch.empty((B, rows, 64), dtype=torch.int32, device=DEV)
    cnt = torch.empty((B, rows), dtype=torch.int32, device=DEV)
    opts = binding.quest_opts(per_q_head=bool(per_q_head))

    def score():
        s = torch.empty((B, rows, pages), device=DEV)
        if per_q_head:
            binding.sv_quest_select_ex(cache, q, table, lens, 64, opts, idx, cnt, scores_out=s)
        else:
            binding.sv_quest_score(cache, q, table, lens, s)
        return s
    repeats(score)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("budget", [0, 48])            # every page; selected ones
def test_sparse_decode_repeats_exactly_beside_scattered_stores(budget, fp8):
    case = PagedCase([1500 + 37 * i for i in range(24)], 2, fp8=fp8)
    cache, table = case.cache(), case.table.clamp_min(0).to(DEV)
    lens = torch.tensor(case.lens, dtype=torch.int32, device=DEV)
    q = torch.randn((24, 16, DIM), device=DEV).bfloat16()
    pages = budget or case.max_pages
    sel = cnt = None
    if budget:
        sel = torch.stack([torch.randperm(90, device=DEV)[:budget].sort().values for _ in range(48)]).int().view(24, 2, budget).contiguous()
        cnt = torch.full((24, 2), budget, dtype=torch.int32, device=DEV)
    ws = torch.empty(binding.sv_sparse_decode_workspace_size(24, 16, 2, pages), dtype=torch.uint8, device=DEV)

    def call():
        out, lse = torch.empty_like(q), torch.empty((24, 16), device=DEV)
        binding.sv_sparse_decode(cache, q, table, lens, sel, cnt, out, lse, ws)
        return torch.cat([out.float().flatten(), lse.flatten()])
    repeats(call)
