"""sv_pages_* where lists and tables hold what they should not, and called right before the calls that read what
they write."""
from __future__ import annotations

import pytest
import torch

from attend_ref import DIM, PAGE, attend, check, window_seen
from query_aware_sparse_quest_gb300 import binding
from test_gpu_pages import Device, Model, ints

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("first", [2 ** 31 - 1, 2 ** 31 - 200, 2 ** 30, 7])
@pytest.mark.parametrize("end", [2 ** 31 - 1, 9, -2 ** 31])
def test_freeing_pages_behind_a_row_does_nothing(first, end):
    d = Device(Model(40, 3, 12))
    d.reserve([0, 1], [100, 190])
    d.free([0, 1, 0], [first, max(first, 12), first], [end] * 3)
    d.same()


def test_as_many_slots_as_an_index_counts():
    """A refused request for 2^31 - 6 tokens, behind one of 5: its slots are -1, up to the list's last."""
    most = 2 ** 31 - 1
    d = Device(Model(40, 3, 12))
    d.reserve([0], [10])
    slots = torch.full((most,), -99, dtype=torch.int32, device=DEV)
    binding.sv_pages_reserve(d.table, d.lens, d.counts, ints([0, 1]), ints([5, most - 5]), slots, d.ws)
    torch.cuda.synchronize()
    assert slots[:5].tolist() == d.m.reserve([0], [5])
    assert (slots[5:2 ** 30] == -1).all() and (slots[2 ** 30:] == -1).all()
    d.same(0x8)


@pytest.mark.parametrize("page", [0, 2])
@pytest.mark.parametrize("entry", [-1, 40, 2 ** 31 - 1, -2 ** 31])
def test_a_row_with_a_page_that_is_none_is_not_forked(entry, page):
    """Page 2 is partly filled, so a fork wants a copy of it; page 0 is shared, or was let go of behind a window."""
    d = Device(Model(40, 6, 5))
    d.reserve([0, 1], [40, 37])
    d.table[0, page] = entry
    d.m.table[0][page] = entry
    binding.sv_pages_fork(d.list, d.table, d.lens, d.counts, ints([1, 0, 0]), ints([3, 2, 4]), d.ws)
    made = page == 0 and entry == -1
    d.m.fork([1, 0, 0] if made else [1], [3, 2, 4] if made else [3])
    d.same(0 if made else 0x1)


@pytest.mark.parametrize("count", [0, -3])
@pytest.mark.parametrize("page", [0, 1, 2])
@pytest.mark.parametrize("rows", [8, 5000])
def test_a_row_with_a_free_page_is_not_forked(rows, page, count):
    """Its pages could be another row's next."""
    d = Device(Model(40, rows, 5))
    d.reserve([0, 1], [40, 37])
    p = d.m.table[0][page]
    d.counts[p] = count
    binding.sv_pages_fork(d.list, d.table, d.lens, d.counts, ints([1, 0, 0]), ints([3, 2, 4]), d.ws)
    d.m.counts[p] = 0
    d.m.fork([1], [3])                       # takes the free page, which is the lowest
    d.same(0x100)


@pytest.mark.parametrize("page", [0, 31, 32, 255, 256, 299])
def test_one_free_page_among_many_is_found(page):
    """Forks of every row but one, more than a cluster has warps; row 100 lists a free page."""
    rows, per = 300, 300
    d = Device(Model(rows + per + 9, 2 * rows, per), heads=(1,), fp8=(False,))
    d.reserve(list(range(rows)), [PAGE] * rows)
    d.reserve([100], [(per - 1) * PAGE])
    p = d.m.table[100][page]
    d.counts[p] = 0
    d.m.counts[p] = 0
    binding.sv_pages_fork(d.list, d.table, d.lens, d.counts, ints(list(range(rows))), ints(list(range(rows, 2 * rows))), d.ws)
    others = [r for r in range(rows) if r != 100]
    d.m.fork(others, [rows + r for r in others])
    d.same(0x100)


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("pool,rows,max_pages", [(24, 4, 3), (9001, 30, 200)])
def test_pages_held_outside_the_rows_are_found_after_a_compaction(pool, rows, max_pages, inplace):
    """A prefix cache holds pages by their counts alone: the map says where they, and all others, went."""
    d = Device(Model(pool, rows, max_pages))
    g = torch.Generator().manual_seed(pool)
    most = min(max_pages * PAGE, 2 * pool * PAGE // rows)
    d.reserve(list(range(rows)), [int(torch.randint(0, most, (1,), generator=g)) for _ in range(rows)])
    kept = sorted({p for r in range(0, rows, 2) for p in d.m.table[r][-(-d.m.lens[r] // PAGE) // 2:-(-d.m.lens[r] // PAGE)]})
    for p in kept:
        d.counts[p] += 1
        d.m.counts[p] += 1
    d.free(list(range(0, rows, 2)) + [1])
    d.same()
    held = [p for p in range(pool) if d.m.counts[p]]
    assert set(kept) <= set(held)
    data = list(d.m.data)
    live = d.m.compact()
    assert any(p >= live for p in kept)
    got, page_map = ints([0]), torch.full((pool,), -99, dtype=torch.int32, device=DEV)
    table, counts = (d.table, d.counts) if inplace else (torch.empty_like(d.table), torch.empty_like(d.counts))
    binding.sv_pages_compact(d.list, d.table, d.lens, d.counts, table, counts, got, d.ws, page_map=page_map)
    d.table, d.counts = table, counts
    d.same()
    to = page_map.tolist()
    assert [p for p in range(pool) if to[p] >= 0] == held and sorted(to[p] for p in held) == list(range(live))
    assert all(t == -1 for p, t in enumerate(to) if p not in set(held))
    assert [d.m.data[to[p]] for p in held] == [data[p] for p in held]


@pytest.mark.parametrize("fp8", [False, True])
def test_decodes_right_behind_the_calls_that_lengthen_rows(fp8):
    """Nothing between sv_pages_reserve or sv_pages_fork and the decode that reads the lengths and pages they wrote:
    the same as with the device idle in between."""
    rows, max_pages, hkv, group, pool = 64, 64, 4, 8, 6000
    hq = hkv * group
    g = torch.Generator(device=DEV).manual_seed(2)
    shape = (pool, hkv, PAGE, DIM)
    meta = torch.zeros((pool, hkv, 2, DIM), dtype=torch.bfloat16, device=DEV)
    if fp8:
        scale = torch.full(shape[:3], 0.01, device=DEV)
        codes = [torch.randint(0, 0x70, shape, generator=g, device=DEV, dtype=torch.uint8) for _ in range(2)]
        cache = binding.Cache(*codes, meta, scale, scale.clone())
    else:
        cache = binding.Cache(*[torch.randn(shape, generator=g, device=DEV).bfloat16() for _ in range(2)], meta)
    table = torch.full((rows, max_pages), -1, dtype=torch.int32, device=DEV)
    lens, counts, all_rows = ints([0] * rows), ints([0] * pool), ints(list(range(rows)))
    ws = torch.empty(binding.sv_pages_workspace_size(pool, rows, rows), dtype=torch.uint8, device=DEV)
    aw = torch.empty(binding.sv_window_attention_workspace_size(rows, hq, hkv, rows), dtype=torch.uint8, device=DEV)
    pw = torch.empty(binding.sv_prefix_decode_workspace_size(rows, hq, hkv, 1), dtype=torch.uint8, device=DEV)
    add, slots = ints([13] * rows), torch.empty(13 * rows, dtype=torch.int32, device=DEV)
    q = torch.randn((rows, hq, DIM), generator=g, device=DEV).bfloat16()
    groups, none = ints([0, rows]), ints([0])

    def both():
        o = [(torch.empty_like(q), torch.empty((rows, hq), device=DEV)) for _ in range(2)]
        binding.sv_window_attention(cache, q, table, lens, 200, 4, *o[0], aw)
        binding.sv_prefix_decode(cache, q, table, lens, groups, none, *o[1], pw)
        return [x for y in o for x in y]

    for step in range(40):
        torch.cuda.synchronize()
        if step % 10 == 9:                   # forks of row 0 in place of the others
            kids = all_rows[1:].contiguous()
            binding.sv_pages_free(table, lens, counts, kids)
            binding.sv_pages_fork(cache, table, lens, counts, ints([0] * (rows - 1)), kids, ws)
        else:
            binding.sv_pages_reserve(table, lens, counts, all_rows, add, slots, ws)
        got = both()
        torch.cuda.synchronize()
        for x, y in zip(got, both()):
            assert torch.equal(x, y), step
    assert lens.tolist() == [13 * 36] * rows
    assert binding.sv_get_device_error() == 0
