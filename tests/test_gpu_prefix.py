"""sv_prefix_decode against the definition in 64 bits."""
from __future__ import annotations

import pytest
import torch

from attend_ref import DIM, PAGE, PagedCase, attend, check
from query_aware_sparse_quest_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def share(case, starts, shared):
    """The first pages of every request of a group become those of the group's first request."""
    for g in range(len(shared)):
        for b in range(starts[g] + 1, starts[g + 1]):
            case.table[b, :shared[g]] = case.table[starts[g], :shared[g]]


@pytest.fixture(params=["narrow", "wide"], autouse=True)
def width(request):
    """Small batches over a narrow page table read every request alone, those over a wide one share the prefix's pages."""
    run.wide = request.param == "wide"


def table_of(case):
    table = case.table.to(DEV)
    return torch.nn.functional.pad(table, (0, 5000), value=-1) if run.wide else table


def run(case, q, starts, shared, scale=None):
    B, Hq, _ = q.shape
    out, lse = torch.full_like(q, 7.0), torch.full((B, Hq), 7.0, device=DEV)
    ws = torch.full((binding.sv_prefix_decode_workspace_size(B, Hq, case.hkv, len(shared)),), 0xFF, dtype=torch.uint8, device=DEV)
    binding.sv_prefix_decode(case.cache(), q, table_of(case), ints(case.lens), ints(starts), ints(shared), out, lse, ws,
                             softmax_scale=scale)
    torch.cuda.synchronize()
    return out, lse


def reference(case, q, rows, scale=DIM ** -0.5):
    ref = [attend(q[b:b + 1], *case.tokens(b), torch.ones((1, case.lens[b]), dtype=torch.bool, device=DEV), scale) for b in rows]
    return [torch.cat(x) for x in zip(*ref)]


def queries(case, group, seed=5):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((len(case.lens), case.hkv * group, DIM), generator=g).bfloat16().to(DEV)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group,starts,shared,tails", [
    (8, [0, 1], [3], [5]),                                        # a group of one
    (4, [0, 4], [8], [1, 16, 17, 100]),
    (8, [0, 16], [9], list(range(1, 17))),                        # 128 rows
    (8, [0, 17], [20], [0] * 17),                                 # 136 rows, nothing but the prefix
    (8, [0, 33], [40], [3 * i for i in range(33)]),               # 264 rows: two row tiles
    (7, [0, 3, 3, 40, 41], [5, 2, 30, 0], [(11 * i) % 70 for i in range(40)] + [50]),   # an empty group, one without prefix
    (1, [0, 300], [12], [i % 5 for i in range(300)]),
    (3, [0, 2, 4], [1000, 1], [1, 40, 2000, 3]),
])
def test_groups(group, starts, shared, tails, fp8):
    of = [g for g in range(len(shared)) for _ in range(starts[g], starts[g + 1])]
    case = PagedCase([shared[of[b]] * PAGE + t for b, t in enumerate(tails)], 2, fp8=fp8, spare=1)
    share(case, starts, shared)
    q = queries(case, group)
    out, lse = run(case, q, starts, shared)
    assert binding.sv_get_device_error() == 0
    check(out, lse, reference(case, q, range(len(tails))))


def test_equals_dense_decode():
    """The same call as dense sparse_decode, within both kernels' bounds."""
    starts, shared = [0, 5, 8], [64, 10]
    lens = [64 * PAGE + 9 * i + 1 for i in range(5)] + [10 * PAGE + 5 * i for i in range(1, 4)]
    case = PagedCase(lens, 4)
    share(case, starts, shared)
    q = queries(case, 8)
    out, lse = run(case, q, starts, shared)
    ref = reference(case, q, range(8))
    check(out, lse, ref)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    ws = torch.empty(binding.sv_sparse_decode_workspace_size(8, 32, 4, case.max_pages), dtype=torch.uint8, device=DEV)
    binding.sv_sparse_decode(case.cache(), q, case.table.clamp_min(0).to(DEV), ints(lens), None, None, o2, l2, ws)
    torch.cuda.synchronize()
    check(o2, l2, ref)


def test_padded_and_invalid_requests():
    starts, shared = [0, 3, 5], [4, 0]
    case = PagedCase([70, 64, 90, 20, 33, 40], 2)
    share(case, starts, shared)
    q = queries(case, 8)
    good = reference(case, q, [0, 2, 3, 4])
    for n, flag in ((0, 0), (63, 0x40), (-1, 0x8), (table_of(case).shape[1] * PAGE + 1, 0x8)):
        held, case.lens[1] = case.lens[1], n
        out, lse = run(case, q, starts, shared)
        case.lens[1] = held
        assert binding.sv_get_device_error() & ~0x40 == flag & ~0x40
        check(out[[0, 2, 3, 4]], lse[[0, 2, 3, 4]], good)
        assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
        assert (out[5] == 7).all() and (lse[5] == 7).all()      # in no group
    binding.sv_get_device_error()


@pytest.mark.parametrize("starts,shared", [
    ([0, 3, 2], [4, 0]), ([0, -3, 5], [4, 0]), ([0, 3, 99], [4, 0]), ([0, 3, 5], [4, -1]), ([0, 3, 5], [4, 77]),
    ([-2, 3, 5], [4, 0]),
])
def test_invalid_groups_stay_in_bounds(starts, shared):
    case = PagedCase([70, 64, 90, 20, 33], 2)
    share(case, [0, 3, 5], [4, 0])
    q = queries(case, 8)
    out, lse = run(case, q, starts, shared)
    assert binding.sv_get_device_error() & 0x40
    assert torch.isfinite(out).all()
    for b in range(5):     # each request is either right, empty, or not touched
        r = reference(case, q, [b])
        if not ((out[b] == 0).all() or (out[b] == 7).all()):
            check(out[b:b + 1], lse[b:b + 1], r)


def test_bad_page_is_masked():
    case = PagedCase([70, 64], 1)
    share(case, [0, 2], [3])
    q = queries(case, 8)
    ref = []
    for b in range(2):
        seen = torch.ones((1, case.lens[b]), dtype=torch.bool, device=DEV)
        seen[:, 16:32] = False
        ref.append(attend(q[b:b + 1], *case.tokens(b), seen, DIM ** -0.5))
    case.table[:, 1] = case.k.shape[0]
    out, lse = run(case, q, [0, 2], [3])
    assert binding.sv_get_device_error() == 0x1
    check(out, lse, [torch.cat(x) for x in zip(*ref)])


@pytest.mark.parametrize("fp8", [False, True])
def test_repeats_and_graph(fp8):
    """Calls in a row on one workspace, and a captured one with other lengths, give what a call alone gives."""
    starts, shared = [0, 20, 23], [30, 4]
    lens = [30 * PAGE + 7 * i for i in range(20)] + [4 * PAGE + 3 * i for i in range(3)]
    case = PagedCase(lens, 2, fp8=fp8, max_pages=50)
    share(case, starts, shared)
    q = queries(case, 7)
    first = run(case, q, starts, shared)
    cache, table, gs, sp, ls = case.cache(), table_of(case), ints(starts), ints(shared), ints(lens)
    ws = torch.full((binding.sv_prefix_decode_workspace_size(23, 14, 2, 2),), 0xFF, dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q), torch.empty((23, 14), device=DEV)

    def call():
        binding.sv_prefix_decode(cache, q, table, ls, gs, sp, out, lse, ws)
    for _ in range(20):
        call()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        for _ in range(3):
            call()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    # other groups in the same graph: everyone for itself
    sp.zero_()
    graph.replay()
    torch.cuda.synchronize()
    check(out, lse, reference(case, q, range(23)))
    assert binding.sv_get_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [3, 8])
def test_many_requests(group, fp8):
    """Enough rows that the parts behind the prefixes join them: groups of all sizes, one without shared pages, padded
    requests, one short of its group's pages, requests in no group, and one behind groups out of order."""
    starts, shared = [0, 1, 20, 20, 43, 45], [7, 30, 5, 0, 2]
    lens = []
    for g in range(5):
        lens += [shared[g] * PAGE + (17 * i) % 70 + (g == 3) for i in range(starts[g + 1] - starts[g])]
    lens += [40, 50]
    case = PagedCase(lens, 2, fp8=fp8)
    share(case, starts, shared)
    q = queries(case, group)
    ref = reference(case, q, range(45))
    out, lse = run(case, q, starts, shared)
    assert binding.sv_get_device_error() == 0
    check(out[:45], lse[:45], ref)
    assert (out[45:] == 7).all() and (lse[45:] == 7).all()
    good = [b for b in range(45) if b not in (5, 9, 30)]
    case.lens[5], case.lens[9], case.lens[30] = 0, 30 * PAGE - 1, -4
    out, lse = run(case, q, starts, shared)
    assert binding.sv_get_device_error() == 0x48
    check(out[good], lse[good], [x[good] for x in ref])
    assert (out[[5, 9, 30]] == 0).all() and torch.isneginf(lse[[5, 9, 30]]).all()
    # Group 1 ends behind where group 3 begins: group 3's rows that are not group 1's are empty.
    case.lens = lens
    out, lse = run(case, q, [0, 1, 20, 11, 43, 45], shared)
    assert binding.sv_get_device_error() & 0x40
    for b in range(45):
        if not ((out[b] == 0).all() and torch.isneginf(lse[b]).all()):
            check(out[b:b + 1], lse[b:b + 1], [x[b:b + 1] for x in ref])
    assert (out[25] == 0).all() and torch.isneginf(lse[25]).all()
