"""sv_window_attention against the definition in 64 bits."""
from __future__ import annotations

import pytest
import torch

from attend_ref import DIM, PAGE, PagedCase, attend, check, window_seen
from query_aware_sparse_quest_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(case, q, window, sink, starts=None, scale=None, rows=None, stream=None):
    cache = case.cache()
    T, Hq, _ = q.shape
    out = torch.full_like(q, 7.0)
    lse = torch.full((T, Hq), 7.0, device=DEV)
    B = len(case.lens)
    ws = torch.full((binding.sv_window_attention_workspace_size(B, Hq, case.hkv, T),), 0xFF, dtype=torch.uint8, device=DEV)
    binding.sv_window_attention(cache, q, case.table.to(DEV), torch.tensor(case.lens, dtype=torch.int32, device=DEV), window,
                                sink, out, lse, ws,
                                q_start=None if starts is None else torch.tensor(starts, dtype=torch.int32, device=DEV),
                                softmax_scale=scale, stream=stream)
    torch.cuda.synchronize()
    return out, lse


def hide_unseen(case, sizes, window, sink):
    """NaN in what no query token sees, -1 for the pages that none reads."""
    if not window:
        return
    for b, (n, size) in enumerate(zip(case.lens, sizes)):
        if size == 0 or n == 0:
            continue
        lo = max(0, n - size - window + 1)
        case.hide_tokens(b, range(min(sink, lo), lo))
        first, sinks = lo // PAGE, -(-sink // PAGE)
        if sinks < first:
            case.table[b, sinks:first] = -1


def compare(case, sizes, group, window, sink, seed=1, tail=0, decode=False, scale=DIM ** -0.5):
    g = torch.Generator().manual_seed(seed)
    T = sum(sizes)
    q = torch.randn((T + tail, case.hkv * group, DIM), generator=g).bfloat16().to(DEV)
    ref = [attend(q[sum(sizes[:b]):sum(sizes[:b + 1])], *case.tokens(b), window_seen(n, sizes[b], window, sink, DEV), scale)
           for b, n in enumerate(case.lens)]
    hide_unseen(case, sizes, window, sink)
    starts = None if decode else [sum(sizes[:b]) for b in range(len(sizes) + 1)]
    out, lse = run(case, q, window, sink, starts, scale)
    assert binding.sv_get_device_error() == 0
    check(out[:T], lse[:T], [torch.cat(x) for x in zip(*ref)])
    # rows behind the last range are left as they were
    assert (out[T:] == 7.0).all() and (lse[T:] == 7.0).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,window,sink", [
    ([1], 0, 0), ([17], 0, 0), ([128], 0, 0), ([129], 0, 0), ([1000], 0, 0),
    ([1000], 1, 0), ([1000], 16, 1), ([1000], 100, 4), ([1000], 100, 16), ([1000], 333, 40), ([1000], 5000, 4),
    ([5000, 1, 300, 2049], 700, 5),
])
def test_decode_one_token(lens, window, sink, fp8):
    compare(PagedCase(lens, 2, fp8=fp8), [1] * len(lens), 4, window, sink, decode=True)


@pytest.mark.parametrize("group", [1, 2, 3, 5, 6, 7, 8])
def test_decode_groups(group):
    compare(PagedCase([700, 33], 3), [1, 1], group, 200, 3, decode=True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,sizes,group,window,sink", [
    ([1], [1], 1, 0, 0),
    ([16], [16], 8, 0, 0),
    ([40], [40], 8, 0, 0),                       # 320 rows: two tiles
    ([300], [300], 1, 0, 0),                     # no sharing of heads
    ([300], [300], 7, 0, 0),                     # 36 tokens a tile, 252 rows
    ([513], [100], 4, 0, 0),
    ([900], [700], 4, 64, 4),                    # windows shorter than the chunk
    ([900], [700], 8, 1, 0),                     # every token sees itself alone
    ([2000], [500], 4, 300, 37),
    ([2000], [500], 5, 1000, 500),
    ([700, 5, 1, 333], [650, 5, 1, 64], 8, 128, 3),
    ([700, 50, 400], [0, 50, 1], 4, 100, 16),    # a request without query tokens
])
def test_chunks(lens, sizes, group, window, sink, fp8):
    compare(PagedCase(lens, 2, fp8=fp8), sizes, group, window, sink, tail=3)


def test_many_short_requests():
    """More items than CTAs: whole items and cut ones in one call."""
    lens = [1 + (37 * i) % 400 for i in range(90)]
    compare(PagedCase(lens, 4, spare=0), [1] * 90, 2, 90, 7, decode=True)


def test_long_context_few_rows():
    compare(PagedCase([40000], 1), [1], 8, 0, 0, decode=True)
    compare(PagedCase([20000], 1, fp8=True), [3], 8, 0, 0)


def test_large_logits_move_the_base():
    """Logits that grow along the context by hundreds: every tile moves the base."""
    case = PagedCase([1500], 1)
    ramp = torch.linspace(0.1, 30, 1500)
    for t in range(1500):
        case.k[case.table[0, t // PAGE], 0, t % PAGE] *= ramp[t]
    case.k = case.k.bfloat16()
    compare(case, [200], 4, 0, 0)
    case = PagedCase([1500], 1)
    for t in range(1500):
        case.k[case.table[0, t // PAGE], 0, t % PAGE] *= ramp[1499 - t]
    compare(case, [200], 4, 0, 0, scale=0.5)


def test_padded_and_invalid_requests():
    case = PagedCase([50, 20, 300], 2)
    q = torch.randn((3, 8, DIM), generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    for bad, flag in ((0, 0), (-4, 0x8), (19 * PAGE + 1, 0x8)):
        refs = [attend(q[b:b + 1], *case.tokens(b), window_seen(n, 1, 0, 0, DEV), DIM ** -0.5) for b, n in ((0, 50), (2, 300))]
        held, case.lens[1] = case.lens[1], bad
        out, lse = run(case, q, 0, 0)
        case.lens[1] = held
        assert binding.sv_get_device_error() == flag
        check(out[[0, 2]], lse[[0, 2]], [torch.cat(x) for x in zip(*refs)])
        assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()


def test_bad_pages_are_masked():
    case = PagedCase([100, 260], 2)
    for entry in (-1, case.k.shape[0], 2 ** 31 - 1):
        keep = case.table.clone()
        ref = []
        q = torch.randn((11, 8, DIM), generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
        for b, (n, size) in enumerate(((100, 1), (260, 10))):
            seen = window_seen(n, size, 0, 0, DEV)
            seen[:, 32:48] = False
            ref.append(attend(q[b:b + size] if b else q[:1], *case.tokens(b), seen, DIM ** -0.5))
        case.table[:, 2] = entry
        out, lse = run(case, q, 0, 0, starts=[0, 1, 11])
        case.table = keep
        assert binding.sv_get_device_error() == 0x1
        check(out, lse, [torch.cat(x) for x in zip(*ref)])


def test_bad_starts_are_skipped():
    case = PagedCase([100, 200, 64], 1)
    q = torch.randn((20, 4, DIM), generator=torch.Generator().manual_seed(3)).bfloat16().to(DEV)
    ref = attend(q[:5], *case.tokens(0), window_seen(100, 5, 0, 0, DEV), DIM ** -0.5)
    for starts in ([0, 5, 3, 900], [0, 5, 25, 21], [0, 5, -1, -7]):
        out, lse = run(case, q, 0, 0, starts=starts)
        assert binding.sv_get_device_error() & 0x20
        check(out[:5], lse[:5], ref)
    # a chunk longer than its request
    out, lse = run(case, q, 0, 0, starts=[0, 5, 10, 20])
    assert binding.sv_get_device_error() == 0
    case.lens[2] = 9
    out, lse = run(case, q, 0, 0, starts=[0, 5, 10, 20])
    assert binding.sv_get_device_error() == 0x20
    check(out[:5], lse[:5], ref)
    assert (out[10:] == 0).all() and torch.isneginf(lse[10:]).all()
    # starts that would list the same rows many times over
    case = PagedCase([256] * 40, 1)
    q = torch.randn((256, 8, DIM)).bfloat16().to(DEV)
    run(case, q, 0, 0, starts=[0, 256] * 20 + [0])
    assert binding.sv_get_device_error() == 0x20


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [3, 7])
def test_part_filled_row_tiles_repeat_exactly(group, fp8):
    """Row tiles that leave threads without a row: what those hold changes nothing."""
    lens, sizes = [700, 90, 1500, 33], [300, 1, 41, 33]
    case = PagedCase(lens, 3, fp8=fp8)
    q = torch.randn((sum(sizes), 3 * group, DIM), generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    starts = [sum(sizes[:b]) for b in range(5)]
    first = run(case, q, 200, 5, starts)
    other = PagedCase([4000], 1)
    for i in range(4):     # other work in between leaves other values in shared memory
        run(other, torch.full((400, 8, DIM), 10.0 ** i, dtype=torch.bfloat16, device=DEV), 0, 0, [0, 400])
        again = run(case, q, 200, 5, starts)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert binding.sv_get_device_error() == 0


def test_workspace_at_sixteen_bytes_and_rows_inside_a_tensor():
    case = PagedCase([500, 77], 2)
    q = torch.randn((60, 6, DIM), generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    first = run(case, q, 100, 4, [0, 50, 60])
    need = binding.sv_window_attention_workspace_size(2, 6, 2, 60)
    whole = torch.full((need + 16,), 0xFF, dtype=torch.uint8, device=DEV)
    out, lse = torch.full((64, 6, DIM), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((64, 6), 7.0, device=DEV)
    binding.sv_window_attention(case.cache(), q, case.table.to(DEV), torch.tensor(case.lens, dtype=torch.int32, device=DEV), 100, 4,
                                out[1:61], lse[1:61], whole[16:], q_start=torch.tensor([0, 50, 60], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(out[1:61], first[0]) and torch.equal(lse[1:61], first[1])
    assert (out[:1] == 7).all() and (out[61:] == 7).all() and (lse[61:] == 7).all()


def test_repeats_are_identical_and_replays_in_a_graph():
    case = PagedCase([3000, 500], 2)
    cache, table = case.cache(), case.table.to(DEV)
    lens = torch.tensor(case.lens, dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 100, 133], dtype=torch.int32, device=DEV)
    q = torch.randn((133, 16, DIM), device=DEV).bfloat16()
    ws = torch.empty(binding.sv_window_attention_workspace_size(2, 16, 2, 133), dtype=torch.uint8, device=DEV)

    def call(out, lse):
        binding.sv_window_attention(cache, q, table, lens, 700, 4, out, lse, ws, q_start=starts)
    first = torch.empty_like(q), torch.empty((133, 16), device=DEV)
    call(*first)
    out, lse = torch.empty_like(q), torch.empty((133, 16), device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(out, lse)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    # other lengths and queries in the same graph
    lens.copy_(torch.tensor([2100, 33], dtype=torch.int32))
    q.normal_()
    graph.replay()
    call(*first)
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert binding.sv_get_device_error() == 0


def test_empty_calls():
    case = PagedCase([50], 2)
    q = torch.empty((0, 8, DIM), dtype=torch.bfloat16, device=DEV)
    out, lse = run(case, q, 0, 0, [0, 0])
    assert out.shape == (0, 8, DIM) and binding.sv_get_device_error() == 0


def test_two_streams_at_once():
    """Two calls with workspaces of their own, at the same time on two streams."""
    cases = [PagedCase([3000, 70], 2, seed=1), PagedCase([900] * 20, 2, fp8=True, seed=2)]
    sizes = [[500, 3], [30] * 20]
    args = []
    for case, size in zip(cases, sizes):
        T, B = sum(size), len(size)
        q = torch.randn((T, 8, DIM), device=DEV).bfloat16()
        args.append(dict(cache=case.cache(), q=q, page_table=case.table.to(DEV), window=256, sink_tokens=4,
                         seq_lens=torch.tensor(case.lens, dtype=torch.int32, device=DEV),
                         q_start=torch.tensor([sum(size[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV),
                         workspace=torch.empty(binding.sv_window_attention_workspace_size(B, 8, 2, T), dtype=torch.uint8, device=DEV)))
    alone = []
    for a in args:
        o = torch.empty_like(a["q"]), torch.empty(a["q"].shape[:2], device=DEV)
        binding.sv_window_attention(**a, out=o[0], lse=o[1])
        alone.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        both = [(torch.empty_like(a["q"]), torch.empty(a["q"].shape[:2], device=DEV)) for a in args]
        torch.cuda.synchronize()
        for _ in range(4):
            for a, o, st in zip(args, both, streams):
                binding.sv_window_attention(**a, out=o[0], lse=o[1], stream=st)
        torch.cuda.synchronize()
        for o, r in zip(both, alone):
            assert torch.equal(o[0], r[0]) and torch.equal(o[1], r[1])
    assert binding.sv_get_device_error() == 0


@pytest.mark.parametrize("fp8,poison", [(False, "nan"), (False, "inf"), (True, "nan"), (True, "scale")])
@pytest.mark.parametrize("lens,sizes,group,window,sink", [
    ([300], [300], 8, 0, 0),
    ([2000], [500], 4, 300, 37),
    ([2000], [500], 1, 300, 37),
    ([40] * 100, [40] * 100, 4, 0, 0),           # whole items
    ([20000], [9], 8, 0, 0),                     # an item in many pieces
    ([700, 5, 1, 333], [650, 5, 1, 64], 7, 128, 3),
])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(lens, sizes, group, window, sink, fp8, poison):
    case = PagedCase(lens, 2, fp8=fp8)
    g = torch.Generator().manual_seed(3)
    q = torch.randn((sum(sizes), 2 * group, DIM), generator=g).bfloat16().to(DEV)
    seen = [window_seen(n, sizes[b], window, sink, DEV) for b, n in enumerate(lens)]
    ref = [attend(q[sum(sizes[:b]):sum(sizes[:b + 1])], *case.tokens(b), seen[b], DIM ** -0.5) for b in range(len(lens))]
    hit = []                                     # (row, channel) that see such a value
    for b, (n, size) in enumerate(zip(lens, sizes)):
        h = torch.zeros((size, DIM), dtype=torch.bool, device=DEV)
        places = {n - 1: 3, n - size + size // 2: 64, max(0, n - size - window // 2): 127}
        for t, channel in places.items():
            page, at = case.table[b, t // PAGE], t % PAGE
            if poison == "scale":
                case.vs[page, :, at] = float("nan")
                h |= seen[b][:, t, None]
            else:
                case.v[page, :, at, channel] = 0x7F if fp8 else float(poison)
                h[:, channel] |= seen[b][:, t]
        hit.append(h)
    hit = torch.cat(hit)[:, None].expand(-1, 2 * group, -1)
    out, lse = run(case, q, window, sink, [sum(sizes[:b]) for b in range(len(sizes) + 1)])
    assert binding.sv_get_device_error() == 0
    assert hit.any()
    bad = out.isposinf() if poison == "inf" else out.isnan()
    assert torch.equal(bad, hit)
    o, ls, tol, tol_lse = (torch.cat(x) for x in zip(*ref))
    check(torch.where(hit, 0, out), lse, (torch.where(hit, 0, o), ls, tol, tol_lse))


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(fp8):
    """A pool of more than 2^31 elements, used at its end: chunks, single tokens, a shared prefix, and page copies."""
    lens, sizes = [300, 77, 300], [100, 1, 40]
    case = PagedCase(lens, 4, fp8=fp8)
    case.table[2, :5] = case.table[0, :5]                                    # requests 0 and 2 share pages
    g = torch.Generator().manual_seed(6)
    q = torch.randn((sum(sizes), 8, DIM), generator=g).bfloat16().to(DEV)
    ref = [attend(q[sum(sizes[:b]):sum(sizes[:b + 1])], *case.tokens(b), window_seen(n, sizes[b], 90, 5, DEV), DIM ** -0.5)
           for b, n in enumerate(lens)]
    every = [attend(q[b:b + 1], *case.tokens(b), torch.ones((1, n), dtype=torch.bool, device=DEV), DIM ** -0.5)
             for b, n in enumerate(lens)]
    case.spread(270000)
    assert case.k.numel() > 2 ** 31
    out, lse = run(case, q, 90, 5, [sum(sizes[:b]) for b in range(4)])
    check(out, lse, [torch.cat(x) for x in zip(*ref)])
    out, lse = run(case, q[:3], 0, 0)
    check(out, lse, [torch.cat(x) for x in zip(*every)])
    order = [0, 2, 1]
    cache, table = case.cache(), case.table[order].to(DEV).contiguous()
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    ws = torch.empty(binding.sv_prefix_decode_workspace_size(3, 8, 4, 2), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(q[:3]), torch.empty((3, 8), device=DEV)
    for wide in (0, 5000):                                                    # each request alone; the prefix once
        binding.sv_prefix_decode(cache, q[order].contiguous(), torch.nn.functional.pad(table, (0, wide), value=-1),
                                 ints([lens[b] for b in order]), ints([0, 2, 3]), ints([5, 0]), out, lse, ws)
        check(out, lse, [torch.cat([x[b] for b in order]) for x in zip(*every)])
    page = case.table[0, 3].item()
    binding.sv_pages_copy(cache, ints([page, page]), ints([1, 260001]))
    for to in (1, 260001):
        for x in (cache.k_pool, cache.v_pool, cache.k_scale, cache.v_scale):
            assert x is None or torch.equal(x[to], x[page])
    assert binding.sv_get_device_error() == 0
