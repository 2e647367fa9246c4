"""sv_pages_* against the same bookkeeping in Python, and the calls used together."""
from __future__ import annotations

import pytest
import torch

from attend_ref import DIM, PAGE, attend, check, window_seen
from query_aware_sparse_quest_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Model:
    """Rows, lengths and counts as Python lists; the data of page p as where it came from."""

    def __init__(self, pool, rows, max_pages):
        self.pool, self.max_pages = pool, max_pages
        self.table = [[-7] * max_pages for _ in range(rows)]
        self.lens, self.counts = [0] * rows, [0] * pool
        self.data = list(range(pool))

    def take(self):
        p = next((i for i, c in enumerate(self.counts) if c == 0), None)
        if p is not None:
            self.counts[p] = 1
        return p

    def free(self, rows, first=None, end=None):
        for i, r in enumerate(rows):
            n = -(-self.lens[r] // PAGE)
            for p in range(max(0, first[i]) if first else 0, min(n, end[i]) if end else n):
                e, self.table[r][p] = self.table[r][p], -1
                if e >= 0:
                    self.counts[e] -= 1
            if not first:
                self.lens[r] = 0

    def fork(self, parents, children):
        free = [i for i, c in enumerate(self.counts) if c == 0]
        for p, c in zip(parents, children):
            n = self.lens[p]
            new = None
            if n % PAGE:
                if not free:
                    continue
                new = free.pop(0)
                self.counts[new] = 1
                self.data[new] = self.data[self.table[p][n // PAGE]]
            for i in range(n // PAGE):
                e = self.table[c][i] = self.table[p][i]
                if e >= 0:
                    self.counts[e] += 1
            if n % PAGE:
                self.table[c][n // PAGE] = new
            self.lens[c] = n

    def reserve(self, rows, add):
        slots = []
        free, used, full = [i for i, c in enumerate(self.counts) if c == 0], 0, False
        for r, a in zip(rows, add):
            n = self.lens[r]
            if -(-(n + a) // PAGE) > self.max_pages:
                slots += [-1] * a
                continue
            need = -(-(n + a) // PAGE) - -(-n // PAGE)
            used += need
            if need and used > len(free):
                slots += [-1] * a
                continue
            for k in range(need):
                p = free[used - need + k]
                self.counts[p] = 1
                self.table[r][-(-n // PAGE) + k] = p
            slots += [self.table[r][t // PAGE] * PAGE + t % PAGE for t in range(n, n + a)]
            self.lens[r] = n + a
        return slots

    def compact(self):
        live = sum(c > 0 for c in self.counts)
        holes = [i for i in range(live) if self.counts[i] == 0]
        movers = [i for i in range(live, self.pool) if self.counts[i] > 0]
        to = {m: h for h, m in zip(holes, movers)}
        for m, h in to.items():
            self.data[h], self.counts[h], self.counts[m] = self.data[m], self.counts[m], 0
        for r, row in enumerate(self.table):
            for p in range(-(-self.lens[r] // PAGE)):
                row[p] = to.get(row[p], row[p])
        return live


class Device:
    """The same on the device, with caches whose pages hold their first number."""

    def __init__(self, m, heads=(2, 1), fp8=(False, True)):
        self.m = m
        self.table, self.lens, self.counts = ints(m.table), ints(m.lens), ints(m.counts)
        self.caches = []
        g = torch.Generator().manual_seed(11)
        for h, f in zip(heads, fp8):
            def values(*shape):
                return torch.randint(-128, 127, (m.pool, h, *shape), generator=g).to(DEV)
            k, v = values(PAGE, DIM), values(PAGE, DIM)
            meta = values(2, DIM).bfloat16()
            if f:
                self.caches.append(binding.Cache(k.to(torch.uint8), v.to(torch.uint8), meta, values(PAGE).float(), values(PAGE).float()))
            else:
                self.caches.append(binding.Cache(k.bfloat16(), v.bfloat16(), meta))
        self.first = [[None if x is None else x.clone() for x in self.parts(c)] for c in self.caches]
        self.list = binding.CacheList(self.caches)
        self.ws = torch.full((binding.sv_pages_workspace_size(m.pool, len(m.lens), 3000),), 0xFF, dtype=torch.uint8, device=DEV)

    @staticmethod
    def parts(c):
        return c.k_pool, c.v_pool, c.meta, c.k_scale, c.v_scale

    def same(self, flags=0):
        torch.cuda.synchronize()
        assert binding.sv_get_device_error() == flags
        assert self.lens.tolist() == self.m.lens
        assert self.counts.tolist() == self.m.counts
        assert self.table.tolist() == self.m.table
        at = torch.tensor(self.m.data, device=DEV)
        for c, first in zip(self.caches, self.first):
            for x, y in zip(self.parts(c), first):
                assert x is None or torch.equal(x, y[at])

    def free(self, rows, first=None, end=None):
        self.m.free(rows, first, end)
        binding.sv_pages_free(self.table, self.lens, self.counts, ints(rows), None if first is None else ints(first),
                              None if end is None else ints(end))

    def fork(self, parents, children):
        self.m.fork(parents, children)
        binding.sv_pages_fork(self.list, self.table, self.lens, self.counts, ints(parents), ints(children), self.ws)

    def reserve(self, rows, add, spare=3):
        want = self.m.reserve(rows, add)
        slots = torch.full((sum(add) + spare,), -99, dtype=torch.int32, device=DEV)
        binding.sv_pages_reserve(self.table, self.lens, self.counts, ints(rows), ints(add), slots, self.ws)
        assert slots.tolist() == want + [-99] * spare

    def compact(self, inplace=True):
        live = self.m.compact()
        got = torch.zeros(1, dtype=torch.int32, device=DEV)
        table, counts = (self.table, self.counts) if inplace else (torch.empty_like(self.table), torch.empty_like(self.counts))
        before = self.table.clone(), self.counts.clone()
        binding.sv_pages_compact(self.list, self.table, self.lens, self.counts, table, counts, got, self.ws)
        assert got.item() == live
        if not inplace:
            assert torch.equal(before[0], self.table) and torch.equal(before[1], self.counts)
        self.table, self.counts = table, counts


@pytest.mark.parametrize("pool,rows,max_pages", [(9, 4, 3), (500, 12, 40), (9001, 30, 300)])
def test_calls_in_turn(pool, rows, max_pages):
    d = Device(Model(pool, rows, max_pages))
    g = torch.Generator().manual_seed(pool)
    held = list(range(rows // 2))
    most = min(max_pages * PAGE, 2 * pool * PAGE // rows)
    d.reserve(held, [int(torch.randint(0, most, (1,), generator=g)) for _ in held])
    d.same()
    d.reserve(held[::-1], [i % 3 for i in range(len(held))])
    d.same()
    kids = [held[-1] + 1 + i for i in range(rows // 4)]
    d.fork([held[i % 2] for i in range(len(kids))], kids)
    d.same()
    d.reserve(kids, [1] * len(kids))
    d.same()
    d.free([held[0], kids[0]])
    d.same()
    d.compact()
    d.same()
    d.free(kids[-1:] + held[1:2])
    d.compact(inplace=False)
    d.same()
    d.reserve([held[0]], [17])
    d.same()


def test_windows_let_go_of_pages():
    d = Device(Model(64, 4, 20))
    d.reserve([0, 1], [300, 150])
    d.free([0, 1, 0], [2, -4, 2], [9, 3, 9])       # row 0 twice
    d.same()
    d.free([1], [5], [99])
    d.free([1], [7], [2])
    d.same()
    d.fork([0], [2])                                # holes are inherited, without a count
    d.same()
    d.free([0])
    d.free([0])                                     # again: nothing is held
    d.same()
    d.compact()
    d.same()


def test_duplicates_free_once():
    d = Device(Model(40, 3, 12))
    d.reserve([0, 1], [100, 190])
    d.m.free([1])
    binding.sv_pages_free(d.table, d.lens, d.counts, ints([1, 1, 1, 1]))
    d.same()


def test_exhausted_pool():
    d = Device(Model(10, 4, 10))
    d.reserve([0, 1], [70, 60])                     # 5 + 4 pages
    d.same()
    d.reserve([2, 0, 1], [17, 9, 4])                # 2 pages: not there; row 0 has room for 9, row 1 for 4
    d.same(0x200)
    d.reserve([2], [16])
    d.fork([1], [3])                                # row 1 is full to the page: no page needed
    d.same()
    d.free([3, 1])
    d.reserve([1], [60])
    d.same()
    d.fork([1, 0], [3, 2])                          # row 1 ends inside a page and none is left
    d.same(0x200)


@pytest.mark.parametrize("n,rows", [(128, 257), (1300, 4096), (1300, 4097)])
def test_long_lists(n, rows):
    """Lists past one block, tables around the size where the check for repeated rows changes."""
    d = Device(Model(4 * n + 40, rows, 5), heads=(1,), fp8=(False,))
    d.reserve(list(range(n)), [1 + (7 * i) % 40 for i in range(n)])
    d.same()
    d.fork([(3 * i) % n for i in range(n)], list(range(n, 2 * n)))
    d.same()
    d.reserve(list(range(2 * n - 1, -1, -1)), [i % 3 for i in range(2 * n)])
    d.same()
    # the same row twice, at both ends of the list
    slots = torch.full((n,), -99, dtype=torch.int32, device=DEV)
    rows = list(range(n - 1)) + [0]
    binding.sv_pages_reserve(d.table, d.lens, d.counts, ints(rows), ints([1] * n), slots, d.ws)
    want = d.m.reserve(rows[:-1], [1] * (n - 1)) + [-1]
    assert slots.tolist() == want
    d.same(0x80)
    d.free(list(range(n, 2 * n)))
    binding.sv_pages_fork(d.list, d.table, d.lens, d.counts, ints([0] * n), ints(list(range(n, 2 * n - 1)) + [n]), d.ws)
    d.m.fork([0] * (n - 1), list(range(n, 2 * n - 1)))
    d.same(0x80)


def test_refused_entries():
    d = Device(Model(50, 6, 8))
    d.reserve([0, 1], [20, 40])
    m = d.m
    # rows out of range, a child twice, a child that is a parent
    binding.sv_pages_fork(d.list, d.table, d.lens, d.counts, ints([0, 0, -1, 0, 0, 3]), ints([2, 2, 4, 6, 1, 5]), d.ws)
    assert binding.sv_get_device_error() == 0x80
    m.fork([0, 3], [2, 5])
    # the child 1 is no parent here, so its fork is made, over what the row held
    m.fork([0], [1])
    d.same()
    binding.sv_pages_fork(d.list, d.table, d.lens, d.counts, ints([2, 0]), ints([4, 2]), d.ws)
    m.fork([2], [4])
    d.same(0x80)
    slots = torch.full((9,), -99, dtype=torch.int32, device=DEV)
    # out of range, negative, twice, too long for the row, past the slots
    binding.sv_pages_reserve(d.table, d.lens, d.counts, ints([9, 0, 0, 4, 5, 2]), ints([1, -3, 2, 2, 200, 2]), slots, d.ws)
    torch.cuda.synchronize()
    assert binding.sv_get_device_error() == 0x80 | 0x8 | 0x4
    assert d.lens.tolist()[4] == m.lens[4] + 2
    m.reserve([4], [2])
    d.same()
    # a partly filled page that somebody else holds too is not written on
    p = m.table[0][m.lens[0] // PAGE]
    d.counts[p] = 2
    d.m.counts[p] = 2
    binding.sv_pages_reserve(d.table, d.lens, d.counts, ints([0]), ints([1]), slots, d.ws)
    d.same(0x100)
    # a count that is zero already
    e = m.table[1][0]
    d.counts[e] = 0
    binding.sv_pages_free(d.table, d.lens, d.counts, ints([1, 7]), ints([0, 0]), ints([1, 1]))
    torch.cuda.synchronize()
    assert binding.sv_get_device_error() == 0x100 | 0x80
    assert d.counts[e].item() == 0
    # pages out of the pool
    d.table[4, 0] = 50
    binding.sv_pages_free(d.table, d.lens, d.counts, ints([4]))
    torch.cuda.synchronize()
    assert binding.sv_get_device_error() == 0x1
    # lengths out of the table
    d.lens[2] = 8 * PAGE + 1
    binding.sv_pages_free(d.table, d.lens, d.counts, ints([2]))
    binding.sv_pages_fork(d.list, d.table, d.lens, d.counts, ints([2]), ints([3]), d.ws)
    torch.cuda.synchronize()
    assert binding.sv_get_device_error() == 0x8


def test_copy():
    d = Device(Model(300, 2, 4), heads=(3, 2, 1), fp8=(False, True, False))
    src, dst = [5, 7, 299, 8], [100, 0, 9, 8]
    binding.sv_pages_copy(d.list, ints(src), ints(dst))
    for s, t in zip(src, dst):
        d.m.data[t] = s
    d.same()
    binding.sv_pages_copy(d.list, ints([1, 300, -1]), ints([2, 3, 4]))
    d.m.data[2] = 1
    d.same(0x1)
    binding.sv_pages_copy(d.caches[0], ints([]), ints([]))
    d.same()


def test_empty_lists_and_empty_pool():
    d = Device(Model(20, 2, 4))
    d.free([])
    d.fork([], [])
    d.reserve([], [])
    d.compact()
    d.same()
    d.reserve([0], [64])
    d.fork([0], [1])
    d.free([0])
    d.compact()
    d.same()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_request_s_life(fp8):
    """Reserve, append, prefill in chunks, fork, append different tokens, decode
    with the shared prefix and with a window, free behind the window, compact,
    decode again: always what the definition gives for the tokens appended."""
    g = torch.Generator().manual_seed(4)
    rows, max_pages, hkv, group, pool = 6, 40, 2, 4, 90
    hq = hkv * group
    shape = (pool, hkv, PAGE, DIM)
    meta = torch.zeros((pool, hkv, 2, DIM), dtype=torch.bfloat16, device=DEV)
    if fp8:
        codes = torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV)
        scale = torch.full(shape[:3], float("nan"), device=DEV)
        cache = binding.Cache(codes, codes.clone(), meta, scale, scale.clone())
    else:
        nan = torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)
        cache = binding.Cache(nan, nan.clone(), meta)
    table = torch.full((rows, max_pages), -1, dtype=torch.int32, device=DEV)
    lens, counts = torch.zeros(rows, dtype=torch.int32, device=DEV), torch.zeros(pool, dtype=torch.int32, device=DEV)
    ws = torch.empty(binding.sv_pages_workspace_size(pool, rows, rows), dtype=torch.uint8, device=DEV)
    held = [[torch.zeros((0, hkv, DIM)), torch.zeros((0, hkv, DIM))] for _ in range(rows)]

    def stored(x):
        x = x.float()
        if not fp8:
            return x
        s = x.abs().amax(-1, keepdim=True) / 448.0
        return (x / s).to(torch.float8_e4m3fn).float() * s

    def append(which, sizes):
        slots = torch.empty(sum(sizes), dtype=torch.int32, device=DEV)
        binding.sv_pages_reserve(table, lens, counts, ints(which), ints(sizes), slots, ws)
        k, v = (torch.randn((sum(sizes), hkv, DIM), generator=g).bfloat16() for _ in range(2))
        binding.sv_quest_update_meta(cache, k.to(DEV), v.to(DEV), slots)
        at = 0
        for r, n in zip(which, sizes):
            held[r] = [torch.cat([a, stored(b[at:at + n])]) for a, b in zip(held[r], (k, v))]
            at += n

    def reference(r, q, window=0, sink=0):
        k, v = (x.double().transpose(0, 1).to(DEV) for x in held[r])
        return attend(q, k, v, window_seen(k.shape[1], q.shape[0], window, sink, DEV), DIM ** -0.5)

    def queries(n):
        return torch.randn((n, hq, DIM), generator=g).bfloat16().to(DEV)

    def window(which, sizes, w, sink):
        q = queries(sum(sizes))
        out, lse = torch.empty_like(q), torch.empty((sum(sizes), hq), device=DEV)
        aw = torch.empty(binding.sv_window_attention_workspace_size(len(which), hq, hkv, sum(sizes)), dtype=torch.uint8, device=DEV)
        starts = ints([sum(sizes[:i]) for i in range(len(sizes) + 1)])
        binding.sv_window_attention(cache, q, table[which].contiguous(), lens[which].contiguous(), w, sink, out, lse, aw, q_start=starts)
        refs = [reference(r, q[sum(sizes[:i]):sum(sizes[:i + 1])], w, sink) for i, r in enumerate(which)]
        check(out, lse, [torch.cat(x) for x in zip(*refs)])

    append([0, 1], [100, 37])
    window([0, 1], [100, 37], 0, 0)
    append([0, 1], [161, 3])
    window([0, 1], [161, 3], 50, 4)
    binding.sv_pages_fork(cache, table, lens, counts, ints([0, 0, 0, 1]), ints([2, 3, 4, 5]), ws)
    for c, p in ((2, 0), (3, 0), (4, 0), (5, 1)):
        held[c] = list(held[p])
    which = [0, 2, 3, 4, 1, 5]
    for step in range(3):
        append(which, [1 + step, 1, 20, 1, 1, 2])
        q = queries(6)
        out, lse = torch.empty_like(q), torch.empty((6, hq), device=DEV)
        pw = torch.empty(binding.sv_prefix_decode_workspace_size(6, hq, hkv, 2), dtype=torch.uint8, device=DEV)
        binding.sv_prefix_decode(cache, q, table[which].contiguous(), lens[which].contiguous(), ints([0, 4, 6]),
                                 ints([261 // PAGE, 40 // PAGE]), out, lse, pw)
        check(out, lse, [torch.cat(x) for x in zip(*[reference(r, q[i:i + 1]) for i, r in enumerate(which)])])
    # a window of 60 tokens and 5 sinks from here on: the pages between are let go
    low = [max(0, len(held[r][0]) + 1 - 60) // PAGE for r in which]
    binding.sv_pages_free(table, lens, counts, ints(which), ints([1] * 6), ints(low))
    append(which, [1] * 6)
    window(which, [1] * 6, 60, 5)
    live = torch.zeros(1, dtype=torch.int32, device=DEV)
    binding.sv_pages_compact(cache, table, lens, counts, table, counts, live, ws)
    assert (counts[: live.item()] > 0).all() and (counts[live.item():] == 0).all()
    window(which, [1] * 6, 60, 5)
    binding.sv_pages_free(table, lens, counts, ints(list(range(rows))))
    assert (counts == 0).all() and (lens == 0).all()
    assert binding.sv_get_device_error() == 0


def test_as_many_caches_as_a_call_takes():
    heads = [1 + i % 2 for i in range(128)]
    d = Device(Model(40, 4, 6), heads=heads, fp8=[i % 3 == 0 for i in range(128)])
    d.reserve([0, 1], [70, 33])
    d.fork([0, 1], [2, 3])
    d.same()
    d.free([0])
    d.compact()
    d.same()


def test_decode_steps_replay_as_a_graph():
    """Reserve, append and both decodes of a step as one graph, over page boundaries: what the calls give one by one."""
    rows, max_pages, hkv, group, pool = 5, 12, 2, 4, 60
    hq = hkv * group
    lens0 = [70, 70, 70, 15, 16]
    g = torch.Generator().manual_seed(9)

    def values(*shape):
        return torch.randn(shape, generator=g).bfloat16().to(DEV)
    prompt = values(sum(lens0), hkv, DIM), values(sum(lens0), hkv, DIM)
    q, kv = values(rows, hq, DIM), [(values(rows, hkv, DIM), values(rows, hkv, DIM)) for _ in range(20)]

    def state():
        shape = (pool, hkv, PAGE, DIM)
        s = dict(cache=binding.Cache(torch.zeros(shape, dtype=torch.bfloat16, device=DEV),
                                     torch.zeros(shape, dtype=torch.bfloat16, device=DEV),
                                     torch.zeros((pool, hkv, 2, DIM), dtype=torch.bfloat16, device=DEV)),
                 table=torch.full((rows, max_pages), -1, dtype=torch.int32, device=DEV), lens=ints([0] * rows),
                 counts=ints([0] * pool), which=ints(list(range(rows))), ones=ints([1] * rows), groups=ints([0, 3, 5]),
                 shared=ints([0, 0]), slots=ints([0] * rows), k=torch.empty_like(kv[0][0]), v=torch.empty_like(kv[0][1]),
                 ws=torch.empty(binding.sv_pages_workspace_size(pool, rows, rows), dtype=torch.uint8, device=DEV),
                 pw=torch.empty(binding.sv_prefix_decode_workspace_size(rows, hq, hkv, 2), dtype=torch.uint8, device=DEV),
                 aw=torch.empty(binding.sv_window_attention_workspace_size(rows, hq, hkv, rows), dtype=torch.uint8, device=DEV),
                 got=[torch.zeros((rows, hq, DIM), dtype=torch.bfloat16, device=DEV) for _ in range(2)],
                 lse=[torch.zeros((rows, hq), device=DEV) for _ in range(2)])
        slots = torch.empty(sum(lens0), dtype=torch.int32, device=DEV)
        binding.sv_pages_reserve(s["table"], s["lens"], s["counts"], s["which"], ints(lens0), slots, s["ws"])
        binding.sv_quest_update_meta(s["cache"], *prompt, slots)
        return s

    def step(s):
        binding.sv_pages_reserve(s["table"], s["lens"], s["counts"], s["which"], s["ones"], s["slots"], s["ws"])
        binding.sv_quest_update_meta(s["cache"], s["k"], s["v"], s["slots"])
        binding.sv_prefix_decode(s["cache"], q, s["table"], s["lens"], s["groups"], s["shared"], s["got"][0], s["lse"][0], s["pw"])
        binding.sv_window_attention(s["cache"], q, s["table"], s["lens"], 40, 3, s["got"][1], s["lse"][1], s["aw"])

    a, b = state(), state()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step(b)
    for k, v in kv:
        for s in (a, b):
            s["k"].copy_(k)
            s["v"].copy_(v)
        step(a)
        graph.replay()
        for x, y in zip(a["got"] + a["lse"] + [a["slots"]], b["got"] + b["lse"] + [b["slots"]]):
            assert torch.equal(x, y)
    assert a["lens"].tolist() == b["lens"].tolist() == [n + 20 for n in lens0]
    assert torch.equal(a["table"], b["table"]) and torch.equal(a["counts"], b["counts"])
    assert binding.sv_get_device_error() == 0
