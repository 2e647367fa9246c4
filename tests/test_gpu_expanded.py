"""sv_expanded_attention against its definition in 64 bits."""
from __future__ import annotations

import pytest
import torch

from latent_ref import attend, causal_seen, check

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5
DEV = "cuda"


@pytest.fixture(autouse=True)
def errors(cuda_ok):
    from query_aware_sparse_quest_gb300 import binding
    binding.sv_get_device_error()
    yield
    assert binding.sv_get_device_error() == 0


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def starts_of(sizes):
    return [sum(sizes[:i]) for i in range(len(sizes) + 1)]


class Rows:
    """q, and k, v, rope in one of the layouts that an expansion leaves; rows behind the last token hold NaN."""

    def __init__(self, sizes, lens, heads, layout="halves", seed=0, mean=0.0, size=1.0, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.sizes, self.lens, self.heads = sizes, lens, heads
        t, s = sum(sizes) + spare, sum(lens) + spare
        self.q = (torch.randn((t, heads, 192), generator=g) * size).bfloat16().to(DEV)
        k, v = (torch.randn((s, heads, 128), generator=g) for _ in range(2))
        rope = torch.randn((s, 64), generator=g)
        for x in (k, v, rope):
            x[sum(lens):] = float("nan")
        k, v, rope = k.bfloat16().to(DEV), (v + mean).bfloat16().to(DEV), rope.bfloat16().to(DEV)
        if layout == "halves":        # [token][head][key | value]
            kv = torch.cat((k, v), -1)
            self.k, self.v = kv[..., :128], kv[..., 128:]
            self.rope = rope
        elif layout == "heads first":
            self.k, self.v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (k, v))
            self.rope = torch.cat((torch.zeros((s, 512), dtype=torch.bfloat16, device=DEV), rope), 1)[:, 512:]
        else:
            self.k, self.v, self.rope = k, v, rope

    def call(self, causal=True, q_start=None, kv_start=None, stream=None):
        from query_aware_sparse_quest_gb300 import binding
        t = self.q.shape[0]
        out = torch.full((t, self.heads, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((t, self.heads), 7.0, device=DEV)
        ws = torch.empty(binding.sv_expanded_attention_workspace_size(len(self.sizes), self.heads, t), dtype=torch.uint8, device=DEV)
        ws.fill_(0xFF)
        binding.sv_expanded_attention(self.q, self.k, self.rope, self.v, ints(q_start or starts_of(self.sizes)),
                                      ints(kv_start or starts_of(self.lens)), out, lse, ws, causal=causal, stream=stream)
        return out, lse

    def reference(self, b, causal=True, rows=None):
        q0, k0, size, n = sum(self.sizes[:b]), sum(self.lens[:b]), self.sizes[b], self.lens[b]
        seen = causal_seen(n, size, DEV) if causal else torch.ones((size, n), dtype=torch.bool, device=DEV)
        rows = slice(None) if rows is None else rows
        k = torch.cat((self.k[k0:k0 + n].double(), self.rope[k0:k0 + n, None].double().expand(-1, self.heads, -1)), -1)
        return attend(self.q[q0:q0 + size][rows], k, self.v[k0:k0 + n].double(), seen[rows], SCALE)

    def check(self, out, lse, causal=True):
        for b, n in enumerate(self.lens):
            at, size = sum(self.sizes[:b]), self.sizes[b]
            if n == 0:
                assert (out[at:at + size] == 0).all() and (lse[at:at + size] == -float("inf")).all()
            elif size:
                check(out[at:at + size], lse[at:at + size], self.reference(b, causal))
        end = sum(self.sizes)
        assert (out[end:] == 7).all() and (lse[end:] == 7).all()


@pytest.mark.parametrize("layout", ["halves", "heads first", "packed"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [1, 3, 16])
@pytest.mark.parametrize("sizes,lens", [
    ([1], [1]),
    ([17, 1, 0, 5], [17, 300, 9, 0]),
    ([127, 128, 129], [127, 128, 129]),
    ([256, 255, 257, 1], [256, 511, 700, 129]),
])
def test_rows(sizes, lens, heads, causal, layout):
    r = Rows(sizes, lens, heads, layout, seed=heads)
    r.check(*r.call(causal), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("sizes,lens,heads", [
    ([1000], [5000], 4),
    ([513, 1, 700], [4097, 9000, 700], 2),
    ([3] * 150, [50] * 150, 2),
    ([1], [20000], 5),
])
def test_long_and_many(sizes, lens, heads, causal):
    r = Rows(sizes, lens, heads, seed=2)
    r.check(*r.call(causal), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("sizes,lens,heads", [
    ([2100, 0, 700, 300], [2100, 40, 700, 1000], 64),   # items of 1 to 17 key tiles
    ([2000], [4000], 40),                               # 320 items, nearly alike: two waves
    ([256], [1100], 152),                               # as many items as SMs, or about
    ([30], [900], 310),
])
def test_items_in_waves(sizes, lens, heads, causal):
    """Sizes whose keys and values do not fit the L2, where CTAs first take whole items in step."""
    r = Rows(sizes, lens, heads, seed=3)
    r.check(*r.call(causal), causal)


def test_more_query_tokens_than_tokens_without_a_mask():
    r = Rows([300, 40], [7, 200], 3)
    r.check(*r.call(False), False)


@pytest.mark.parametrize("size", [0.0, 1e-3, 30.0, 1000.0])
def test_logits_of_any_size(size):
    r = Rows([200], [1000], 2, mean=1.0, size=size)
    r.check(*r.call())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("what", ["k", "v", "rope"])
def test_values_that_are_not_finite_stay_with_rows_that_see_them(what, value):
    sizes, lens, bad = [300, 20], [400, 90], 333
    r = Rows(sizes, lens, 2, seed=4)
    clean, lse0 = r.call()
    getattr(r, what)[bad] = value
    out, lse = r.call()
    first = bad - (lens[0] - sizes[0])
    check(out[:first], lse[:first], r.reference(0, rows=slice(0, first)))
    if what == "v":
        assert not torch.isfinite(out[first:sizes[0]]).any()
    at = sizes[0]
    assert torch.equal(out[at:], clean[at:]) and torch.equal(lse[at:], lse0[at:])


def test_broken_ranges():
    from query_aware_sparse_quest_gb300 import binding
    r = Rows([10, 20, 30], [40, 20, 50], 2, seed=1)
    good, lse0 = r.call()
    # A kv range out of order, one behind the end, a request longer than its tokens: 0 and -inf.
    for kv, hit in (([0, 40, 30, 110], 1), ([0, 40, 60, 10 ** 6], 2), ([0, 5, 60, 110], 0)):
        out, lse = r.call(kv_start=kv)
        assert binding.sv_get_device_error() == 0x20
        at = starts_of(r.sizes)
        assert (out[at[hit]:at[hit + 1]] == 0).all() and (lse[at[hit]:at[hit + 1]] == -float("inf")).all()
    # A query range that is not one is skipped.
    out, lse = r.call(q_start=[0, 10, 30, 10 ** 6])
    assert binding.sv_get_device_error() == 0x20
    assert torch.equal(out[:30], good[:30]) and torch.equal(lse[:30], lse0[:30])
    assert (out[30:] == 7).all()


def test_no_tokens_at_all_and_no_query():
    from query_aware_sparse_quest_gb300 import binding
    q = torch.zeros((2, 3, 192), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((0, 3, 128), dtype=torch.bfloat16, device=DEV)
    rope = torch.zeros((0, 64), dtype=torch.bfloat16, device=DEV)
    out, lse = torch.full((2, 3, 128), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((2, 3), 7.0, device=DEV)
    ws = torch.empty(binding.sv_expanded_attention_workspace_size(1, 3, 2), dtype=torch.uint8, device=DEV)
    binding.sv_expanded_attention(q, k, rope, k, ints([0, 2]), ints([0, 0]), out, lse, ws)
    assert (out == 0).all() and (lse == -float("inf")).all()
    k, rope = torch.zeros((4, 3, 128), dtype=torch.bfloat16, device=DEV), torch.zeros((4, 64), dtype=torch.bfloat16, device=DEV)
    binding.sv_expanded_attention(q[:0], k, rope, k, ints([0, 0]), ints([0, 4]), out[:0], lse[:0], ws)


def test_two_streams_and_a_captured_graph():
    from query_aware_sparse_quest_gb300 import binding
    rows = [Rows([300, 1], [900, 400], 3, seed=s) for s in range(2)]
    ref = [r.call() for r in rows]
    streams = [torch.cuda.Stream() for _ in rows]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(rows[i].call())
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, ref[i][0]) and torch.equal(lse, ref[i][1])
    r = rows[0]
    t = r.q.shape[0]
    q_start, kv_start = ints([0, 300, 301]), ints([0, 900, 1300])
    out, lse = torch.empty((t, 3, 128), dtype=torch.bfloat16, device=DEV), torch.empty((t, 3), device=DEV)
    ws = torch.empty(binding.sv_expanded_attention_workspace_size(2, 3, t), dtype=torch.uint8, device=DEV)
    args = (r.q, r.k, r.rope, r.v, q_start, kv_start, out, lse, ws)
    binding.sv_expanded_attention(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.sv_expanded_attention(*args)
    for sizes, lens in (([300, 1], [900, 400]), ([4, 250], [70, 1000]), ([0, 64], [0, 64])):
        q_start.copy_(ints(starts_of(sizes)))
        kv_start.copy_(ints(starts_of(lens)))
        out.fill_(7.0)
        lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        r.sizes, r.lens = sizes, lens
        r.check(out, lse)


def test_rows_further_apart_than_2_31_elements():
    from query_aware_sparse_quest_gb300 import binding
    n, heads = 300, 2
    wide = torch.empty((heads, n, 1 << 22), dtype=torch.bfloat16, device=DEV)      # 2^22 elements between tokens
    r = Rows([n], [n], heads, seed=3, spare=0)
    k, v, rope = wide[..., :128].transpose(0, 1), wide[..., 128:256].transpose(0, 1), wide[1, :, 256:320]
    k.copy_(r.k)
    v.copy_(r.v)
    rope.copy_(r.rope)
    r.k, r.v, r.rope = k, v, rope
    r.check(*r.call())


def test_sums_of_more_than_65536_tokens():
    """Heads that overlap in memory (a token's row is the next head's of the token before) keep long rows small."""
    n, heads, size = 140000, 160, 70
    r = Rows([size], [n], 1, seed=5, mean=2.0, spare=heads)
    r.heads = heads
    g = torch.Generator().manual_seed(6)
    r.q = torch.randn((size, heads, 192), generator=g).bfloat16().to(DEV)
    flat_k, flat_v = (torch.nan_to_num(x.reshape(-1, 128).contiguous()) for x in (r.k, r.v))
    r.k, r.v = (x.as_strided((n, heads, 128), (128, 128, 1)) for x in (flat_k, flat_v))
    r.rope = r.rope[:n]
    out, lse = r.call()
    pick = [0, 1, 79, 159]
    q, k, v = r.q[:, pick], r.k[:, pick], r.v[:, pick]
    k = torch.cat((k.double(), r.rope[:, None].double().expand(-1, len(pick), -1)), -1)
    check(out[:, pick], lse[:, pick], attend(q, k, v.double(), causal_seen(n, size, DEV), SCALE))


@pytest.mark.parametrize("size,n,spikes", [
    (70, 270000, ((1500, 100.0), (1501, 100.0), (2080, 186.0), (2081, 186.0))),   # even and odd tiles: 1055 a stream
    (200, 140000, ((700, 100.0), (1050, 186.0))),                                 # two row halves: 1094 each
])
def test_sums_that_leave_the_tensor_memory_more_than_once(size, n, spikes):
    """As above, with tokens in some tiles whose logits move the bases: what was summed before is part of the average."""
    heads = 160
    r = Rows([size], [n], 1, seed=7, mean=2.0, spare=heads)
    r.heads = heads
    g = torch.Generator().manual_seed(8)
    r.q = (torch.randn((size, heads, 192), generator=g) * 0.1).bfloat16().to(DEV)
    r.q[..., 128] = 1.0
    flat_k, flat_v = (torch.nan_to_num(x.reshape(-1, 128).contiguous()) for x in (r.k, r.v))
    r.k, r.v = (x.as_strided((n, heads, 128), (128, 128, 1)) for x in (flat_k, flat_v))
    r.rope = r.rope[:n]
    for tile, value in spikes:
        r.rope[tile * 128 + 77, 0] = value
    out, lse = r.call()
    pick = [0, 1, 79, 159]
    q, k, v = r.q[:, pick], r.k[:, pick], r.v[:, pick]
    k = torch.cat((k.double(), r.rope[:, None].double().expand(-1, len(pick), -1)), -1)
    check(out[:, pick], lse[:, pick], attend(q, k, v.double(), causal_seen(n, size, DEV), SCALE))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("sizes,lens,heads", [
    ([5000, 0, 2100, 300], [5000, 40, 2100, 1000], 40),
    ([1600, 1536, 1537], [1700, 1536, 5000], 24),
    ([1550], [1550], 152),
])
def test_long_prompts_in_waves(sizes, lens, heads, causal):
    """Prompts of several row tiles a head, whose keys and values do not fit the L2: whole items first, in step."""
    r = Rows(sizes, lens, heads, seed=4)
    r.check(*r.call(causal), causal)
