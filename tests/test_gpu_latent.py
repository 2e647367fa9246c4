"""sv_latent_attention, sv_latent_append and sv_latent_gather against their definitions in 64 bits."""
from __future__ import annotations

import pytest
import torch

from latent_ref import LATENT, PAGE, ROPE, LatentCase, attend, causal_seen, check, code

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


def queries(rows, heads, seed=0, size=1.0):
    g = torch.Generator().manual_seed(seed + 77)
    return (torch.randn((rows, heads, LATENT + ROPE), generator=g) * size).bfloat16().to(DEV)


def call(case, q, sizes=None, cache=None, total=None, stream=None, ws=None):
    """out, lse of sv_latent_attention; rows that no request holds keep 7."""
    from query_aware_sparse_quest_gb300 import binding
    rows, heads, _ = q.shape
    out = torch.full((rows, heads, LATENT), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((rows, heads), 7.0, device=DEV)
    if ws is None:
        ws = torch.empty(binding.sv_latent_attention_workspace_size(len(case.lens), heads, rows), dtype=torch.uint8, device=DEV)
        ws.fill_(0xFF)
    binding.sv_latent_attention(cache or case.cache(), q, case.table.to(DEV), ints(case.lens), out, lse, ws,
                                softmax_scale=SCALE, q_start=None if sizes is None else ints(starts_of(sizes)), stream=stream)
    return out, lse


def reference(case, q, sizes, b):
    at, n, size = sum(sizes[:b]), case.lens[b], sizes[b]
    c, r = case.tokens(b)
    return attend(q[at:at + size], torch.cat((c, r), 1), c, causal_seen(n, size, DEV), SCALE)


def check_all(case, q, sizes, out, lse):
    for b, n in enumerate(case.lens):
        at, size = sum(sizes[:b]), sizes[b]
        if n == 0:
            assert (out[at:at + size] == 0).all() and (lse[at:at + size] == -float("inf")).all()
        elif size:
            check(out[at:at + size], lse[at:at + size], reference(case, q, sizes, b))
    end = sum(sizes)
    assert (out[end:] == 7).all() and (lse[end:] == 7).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [1, 3, 16, 17, 32, 33, 64, 65, 100, 128])
@pytest.mark.parametrize("lens", [[1], [15, 16, 17, 0, 1], [63, 64, 65, 127, 128, 129, 200], [1023, 3, 700]])
def test_single_tokens(lens, heads, fp8):
    case = LatentCase(lens, fp8=fp8, seed=heads)
    q = queries(len(lens), heads, seed=heads)
    out, lse = call(case, q)
    check_all(case, q, [1] * len(lens), out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,sizes", [
    ([1], [1]),
    ([5], [5]),
    ([16, 40, 0, 3], [16, 7, 2, 0]),
    ([300, 64, 129, 1], [300, 1, 65, 1]),
    ([513, 512, 2, 77], [2, 130, 2, 77]),
])
@pytest.mark.parametrize("heads", [1, 5, 16, 48, 128])
def test_chunks(lens, sizes, heads, fp8):
    case = LatentCase(lens, fp8=fp8, seed=len(lens), max_pages=40)
    q = queries(sum(sizes) + 2, heads, seed=3)
    out, lse = call(case, q, sizes)
    check_all(case, q, sizes, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,lens,sizes", [
    (16, [20011], [1]),
    (128, [9000, 31], [1, 1]),
    (16, [5000, 4000, 6001], [1, 200, 3]),
    (8, [300] * 40, [1] * 40),
    (128, [700], [300]),
    (2, [40] * 200, [3] * 200),
])
def test_long_and_many(heads, lens, sizes, fp8):
    case = LatentCase(lens, fp8=fp8, seed=5)
    q = queries(sum(sizes), heads, seed=5)
    out, lse = call(case, q, sizes)
    check_all(case, q, sizes, out, lse)
    if all(n == 1 for n in sizes):
        again, lse2 = call(case, q)
        check_all(case, q, sizes, again, lse2)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch", [256, 257, 300])
def test_single_tokens_of_many_requests(batch, fp8):
    """Up to 256 requests every CTA plans for itself, behind that a kernel does; some have no tokens."""
    lens = [(7 * i) % 50 for i in range(batch)]
    case = LatentCase(lens, fp8=fp8, seed=6)
    q = queries(batch, 2, seed=6)
    out, lse = call(case, q)
    check_all(case, q, [1] * batch, out, lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_logits_of_any_size(fp8):
    """Weights that are all equal, that fall on one token, and that grow along the row."""
    case = LatentCase([1000, 1000, 1000], fp8=fp8, seed=2, mean=1.0)
    for size in (0.0, 1e-3, 30.0, 1000.0):
        q = queries(3, 16, size=size)
        out, lse = call(case, q)
        check_all(case, q, [1, 1, 1], out, lse)


@pytest.mark.parametrize("fp8", [False, True])
def test_latents_of_any_scale(fp8):
    for scale in (2.0 ** -60, 2.0 ** 40):
        case = LatentCase([130, 17], fp8=fp8, seed=2)
        if fp8:
            case.scale *= scale
        else:
            case.latent *= scale
        q = queries(2, 16)
        q[..., :LATENT] /= scale
        out, lse = call(case, q)
        check_all(case, q, [1, 1], out, lse)


@pytest.mark.parametrize("heads", [1, 16, 20, 128])
def test_scales_of_one_request_far_apart(heads):
    """Tokens whose scales are up to 2^60 apart, and tiles of zero tokens (scale 0) before the first other one.

    A token's weight times its scale is rounded to fp16 in a unit that is at most the largest of the row: below 2^-14 of
    that the rounding is off by up to 2^-25 of it, whatever the product, which comes on top of the bounds of `attend`."""
    lens = [300, 130, 200]
    case = LatentCase(lens, fp8=True, seed=5)
    g = torch.Generator().manual_seed(9)
    case.scale *= torch.exp2(torch.randint(-30, 31, case.scale.shape, generator=g).float())
    for t in range(140):
        page = case.table[2, t // PAGE]
        case.latent[page, t % PAGE], case.scale[page, t % PAGE] = 0, 0.0
    q = queries(3, heads)
    q[..., :LATENT] *= 2.0 ** -32                # the largest scales' logits are of the rotary part's size
    out, lse = call(case, q)
    for b, n in enumerate(lens):
        o, l, tol, tol_lse = reference(case, q, [1, 1, 1], b)
        page = case.table[b, : -(-n // PAGE)].long()
        size = case.scale[page].flatten()[:n].double().to(DEV)
        codes = case.latent[page].flatten(0, 1)[:n].to(DEV).view(torch.float8_e4m3fn).double().abs()
        c, r = case.tokens(b)
        z = (q[b].double() @ torch.cat((c, r), 1).T) * SCALE
        largest = (torch.exp(z - l[0][:, None]) * size).amax(1)
        check(out[b:b + 1], lse[b:b + 1], (o, l, tol + 2.0 ** -25 * largest[None, :, None] * codes.sum(0), tol_lse))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("heads", [16, 128])
def test_values_that_are_not_finite_stay_with_rows_that_see_them(value, heads, fp8):
    lens, sizes, bad = [200, 90], [40, 3], 180
    case = LatentCase(lens, fp8=fp8, seed=9)
    q = queries(sum(sizes), heads)
    clean, lse0 = call(case, q, sizes)
    case.fill_tokens(0, [bad], value)
    out, lse = call(case, q, sizes)
    first = bad - (lens[0] - sizes[0])      # the first row that sees it
    c, r = case.tokens(0)
    ref = attend(q[:first], torch.cat((c, r), 1), c, causal_seen(lens[0], sizes[0], DEV)[:first], SCALE)
    check(out[:first], lse[:first], ref)
    assert not torch.isfinite(out[first:sizes[0]]).any()
    assert torch.equal(out[sizes[0]:], clean[sizes[0]:]) and torch.equal(lse[sizes[0]:], lse0[sizes[0]:])


def test_pages_that_the_table_does_not_give():
    from query_aware_sparse_quest_gb300 import binding
    case = LatentCase([100, 50], seed=1)
    q = queries(2, 16)
    table = case.table.clone()
    table[0, 2], table[1, 0] = -1, 10 ** 6
    hidden = [list(range(32, 48)), list(range(16))]
    cache = case.cache()
    good, case.table = case.table, table
    out, lse = call(case, q, cache=cache)
    assert binding.sv_get_device_error() == 0x1
    case.table = good
    for b in range(2):
        c, r = case.tokens(b)
        seen = torch.ones((1, case.lens[b]), dtype=torch.bool, device=DEV)
        seen[:, hidden[b]] = False
        check(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], torch.cat((c, r), 1), c, seen, SCALE))


def test_bad_lengths_and_starts():
    from query_aware_sparse_quest_gb300 import binding
    case = LatentCase([100, 50, 20], seed=1)
    q = queries(3, 16)
    for lens, bits in (([100, -1, 20], 0x8), ([100, 1 << 30, 20], 0x8)):
        kept, case.lens = case.lens, lens
        cache = LatentCase([100, 50, 20], seed=1).cache()
        out, lse = call(case, q, cache=cache)
        assert binding.sv_get_device_error() == bits
        assert (out[1] == 0).all() and (lse[1] == -float("inf")).all()
        case.lens = kept
        for b in (0, 2):   # (how a request is cut, and so its last bits, goes by the batch)
            check(out[b:b + 1], lse[b:b + 1], reference(case, q, [1, 1, 1], b))
    out = torch.full((6, 16, LATENT), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((6, 16), 7.0, device=DEV)
    ws = torch.empty(binding.sv_latent_attention_workspace_size(3, 16, 6), dtype=torch.uint8, device=DEV)
    q = queries(6, 16)
    # The second chunk is out of order, the third longer than the pool of rows.
    binding.sv_latent_attention(case.cache(), q, case.table.to(DEV), ints(case.lens), out, lse, ws, softmax_scale=SCALE,
                                q_start=ints([0, 3, 2, 9]))
    assert binding.sv_get_device_error() == 0x20
    check(out[:2], lse[:2], tuple(x[:2] for x in reference(case, q, [3, 0, 0], 0)))
    # A chunk longer than its request.
    case.lens = [2, 50, 20]
    binding.sv_latent_attention(case.cache(), q, case.table.to(DEV), ints(case.lens), out, lse, ws, softmax_scale=SCALE,
                                q_start=ints([0, 3, 4, 5]))
    assert binding.sv_get_device_error() == 0x20
    assert (out[:3] == 0).all() and (lse[:3] == -float("inf")).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_pool_of_more_than_2_31_elements(fp8):
    case = LatentCase([500, 33], fp8=fp8, seed=4)
    case.spread(300000 if not fp8 else 600000)
    q = queries(2, 16)
    cache = case.cache()
    out, lse = call(case, q, cache=cache)
    check_all(case, q, [1, 1], out, lse)
    # What is written and read back there.
    from query_aware_sparse_quest_gb300 import binding
    n = case.latent.shape[0]
    slots = ints([n * PAGE - 1, (n - 2) * PAGE])
    rows = torch.randn((2, LATENT + ROPE), device=DEV).bfloat16()
    binding.sv_latent_append(cache, rows[:, :LATENT], rows[:, LATENT:], slots)
    table = ints([[n - 2], [n - 1]])
    back, rope = torch.empty((2, LATENT), dtype=torch.bfloat16, device=DEV), torch.empty((2, ROPE), dtype=torch.bfloat16, device=DEV)
    binding.sv_latent_gather(cache, table, ints([1, 16]), ints([0, 1, 2]), back, rope, first_token=ints([0, 15]))
    assert torch.equal(rope.flip(0), rows[:, LATENT:])
    if not fp8:
        assert torch.equal(back.flip(0), rows[:, :LATENT])


def test_two_streams_and_a_captured_graph():
    from query_aware_sparse_quest_gb300 import binding
    cases = [LatentCase([900, 30, 411], seed=s, fp8=s == 1) for s in range(2)]
    qs = [queries(3, 16, seed=s) for s in range(2)]
    ref = [call(c, q) for c, q in zip(cases, qs)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    caches = [c.cache() for c in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call(cases[i], qs[i], cache=caches[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, ref[i][0]) and torch.equal(lse, ref[i][1])
    # A captured call sees new lengths and queries on replay.
    case, q = cases[0], qs[0].clone()
    lens, table = ints(case.lens), case.table.to(DEV)
    out = torch.empty((3, 16, LATENT), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((3, 16), device=DEV)
    ws = torch.empty(binding.sv_latent_attention_workspace_size(3, 16, 3), dtype=torch.uint8, device=DEV)
    binding.sv_latent_attention(caches[0], q, table, lens, out, lse, ws, softmax_scale=SCALE)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.sv_latent_attention(caches[0], q, table, lens, out, lse, ws, softmax_scale=SCALE)
    for new in ([900, 30, 411], [17, 0, 400], [640, 30, 1]):
        lens.copy_(ints(new))
        q.copy_(queries(3, 16, seed=sum(new)))
        graph.replay()
        torch.cuda.synchronize()
        for b, n in enumerate(new):
            if n == 0:
                assert (out[b] == 0).all() and (lse[b] == -float("inf")).all()
                continue
            c, r = case.tokens(b, n)
            check(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], torch.cat((c, r), 1), c,
                                                     torch.ones((1, n), dtype=torch.bool, device=DEV), SCALE))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens", [1, 7, 16, 1000])
@pytest.mark.parametrize("packed", [False, True])
def test_append_and_gather(tokens, packed, fp8):
    from query_aware_sparse_quest_gb300 import binding
    g = torch.Generator().manual_seed(tokens)
    pages = -(-tokens // PAGE) + 5
    cache = binding.LatentCache.empty(pages, fp8=fp8)
    filler = 0x5A if fp8 else 3.0
    cache.latent.fill_(filler)
    cache.rope.fill_(3.0)
    if fp8:
        cache.scale.fill_(3.0)
    rows = torch.randn((tokens, LATENT + ROPE), generator=g) * torch.randn((tokens, 1), generator=g).mul(3).exp()
    rows[0, :LATENT] = 0                       # a row of zeros codes as scale 0
    rows = rows.bfloat16().to(DEV)
    latent, rope = rows[:, :LATENT], rows[:, LATENT:]
    if packed:
        latent, rope = latent.contiguous(), rope.contiguous()
    order = torch.randperm(pages * PAGE, generator=g)[:tokens].int().to(DEV)
    binding.sv_latent_append(cache, latent, rope, order)
    untouched = torch.ones(pages * PAGE, dtype=torch.bool, device=DEV)
    untouched[order.long()] = False
    assert torch.equal(cache.rope.view(-1, ROPE)[order.long()], rope)
    assert (cache.rope.view(-1, ROPE)[untouched] == 3).all() and (cache.latent.view(-1, LATENT)[untouched] == filler).all()
    if fp8:
        want, scale = code(latent)
        assert torch.equal(cache.scale.view(-1)[order.long()], scale)
        assert torch.equal(cache.latent.view(-1, LATENT)[order.long()], want)
        assert (cache.scale.view(-1)[untouched] == 3).all()
        back = (want.view(torch.float8_e4m3fn).float() * scale[:, None]).bfloat16()
    else:
        assert torch.equal(cache.latent.view(-1, LATENT)[order.long()], latent)
        back = latent
    # Each token as a request of its own page and place, into rows of a wider tensor, some of which nobody holds.
    table = (order // PAGE)[:, None].contiguous()
    place = (order % PAGE).int()
    wide = torch.full((tokens + 3, LATENT + ROPE + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    binding.sv_latent_gather(cache, table, place + 1, torch.arange(1, tokens + 2, device=DEV).int(), wide[:, :LATENT],
                             wide[:, LATENT:LATENT + ROPE], first_token=place)
    assert torch.equal(wide[1:tokens + 1, :LATENT], back) and torch.equal(wide[1:tokens + 1, LATENT:-8], rope)
    assert (wide[0] == 7).all() and (wide[tokens + 1:] == 7).all() and (wide[:, -8:] == 7).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_gather_ranges(fp8):
    from query_aware_sparse_quest_gb300 import binding
    case = LatentCase([100, 0, 17, 333], fp8=fp8, seed=6)
    cache = case.cache()
    firsts, sizes = [5, 0, 16, 0], [90, 0, 1, 333]
    total = sum(sizes)
    latent = torch.full((total + 1, LATENT), 7.0, dtype=torch.bfloat16, device=DEV)
    rope = torch.full((total + 1, ROPE), 7.0, dtype=torch.bfloat16, device=DEV)
    binding.sv_latent_gather(cache, case.table.to(DEV), ints(case.lens), ints(starts_of(sizes)), latent, rope, first_token=ints(firsts))
    for b, (f, n) in enumerate(zip(firsts, sizes)):
        c, r = case.tokens(b)
        at = sum(sizes[:b])
        # value(code) * scale is rounded to fp32 and then to bf16: half a step of each.
        assert ((latent[at:at + n].double() - c[f:f + n]).abs() <= c[f:f + n].abs() * (2.0 ** -8 + 2.0 ** -23) * (1 if fp8 else 0)).all()
        assert torch.equal(rope[at:at + n].double(), r[f:f + n])
    assert (latent[total:] == 7).all() and (rope[total:] == 7).all()
    # From the first token on; tokens behind a request's last read as zeros, with an error.
    binding.sv_latent_gather(cache, case.table.to(DEV), ints(case.lens), ints([0, 0, 0, 20, 20]), latent, rope)
    assert binding.sv_get_device_error() == 0x8
    assert torch.equal(rope[:17].double(), case.tokens(2)[1]) and (rope[17:20] == 0).all() and (latent[17:20] == 0).all()
    # Broken ranges are skipped, pages that are not there read as zeros.
    latent.fill_(7.0)
    binding.sv_latent_gather(cache, case.table.to(DEV), ints(case.lens), ints([0, 4, 2, 3, 10 ** 6]), latent, rope)
    assert binding.sv_get_device_error() & 0x20
    assert (latent[3:] == 7).all()
    table = case.table.to(DEV)
    table[0, 1] = -1
    binding.sv_latent_gather(cache, table, ints(case.lens), ints([0, 40, 40, 40, 40]), latent, rope)
    assert binding.sv_get_device_error() == 0x1
    assert (latent[16:32] == 0).all() and (rope[16:32] == 0).all()
    assert torch.equal(rope[:16].double(), case.tokens(0)[1][:16]) and torch.equal(rope[32:40].double(), case.tokens(0)[1][32:40])


@pytest.mark.parametrize("fp8", [False, True])
def test_gather_many_rows(fp8):
    """More rows than a warp takes one by one: odd range ends, a request without rows, a page that is not there."""
    from query_aware_sparse_quest_gb300 import binding
    case = LatentCase([20011, 50, 15000, 9, 3], fp8=fp8, seed=8)
    cache, table = case.cache(), case.table.to(DEV)
    firsts, sizes = [37, 0, 1, 0, 0], [19973, 0, 14999, 9, 3]
    table[2, 500] = -1
    total = sum(sizes)
    latent = torch.full((total + 5, LATENT), 7.0, dtype=torch.bfloat16, device=DEV)
    rope = torch.full((total + 5, ROPE), 7.0, dtype=torch.bfloat16, device=DEV)
    binding.sv_latent_gather(cache, table, ints(case.lens), ints(starts_of(sizes)), latent, rope, first_token=ints(firsts))
    assert binding.sv_get_device_error() == 0x1
    for b, (f, n) in enumerate(zip(firsts, sizes)):
        c, r = (x.clone() for x in case.tokens(b))
        if b == 2:
            c[500 * PAGE:501 * PAGE] = r[500 * PAGE:501 * PAGE] = 0.0
        at = sum(sizes[:b])
        assert ((latent[at:at + n].double() - c[f:f + n]).abs() <= c[f:f + n].abs() * (2.0 ** -8 + 2.0 ** -23) * (1 if fp8 else 0)).all()
        assert torch.equal(rope[at:at + n].double(), r[f:f + n])
    assert (latent[total:] == 7).all() and (rope[total:] == 7).all()


def test_append_leaves_out_slots_outside_the_pool_and_codes_rows_that_are_not_finite():
    from query_aware_sparse_quest_gb300 import binding
    cache = binding.LatentCache.empty(2, fp8=True)
    rows = torch.randn((4, LATENT + ROPE), device=DEV).bfloat16()
    rows[2, 100], rows[3, 7] = float("inf"), float("nan")
    binding.sv_latent_append(cache, rows[:, :LATENT], rows[:, LATENT:], ints([32, 5, 0, 31]))
    assert binding.sv_get_device_error() == 0x4
    binding.sv_latent_append(cache, rows[:1, :LATENT], rows[:1, LATENT:], ints([-1]))
    assert binding.sv_get_device_error() == 0x4
    latent = torch.empty((32, LATENT), dtype=torch.bfloat16, device=DEV)
    rope = torch.empty((32, ROPE), dtype=torch.bfloat16, device=DEV)
    binding.sv_latent_gather(cache, ints([[0, 1]]), ints([32]), ints([0, 32]), latent, rope)
    assert torch.isnan(latent[[0, 31]].float()).all()
    rest = torch.ones(32, dtype=torch.bool)
    rest[[0, 5, 31]] = False
    assert (latent[rest] == 0).all() and (latent[5] != 0).any()
    assert torch.equal(rope[[5, 0, 31]], rows[1:, LATENT:])


@pytest.mark.parametrize("fp8", [False, True])
def test_a_request_from_prompt_to_fork(fp8):
    """Reserve, append, a chunk, forks, single tokens, compaction: the calls together, as a server makes them."""
    from query_aware_sparse_quest_gb300 import binding
    heads, pool, rows, prompt = 16, 40, 4, 133
    g = torch.Generator().manual_seed(1)
    layers = [binding.LatentCache.empty(pool, fp8=fp8) for _ in range(2)]
    for c in layers:
        c.rope.fill_(float("nan"))
        (c.scale if fp8 else c.latent).fill_(float("nan"))
    every = binding.CacheList(layers)
    table = torch.full((rows, 20), -1, dtype=torch.int32, device=DEV)
    lens, counts = torch.zeros(rows, dtype=torch.int32, device=DEV), torch.zeros(pool, dtype=torch.int32, device=DEV)
    ws = torch.empty(binding.sv_pages_workspace_size(pool, rows, rows), dtype=torch.uint8, device=DEV)
    aws = torch.empty(binding.sv_latent_attention_workspace_size(rows, heads, prompt), dtype=torch.uint8, device=DEV)
    history = [[[] for _ in range(rows)] for _ in layers]

    def new(n):
        return torch.randn((n, LATENT + ROPE), generator=g).bfloat16().to(DEV)

    def append(slots, owners):
        for i, c in enumerate(layers):
            x = new(len(owners))
            binding.sv_latent_append(c, x[:, :LATENT], x[:, LATENT:], slots)
            for t, r in enumerate(owners):
                history[i][r].append(x[t])

    def tokens(i, r):
        x = torch.stack(history[i][r])
        c = x[:, :LATENT].double()
        if fp8:
            q, s = code(x[:, :LATENT])
            c = q.view(torch.float8_e4m3fn).double() * s.double()[:, None]
        return c, x[:, LATENT:].double()

    def step(sizes):
        q = queries(sum(sizes), heads, seed=sum(sizes))
        for i, c in enumerate(layers):
            out = torch.empty((sum(sizes), heads, LATENT), dtype=torch.bfloat16, device=DEV)
            lse = torch.empty((sum(sizes), heads), device=DEV)
            binding.sv_latent_attention(c, q, table, lens, out, lse, aws, softmax_scale=SCALE, q_start=ints(starts_of(sizes)))
            for r, n in enumerate(sizes):
                if n:
                    k, x = tokens(i, r)
                    at = sum(sizes[:r])
                    check(out[at:at + n], lse[at:at + n],
                          attend(q[at:at + n], torch.cat((k, x), 1), k, causal_seen(k.shape[0], n, DEV), SCALE))

    slots = torch.empty(prompt, dtype=torch.int32, device=DEV)
    binding.sv_pages_reserve(table, lens, counts, ints([0]), ints([prompt]), slots, ws)
    append(slots, [0] * prompt)
    step([prompt, 0, 0, 0])
    binding.sv_pages_fork(every, table, lens, counts, ints([0, 0]), ints([1, 2]), ws)
    for h in history:
        h[1], h[2] = list(h[0]), list(h[0])
    slots = torch.empty(3, dtype=torch.int32, device=DEV)
    for _ in range(20):
        binding.sv_pages_reserve(table, lens, counts, ints([0, 1, 2]), ints([1, 1, 1]), slots, ws)
        append(slots, [0, 1, 2])
    step([1, 1, 1, 0])
    binding.sv_pages_free(table, lens, counts, ints([0]))
    for h in history:
        h[0] = []
    live = torch.empty(1, dtype=torch.int32, device=DEV)
    binding.sv_pages_compact(every, table, lens, counts, table, counts, live, ws)
    step([0, 1, 1, 0])
    # The cache read back is what the expansion starts from.
    for i, c in enumerate(layers):
        n = [0, len(history[i][1]), len(history[i][2]), 0]
        latent = torch.empty((sum(n), LATENT), dtype=torch.bfloat16, device=DEV)
        rope = torch.empty((sum(n), ROPE), dtype=torch.bfloat16, device=DEV)
        binding.sv_latent_gather(c, table, lens, ints(starts_of(n)), latent, rope)
        assert torch.equal(rope[: n[1]].double(), tokens(i, 1)[1])


def test_absorbed_and_expanded_forms_agree():
    """A small model's layer both ways: the query times the key expansion over the latents, and heads of their own."""
    from query_aware_sparse_quest_gb300 import binding
    heads, n, size = 8, 150, 40
    case = LatentCase([n], seed=3)
    g = torch.Generator().manual_seed(8)
    up = (torch.randn((heads, 256, LATENT), generator=g) / LATENT ** 0.5).bfloat16().to(DEV)   # key and value expansion
    q = torch.randn((size, heads, 192), generator=g).bfloat16().to(DEV)
    cache = case.cache()
    latent = torch.empty((n, LATENT), dtype=torch.bfloat16, device=DEV)
    rope = torch.empty((n, ROPE), dtype=torch.bfloat16, device=DEV)
    binding.sv_latent_gather(cache, case.table.to(DEV), ints([n]), ints([0, n]), latent, rope)
    kv = torch.einsum("tc,hdc->thd", latent.float(), up.float()).bfloat16()
    out, lse = torch.empty((size, heads, 128), dtype=torch.bfloat16, device=DEV), torch.empty((size, heads), device=DEV)
    ws = torch.empty(binding.sv_expanded_attention_workspace_size(1, heads, size), dtype=torch.uint8, device=DEV)
    binding.sv_expanded_attention(q, kv[..., :128], rope, kv[..., 128:], ints([0, size]), ints([0, n]), out, lse, ws)
    absorbed = torch.cat((torch.einsum("thd,hdc->thc", q[..., :128].float(), up[:, :128].float()), q[..., 128:].float()), -1).bfloat16()
    mid, lse2 = call(case, absorbed.contiguous(), [size], cache=cache)
    other = torch.einsum("thc,hdc->thd", mid.float(), up[:, 128:].float())
    # Each form rounds its own intermediates to bf16 (keys, values and the absorbed query: 2^-8 each): logits of about
    # 1.4 move by 2^-8 sqrt(2) / sqrt(192) of the sum of 192 magnitudes at the most, outputs by a few 2^-8 of values of 1.
    assert (lse - lse2).abs().max() < 0.05
    assert (out.float() - other).abs().max() < 0.1


@pytest.mark.parametrize("fp8", [False, True])
def test_sums_of_more_than_65536_tokens(fp8):
    """Many requests over the same pages, so that a CTA's run is longer than the sums stay in TMEM."""
    n, batch = 70016, 160
    case = LatentCase([n], fp8=fp8, seed=12, mean=2.0)
    one = case.lens
    q = queries(batch, 16, seed=12)
    case.lens, case.table = one * batch, case.table.expand(batch, -1).contiguous()
    out, lse = call(case, q)
    case.lens, case.table = one, case.table[:1]
    c, r = case.tokens(0)
    for b in (0, 1, 77, 159):
        check(out[b:b + 1], lse[b:b + 1], attend(q[b:b + 1], torch.cat((c, r), 1), c,
                                                 torch.ones((1, n), dtype=torch.bool, device=DEV), SCALE))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("how", ["page", "logit"])
@pytest.mark.parametrize("heads,lens,sizes", [
    (16, [5000], None),                  # runs of a few tiles each
    (128, [5000, 70, 400], None),
    (16, [200, 330] * 100, None),        # whole requests and cut ones
    (5, [130, 3000, 260], [3, 40, 1]),
    (128, [500, 1000], [40, 1]),
])
def test_rows_that_see_nothing_in_their_first_tiles(heads, lens, sizes, how, fp8):
    """The first tokens are not there (64 make a key tile: the table does not give their pages, or their logits are
    -inf), and what follows has logits of any size, below 0 too; over codes the next tokens are zeros (scale 0)."""
    from query_aware_sparse_quest_gb300 import binding
    steps = [1] * len(lens) if sizes is None else sizes
    case = LatentCase(lens, fp8=fp8, seed=21)
    if fp8:
        for b in range(0, len(lens), 2):
            for t in range(min(130, lens[b] - 70)):
                page = case.table[b, t // PAGE]
                case.latent[page, t % PAGE], case.scale[page, t % PAGE] = 0, 0.0
    case.rope[..., 0] = 64.0
    for hidden in (64, 128):
        keep = case.rope.clone()
        table = case.table.clone()
        if how == "page":
            table[:, : hidden // PAGE] = -1
        else:
            for b, n in enumerate(lens):
                for t in range(min(hidden, n)):
                    case.rope[case.table[b, t // PAGE], t % PAGE, 1] = -float("inf")
        cache = case.cache()
        for size, shift in ((1.0, 0.0), (0.03, 0.0), (0.3, -0.8), (0.3, -40.0)):
            q = queries(sum(steps), heads, seed=hidden, size=size)
            q[..., LATENT], q[..., LATENT + 1] = shift, 0.5
            good, case.table = case.table, table
            out, lse = call(case, q, sizes, cache=cache)
            case.table = good
            assert binding.sv_get_device_error() == (0x1 if how == "page" else 0)
            for b in list(range(len(lens)))[:6]:
                n, at = lens[b], sum(steps[:b])
                c, r = case.tokens(b)
                seen = causal_seen(n, steps[b], DEV)
                seen[:, :hidden] = False
                r = torch.nan_to_num(r, neginf=0.0)
                check(out[at:at + steps[b]], lse[at:at + steps[b]],
                      attend(q[at:at + steps[b]], torch.cat((c, r), 1), c, seen, SCALE))
        case.rope = keep


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,batch", [(16, 160), (128, 80)])
def test_sums_that_leave_the_tensor_memory_more_than_once(heads, batch, fp8):
    """Runs of 3200 tiles, with a token at tile 1500 and one at 2600 whose logits move the bases: what was summed before
    is a quarter of the average."""
    n = 204805
    count = -(-n // PAGE)
    case = LatentCase([642 * PAGE], fp8=fp8, seed=12, mean=2.0)
    at = torch.arange(count) * 640 // count
    for i, (tile, size) in enumerate(((1500, 100.0), (2600, 186.0))):
        at[4 * tile] = 640 + i
        case.rope[case.table[0, 640 + i], 3, 0] = size
    case.table = case.table[:1, at].contiguous()
    q = queries(batch, heads, seed=13, size=0.1)
    q[..., LATENT] = 1.0
    case.lens, case.table = [n] * batch, case.table.expand(batch, -1).contiguous()
    out, lse = call(case, q)
    case.lens, case.table = [n], case.table[:1]
    c, r = case.tokens(0)
    seen = torch.ones((1, n), dtype=torch.bool, device=DEV)
    pick = sorted({0, heads // 2 - 1, heads // 2, heads - 1})
    for b in (0, 1, batch // 2, batch - 1):
        check(out[b:b + 1, pick], lse[b:b + 1, pick], attend(q[b:b + 1, pick], torch.cat((c, r), 1), c, seen, SCALE))


def pools(pages, kinds, seed):
    """Caches of the given formats whose pages hold anything, and all their tensors."""
    from query_aware_sparse_quest_gb300 import binding
    g = torch.Generator().manual_seed(seed)

    def new(dtype, *shape):
        size = {torch.uint8: 1, torch.bfloat16: 2, torch.float32: 4}[dtype]
        return torch.randint(0, 256, (pages, *shape[:-1], shape[-1] * size), generator=g, dtype=torch.uint8).to(DEV).view(dtype)
    caches, tensors = [], []
    for kind in kinds:
        code = torch.uint8 if kind.endswith("e4m3") else torch.bfloat16
        if kind.startswith("latent"):
            t = [new(code, PAGE, LATENT), new(torch.bfloat16, PAGE, ROPE)] + ([new(torch.float32, PAGE)] if code == torch.uint8 else [])
            caches.append(binding.LatentCache(*t))
        else:
            t = [new(code, 2, PAGE, 128), new(code, 2, PAGE, 128), new(torch.bfloat16, 2, 2, 128)]
            t += [new(torch.float32, 2, PAGE) for _ in range(2)] if code == torch.uint8 else []
            caches.append(binding.Cache(*t))
        tensors += t
    return caches, tensors


@pytest.mark.parametrize("kinds", [["latent"], ["latent e4m3"], ["latent", "heads", "latent e4m3", "heads e4m3"]])
def test_pages_of_any_formats_are_copied(kinds):
    """One latent cache as it is, and caches of all formats in one list: every byte of a copied page, and no other."""
    from query_aware_sparse_quest_gb300 import binding
    pages = 9
    caches, tensors = pools(pages, kinds, seed=len(kinds))
    src, dst = [0, 8, 5], [3, 1, 7]
    want = []
    for t in tensors:
        w = t.view(torch.uint8).clone()
        w[dst] = w[src]
        want.append(w)
    binding.sv_pages_copy(caches[0] if len(caches) == 1 else caches, ints(src), ints(dst))
    for t, w in zip(tensors, want):
        assert torch.equal(t.view(torch.uint8), w)
    # A fork copies the partly filled page of its row.
    table = ints([[2, 4, -1], [-1, -1, -1]])
    lens, counts = ints([20, 0]), ints([0, 0, 1, 0, 1, 0, 0, 0, 0])
    ws = torch.empty(binding.sv_pages_workspace_size(pages, 2, 1), dtype=torch.uint8, device=DEV)
    binding.sv_pages_fork(caches[0] if len(caches) == 1 else caches, table, lens, counts, ints([0]), ints([1]), ws)
    new = int(table[1, 1])
    assert table[1, 0] == 2 and new not in (2, 4) and lens.tolist() == [20, 20] and counts[2] == 2
    for t, w in zip(tensors, want):
        w[new] = w[4]
        assert torch.equal(t.view(torch.uint8), w)
