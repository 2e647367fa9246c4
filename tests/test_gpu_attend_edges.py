"""sv_window_attention and sv_prefix_decode where a row sees nothing, over queries and weights of any size, and
over values that are not finite."""
from __future__ import annotations

import pytest
import torch

import test_gpu_prefix as prefix
from attend_ref import DIM, PAGE, PagedCase, attend, check, window_seen
from query_aware_sparse_quest_gb300 import binding
from test_gpu_window import compare, run

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def gauss(*shape, seed=3):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("lens,group,window,sink", [
    ([2, 3, 5, 17], 8, 0, 0), ([300, 77], 7, 0, 0), ([5000, 1, 40], 4, 333, 5), ([3000], 1, 0, 0), ([20000] * 3, 2, 0, 0),
])
def test_single_tokens_over_bf16_keep_their_weights(lens, group, window, sink):
    """Weights enter the product as two bf16 parts: the second is less than 2^-7 of a weight and off by 2^-8 of itself."""
    case = PagedCase(lens, 2)
    q = (3 * gauss(len(lens), 2 * group, DIM)).bfloat16().to(DEV)
    seen = [window_seen(n, 1, window, sink, DEV) for n in lens]
    tokens = [case.tokens(b) for b in range(len(lens))]
    o, ls, tol, tol_lse = (torch.cat(x) for x in zip(*[attend(q[b:b + 1], *tokens[b], seen[b], DIM ** -0.5) for b in range(len(lens))]))
    size = torch.cat([attend(q[b:b + 1], k, torch.nan_to_num(v).abs(), seen[b], DIM ** -0.5)[0] for b, (k, v) in enumerate(tokens)])
    # attend()'s bound with 2^-15 in place of P's 2^-8, in the output's own rounding too
    tol = tol - (2.0 ** -8 - 2.0 ** -15) * (1 + 2.0 ** -8) * size
    check(*run(case, q, window, sink), (o, ls, tol, tol_lse))


def test_small_weights_over_e4m3_count_in_the_output():
    """One token of value 0 outweighs the others of its page by 2^26; the output is theirs alone.

    A weight is held in f16 relative to 2^-7 of the largest of its page, in steps of 2^-24 at least: off by at
    most 2^-32 of the largest, and in 15 tokens of value 1 by 15 of those."""
    case = PagedCase([PAGE], 1, fp8=True)
    page = case.table[0, 0]
    case.k[page], case.v[page] = 0, 0x7E                     # 448
    case.v[page, 0, 0] = 0
    case.ks[page], case.vs[page] = 1.0, 1 / 448
    q = torch.zeros((1, 4, DIM), dtype=torch.bfloat16, device=DEV)
    q[:, :, 0] = 1
    lift = torch.tensor([26 * 0.6931471805599453 / 448])
    case.k[page, 0, 1:, 0] = 0xFE                            # -448
    case.ks[page, 0, 1:] = lift
    ref = attend(q, *case.tokens(0), window_seen(PAGE, 1, 0, 0, DEV), 1.0)
    assert (ref[0] - 15 * 2.0 ** -26).abs().max() < 1e-10
    ref[2].add_(15 * 2.0 ** -32)
    check(*run(case, q, 0, 0, scale=1.0), ref)


# Queries of every size a bf16 has, with a scale that makes ordinary logits of them.
SIZES = {"1e-6": (1e-6, 1e5), "1e-30": (1e-30, 1e28), "3e4": (3e4, 3e-6), "1e30": (1e30, 1e-31),
         "mixed": (None, 1.0)}


def sized(q, name):
    size, scale = SIZES[name]
    if size is None:                     # channels over 20 powers of two, the largest near 1
        return (q * torch.exp2(-(torch.arange(DIM) * 7 % 20).float())).bfloat16(), scale
    return (q * size).bfloat16(), scale


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", list(SIZES))
def test_queries_of_any_size(name, fp8):
    """A token alone, the same one as a chunk, and behind a prefix, read alone or in tiles."""
    lens, group = [700, 33, 260], 4
    case = PagedCase(lens, 2, fp8=fp8)
    q, scale = sized(gauss(3, 2 * group, DIM), name)
    q = q.to(DEV)
    ref = [torch.cat(x) for x in zip(*[attend(q[b:b + 1], *case.tokens(b), window_seen(n, 1, 0, 0, DEV), scale)
                                       for b, n in enumerate(lens)])]
    for starts in (None, [0, 1, 2, 3]):
        out, lse = run(case, q, 0, 0, starts, scale)
        check(out, lse, ref)
    cache, lens = case.cache(), ints(lens)
    ws = torch.empty(binding.sv_prefix_decode_workspace_size(3, 2 * group, 2, 3), dtype=torch.uint8, device=DEV)
    for wide in (0, 5000):
        table = torch.nn.functional.pad(case.table, (0, wide), value=-1).to(DEV)
        binding.sv_prefix_decode(cache, q, table, lens, ints([0, 1, 2, 3]), ints([20, 1, 0]), out, lse, ws, softmax_scale=scale)
        check(out, lse, ref)
    assert binding.sv_get_device_error() == 0


def test_queries_of_infinity_and_nan_over_e4m3():
    """They give NaN to their own heads alone."""
    case = PagedCase([100], 2, fp8=True)
    q = gauss(1, 8, DIM).bfloat16().to(DEV)
    ref = attend(q, *case.tokens(0), window_seen(100, 1, 0, 0, DEV), DIM ** -0.5)
    q[0, 2, 9], q[0, 5, 0] = float("inf"), float("nan")
    out, lse = run(case, q, 0, 0)
    good = [0, 1, 3, 4, 6, 7]
    check(out[:, good], lse[:, good], [x[:, good] for x in ref])
    assert out[:, [2, 5]].isnan().all() and not lse[:, [2, 5]].isfinite().any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("requests", [1, 100])         # items that are cut; whole ones
def test_rows_that_see_nothing_beside_a_nan(requests, fp8):
    """A missing page empties some rows of a tile; others of the tile see a NaN.  The empty ones are 0, -inf."""
    n, size, group, window = 200, 64, 4, 8
    case = PagedCase([n] * requests, 2, fp8=fp8)
    q = gauss(requests * size, 2 * group, DIM).bfloat16().to(DEV)
    seen = window_seen(n, size, window, 0, DEV)
    seen[:, 144:160] = False
    ref = [attend(q[b * size:(b + 1) * size], *case.tokens(b), seen, DIM ** -0.5) for b in range(requests)]
    nan = 163
    for b in range(requests):
        case.v[case.table[b, nan // PAGE], :, nan % PAGE, 5] = 0x7F if fp8 else float("nan")
        case.table[b, 144 // PAGE] = -1
    out, lse = run(case, q, window, 0, [b * size for b in range(requests + 1)])
    assert binding.sv_get_device_error() == 0x1
    empty = (~seen.any(1)).repeat(requests)
    assert empty.sum() == 9 * requests
    assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    hit = torch.zeros((n - (n - size), DIM), dtype=torch.bool, device=DEV)
    hit[:, 5] = seen[:, nan]
    hit = hit.repeat(requests, 1)[:, None].expand(-1, 2 * group, -1)
    assert torch.equal(out.isnan(), hit)
    o, ls, tol, tol_lse = (torch.cat(x) for x in zip(*ref))
    check(torch.where(hit, 0, out), lse, (torch.where(hit, 0, o), ls, tol, tol_lse))


def test_a_cta_waits_as_long_as_an_item_takes():
    """Items of 1.35 million key tiles (173 million tokens, 2.3 s), with short requests behind the first, so that its
    CTA's scheduler waits for all of it.  The first page outweighs the others by 2^184, so it is the answer."""
    pages, group, tile = 1_350_000 * 8, 8, 32            # 32 tokens x 8 heads are a row tile
    case = PagedCase([PAGE, PAGE], 1)
    first, rest = (int(case.table[b, 0]) for b in range(2))
    case.k[first, ..., 0], case.k[rest, ..., 0] = 8, -8
    short = 5
    table = torch.full((short + 2, pages), rest, dtype=torch.int32, device=DEV)
    table[:, 0] = first
    sizes = [tile] + [1] * short + [151 * tile]           # 152 CTAs: the last request's items fill the other 151
    lens = [(pages - 64 * 8) * PAGE] + [PAGE] * short + [pages * PAGE]
    q = gauss(sum(sizes), group, DIM).bfloat16().to(DEV)
    q[..., 0] = 8
    ref = attend(q, *case.tokens(0), torch.ones((sum(sizes), PAGE), dtype=torch.bool, device=DEV), 1.0)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    ws = torch.empty(binding.sv_window_attention_workspace_size(len(sizes), group, 1, sum(sizes)), dtype=torch.uint8, device=DEV)
    binding.sv_window_attention(case.cache(), q, table, ints(lens), 0, 0, out, lse, ws, softmax_scale=1.0,
                                q_start=ints([sum(sizes[:b]) for b in range(len(sizes) + 1)]))
    torch.cuda.synchronize()
    assert binding.sv_get_device_error() == 0
    check(out, lse, ref)


@pytest.mark.parametrize("lens,sizes,group", [
    ([500 + 7 * i % 100 for i in range(700)], [32] * 700, 8),        # whole items and cut ones, 256 rows each
    ([900 + 7 * i % 100 for i in range(700)], [16] * 700, 8),        # 128 rows: both streams take tiles in turn
    ([260] * 1500, [1 + i % 40 for i in range(1500)], 7),
])
def test_e4m3_tiles_repeat_exactly_while_rows_are_written(lens, sizes, group):
    """Several items a CTA: rows of one are written while the next one's codes are widened."""
    case = PagedCase(lens, 2, fp8=True)
    q = gauss(sum(sizes), 2 * group, DIM).bfloat16().to(DEV)
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + n)
    cache, table, ls, qs = case.cache(), case.table.to(DEV), ints(lens), ints(starts)
    ws = torch.empty(binding.sv_window_attention_workspace_size(len(lens), 2 * group, 2, len(q)), dtype=torch.uint8, device=DEV)

    def call():
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        binding.sv_window_attention(cache, q, table, ls, 0, 0, out, lse, ws, q_start=qs)
        return out, lse
    first = call()
    for b in range(0, len(lens), 97):
        rows = slice(starts[b], starts[b + 1])
        check(first[0][rows], first[1][rows], attend(q[rows], *case.tokens(b), window_seen(lens[b], sizes[b], 0, 0, DEV), DIM ** -0.5))
    for _ in range(60):
        out, lse = call()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert binding.sv_get_device_error() == 0
def repeated(levels, step, seed=8):
    """64 pages a level, whose logits rise by `step` nats a level (channel 0, where q is 1, at a scale of 0.1)."""
    n = 64 * levels
    k = gauss(n, 1, PAGE, DIM, seed=seed)
    k[..., 0] = 10 * step * torch.arange(n).div(64, rounding_mode="floor")[:, None, None]
    v = gauss(n, 1, PAGE, DIM, seed=seed + 1) + 2
    return k, v


def held(k, v, fp8):
    """The cache of K and V (fp32), and what it holds, in 64 bits."""
    meta = torch.zeros((k.shape[0], 1, 2, DIM), dtype=torch.bfloat16, device=DEV)
    if not fp8:
        k, v = k.bfloat16().to(DEV), v.bfloat16().to(DEV)
        return binding.Cache(k, v, meta), k.double().view(-1, DIM), v.double().view(-1, DIM)
    (kc, ks), (vc, vs) = PagedCase._code(k), PagedCase._code(v)
    kc, ks, vc, vs = (x.to(DEV).contiguous() for x in (kc, ks, vc, vs))
    wide = [(x.view(torch.float8_e4m3fn).double() * s.double()[..., None]).view(-1, DIM) for x, s in ((kc, ks), (vc, vs))]
    return binding.Cache(kc, vc, meta, ks, vs), *wide


def weighted(q, k, v, w, scale):
    """attend() of tokens that a row sees w [n, L] times.  The sums: 512 tiles of 128 tokens at a time, cut off at
    fp32's last bit by the MMAs 8 times a tile (2^-23 of the sum each), then those sums, rounded; l: rounded."""
    z = torch.einsum("nhd,ld->nhl", q.double(), k) * scale
    mag = (torch.einsum("nhd,ld->nhl", q.double().abs(), k.abs()) * scale).amax(-1)
    z = z + w.double().log()[:, None]
    ls = torch.logsumexp(z, -1)
    p = torch.exp(z - ls[..., None])
    o, a = p @ v, p @ v.abs()
    ez = 130 * 2.0 ** -24 * mag
    folds = w.sum(1).max().item() / 65536
    tol = (2.0 ** -8 + 2 * ez[..., None] + 2.0 ** -11 + folds * 2.0 ** -24 + 2.0 ** -20) * a + 2.0 ** -8 * (o.abs() + 2.0 ** -8 * a)
    return o, ls, tol, ez + 2.0 ** -21 + 2.0 ** -20 + (512 + folds) * 2.0 ** -24 + 2.0 ** -23 * ls.abs()


LONG = 1 << 20


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("form", ["halves", "joined", "cut", "prefix"])
def test_long_sums_of_one_sign_lose_nothing(form, fp8):
    """A million values 1 a row: the average is 1.  Row tiles of 256 rows and of 128, whole and cut; prefixes."""
    pages, group = LONG // PAGE, 8
    k = gauss(64, 1, PAGE, DIM)
    cache, k64, _ = held(k, torch.ones_like(k), fp8)
    batch, size = {"halves": (1, 152 * 32), "joined": (152, 16), "cut": (1, 100 * 32), "prefix": (320, 1)}[form]
    table = (torch.arange(pages + 1, dtype=torch.int32, device=DEV) % 64).repeat(batch, 1)
    q = gauss(batch * size, group, DIM, seed=4).bfloat16().to(DEV)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    length = LONG + (5 if form == "prefix" else 0)
    lens = ints([length] * batch)
    if form == "prefix":
        ws = torch.empty(binding.sv_prefix_decode_workspace_size(batch, group, 1, 10), dtype=torch.uint8, device=DEV)
        binding.sv_prefix_decode(cache, q, table, lens, ints([32 * g for g in range(11)]), ints([pages] * 10), out, lse, ws)
    else:
        ws = torch.empty(binding.sv_window_attention_workspace_size(batch, group, 1, batch * size), dtype=torch.uint8, device=DEV)
        binding.sv_window_attention(cache, q, table, lens, 0, 0, out, lse, ws, q_start=ints([b * size for b in range(batch + 1)]))
    assert binding.sv_get_device_error() == 0
    assert (out == 1).all(), (out.double() - 1).abs().max().item()
    rows = torch.tensor([0, size // 2, batch * size - 1], device=DEV)
    pos = length - size + rows % size
    w = (pos[:, None] + 1) // 1024 + (torch.arange(1024, device=DEV) < (pos[:, None] + 1) % 1024)
    _, ls, _, tol = weighted(q[rows], k64, torch.ones_like(k64), w, DIM ** -0.5)
    assert ((lse[rows] - ls).abs() <= tol).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("form", ["halves", "joined"])
@pytest.mark.parametrize("step", [3.0, -0.5])
def test_long_contexts_whose_logits_rise_and_fall(step, form, fp8):
    """16 levels of 65536 tokens each: the base moves between the sums that a row is folded into."""
    levels, group = 16, 8
    k, v = repeated(levels, step)
    cache, k64, v64 = held(k, v, fp8)
    pages = LONG // PAGE
    at = torch.arange(pages, device=DEV)
    batch, size = (1, 152 * 32) if form == "halves" else (152, 16)
    table = (at // 4096 * 64 + at % 64).int().repeat(batch, 1)
    q = gauss(batch * size, group, DIM, seed=5).bfloat16().to(DEV)
    q[..., 0] = 1
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    ws = torch.empty(binding.sv_window_attention_workspace_size(batch, group, 1, batch * size), dtype=torch.uint8, device=DEV)
    binding.sv_window_attention(cache, q, table, ints([LONG] * batch), 0, 0, out, lse, ws, softmax_scale=0.1,
                                q_start=ints([b * size for b in range(batch + 1)]))
    assert binding.sv_get_device_error() == 0
    rows = torch.arange(0, batch * size, 37, device=DEV)
    seen = LONG - size + rows % size + 1
    level = torch.arange(levels, device=DEV).repeat_interleave(1024)
    token = torch.arange(1024, device=DEV).repeat(levels)
    inside = (seen[:, None] - 65536 * level).clamp(0, 65536)
    check(out[rows], lse[rows], weighted(q[rows], k64, v64, inside // 1024 + (token < inside % 1024), 0.1))


def test_a_nan_behind_a_long_context():
    """Only the last token's rows see it; the others of its tile, which have folded sums, do not."""
    length, size, group = 1 << 17, 152 * 32, 8
    k = gauss(65, 1, PAGE, DIM)
    v = torch.ones_like(k)
    v[64, 0, 15, 5] = float("nan")
    cache, _, _ = held(k, v, False)
    table = (torch.arange(length // PAGE, dtype=torch.int32, device=DEV) % 64)[None].contiguous()
    table[0, -1] = 64
    q = gauss(size, group, DIM, seed=4).bfloat16().to(DEV)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    ws = torch.empty(binding.sv_window_attention_workspace_size(1, group, 1, size), dtype=torch.uint8, device=DEV)
    binding.sv_window_attention(cache, q, table, ints([length]), 0, 0, out, lse, ws, q_start=ints([0, size]))
    assert binding.sv_get_device_error() == 0
    assert out[-1, :, 5].isnan().all() and lse.isfinite().all()
    out[-1, :, 5] = 1
    assert (out == 1).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("length", [LONG, 4 * LONG])
def test_long_sums_of_one_sign_in_single_tokens(length, fp8):
    """Enough requests that one split reads all of a row: the average of 4 million values 1 is 1."""
    batch, group = 152 * 4, 8
    k = gauss(64, 1, PAGE, DIM)
    cache, k64, _ = held(k, torch.ones_like(k), fp8)
    table = (torch.arange(length // PAGE, dtype=torch.int32, device=DEV) % 64).repeat(batch, 1)
    q = gauss(batch, group, DIM, seed=4).bfloat16().to(DEV)
    out, lse = torch.empty_like(q), torch.empty((batch, group), device=DEV)
    ws = torch.empty(binding.sv_window_attention_workspace_size(batch, group, 1, batch), dtype=torch.uint8, device=DEV)
    binding.sv_window_attention(cache, q, table, ints([length] * batch), 0, 0, out, lse, ws)
    assert binding.sv_get_device_error() == 0
    assert (out == 1).all(), (out.double() - 1).abs().max().item()
    _, ls, _, _ = weighted(q, k64, torch.ones_like(k64), torch.full((batch, 1024), length // 1024, device=DEV), DIM ** -0.5)
    # a lane's sum of length / 64 pages' weights, each addition rounded
    assert ((lse - ls).abs() <= 1e-5 + length / 64 * 2.0 ** -24).all()


@pytest.mark.parametrize("wide", [0, 5000])
@pytest.mark.parametrize("length,flag", [(70, 0), (64, 0), (0, 0), (63, 0x40), (1, 0x40), (-1, 0x8), (-2 ** 31, 0x8), (None, 0x8)])
def test_prefix_decode_says_exactly_what_is_wrong(length, flag, wide):
    """A request of a group with 4 shared pages, of every length."""
    starts, shared = [0, 3, 5], [4, 0]
    case = PagedCase([70, 70, 90, 20, 33, 40], 2)
    prefix.share(case, starts, shared)
    prefix.run.wide = False
    q = prefix.queries(case, 8)
    ref = prefix.reference(case, q, range(5))
    table = torch.nn.functional.pad(case.table, (0, wide), value=-1).to(DEV)
    lens = list(case.lens)
    lens[1] = table.shape[1] * PAGE + 1 if length is None else length
    if length == 64:
        k, v = case.tokens(1, 64)
        ref = [torch.cat([x[:1], y, x[2:]]) for x, y in zip(ref, attend(q[1:2], k, v, window_seen(64, 1, 0, 0, DEV), DIM ** -0.5))]
    out, lse = torch.full_like(q, 7.0), torch.full((6, 16), 7.0, device=DEV)
    ws = torch.empty(binding.sv_prefix_decode_workspace_size(6, 16, 2, 2), dtype=torch.uint8, device=DEV)
    binding.sv_prefix_decode(case.cache(), q, table, ints(lens), ints(starts), ints(shared), out, lse, ws)
    assert binding.sv_get_device_error() == flag
    right = [0, 1, 2, 3, 4] if lens[1] in (70, 64) else [0, 2, 3, 4]
    check(out[right], lse[right], [x[right] for x in ref])
    if 1 not in right:
        assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()
    assert (out[5] == 7).all() and (lse[5] == 7).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("v_mean", [0.0, 3.0])        # outputs that are averages near 0, and that are not
def test_many_short_requests_in_tiles(v_mean, fp8):
    """More items than CTAs: whole items and cut ones in one call of the tiles."""
    lens = [1 + (37 * i) % 400 for i in range(90)]
    compare(PagedCase(lens, 4, spare=0, fp8=fp8, v_mean=v_mean), [1] * 90, 2, 90, 7)
    lens = [1 + (337 * i) % 4000 for i in range(40)]
    compare(PagedCase(lens, 4, spare=0, fp8=fp8, v_mean=v_mean), [min(n, 1 + 11 * i % 70) for i, n in enumerate(lens)], 8, 0, 0)


@pytest.mark.parametrize("fp8,poison", [(False, "nan"), (False, "inf"), (True, "nan"), (True, "scale")])
@pytest.mark.parametrize("form", ["window", "alone", "tiles"])
def test_values_that_are_not_finite_in_single_tokens(form, fp8, poison):
    """They reach the requests that see them: one token of a request's own, one of a shared prefix."""
    starts, shared = [0, 3, 6], [4, 6]
    case = PagedCase([100, 64, 90, 700, 96, 97], 2, fp8=fp8)
    window, sink = (0, 0) if form != "window" else (60, 3)
    if form != "window":
        prefix.share(case, starts, shared)
    q = prefix.queries(case, 4)
    seen = [window_seen(n, 1, window, sink, DEV) for n in case.lens]
    ref = [torch.cat(x) for x in zip(*[attend(q[b:b + 1], *case.tokens(b), seen[b], DIM ** -0.5) for b in range(6)])]
    hit = torch.zeros((6, DIM), dtype=torch.bool, device=DEV)
    for b, t, channel in ((2, 85, 3), (3, 690, 127), (0, 20, 64)):
        page, at = case.table[b, t // PAGE], t % PAGE
        if poison == "scale":
            case.vs[page, :, at] = float("nan")
        else:
            case.v[page, :, at, channel] = 0x7F if fp8 else float(poison)
        for r in range(6):
            same = r == b or (form != "window" and t < PAGE * shared[0 if r < 3 else 1] and case.table[r, t // PAGE] == page)
            if same and t < case.lens[r] and seen[r][0, t]:
                hit[r, slice(None) if poison == "scale" else channel] = True
    assert hit.any(1).sum() >= 2 and not hit.all(1).all()
    if form == "window":
        out, lse = run(case, q, window, sink)
    else:
        prefix.run.wide = form == "tiles"
        out, lse = prefix.run(case, q, starts, shared)
    assert binding.sv_get_device_error() == 0
    hit = hit[:, None].expand(-1, 8, -1)
    assert torch.equal(out.isposinf() if poison == "inf" else out.isnan(), hit)
    check(torch.where(hit, 0, out), lse, (torch.where(hit, 0, ref[0]), *ref[1:]))


@pytest.mark.parametrize("fp8", [False, True])
def test_prefixes_of_many_groups(fp8):
    """Groups in every round of 32 that the scheduler looks at: empty ones, ones that share nothing, ones out of order."""
    rng = torch.Generator().manual_seed(9)
    sizes = torch.randint(0, 7, (300,), generator=rng).tolist()
    shared = [0 if i % 11 == 5 else 1 + i % 13 for i in range(300)]
    sizes[64:96] = [0] * 32
    starts = [sum(sizes[:g]) for g in range(301)]
    of = [g for g in range(300) for _ in range(sizes[g])]
    lens = [shared[g] * PAGE + 1 + 5 * b % 40 for b, g in enumerate(of)]
    case = PagedCase(lens, 2, fp8=fp8)
    prefix.share(case, starts, shared)
    prefix.run.wide = True
    q = prefix.queries(case, 4)
    ref = prefix.reference(case, q, range(len(lens)))
    out, lse = prefix.run(case, q, starts, shared)
    assert binding.sv_get_device_error() == 0
    check(out, lse, ref)
    g = next(g for g in range(200, 290) if sizes[g] > 0 and sizes[g + 1] > 1)
    broken = list(starts)
    broken[g] = starts[g + 1] + 1          # group g ends before it begins, group g - 1 takes its requests and one more
    out, lse = prefix.run(case, q, broken, shared)
    assert binding.sv_get_device_error() & 0x40
    right = [b for b in range(len(lens)) if of[b] not in (g - 1, g, g + 1)]
    check(out[right], lse[right], [x[right] for x in ref])
