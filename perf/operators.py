"""What the paged-cache operators are measured on: sliding-window attention with
sinks over a paged KV cache (chunks and single tokens), decode of a batch that
shares a prefix, and the page owner's calls (fork, reserve, free, compact).

A case is a dict of plain values; `run` makes one pass through an operator, in
plain torch operations, or (where `own` is true) through the library's calls.
"""
import math

import torch

own = False

PAGE = 16
DIM = 128
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The smallest decode: one request of the tiny 4-query-head geometry; latency counts.
        dict(name="window decode b1", kind="window", batch=1, hkv=1, group=4, ctx=4096, ragged=0, chunk=1, window=1024,
             sink=4, fp8=False),
        # A decode step of the 128k batch-8 serving batch in a layer with a 4096-token window.
        dict(name="window decode b8 128k", kind="window", batch=8, hkv=4, group=8, ctx=128000, ragged=0, chunk=1,
             window=4096, sink=16, fp8=False),
        # The ragged serving batch (8k to 128k tokens) over an e4m3 pool, odd sinks.
        dict(name="window decode b32 fp8", kind="window", batch=32, hkv=4, group=8, ctx=131072, ragged=1, chunk=1,
             window=2048, sink=5, fp8=True),
        # One 4096-token chunk of a chunked prefill at 32k tokens, windowed layer.
        dict(name="window prefill 4096", kind="window", batch=1, hkv=4, group=8, ctx=32768, ragged=0, chunk=4096,
             window=4096, sink=16, fp8=False),
        # A mixed batch: chunks of odd lengths with single tokens among them, 7 query heads a kv head, e4m3 pool.
        dict(name="ragged chunks b7 fp8", kind="window", batch=7, hkv=4, group=7, ctx=4000, ragged=1, chunk=777,
             window=1000, sink=3, fp8=True),
        # The largest: the same chunk in a layer without a window (every earlier token visible).
        dict(name="causal prefill 4096 at 32k", kind="window", batch=1, hkv=4, group=8, ctx=32768, ragged=0, chunk=4096,
             window=0, sink=0, fp8=False),
        # Four samples of one short prompt, tiny geometry.
        dict(name="prefix decode b4", kind="prefix", batch=4, hkv=1, group=4, groups=1, shared=128, suffix=100,
             fp8=False),
        # 32 requests behind one 32k-token system prompt.
        dict(name="prefix decode b32 32k", kind="prefix", batch=32, hkv=4, group=8, groups=1, shared=2048, suffix=1024,
             fp8=False),
        # 61 requests over 5 prompts of 8k tokens and less, e4m3 pool.
        dict(name="prefix decode b61 fp8", kind="prefix", batch=61, hkv=4, group=8, groups=5, shared=512, suffix=700,
             fp8=True),
        # A beam step of 8 beams on one layer: latency counts.
        dict(name="fork 8 of 1, one layer", kind="fork", rows=16, parents=1, children=8, hkv=4, layers=1, ctx=4096,
             pool=8192),
        # A beam step of 64 children from 16 parents in 8 layers.
        dict(name="fork 64 of 16, 8 layers", kind="fork", rows=96, parents=16, children=64, hkv=4, layers=8, ctx=8000,
             pool=16384),
        # A pool at 60 per cent, in holes, packed in 4 layers.
        dict(name="compact 16384 pages", kind="compact", rows=48, hkv=4, layers=4, ctx=4096, pool=16384, live=60),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("window", "window", "prefix", "fork", "compact"))
    hkv = rng.choice((1, 2, 4, 8))
    group = rng.randint(1, 8)
    if kind == "window":
        c = dict(kind=kind, batch=_log(rng, 1, 32), hkv=hkv, group=group, ctx=_log(rng, 64, 32768),
                 ragged=rng.randint(0, 1), chunk=1 if rng.random() < 0.4 else _log(rng, 2, 2048),
                 window=0 if rng.random() < 0.25 else _log(rng, 1, 8192), sink=rng.choice((0, 1, 4, 16, rng.randint(0, 100))),
                 fp8=rng.random() < 0.4)
        c["chunk"] = min(c["chunk"], c["ctx"])
        while c["batch"] > 1 and c["batch"] * c["chunk"] * c["ctx"] * hkv * group > 1 << 31:
            c["batch"] //= 2
        while c["batch"] * c["chunk"] * c["ctx"] * hkv * group > 1 << 31:
            c["chunk"] = c["chunk"] * 2 // 3
        return c
    if kind == "prefix":
        batch = _log(rng, 1, 64)
        return dict(kind=kind, batch=batch, hkv=rng.choice((1, 2, 4)), group=group, groups=rng.randint(1, min(batch, 6)),
                    shared=_log(rng, 1, 1024), suffix=_log(rng, 1, 1000), fp8=rng.random() < 0.4)
    if kind == "fork":
        parents = rng.randint(1, 12)
        children = rng.randint(1, 48)
        return dict(kind=kind, rows=parents + children + rng.randint(0, 8), parents=parents, children=children,
                    hkv=hkv, layers=rng.randint(1, 6), ctx=_log(rng, 20, 4000), pool=_log(rng, 6000, 12000))
    return dict(kind=kind, rows=rng.randint(3, 40), hkv=rng.choice((1, 2, 4)), layers=rng.randint(1, 4),
                ctx=_log(rng, 20, 2000), pool=_log(rng, 6000, 12000), live=rng.randint(20, 90))


# ------------------------------------------------------------------ inputs
def _lens(c):
    """Lengths that the case fixes (the seed draws values, not sizes)."""
    if not c["ragged"]:
        return [c["ctx"]] * c["batch"]
    lo = max(1, c["ctx"] // 16)
    return [lo + (c["ctx"] - lo) * ((i * 7919 + 13) % 101) // 100 for i in range(c["batch"])]


def _chunks(c):
    lens = _lens(c)
    if c["chunk"] == 1 or not c["ragged"]:
        return [min(c["chunk"], n) for n in lens]
    return [1 if i % 3 == 2 else min(n, 1 + (c["chunk"] - 1) * ((i * 5 + 7) % 8) // 7) for i, n in enumerate(lens)]


def _group_sizes(c):
    left, sizes = c["batch"], []
    for g in range(c["groups"]):
        most = left - (c["groups"] - 1 - g)
        n = most if g == c["groups"] - 1 else max(1, min(most, c["batch"] // c["groups"] + (3 if g % 2 else -2)))
        sizes.append(n)
        left -= n
    return sizes


def _prefixes(c):
    """(shared pages of each group, suffix tokens of each request)"""
    shared = [max(1, c["shared"] - g * (c["shared"] // 7)) for g in range(c["groups"])]
    return shared, [1 + (c["suffix"] - 1) * ((b * 11 + 5) % 16) // 15 for b in range(c["batch"])]


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _values(gen, shape, scale=None):
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    return (x if scale is None else x * scale).bfloat16()


def _coded(x):
    """e4m3 codes and one scale a row, as the cache keeps them."""
    x = x.float()
    s = x.abs().amax(-1) / 448.0
    return (x / s[..., None].clamp_min(1e-30)).to(torch.float8_e4m3fn).view(torch.uint8), s


def _pool(c, gen, pages):
    """K/V pages with outlier key channels, and what a cache keeps of them."""
    shape = (pages, c["hkv"], PAGE, DIM)
    channel = torch.randn((1, c["hkv"], 1, DIM), generator=gen, device=DEV).mul(0.5).exp()
    k, v = _values(gen, shape, channel), _values(gen, shape)
    meta = torch.stack((k.amin(2), k.amax(2)), 2).contiguous()
    s = dict(k=k, v=v, meta=meta, ks=None, vs=None)
    if c["fp8"]:
        s["k"], s["ks"] = _coded(k)
        s["v"], s["vs"] = _coded(v)
    return s


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    if c["kind"] in ("fork", "compact"):
        return _prepare_pages(c, gen)
    hq = c["hkv"] * c["group"]
    if c["kind"] == "window":
        lens, chunks = _lens(c), _chunks(c)
        counts = [-(-n // PAGE) for n in lens]
        order = torch.randperm(sum(counts), generator=gen, device=DEV).int()
        table = torch.zeros((c["batch"], max(counts)), dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(counts):
            table[b, :n] = order[at:at + n]
            at += n
        s = _pool(c, gen, sum(counts))
        starts = [sum(chunks[:i]) for i in range(c["batch"] + 1)]
        rows = starts[-1]
        s.update(starts=None if c["chunk"] == 1 else _int(starts), most=max(chunks), longest=max(lens))
    else:
        sizes = _group_sizes(c)
        shared, suffix = _prefixes(c)
        of = [g for g, n in enumerate(sizes) for _ in range(n)]
        lens = [shared[of[b]] * PAGE + suffix[b] for b in range(c["batch"])]
        tails = [-(-n // PAGE) for n in suffix]
        total = sum(shared) + sum(tails)
        order = torch.randperm(total, generator=gen, device=DEV).int()
        table = torch.zeros((c["batch"], max(-(-n // PAGE) for n in lens)), dtype=torch.int32, device=DEV)
        heads = [sum(shared[:g]) for g in range(c["groups"])]
        at = sum(shared)
        for b in range(c["batch"]):
            g = of[b]
            table[b, :shared[g]] = order[heads[g]:heads[g] + shared[g]]
            table[b, shared[g]:shared[g] + tails[b]] = order[at:at + tails[b]]
            at += tails[b]
        s = _pool(c, gen, total)
        rows = c["batch"]
        s.update(group_start=_int([sum(sizes[:g]) for g in range(c["groups"] + 1)]), shared=_int(shared),
                 group_of=torch.tensor(of, device=DEV), longest_shared=max(shared), longest_tail=max(tails))
    s.update(case=c, table=table, lens=_int(lens), q=_values(gen, (rows, hq, DIM)), scale=DIM ** -0.5)
    if own:  # the cache handle and the workspace that a serving program keeps
        from query_aware_sparse_quest_gb300 import binding
        s["cache"] = binding.Cache(s["k"], s["v"], s["meta"], s["ks"], s["vs"])
        size = (binding.sv_window_attention_workspace_size(c["batch"], hq, c["hkv"], rows) if c["kind"] == "window" else
                binding.sv_prefix_decode_workspace_size(c["batch"], hq, c["hkv"], c["groups"]))
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s


def _prepare_pages(c, gen):
    pool, rows = c["pool"], c["rows"]
    shape = (c["layers"], pool, c["hkv"], PAGE, DIM)
    s = dict(case=c, k=_values(gen, shape), v=_values(gen, shape),
             meta=_values(gen, (c["layers"], pool, c["hkv"], 2, DIM)))
    order = torch.randperm(pool, generator=gen, device=DEV).int()
    most = -(-(c["ctx"] + 1) // PAGE)
    s["table"] = torch.full((rows, most), -1, dtype=torch.int32, device=DEV)
    lens = [0] * rows
    if c["kind"] == "fork":
        at = 0
        for r in range(c["parents"]):
            lens[r] = max(1, c["ctx"] - 13 * r)
            n = -(-lens[r] // PAGE)
            s["table"][r, :n] = order[at:at + n]
            at += n
        s["counts"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
        s["counts"][order[:at].long()] = 1
        s["parents"] = _int([i * 7 % c["parents"] for i in range(c["children"])])
        s["children"] = _int([c["parents"] + i for i in range(c["children"])])
        s["ones"] = torch.ones(c["children"], dtype=torch.int32, device=DEV)
        s["slots"] = torch.empty(c["children"], dtype=torch.int32, device=DEV)
        s["lens"] = _int(lens)
    else:
        share = pool * c["live"] // 100
        at = 0
        for r in range(rows):
            n = min(most - 1, share - at)
            lens[r] = max(0, n * PAGE - (r * 5) % PAGE)
            s["table"][r, :n] = order[at:at + n]
            at += n
        # pages that a prefix cache holds beside the rows
        s["counts"] = torch.zeros(pool, dtype=torch.int32, device=DEV)
        s["counts"][order[:share].long()] = 1
        s["lens"] = _int(lens)
        s["table_out"], s["counts_out"] = torch.empty_like(s["table"]), torch.empty_like(s["counts"])
        s["live"] = torch.empty(1, dtype=torch.int32, device=DEV)
    if own:  # the cache handles (one a layer) and the workspace that a serving program keeps
        from query_aware_sparse_quest_gb300 import binding
        s["caches"] = binding.CacheList([binding.Cache(s["k"][i], s["v"][i], s["meta"][i]) for i in range(c["layers"])])
        s["ws"] = torch.empty(binding.sv_pages_workspace_size(pool, rows, c.get("children", 1)), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ the plain forms
def _attend(q, k, v, seen, scale):
    """q [.., n, D], k / v [.., L, D], seen [.., n, L] -> sums relative to the largest logit, in 32 bits."""
    z = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = z.sub_(m.clamp_min(-1e30)).exp_()
    return p @ v, p.sum(-1, keepdim=True), m


def _gather(s, phys, heads_first=True):
    """The K and V of pages phys [.., n] as fp32 [.., Hkv, 16 n, D]."""
    def one(pool, scale):
        x = pool[phys]
        x = x.float() if scale is None else x.view(torch.float8_e4m3fn).float() * scale[phys][..., None]
        return x.transpose(-4, -3).flatten(-3, -2)
    return one(s["k"], s["ks"]), one(s["v"], s["vs"])


def _window_plain(s):
    c = s["case"]
    hkv, group, n = c["hkv"], c["group"], s["most"]
    lens = s["lens"].long()
    batch = lens.numel()
    starts = torch.arange(batch + 1, device=DEV) if s["starts"] is None else s["starts"].long()
    size = starts[1:] - starts[:-1]
    step = torch.arange(n, device=DEV)
    row = (starts[:-1, None] + step).clamp_max(s["q"].shape[0] - 1)          # [B, n]
    there = step < size[:, None]
    pos = lens[:, None] - size[:, None] + step                               # position of each query token
    # Pages some row sees: the sinks' and those from the first row's window on.
    first = torch.zeros_like(lens) if not c["window"] else (lens - size + 1 - c["window"]).clamp_min(0) // PAGE
    sinks = torch.zeros_like(lens) if not c["window"] else first.clamp_max(-(-c["sink"] // PAGE))
    last = -(-lens // PAGE)
    most = int(-(-s["longest"] // PAGE) if not c["window"] else
               min(-(-s["longest"] // PAGE), -(-c["sink"] // PAGE) + (c["window"] + n - 2) // PAGE + 2))
    i = torch.arange(most, device=DEV)
    page = torch.where(i < sinks[:, None], i, first[:, None] + i - sinks[:, None])
    page = page.clamp_max(s["table"].shape[1] - 1)
    token = (torch.where(i < (sinks + last - first)[:, None], page * PAGE, 1 << 30)[..., None] +
             torch.arange(PAGE, device=DEV)).flatten(1)                      # [B, L]
    k, v = _gather(s, s["table"].gather(1, page).long())                     # [B, Hkv, L, D]
    q = s["q"].float()[row].unflatten(2, (hkv, group)).permute(0, 2, 3, 1, 4).flatten(2, 3)   # [B, Hkv, G n, D]
    seen = token[:, None] <= pos[..., None]
    if c["window"]:
        seen &= (token[:, None] > pos[..., None] - c["window"]) | (token[:, None] < c["sink"])
    seen = seen[:, None].repeat(1, 1, group, 1)
    o, l, m = _attend(q, k, v, seen, s["scale"])
    o = (o / l).unflatten(2, (group, n)).permute(0, 3, 1, 2, 4).flatten(2, 3)                 # [B, n, Hq, D]
    lse = (l.log() + m).unflatten(2, (group, n)).permute(0, 3, 1, 2, 4).reshape(batch, n, -1)
    return o[there].bfloat16(), lse[there]


def _prefix_plain(s):
    c = s["case"]
    hkv, group = c["hkv"], c["group"]
    lens, of = s["lens"].long(), s["group_of"]
    shared = s["shared"].long()
    batch = lens.numel()
    q = s["q"].float().unflatten(1, (hkv, group))                            # [B, Hkv, G, D]
    lead = s["group_start"].long()[:-1]
    # The prefix: every group's rows against its pages, read once.
    i = torch.arange(s["longest_shared"], device=DEV)
    page = torch.where(i < shared[:, None], i, 0)
    k, v = _gather(s, s["table"][lead].gather(1, page).long())               # [groups, Hkv, L, D]
    size = s["group_start"].long().diff()
    most = batch if c["groups"] == 1 else max(_group_sizes(c))
    slot = (lead[:, None] + torch.arange(most, device=DEV)).clamp_max(batch - 1)
    at = torch.arange(batch, device=DEV) - lead[of]
    qg = q[slot].permute(0, 2, 1, 3, 4).flatten(2, 3)                        # [groups, Hkv, most G, D]
    seen = (torch.arange(k.shape[2], device=DEV) < shared[:, None] * PAGE)[:, None, None]
    o1, l1, m1 = (x.unflatten(2, (most, group)).transpose(1, 2)[of, at] for x in _attend(qg, k, v, seen, s["scale"]))
    # The rest of each request.
    i = torch.arange(s["longest_tail"], device=DEV)
    page = (shared[of][:, None] + i).clamp_max(s["table"].shape[1] - 1)
    k, v = _gather(s, s["table"].gather(1, page).long())
    token = (shared[of][:, None] + i)[..., None] * PAGE + torch.arange(PAGE, device=DEV)
    seen = (token.flatten(1) < lens[:, None])[:, None, None]
    o2, l2, m2 = _attend(q, k, v, seen, s["scale"])
    m = torch.maximum(m1, m2)
    e1, e2 = (m1 - m).exp(), (m2 - m).exp()
    l = l1 * e1 + l2 * e2
    return ((o1 * e1 + o2 * e2) / l).flatten(1, 2).bfloat16(), (l.log() + m).flatten(1)


def _fork_plain(s):
    table, lens, counts = s["table"], s["lens"], s["counts"]
    kids, parents = s["children"].long(), s["parents"].long()
    i = torch.arange(table.shape[1], device=DEV)
    # Free the rows of the last step.
    held = (i < -(-lens[kids, None] // PAGE)) & (table[kids] >= 0)
    counts.index_add_(0, table[kids].clamp_min(0).flatten().long(), -held.flatten().int())
    table[kids] = torch.where(held, -1, table[kids])
    lens[kids] = 0
    # Fork: full pages are shared, the partial one is copied to the lowest free page.
    n = lens[parents]
    shared = (i < n[:, None] // PAGE) & (table[parents] >= 0)
    part = n % PAGE > 0
    free = (counts == 0).nonzero().flatten()
    new = free[(part.cumsum(0) - 1).clamp_min(0)].int()
    rows = torch.where(shared, table[parents], table[kids])
    old = table[parents, (n // PAGE).clamp_max(table.shape[1] - 1).long()]
    rows = torch.where((i == n[:, None] // PAGE) & part[:, None], new[:, None], rows)
    counts.index_add_(0, rows.clamp_min(0).flatten().long(), (shared | ((i == n[:, None] // PAGE) & part[:, None])).flatten().int())
    table[kids] = rows
    lens[kids] = n
    src, dst = old[part].long(), new[part].long()
    for x in (s["k"], s["v"], s["meta"]):
        x[:, dst] = x[:, src]
    # Reserve one token a child: rows whose last page is full take the next free page.
    full = n % PAGE == 0
    free = (counts == 0).nonzero().flatten()
    new = free[(full.cumsum(0) - 1).clamp_min(0)].int()
    at = (n // PAGE).long()
    table[kids, at] = torch.where(full, new, table[kids, at])
    counts.index_add_(0, new.long(), full.int())
    lens[kids] = n + 1
    slots = table[kids, at] * PAGE + n % PAGE
    return dict(table=table, lens=lens, counts=counts, slots=slots, k=s["k"], v=s["v"], meta=s["meta"])


def _compact_plain(s):
    table, lens, counts = s["table"], s["lens"], s["counts"]
    alive = counts > 0
    live = alive.sum()
    i = torch.arange(counts.numel(), device=DEV)
    holes = (~alive & (i < live)).nonzero().flatten()
    movers = (alive & (i >= live)).nonzero().flatten()
    for x in (s["k"], s["v"], s["meta"]):
        x[:, holes] = x[:, movers]
    to = i.int()
    to[movers] = holes.int()
    held = (torch.arange(table.shape[1], device=DEV) < -(-lens[:, None] // PAGE)) & (table >= 0)
    out = torch.where(held, to[table.clamp_min(0).long()], table)
    left = counts.clone()
    left[holes] = counts[movers]
    left[movers] = 0
    return dict(table=out, counts=left, live=live.int()[None], k=s["k"], v=s["v"], meta=s["meta"])


def run(state):
    s, c = state, state["case"]
    if not own:
        return dict(window=_window_plain, prefix=_prefix_plain, fork=_fork_plain, compact=_compact_plain)[c["kind"]](s)
    from query_aware_sparse_quest_gb300 import binding
    if c["kind"] in ("window", "prefix"):
        out = torch.empty_like(s["q"])
        lse = torch.empty(out.shape[:2], dtype=torch.float32, device=DEV)
        if c["kind"] == "window":
            binding.sv_window_attention(s["cache"], s["q"], s["table"], s["lens"], c["window"], c["sink"], out, lse, s["ws"],
                                        q_start=s["starts"], softmax_scale=s["scale"])
        else:
            binding.sv_prefix_decode(s["cache"], s["q"], s["table"], s["lens"], s["group_start"], s["shared"], out, lse,
                                     s["ws"], softmax_scale=s["scale"])
        return out, lse
    if c["kind"] == "fork":
        binding.sv_pages_free(s["table"], s["lens"], s["counts"], s["children"])
        binding.sv_pages_fork(s["caches"], s["table"], s["lens"], s["counts"], s["parents"], s["children"], s["ws"])
        binding.sv_pages_reserve(s["table"], s["lens"], s["counts"], s["children"], s["ones"], s["slots"], s["ws"])
        return dict(table=s["table"], lens=s["lens"], counts=s["counts"], slots=s["slots"], k=s["k"], v=s["v"],
                    meta=s["meta"])
    binding.sv_pages_compact(s["caches"], s["table"], s["lens"], s["counts"], s["table_out"], s["counts_out"], s["live"],
                             s["ws"])
    return dict(table=s["table_out"], counts=s["counts_out"], live=s["live"], k=s["k"], v=s["v"], meta=s["meta"])


# ------------------------------------------------------------------ what a pass cannot do without
def _visible(n, size, window, sink):
    """(pairs seen by the rows of one request, distinct tokens seen)"""
    pairs = 0
    if not window:
        return size * (n - size) + size * (size + 1) // 2, n
    for p in range(n - size, n):
        lo = max(0, p - window + 1)
        pairs += p - lo + 1 + min(lo, sink)
    lo = max(0, n - size - window + 1)
    return pairs, n - lo + min(lo, sink)


def work(case):
    c = case
    token = 2 * c["hkv"] * ((DIM + 4) if c.get("fp8") else 2 * DIM)   # bytes of one token's K and V
    if c["kind"] == "window":
        lens, chunks = _lens(c), _chunks(c)
        seen = [_visible(n, k, c["window"], c["sink"]) for n, k in zip(lens, chunks)]
        rows = sum(chunks) * c["hkv"] * c["group"]
        return {"bytes": sum(t for _, t in seen) * token + rows * (4 * DIM + 4) + 4 * sum(-(-t // PAGE) for _, t in seen),
                "flops": 4 * DIM * c["hkv"] * c["group"] * sum(p for p, _ in seen)}
    if c["kind"] == "prefix":
        shared, suffix = _prefixes(c)
        of = [g for g, n in enumerate(_group_sizes(c)) for _ in range(n)]
        tokens = sum(shared) * PAGE + sum(suffix)
        pairs = sum(shared[of[b]] * PAGE + suffix[b] for b in range(c["batch"]))
        rows = c["batch"] * c["hkv"] * c["group"]
        return {"bytes": tokens * token + rows * (4 * DIM + 4) + tokens // 4, "flops": 4 * DIM * c["hkv"] * c["group"] * pairs}
    page = c["layers"] * c["hkv"] * (2 * PAGE + 2) * DIM * 2
    if c["kind"] == "fork":
        lens = [max(1, c["ctx"] - 13 * r) for r in range(c["parents"])]
        held = [lens[i * 7 % c["parents"]] for i in range(c["children"])]
        moved = sum(1 for n in held if n % PAGE)
        return {"bytes": 2 * page * moved + 4 * c["pool"] + sum(28 * (-(-n // PAGE)) for n in held), "flops": 0}
    share = c["pool"] * c["live"] // 100
    moved = share * (c["pool"] - share) // c["pool"]
    return {"bytes": 2 * page * moved + 8 * c["pool"] + 8 * c["rows"] * (-(-c["ctx"] // PAGE)), "flops": 0}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _tokens64(s, b, n):
    """K and V of one request's n tokens in 64 bits: [Hkv, n, D]."""
    page = s["table"][b, : -(-n // PAGE)].long()

    def one(pool, scale):
        x = pool[page]
        if scale is not None:
            x = x.view(torch.float8_e4m3fn).double() * scale[page].double().unsqueeze(-1)
        return x.double().permute(1, 0, 2, 3).reshape(x.shape[1], -1, DIM)[:, :n]
    return one(s["k"], s["ks"]), one(s["v"], s["vs"])


def _rows64(s, b, first, size):
    """Rows first .. first + size - 1 of q, the last `size` tokens of request b."""
    c = s["case"]
    n = int(s["lens"][b])
    k, v = _tokens64(s, b, n)
    p = torch.arange(n - size, n, device=DEV)[:, None]
    j = torch.arange(n, device=DEV)[None]
    hidden = j > p
    if c.get("window"):
        hidden = hidden | ((j <= p - c["window"]) & (j >= c["sink"]))
    keep = (~hidden).any(0).nonzero().flatten()
    hidden, k, v = hidden[:, keep], k[:, keep], v[:, keep]
    out = torch.empty((size, c["hkv"] * c["group"], DIM), dtype=torch.float64, device=DEV)
    lse = torch.empty(out.shape[:2], dtype=torch.float64, device=DEV)
    for h in range(out.shape[1]):
        g = h // c["group"]
        z = s["q"][first:first + size, h].double() @ k[g].T * s["scale"]
        z[hidden] = -math.inf
        lse[:, h] = torch.logsumexp(z, 1)
        out[:, h] = torch.exp(z - lse[:, h, None]) @ v[g]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["kind"] in ("window", "prefix"):
        chunks = _chunks(c) if c["kind"] == "window" else [1] * c["batch"]
        parts = [_rows64(s, b, sum(chunks[:b]), n) for b, n in enumerate(chunks)]
        return torch.cat([o for o, _ in parts]), torch.cat([m for _, m in parts])
    counts = s["counts"].tolist()
    moves = {}
    if c["kind"] == "fork":
        free = [p for p, n in enumerate(counts) if n == 0]
        lens, parents = s["lens"].tolist(), s["parents"].tolist()
        for r in parents:
            if lens[r] % PAGE:
                moves[free.pop(0)] = int(s["table"][r, lens[r] // PAGE])
    else:
        live = sum(1 for n in counts if n)
        holes = [p for p in range(live) if not counts[p]]
        moves = dict(zip(holes, [p for p in range(live, len(counts)) if counts[p]]))
    source = list(range(len(counts)))
    for to, frm in moves.items():
        source[to] = frm
    pick = torch.tensor(source, device=DEV)
    after = {x: s[x].double()[:, pick] for x in ("k", "v", "meta")}
    return after
