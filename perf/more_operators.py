"""What the latent-cache operators are measured on: attention over a paged cache
that keeps one shared latent vector and one rotary key a token (absorbed form:
single tokens and chunks), the cache's writes (bf16, or quantised to e4m3) and
its read-back, and attention in the expanded form, with keys and values a head.

A case is a dict of plain values; `run` makes one pass through an operator, in
plain torch operations, or (where `own` is true) through the library's calls.
"""
import math

import torch

own = False

PAGE = 16
LATENT, ROPE = 512, 64          # channels of a token's latent and of its rotary key
NOPE, VALUE = 128, 128          # expanded: key channels without rotation and value channels of a head
SCALE = (NOPE + ROPE) ** -0.5
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The smallest decode: one request, 16 query heads (an eighth of 128); latency counts.
        dict(name="latent decode b1", kind="attend", batch=1, heads=16, ctx=4096, ragged=0, chunk=1, fp8=False),
        # A decode step of the 128k batch-8 serving batch with all 128 query heads on one GPU.
        dict(name="latent decode b8 128k", kind="attend", batch=8, heads=128, ctx=128000, ragged=0, chunk=1, fp8=False),
        # The ragged serving batch (4k to 64k tokens) over an e4m3 pool, a shard of 16 heads.
        dict(name="latent decode b32 fp8", kind="attend", batch=32, heads=16, ctx=65536, ragged=1, chunk=1, fp8=True),
        # A mixed batch: chunks of odd lengths with single tokens among them, an odd number of heads, e4m3 pool.
        dict(name="latent chunks b7 fp8", kind="attend", batch=7, heads=27, ctx=4000, ragged=1, chunk=777, fp8=True),
        # A chunk of a prefill over the cache in the absorbed form, all heads.
        dict(name="latent chunk 512 at 8192", kind="attend", batch=1, heads=128, ctx=8192, ragged=0, chunk=512, fp8=False),
        # A decode step's new tokens: latency counts.
        dict(name="append 8", kind="append", tokens=8, pool=64, fp8=False),
        # A prefill chunk, quantised as it is written.
        dict(name="append 4096 fp8", kind="append", tokens=4096, pool=512, fp8=True),
        # A 4096-token prompt of an e4m3 pool, read back for the expansion.
        dict(name="gather 4096 fp8", kind="gather", batch=1, ctx=4096, ragged=0, skip=0, fp8=True),
        # A ragged batch of prefixes of up to 32k tokens, each from a token inside a page on.
        dict(name="gather b8 32k", kind="gather", batch=8, ctx=32768, ragged=1, skip=37, fp8=False),
        # A short prompt, 16 heads.
        dict(name="expanded 300", kind="expand", batch=1, heads=16, ctx=300, ragged=0, chunk=300, causal=True),
        # Five requests of odd lengths with what they have cached, 8 heads.
        dict(name="expanded ragged b5", kind="expand", batch=5, heads=8, ctx=5003, ragged=1, chunk=1999, causal=True),
        # The largest: one 4096-token chunk of a chunked prefill at 32k tokens, 32 heads.
        dict(name="expanded chunk 4096 at 32k", kind="expand", batch=1, heads=32, ctx=32768, ragged=0, chunk=4096, causal=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("attend", "attend", "attend", "append", "gather", "expand", "expand"))
    if kind == "append":
        tokens = _log(rng, 1, 20000)
        return dict(kind=kind, tokens=tokens, pool=-(-tokens // PAGE) + _log(rng, 1, 400), fp8=rng.random() < 0.5)
    if kind == "gather":
        ctx = _log(rng, 1, 40000)
        return dict(kind=kind, batch=_log(rng, 1, 12), ctx=ctx, ragged=rng.randint(0, 1), skip=rng.randint(0, min(ctx - 1, 100)),
                    fp8=rng.random() < 0.5)
    if kind == "attend":
        c = dict(kind=kind, batch=_log(rng, 1, 40), heads=rng.choice((1, 8, 16, 32, 64, 128, rng.randint(1, 128))),
                 ctx=_log(rng, 1, 70000), ragged=rng.randint(0, 1), chunk=1 if rng.random() < 0.6 else _log(rng, 2, 1024),
                 fp8=rng.random() < 0.5)
        most = 1 << 28      # (row, token) pairs: half of the chunk of 512 at 8192
        tokens = 1 << 20
    else:
        c = dict(kind=kind, batch=_log(rng, 1, 8), heads=rng.choice((1, 4, 8, 16, 32, rng.randint(1, 40))),
                 ctx=_log(rng, 1, 20000), ragged=rng.randint(0, 1), chunk=_log(rng, 1, 4096), causal=rng.random() < 0.8)
        most = 1 << 30
        tokens = 1 << 17
    c["chunk"] = min(c["chunk"], c["ctx"])
    while c["batch"] > 1 and (c["batch"] * c["chunk"] * c["ctx"] * c["heads"] > most or c["batch"] * c["ctx"] > tokens):
        c["batch"] //= 2
    while c["chunk"] > 1 and c["chunk"] * c["ctx"] * c["heads"] > most:
        c["chunk"] = c["chunk"] * 2 // 3
    return c


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


def _skips(c):
    return [min(c["skip"], n - 1) for n in _lens(c)]


def _starts(sizes):
    return [sum(sizes[:i]) for i in range(len(sizes) + 1)]


def _int(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)


def _rows(gen, n):
    """The latents (normalised, times a weight a channel) and rotary keys (of a few large channels) of n tokens: [n, 576]."""
    x = _randn(gen, n, LATENT + ROPE)
    x *= _randn(gen, LATENT + ROPE).mul_(0.4).exp_()
    return x.bfloat16()


def _coded(x):
    """e4m3 codes and one scale a row, as the cache keeps them."""
    x = x.float()
    s = x.abs().amax(-1) / 448.0
    return (x / s[..., None].clamp_min(1e-30)).to(torch.float8_e4m3fn).view(torch.uint8), s


def _pool(c, gen, pages):
    rows = _rows(gen, pages * PAGE).unflatten(0, (pages, PAGE))
    s = dict(latent=rows[..., :LATENT].contiguous(), rope=rows[..., LATENT:].contiguous(), scale=None)
    if c["fp8"]:
        s["latent"], s["scale"] = _coded(s["latent"])
    return s


def _tables(gen, lens):
    """Pages in any order: the page table and how many pages there are."""
    counts = [-(-n // PAGE) for n in lens]
    order = torch.randperm(sum(counts), generator=gen, device=DEV).int()
    table = torch.zeros((len(lens), max(counts)), dtype=torch.int32, device=DEV)
    for b, at in enumerate(_starts(counts)[:-1]):
        table[b, :counts[b]] = order[at:at + counts[b]]
    return table, sum(counts)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    if c["kind"] == "append":
        s = _pool(c, gen, c["pool"])
        # A projection's output: latent and rotary key side by side, in slots of whole pages in any order.
        rows = _rows(gen, c["tokens"])
        pages = torch.randperm(c["pool"], generator=gen, device=DEV)[:-(-c["tokens"] // PAGE)]
        slots = (pages[:, None] * PAGE + torch.arange(PAGE, device=DEV)).flatten()[:c["tokens"]].int()
        s.update(new_latent=rows[:, :LATENT], new_rope=rows[:, LATENT:], slots=slots)
    elif c["kind"] == "expand":
        lens, chunks = _lens(c), _chunks(c)
        h, total, rows = c["heads"], sum(lens), sum(chunks)
        # The expansion's output: a head's key and value channels side by side.
        kv = _randn(gen, total, h, NOPE + VALUE).bfloat16()
        s = dict(q=_randn(gen, rows, h, NOPE + ROPE).bfloat16(), k=kv[..., :NOPE], v=kv[..., NOPE:],
                 rope=_randn(gen, total, ROPE).bfloat16(), q_start=_int(_starts(chunks)), kv_start=_int(_starts(lens)),
                 most_q=max(chunks), most_kv=max(lens))
        if own:
            from query_aware_sparse_quest_gb300 import binding
            s["ws"] = torch.empty(binding.sv_expanded_attention_workspace_size(c["batch"], h, rows), dtype=torch.uint8, device=DEV)
    else:
        lens = _lens(c)
        table, pages = _tables(gen, lens)
        s = _pool(c, gen, pages)
        s.update(table=table, lens=_int(lens), longest=max(lens))
        if c["kind"] == "gather":
            skips = _skips(c)
            sizes = [n - k for n, k in zip(lens, skips)]
            s.update(first=_int(skips), starts=_int(_starts(sizes)), rows=sum(sizes))
        else:
            chunks = _chunks(c)
            s.update(q=_randn(gen, sum(chunks), c["heads"], LATENT + ROPE).bfloat16(), most=max(chunks),
                     starts=None if c["chunk"] == 1 else _int(_starts(chunks)))
            if own:
                from query_aware_sparse_quest_gb300 import binding
                s["ws"] = torch.empty(binding.sv_latent_attention_workspace_size(c["batch"], c["heads"], sum(chunks)),
                                      dtype=torch.uint8, device=DEV)
    if own and c["kind"] != "expand":  # the cache handle that a serving program keeps
        from query_aware_sparse_quest_gb300 import binding
        s["cache"] = binding.LatentCache(s["latent"], s["rope"], s["scale"])
    s["case"] = c
    return s


# ------------------------------------------------------------------ the plain forms
def _attend(q, k, v, seen):
    """q [.., n, D], k / v [.., L, D], seen [.., n, L] -> the average of v and ln of the sum, in 32 bits."""
    z = (q @ k.transpose(-1, -2)).mul_(SCALE).masked_fill_(~seen, -math.inf)
    m = z.amax(-1, keepdim=True).clamp_min(-1e30)
    p = z.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    return (p @ v) / l, (l.log() + m)[..., 0]


def _read(s, page):
    """The tokens of pages [.., n] in 32 bits: latents [.., 16 n, 512] and rotary keys [.., 16 n, 64]."""
    x = s["latent"][page]
    x = x.float() if s["scale"] is None else x.view(torch.float8_e4m3fn).float() * s["scale"][page][..., None]
    return x.flatten(-3, -2), s["rope"][page].float().flatten(-3, -2)


def _attend_plain(s):
    heads, n = s["case"]["heads"], s["most"]
    lens = s["lens"].long()
    batch = lens.numel()
    starts = torch.arange(batch + 1, device=DEV) if s["starts"] is None else s["starts"].long()
    size = starts[1:] - starts[:-1]
    step = torch.arange(n, device=DEV)
    row = (starts[:-1, None] + step).clamp_max(s["q"].shape[0] - 1)              # [B, n]
    there = step < size[:, None]
    pos = lens[:, None] - size[:, None] + step
    latent, rope = _read(s, s["table"].long())                                   # [B, L, ..]
    q = s["q"].float()[row].flatten(1, 2)                                        # [B, n heads, 576]
    seen = torch.arange(latent.shape[1], device=DEV) <= pos[..., None].clamp_min(0)
    o, lse = _attend(q, torch.cat((latent, rope), -1), latent, seen.repeat_interleave(heads, 1))
    return o.unflatten(1, (n, heads))[there].bfloat16(), lse.unflatten(1, (n, heads))[there]


def _expand_plain(s):
    h, n, most = s["case"]["heads"], s["most_q"], s["most_kv"]
    qs, ks = s["q_start"].long(), s["kv_start"].long()
    size, lens = qs.diff(), ks.diff()
    step, token = torch.arange(n, device=DEV), torch.arange(most, device=DEV)
    row = (qs[:-1, None] + step).clamp_max(s["q"].shape[0] - 1)
    at = (ks[:-1, None] + token).clamp_max(s["k"].shape[0] - 1)
    pos = lens[:, None] - size[:, None] + step if s["case"]["causal"] else (lens[:, None] - 1).expand(-1, n)
    seen = (token <= pos[..., None].clamp_min(0)) & (token < lens[:, None, None])
    q = s["q"].float()[row].transpose(1, 2)                                      # [B, H, n, 192]
    k = torch.cat((s["k"].float()[at], s["rope"].float()[at][:, :, None].expand(-1, -1, h, -1)), -1).transpose(1, 2)
    o, lse = _attend(q, k, s["v"].float()[at].transpose(1, 2), seen[:, None])
    there = step < size[:, None]
    return o.transpose(1, 2)[there].bfloat16(), lse.transpose(1, 2)[there]


def _append_plain(s):
    slots = s["slots"].long()
    x = s["new_latent"]
    if s["scale"] is not None:
        x, scale = _coded(x)
        s["scale"].view(-1)[slots] = scale
    s["latent"].view(-1, LATENT)[slots] = x
    s["rope"].view(-1, ROPE)[slots] = s["new_rope"]


def _gather_plain(s):
    starts, first = s["starts"].long(), s["first"].long()
    row = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(starts, row, right=True) - 1
    token = row - starts[b] + first[b]
    page, at = s["table"].long()[b, token // PAGE], token % PAGE
    x = s["latent"][page, at]
    if s["scale"] is not None:
        x = (x.view(torch.float8_e4m3fn).float() * s["scale"][page, at][:, None]).bfloat16()
    return x, s["rope"][page, at]


def _pool_out(s):
    if s["scale"] is None:
        return dict(latent=s["latent"], rope=s["rope"])
    return dict(latent=s["latent"].view(torch.float8_e4m3fn), rope=s["rope"], scale=s["scale"])


def run(state):
    s, c = state, state["case"]
    if not own:
        if c["kind"] == "append":
            _append_plain(s)
            return _pool_out(s)
        return dict(attend=_attend_plain, gather=_gather_plain, expand=_expand_plain)[c["kind"]](s)
    from query_aware_sparse_quest_gb300 import binding
    if c["kind"] == "append":
        binding.sv_latent_append(s["cache"], s["new_latent"], s["new_rope"], s["slots"])
        return _pool_out(s)
    if c["kind"] == "gather":
        latent = torch.empty((s["rows"], LATENT), dtype=torch.bfloat16, device=DEV)
        rope = torch.empty((s["rows"], ROPE), dtype=torch.bfloat16, device=DEV)
        binding.sv_latent_gather(s["cache"], s["table"], s["lens"], s["starts"], latent, rope, first_token=s["first"])
        return latent, rope
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    if c["kind"] == "attend":
        out = torch.empty((*lse.shape, LATENT), dtype=torch.bfloat16, device=DEV)
        binding.sv_latent_attention(s["cache"], s["q"], s["table"], s["lens"], out, lse, s["ws"], softmax_scale=SCALE,
                                    q_start=s["starts"])
    else:
        out = torch.empty((*lse.shape, VALUE), dtype=torch.bfloat16, device=DEV)
        binding.sv_expanded_attention(s["q"], s["k"], s["rope"], s["v"], s["q_start"], s["kv_start"], out, lse, s["ws"],
                                      causal=c["causal"], softmax_scale=SCALE)
    return out, lse


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    token = LATENT + 4 + 2 * ROPE if c.get("fp8") else 2 * (LATENT + ROPE)       # bytes of a cached token
    plain = 2 * (LATENT + ROPE)
    if c["kind"] == "append":
        return {"bytes": c["tokens"] * (plain + token + 4), "flops": 0}
    lens = _lens(c)
    if c["kind"] == "gather":
        rows = sum(lens) - sum(_skips(c))
        return {"bytes": rows * (plain + token), "flops": 0}
    chunks = _chunks(c)
    rows = sum(chunks) * c["heads"]
    if c["kind"] == "attend":
        pairs = sum(k * (n - k) + k * (k + 1) // 2 for n, k in zip(lens, chunks)) * c["heads"]
        return {"bytes": sum(lens) * token + rows * (2 * (2 * LATENT + ROPE) + 4), "flops": 2 * (2 * LATENT + ROPE) * pairs}
    pairs = sum(k * (n - k) + k * (k + 1) // 2 if c["causal"] else k * n for n, k in zip(lens, chunks)) * c["heads"]
    return {"bytes": sum(lens) * 2 * (c["heads"] * (NOPE + VALUE) + ROPE) + rows * (2 * (NOPE + ROPE + VALUE) + 4),
            "flops": 2 * (NOPE + ROPE + VALUE) * pairs}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _softmax64(z, hidden, v):
    z[hidden] = -math.inf
    lse = torch.logsumexp(z, -1)
    return torch.exp(z - lse[..., None]) @ v, lse


def _token64(s, b, i):
    """Tokens i (a tensor) of request b: latents and rotary keys in 64 bits."""
    slot = s["table"][b].long()[i // PAGE] * PAGE + i % PAGE
    c = s["latent"].reshape(-1, LATENT)[slot]
    if s["scale"] is not None:
        c = c.view(torch.float8_e4m3fn).double() * s["scale"].reshape(-1)[slot].double().unsqueeze(1)
    return c.double(), s["rope"].reshape(-1, ROPE)[slot].double()


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] == "append":
        slots = s["slots"].tolist()
        latent, rope = s["latent"], s["rope"].double()
        latent = (latent.view(torch.float8_e4m3fn) if c["fp8"] else latent).double()
        new = s["new_latent"].double()
        after = dict(latent=latent, rope=rope)
        if c["fp8"]:
            size = new.abs().max(1).values / 448
            x = new / size[:, None]
            # The nearest code: 3 mantissa bits from 2^-6 on, steps of 2^-9 below; ties to even.
            step = torch.exp2(torch.log2(x.abs().clamp_min(2.0 ** -6)).floor() - 3)
            new = torch.round(x / step) * step
            after["scale"] = s["scale"].double()
        for i in range(0, len(slots), PAGE):    # a page's tokens are consecutive
            page, n = slots[i] // PAGE, min(PAGE, len(slots) - i)
            latent[page, :n] = new[i:i + n]
            rope[page, :n] = s["new_rope"][i:i + n].double()
            if c["fp8"]:
                after["scale"][page, :n] = size[i:i + n]
        return after
    lens = _lens(c)
    if c["kind"] == "gather":
        parts = [_token64(s, b, torch.arange(k, n, device=DEV)) for b, (n, k) in enumerate(zip(lens, _skips(c)))]
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    chunks = _chunks(c)
    outs, sums = [], []
    for b, (n, size) in enumerate(zip(lens, chunks)):
        at = sum(chunks[:b])
        j = torch.arange(n, device=DEV)
        if c["kind"] == "attend":
            latent, rope = _token64(s, b, j)
            for i0 in range(0, size, 64):
                i1 = min(size, i0 + 64)
                q = s["q"][at + i0:at + i1].double()
                z = (q[..., :LATENT] @ latent.T + q[..., LATENT:] @ rope.T) * SCALE
                last = torch.arange(n - size + i0, n - size + i1, device=DEV)
                o, l = _softmax64(z, (j > last[:, None, None]).expand_as(z), latent)
                outs.append(o)
                sums.append(l)
        else:
            from_, to = sum(lens[:b]), sum(lens[:b + 1])
            last = torch.arange(n - size, n, device=DEV) if c["causal"] else torch.full((size,), n - 1, device=DEV)
            o = torch.empty((size, c["heads"], VALUE), dtype=torch.float64, device=DEV)
            l = torch.empty((size, c["heads"]), dtype=torch.float64, device=DEV)
            for h in range(c["heads"]):
                q = s["q"][at:at + size, h].double()
                z = (q[:, :NOPE] @ s["k"][from_:to, h].double().T + q[:, NOPE:] @ s["rope"][from_:to].double().T) * SCALE
                o[:, h], l[:, h] = _softmax64(z, j > last[:, None], s["v"][from_:to, h].double())
            outs.append(o)
            sums.append(l)
    return torch.cat(outs), torch.cat(sums)
