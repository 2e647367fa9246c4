"""Attention over latents and in the expanded form from its definition, in 64
bits, and the error that the kernels' roundings allow."""
from __future__ import annotations

import torch

PAGE, LATENT, ROPE = 16, 512, 64


def code(x):
    """e4m3 codes and one scale a row (divided as IEEE does, not by a product with 1 / 448)."""
    x = x.float()
    s = (x.abs().amax(-1).double() / 448.0).float()
    return (x / s[..., None].clamp_min(1e-30)).to(torch.float8_e4m3fn).view(torch.uint8), s


class LatentCase:
    """A shuffled pool of latents whose unused slots, and the slots that a test hides, hold NaN."""

    def __init__(self, lens, max_pages=None, fp8=False, seed=0, device="cuda", spare=3, mean=0.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.fp8, self.device = list(lens), fp8, device
        counts = [-(-n // PAGE) for n in lens]
        total = sum(counts) + spare
        self.max_pages = max_pages or max(1, max(counts, default=1))
        order = torch.randperm(total, generator=g)
        self.table = torch.full((len(lens), self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n].int()
            at += n
        self.latent = (torch.randn((total, PAGE, LATENT), generator=g) * torch.randn(LATENT, generator=g).mul(0.4).exp() +
                       mean).bfloat16()
        self.rope = torch.randn((total, PAGE, ROPE), generator=g).bfloat16()
        self.scale = None
        if fp8:
            self.latent, self.scale = code(self.latent)
        used = torch.zeros((total, PAGE), dtype=torch.bool)
        for b, n in enumerate(lens):
            for p in range(counts[b]):
                used[self.table[b, p], : min(PAGE, n - p * PAGE)] = True
        self.fill(~used)

    def fill(self, mask, value=float("nan")):
        """`value` in every channel of the slots of mask [pages, 16]."""
        if self.fp8:
            self.latent[mask] = 0x7F if value != value else 0x38      # NaN, or 1 with the value as its scale
            self.scale[mask] = value
        else:
            self.latent[mask] = value
        self.rope[mask] = value

    def fill_tokens(self, b, tokens, value=float("nan")):
        mask = torch.zeros(self.latent.shape[:2], dtype=torch.bool)
        for t in tokens:
            mask[self.table[b, t // PAGE], t % PAGE] = True
        self.fill(mask, value)

    def cache(self):
        from query_aware_sparse_quest_gb300 import binding
        f = [None if x is None else x.to(self.device).contiguous() for x in (self.latent, self.rope, self.scale)]
        return binding.LatentCache(*f)

    def spread(self, pages):
        """The same cache in a pool of `pages` pages, from the last one down (the others hold whatever was there)."""
        at = pages - 1 - 2 * torch.arange(self.latent.shape[0])
        self.table = torch.where(self.table >= 0, at[self.table.long().clamp_min(0)].int(), self.table)

        def one(x):
            if x is None:
                return None
            big = torch.empty((pages, *x.shape[1:]), dtype=x.dtype, device=self.device)
            big[at.to(self.device)] = x.to(self.device)
            return big
        self.latent, self.rope, self.scale = (one(x) for x in (self.latent, self.rope, self.scale))

    def tokens(self, b, n=None):
        """Latents [n, 512] and rotary keys [n, 64] of request b in 64 bits, on the device."""
        n = self.lens[b] if n is None else n
        page = self.table[b, : -(-n // PAGE)].long().to(self.latent.device)
        c = self.latent[page].to(self.device)
        c = c.double() if self.scale is None else \
            c.view(torch.float8_e4m3fn).double() * self.scale[page].to(self.device).double()[..., None]
        return c.flatten(0, 1)[:n], self.rope[page].to(self.device).double().flatten(0, 1)[:n]


def attend(q, k, v, seen, scale):
    """q [n, H, D], k [L, D] or [L, H, D], v [L, E] or [L, H, E], seen [n, L] -> out, lse, and the bounds of their
    errors (all 64 bits; a row that sees nothing: 0 and -inf).

    Roundings: a weight to bf16, 2^-8 of it, with the average taken over the sum of weights before or after it (2^-8 of
    the average too); the output to bf16 (2^-8 of it); the logits: a product's D / 16 steps and at most two scales in
    fp32, each off by 2^-23 (a step's sum is cut off, not rounded) of the sum of magnitudes, twice, as weights and sum
    both move; the exponential 2^-21; the values' L / 16 steps, cut off at 2^-23, and sums of partial results, 2^-20."""
    n, heads, d = q.shape
    length, e = seen.shape[1], v.shape[-1]
    out = torch.zeros((n, heads, e), dtype=torch.float64, device=q.device)
    lse = torch.full((n, heads), -float("inf"), dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    any_seen = seen.any(1)
    zero, low = (torch.tensor(x, device=q.device, dtype=torch.float64) for x in (0.0, -float("inf")))
    for h in range(heads):
        kk, vv = (torch.nan_to_num(x if x.dim() == 2 else x[:, h], posinf=0.0, neginf=0.0) for x in (k, v))
        qh = q[:, h].double()
        z = torch.where(seen, (qh @ kk.T) * scale, low)
        mag = torch.where(seen, (qh.abs() @ kk.abs().T) * scale, zero)
        mag = mag.amax(1) if length else torch.zeros(n, dtype=torch.float64, device=q.device)
        ls = torch.logsumexp(z, 1)
        p = torch.where(any_seen[:, None], torch.exp(z - torch.where(any_seen, ls, zero)[:, None]), zero)
        o, a = p @ vv, p @ vv.abs()
        ez = (d / 16 + 4) * 2.0 ** -23 * mag
        sums = 2.0 ** -27 * length + 2.0 ** -20
        out[:, h], lse[:, h] = o, torch.where(any_seen, ls, low)
        tol[:, h] = 2.0 ** -8 * (a + o.abs()) + (2 * ez[:, None] + 2.0 ** -20 + sums) * a + 2.0 ** -8 * (o.abs() + 2.0 ** -7 * a) + 1e-30
        tol_lse[:, h] = ez + 2.0 ** -20 + sums + 2.0 ** -23 * torch.where(any_seen, ls.abs(), zero)
    return out, lse, tol, tol_lse


def check(got_out, got_lse, ref):
    out, lse, tol, tol_lse = ref
    got_out, got_lse = got_out.double(), got_lse.double()
    assert torch.isfinite(got_out).all()
    err = (got_out - out).abs()
    assert (err <= tol).all(), (err / tol).max().item()
    empty = torch.isinf(lse)
    assert torch.equal(got_lse[empty], lse[empty])
    e = (got_lse - lse).abs()[~empty]
    assert (e <= tol_lse[~empty]).all(), (e / tol_lse[~empty]).max().item()


def causal_seen(n, size, device):
    """[size, n]: what the last `size` of n tokens see."""
    return torch.arange(n, device=device)[None] <= torch.arange(n - size, n, device=device)[:, None]
