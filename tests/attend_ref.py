"""Attention over a paged cache from its definition, in 64 bits, and the error
that the kernels' roundings allow."""
from __future__ import annotations

import torch

PAGE, DIM = 16, 128


class PagedCase:
    """A shuffled pool whose unused slots, and the slots of tokens that nobody may read, hold NaN."""

    def __init__(self, lens, hkv, max_pages=None, fp8=False, seed=0, device="cuda", spare=3, v_mean=0.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.fp8 = list(lens), hkv, fp8
        counts = [-(-n // PAGE) for n in lens]
        total = sum(counts) + spare
        self.max_pages = max_pages or max(1, max(counts, default=1))
        order = torch.randperm(total, generator=g)
        self.table = torch.full((len(lens), self.max_pages), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n].int()
            at += n
        shape = (total, hkv, PAGE, DIM)
        channel = torch.randn((1, hkv, 1, DIM), generator=g).mul(0.5).exp()
        k = (torch.randn(shape, generator=g) * channel).bfloat16()
        v = (torch.randn(shape, generator=g) + v_mean).bfloat16()
        used = torch.zeros((total, PAGE), dtype=torch.bool)
        for b, n in enumerate(lens):
            for p in range(counts[b]):
                used[self.table[b, p], : min(PAGE, n - p * PAGE)] = True
        self.device = device
        self.k, self.v, self.ks, self.vs = k, v, None, None
        if fp8:
            self.k, self.ks = self._code(k)
            self.v, self.vs = self._code(v)
        self.hide(~used)

    @staticmethod
    def _code(x):
        x = x.float()
        s = x.abs().amax(-1) / 448.0
        return (x / s[..., None].clamp_min(1e-30)).to(torch.float8_e4m3fn).view(torch.uint8), s

    def hide(self, mask):
        """NaN in every row of mask [pages, 16]."""
        m = mask[:, None, :].expand(-1, self.hkv, -1)
        for x, s in ((self.k, self.ks), (self.v, self.vs)):
            if self.fp8:
                x[m] = 0x7F
                s[m] = float("nan")
            else:
                x[m] = float("nan")

    def hide_tokens(self, b, tokens):
        mask = torch.zeros((self.k.shape[0], PAGE), dtype=torch.bool)
        for t in tokens:
            mask[self.table[b, t // PAGE], t % PAGE] = True
        self.hide(mask)

    def cache(self):
        from query_aware_sparse_quest_gb300 import binding
        dev = self.device
        meta = torch.zeros((self.k.shape[0], self.hkv, 2, DIM), dtype=torch.bfloat16, device=dev)
        f = [None if x is None else x.to(dev).contiguous() for x in (self.k, self.v, self.ks, self.vs)]
        return binding.Cache(f[0], f[1], meta, f[2], f[3])

    def spread(self, pages):
        """The same cache in a pool of `pages` pages, from the last one down (the others hold whatever was there)."""
        at = pages - 1 - 2 * torch.arange(self.k.shape[0])
        self.table = torch.where(self.table >= 0, at[self.table.long()].int(), self.table)

        def one(x):
            if x is None:
                return None
            big = torch.empty((pages, *x.shape[1:]), dtype=x.dtype, device=self.device)
            big[at.to(self.device)] = x.to(self.device)
            return big
        self.k, self.v, self.ks, self.vs = (one(x) for x in (self.k, self.v, self.ks, self.vs))

    def tokens(self, b, n=None):
        """K, V [Hkv, n, D] of request b in 64 bits, on the device."""
        n = self.lens[b] if n is None else n
        page = self.table[b, : -(-n // PAGE)].long()

        def one(x, s):
            x = x[page].to(self.device)
            x = x.double() if s is None else x.view(torch.float8_e4m3fn).double() * s[page].to(self.device).double()[..., None]
            return x.transpose(0, 1).flatten(1, 2)[:, :n]
        return one(self.k, self.ks), one(self.v, self.vs)


def attend(q, k, v, seen, scale):
    """q [n, Hq, D], k / v [Hkv, L, D], seen [n, L] -> out, lse, and the bounds of
    their errors (all 64 bits; a row that sees nothing: 0 and -inf).

    Roundings: P to bf16 (at most 2^-8 of each weight), the output to bf16 (2^-8 of
    it), the logits' 128 products and additions and the scale in fp32 (2^-24 each
    of the sum of magnitudes; twice, as P and its sum both move), the exponential
    (2^-22), and the fp32 sums over L tokens, taken as 2^-24 sqrt(L) + 2^-20."""
    n, hq, _ = q.shape
    group = hq // k.shape[0]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full((n, hq), -float("inf"), dtype=torch.float64, device=q.device)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    any_seen = seen.any(1)
    for h in range(hq):
        kk, vv = k[h // group], v[h // group]
        qh = q[:, h].double()
        # A token that a row does not see contributes nothing, whatever it holds.
        z = torch.where(seen, (qh @ torch.nan_to_num(kk).T) * scale, torch.tensor(-float("inf"), device=q.device, dtype=torch.float64))
        mag = torch.where(seen, (qh.abs() @ torch.nan_to_num(kk).abs().T) * scale, torch.zeros((), device=q.device, dtype=torch.float64)).amax(1)
        ls = torch.logsumexp(z, 1)
        p = torch.where(any_seen[:, None], torch.exp(z - torch.where(any_seen, ls, 0.0)[:, None]), 0.0)
        vv = torch.nan_to_num(vv)
        o, a = p @ vv, p @ vv.abs()
        ez = 130 * 2.0 ** -24 * mag
        sums = 2.0 ** -24 * max(1, seen.shape[1]) ** 0.5 + 2.0 ** -20
        out[:, h], lse[:, h] = o, torch.where(any_seen, ls, -float("inf"))
        tol[:, h] = (2.0 ** -8 + 2 * ez[:, None] + sums) * a + 2.0 ** -8 * (o.abs() + 2.0 ** -8 * a) + 1e-30
        tol_lse[:, h] = ez + 2.0 ** -21 + sums + 2.0 ** -23 * torch.where(any_seen, ls.abs(), 0.0)
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


def window_seen(n, size, window, sink, device):
    """[size, n]: what the last `size` of n tokens see."""
    p = torch.arange(n - size, n, device=device)[:, None]
    j = torch.arange(n, device=device)[None]
    seen = j <= p
    if window:
        seen = seen & ((j > p - window) | (j < sink))
    return seen
