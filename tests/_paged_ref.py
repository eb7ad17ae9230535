"""Float64 definitions of the paged cache and packed prompt operators, and their inputs
(test infrastructure; no library code)."""
from __future__ import annotations

import math

import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def half_step(dtype) -> float:
    """Largest relative error of one rounding to nearest."""
    return torch.finfo(dtype).eps / 2


class Pool:
    """Pages holding sequences of given lengths in shuffled order, every row that belongs to
    no sequence poisoned with NaN.  kv: bf16, f16 or fp8; layout "hnd" or "nhd" (strides)."""

    def __init__(self, lens, h_kv, d, page, kv, layout="hnd", seed=0, spare=2, empty=False,
                 max_pages=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.page, self.kv, self.d, self.h_kv = list(lens), page, kv, d, h_kv
        need = [-(-n // page) for n in lens]
        width = max_pages or max(1, max(need))
        self.num_pages = sum(need) + spare
        order = torch.randperm(self.num_pages, generator=g).to(torch.int32)
        # table entries that no position uses are out of range on purpose
        self.pages = torch.full((len(lens), width), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.pages[b, :n] = order[at:at + n]
            at += n
        shape = (self.num_pages, h_kv, page, d)
        if kv == "fp8":
            self.k, self.v = (torch.full(shape, 0x7F, dtype=torch.uint8) for _ in range(2))
            self.k_scale, self.v_scale = (torch.full(shape[:3], math.nan) for _ in range(2))
        else:
            self.k, self.v = (torch.full(shape, math.nan, dtype=TYPES[kv]) for _ in range(2))
            self.k_scale = self.v_scale = None
        for b, n in enumerate(lens):
            if empty or n == 0:
                continue
            pg, r = self.at(b, 0, n)
            for pool, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
                x = torch.randn(n, h_kv, d, generator=g)
                if kv == "fp8":
                    pool[pg, :, r] = x.mul(40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    scale[pg, :, r] = torch.rand(n, h_kv, generator=g) * 0.05 + 0.005
                else:
                    pool[pg, :, r] = x.to(pool.dtype)
        self.layout = layout

    def at(self, b, lo, hi):
        """Pages and rows of positions [lo, hi) of sequence b."""
        pos = torch.arange(lo, hi)
        return self.pages[b][pos // self.page].long(), pos % self.page

    def rows(self, b, lo, hi):
        """float64 K and V [hi - lo, h_kv, d] of positions [lo, hi)."""
        pg, r = self.at(b, lo, hi)
        out = []
        for pool, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
            if self.kv == "fp8":
                x = pool[pg, :, r].view(torch.float8_e4m3fn).double()
                out.append(x * scale[pg, :, r].double()[..., None])
            else:
                out.append(pool[pg, :, r].double())
        return out

    def to(self, dev):
        """(k, v, pages, lens, k_scale, v_scale) on the device, in the pool's layout."""
        def move(t):
            if t is None:
                return None
            if self.layout == "nhd":
                return t.transpose(1, 2).contiguous().to(dev).transpose(1, 2)
            return t.to(dev)
        return (move(self.k), move(self.v), self.pages.to(dev),
                torch.tensor(self.lens, dtype=torch.int32).to(dev), move(self.k_scale),
                move(self.v_scale))


def quantise(x):
    """uint8 codes and float32 scales of rows (last axis) of x, as the library defines them:
    s = amax / 448 and x / s in IEEE float32, rounded to nearest even."""
    x = x.float()
    amax = x.abs().amax(-1)
    s = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    return (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def attend(q, k, v, scale, visible):
    """One head in float64: q [n, d], k, v [m, d], visible [n] keys each.  Returns out, lse,
    the weighted mean of |v| (what roundings of the weights are relative to) and the largest
    sum of |q_i k_i| * scale over the visible pairs (what logit rounding is relative to)."""
    x = (q @ k.T) * scale
    seen = torch.arange(k.shape[0]) < visible[:, None]
    x = torch.where(seen, x, -math.inf)
    lse = torch.logsumexp(x, -1) if k.shape[0] else torch.full((q.shape[0],), -math.inf).double()
    w = torch.where(seen, torch.exp(x - torch.where(torch.isinf(lse), 0.0, lse)[:, None]), 0.0)
    mag = torch.where(seen, (q.abs() @ k.abs().T) * scale, 0.0)
    return w @ v, lse, w @ v.abs(), float(mag.max()) if mag.numel() else 0.0


def check(out, lse, ref, dtype, weights_dtype, n_keys, what=""):
    """Holds one head's results to the definition.  The bound: a float32 logit is off by at
    most e = 160 * 2^-24 of sum |q_i k_i| (up to 128 products added one after another, their
    scaling and the exponent's rounding), which moves every weight by a factor within
    1 +- 2.1 e, the sum of the weights included; each weight is rounded once to `weights_dtype`
    and summed in float32 (64 * 2^-24 for pairwise groups of keys); weights below the type's
    normal range are off by at most 2^-25 of the largest; the result is rounded once."""
    o, z, mean_abs, mag = ref
    e = 160 * 2.0 ** -24 * (mag + 1)
    rel = half_step(weights_dtype) + 4.2 * e + 64 * 2.0 ** -24
    tiny = n_keys * 2.0 ** -25
    bound = (half_step(dtype) * (1 + rel)) * o.abs() + rel * mean_abs + tiny * (mean_abs + 1) + 2.0 ** -24
    bad = (out.double() - o).abs() > bound
    assert not bool(bad.any()) and bool(torch.isfinite(out.double()).all()), \
        f"{what}: off by {((out.double() - o).abs() - bound).max().item()} over the bound"
    empty = torch.isinf(z)
    assert torch.equal(torch.isinf(lse.double()), empty) and bool((lse[empty] < 0).all()), what
    assert bool((out[empty] == 0).all()), what
    off = (lse.double() - z)[~empty].abs()
    lim = 2.1 * e + 2.0 ** -20 + 2.0 ** -22 * z[~empty].abs()
    assert bool((off <= lim).all()), f"{what}: lse off by {off.max().item()}"
