"""The cache with a scale for each block of 16 tokens and head, from its
definition, in numpy (tests only): values in 64 bits, codes kept as the numbers
they stand for."""
import numpy as np
import torch

BLOCK = 16
TOP = {"e4m3fn": 448.0, "e5m2": 57344.0}
TORCH = {"e4m3fn": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "bf16": torch.bfloat16, "f16": torch.float16,
         "f32": torch.float32}


def grid(x, fmt):
    """x to the nearest number of the type, ties to even, saturating; NaN stays."""
    bits, low = {"e4m3fn": (3, -6), "e5m2": (2, -14)}[fmt]
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        clipped = np.clip(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300), -2 * TOP[fmt], 2 * TOP[fmt])
        e = np.maximum(np.frexp(clipped)[1] - 1, low)
        unit = np.ldexp(1.0, e - bits)
        out = np.clip(np.rint(clipped / unit) * unit, -TOP[fmt], TOP[fmt])
    return np.where(np.isnan(x), np.nan, out)


def times(x, by, fmt):
    """Codes of x * by, the product rounded to fp32 first (x holds fp32 numbers)."""
    with np.errstate(invalid="ignore", over="ignore", under="ignore"):
        return grid((np.asarray(x, np.float32) * np.float32(by)).astype(np.float64), fmt)


def own_scale(x, fmt):
    """The block's scale from its new values: the smallest 2^k >= 2^-64 with amax <= TOP 2^k, by trying."""
    x = np.abs(np.asarray(x, np.float64))
    amax = np.max(np.where(np.isfinite(x), x, 0.0), initial=0.0)
    k = -64
    while amax > TOP[fmt] * 2.0 ** k:
        k += 1
    return 2.0 ** k


class Cache:
    """K (or V) of a pool as numbers [pages, page_size, heads, d] with scales [pages, page_size / 16, heads]."""

    def __init__(self, values, scales, fmt):
        self.values, self.scales = (np.array(np.asarray(x), np.float64) for x in (values, scales))
        self.fmt = fmt

    def append(self, x, qo_indptr, cached, kv_indptr, kv_indices):
        ps = self.values.shape[1]
        for b, c in enumerate(cached):
            r0, r1 = qo_indptr[b], qo_indptr[b + 1]
            pos = c
            while r0 < r1:
                m = min(BLOCK - pos % BLOCK, r1 - r0)
                page, slot = kv_indices[kv_indptr[b] + pos // ps], pos % ps
                first, blk = slot // BLOCK * BLOCK, slot // BLOCK
                for h in range(self.values.shape[2]):
                    rows = np.asarray(x[r0:r0 + m, h], np.float64)
                    s = own_scale(rows, self.fmt)
                    if slot > first:
                        old = self.scales[page, blk, h]
                        s = max(s, old)
                        if s > old:
                            self.values[page, first:slot, h] = times(self.values[page, first:slot, h], np.float32(old) / np.float32(s),
                                                                     self.fmt)
                    self.values[page, slot:slot + m, h] = times(rows, np.float32(1) / np.float32(s), self.fmt)
                    self.scales[page, blk, h] = s
                r0, pos = r0 + m, pos + m


def as_tokens(cache, layout):
    """A torch cache in either layout as numbers [pages, page_size, heads, d]."""
    x = cache.double().cpu().numpy()
    return x if layout == "NHD" else x.transpose(0, 2, 1, 3)


def raw(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def in_layout(x, layout):
    """[pages, page_size, heads, d] codes in the layout's order."""
    return x if layout == "NHD" else raw(x).transpose(1, 2).contiguous().view(x.dtype)


def table(lens, page_size, gen, spare=3):
    """A page table of shuffled pages: (kv_indptr, kv_indices, pool)."""
    n = [-(-x // page_size) for x in lens]
    ptr = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
    pool = int(ptr[-1]) + spare
    return ptr, torch.randperm(pool, generator=gen)[:ptr[-1]].numpy(), pool


def random_cache(pool, page_size, heads, d, fmt, gen, powers=True):
    """Codes [pages, page_size, heads, d] with scales of unlike size; powers of two, or any."""
    s = 2.0 ** torch.randint(-12, 4, (pool, page_size // BLOCK, heads), generator=gen).float()
    if not powers:
        s = s * (1 + torch.rand(s.shape, generator=gen))
    x = torch.randn(pool, page_size, heads, d, generator=gen) * (TOP[fmt] / 6)
    return x.clamp(-TOP[fmt], TOP[fmt]).to(TORCH[fmt]), s
