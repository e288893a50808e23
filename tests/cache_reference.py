"""The cache's and the attention's definitions in 64 bits, one row at a time.

Shares no code with the package: e4m3 is decoded from its bit fields and
encoded by rounding to its steps.
"""
import math

import torch

F8_MAX = 448.0


def e4m3_values() -> torch.Tensor:
    c = torch.arange(256)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e.double() - 10))
    v[127] = v[255] = math.nan
    v[128:] = -v[128:]
    return v


VALUES = e4m3_values()


def encode(y: torch.Tensor) -> torch.Tensor:
    """Nearest e4m3 value, ties to even, saturated; NaN -> 0."""
    y = torch.nan_to_num(y.double(), nan=0.0, posinf=F8_MAX, neginf=-F8_MAX).clamp(-F8_MAX, F8_MAX)
    _, x = torch.frexp(y)                       # |y| in [2^(x-1), 2^x)
    step = torch.exp2((x.double() - 1).clamp(min=-6) - 3)
    return (torch.round(y / step) * step).clamp(-F8_MAX, F8_MAX)


def scale_of(x: torch.Tensor) -> float:
    """Smallest 2^e, e in [-48, 48], with |finite x| <= 448 2^e."""
    a = x.double().abs()
    a = a[torch.isfinite(a)]
    top = float(a.max()) if a.numel() else 0.0
    e = -48
    while e < 48 and top > F8_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Cache:
    """The state of one layer: values (64 bits) per page, head and slot, and scales."""

    def __init__(self, pages, heads, page, dim):
        self.x = {n: torch.zeros(pages, heads, page, dim, dtype=torch.float64) for n in "kv"}
        self.s = {n: torch.ones(pages, heads, dtype=torch.float64) for n in "kv"}
        self.page, self.heads = page, heads

    def write(self, new, table, lens, counts):
        """new: {"k", "v"} of [N, heads, dim], packed."""
        at = 0
        for b, (n, c) in enumerate(zip(lens, counts)):
            start = n - c
            for pg in range(start // self.page, (n - 1) // self.page + 1 if c else 0):
                lo, hi = max(start, pg * self.page), min(n, (pg + 1) * self.page)
                s0, s1 = lo - pg * self.page, hi - pg * self.page
                page = int(table[b][pg])
                for name in "kv":
                    fresh = new[name][at + lo - start:at + hi - start].double().transpose(0, 1)
                    for h in range(self.heads):
                        x = torch.cat([self.x[name][page, h, :s0], fresh[h]])
                        s = scale_of(x)
                        self.x[name][page, h, :s1] = encode(x / s) * s
                        self.s[name][page, h] = s
            at += c

    def rows(self, name, table_row, lo, hi):
        """Positions lo..hi of a row: [hi - lo, heads, dim]."""
        j = torch.arange(lo, hi)
        pages = torch.as_tensor(table_row)[j // self.page].long()
        return self.x[name][pages, :, j % self.page]


def attend(q, k, v, first, scale, window=0, sinks=0):
    """q [T, heads, group, dim] at positions first, first + 1, ..; k, v [n, heads, dim].
    Returns the result and sum_j p_j |v_j|, which bounds what rounding p does."""
    z = torch.einsum("thgd,jhd->thgj", q.double(), k) * scale
    p, j = torch.arange(first, first + q.shape[0])[:, None], torch.arange(k.shape[0])[None]
    see = j <= p
    if window:
        see &= (j > p - window) | (j < sinks)
    z = z.masked_fill(~see[:, None, None, :], -math.inf)
    w = torch.softmax(z, -1)
    return torch.einsum("thgj,jhd->thgd", w, v), torch.einsum("thgj,jhd->thgd", w, v.abs())
