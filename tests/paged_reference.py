"""Plain 64-bit statements of the rotating append and of windowed attention, and
paged caches to run them on, for the parity tests.  Nothing here uses the library.

A cache starts poisoned: slots and boxes that no token has hold NaN (E4M3: the NaN
code), block-table entries that no call may read hold an id far out of range.
"""
from __future__ import annotations

import math

import torch

POOL = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.uint8}
VALUE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float16}
F8 = torch.float8_e4m3fn
BAD_PAGE = 1 << 30


def half_step(dtype: torch.dtype) -> float:
    """Largest relative error of one rounding to the type."""
    return torch.finfo(dtype).eps / 2


class Paged:
    """A paged cache of sequences of the given lengths, with room for `reserve` more tokens each."""

    def __init__(self, dtype, lens, hkv, d, page, seed=0, reserve=0, device="cuda", amax_spread=0.0):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.dtype, self.lens, self.hkv, self.d, self.page, self.device = dtype, list(lens), hkv, d, page, device
        pages = [max(0, -(-(L + reserve) // page)) for L in self.lens]
        width = max(1, max(pages, default=1)) + 1
        count = sum(pages) + 3
        order = torch.randperm(count, generator=g)
        table = torch.full((len(self.lens), width), BAD_PAGE, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        self.count = count
        kv = torch.full((2, count, hkv, page, d), 0x7F if dtype == "e4m3" else float("nan"), dtype=POOL[dtype])
        bounds = torch.full((count, hkv, 2, d), 0x7F if dtype == "e4m3" else float("nan"), dtype=POOL[dtype])
        scales = torch.full((count, hkv, 4), float("nan")) if dtype == "e4m3" else None
        for b, L in enumerate(self.lens):
            for i in range(-(-L // page)):
                at, rows = int(table[b, i]), min(page, L - i * page)
                for w in range(2):
                    x = torch.randn((hkv, rows, d), generator=g)
                    if dtype == "e4m3":
                        if amax_spread:
                            x = x * math.exp(amax_spread * (2 * float(torch.rand((), generator=g)) - 1))
                        amax = x.abs().amax(dim=(1, 2))
                        scales[at, :, w] = amax
                        code = (x / (amax / 448.0)[:, None, None]).to(F8).view(torch.uint8)
                        kv[w, at, :, :rows] = torch.where(code == 0x80, torch.zeros_like(code), code)
                    else:
                        kv[w, at, :, :rows] = x.to(POOL[dtype])
                    if w == 0:
                        keys = kv[0, at, :, :rows]
                        keys = (keys.view(F8) if dtype == "e4m3" else keys).float()
                        box = torch.stack((keys.amin(1), keys.amax(1)), 1)
                        bounds[at] = box.to(F8).view(torch.uint8) if dtype == "e4m3" else box.to(POOL[dtype])
        kv = kv.to(device)
        self.k_pool, self.v_pool = kv[0], kv[1]
        self.bounds = bounds.to(device)
        self.scales = scales.to(device) if scales is not None else None
        self.table = table.to(device)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)

    def library(self):
        from query_aware_sparse_append_gb300 import binding as qasa
        return qasa.PagedKVCache(self.k_pool, self.v_pool, self.bounds, self.scales)

    def wide(self, which: int, b: int, length: int) -> torch.Tensor:
        """Keys (0) or values (1) of sequence b in 64 bits, [hkv, length, d]; bad pages are zeros."""
        ids = self.table[b, :-(-length // self.page)].long()
        good = (ids >= 0) & (ids < self.count)
        ids = torch.where(good, ids, torch.zeros_like(ids))
        pool = (self.k_pool, self.v_pool)[which][ids]
        if self.dtype == "e4m3":
            x = pool.view(F8).double() * (self.scales[ids][:, :, which].double() / 448.0)[:, :, None, None]
        else:
            x = pool.double()
        x = torch.where(good[:, None, None, None], x, torch.zeros_like(x))
        return x.transpose(0, 1).reshape(self.hkv, -1, self.d)[:, :length]

    def good_tokens(self, b: int, length: int) -> torch.Tensor:
        ids = self.table[b, :-(-length // self.page)].long()
        return ((ids >= 0) & (ids < self.count)).repeat_interleave(self.page)[:length]


def attention(cache: Paged, q: torch.Tensor, b: int, length: int, n: int, window, sinks: int, scale=None):
    """(out, sum_j p_j |v_j|, largest sum_c |q_c k_jc| of a visible token) of the newest n tokens of sequence b,
    in 64 bits, [n, hq, d], [n, hq, d] and [n, hq].  q [T, hq, d]."""
    hq, d = q.shape[1:]
    G = hq // cache.hkv
    scale = scale or 1.0 / math.sqrt(d)
    dev = q.device
    if n == 0 or length == 0:
        z = torch.zeros((n, hq, d), dtype=torch.float64, device=dev)
        return z, z, z[..., 0]
    i = torch.arange(length - n, length, device=dev)[:, None]
    j = torch.arange(length, device=dev)[None, :]
    seen = j <= i
    if window is not None:
        seen &= (j < sinks) | (j > i - window)
    seen &= cache.good_tokens(b, length)[None]
    anybody = seen.any(0)
    k = torch.where(anybody[None, :, None], cache.wide(0, b, length), torch.zeros((), dtype=torch.float64, device=dev))
    v = torch.where(anybody[None, :, None], cache.wide(1, b, length), torch.zeros((), dtype=torch.float64, device=dev))
    k, v = k.repeat_interleave(G, 0), v.repeat_interleave(G, 0)
    x = q[:n].double().transpose(0, 1)
    s = (x @ k.transpose(1, 2) * scale).masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top.isinf(), torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    size = (x.abs() @ k.abs().transpose(1, 2)).masked_fill(~seen, 0.0).amax(-1)
    return (p @ v).transpose(0, 1), (p @ v.abs()).transpose(0, 1), size.transpose(0, 1)


def attention_tolerance(out, weighed, size, d, dtype: torch.dtype, scale=None):
    """|error| allowed of an output in `dtype`: its own rounding, one rounding of the weights to the type and one
    of E4M3 values times their scale (2 u of sum p |v|), and what the scores are off by, which moves every weight by
    that share: d products summed in fp32 in any order, 2^-23 each for the adder and the scaling, twice (numerator
    and denominator), and 2^-20 for the exponential of either."""
    u = half_step(dtype)
    off = (scale or 1.0 / math.sqrt(d)) * size * (d + 4) * 2.0 ** -23
    return u * out.abs() + (2 * u + 2 * off[..., None] + 2.0 ** -20) * weighed + 2.0 ** -24


def rotate(x: torch.Tensor, table: torch.Tensor, first: int, interleaved: bool) -> torch.Tensor:
    """x [n, H, d] at positions first .. in 64 bits."""
    half = table.shape[2]
    cs = table[first:first + x.shape[0]].double()
    cos, sin = cs[:, None, 0], cs[:, None, 1]
    y = x.double().clone()
    a = y[..., 0:2 * half:2] if interleaved else y[..., :half]
    b = y[..., 1:2 * half:2] if interleaved else y[..., half:2 * half]
    ya, yb = a * cos - b * sin, b * cos + a * sin
    a.copy_(ya)
    b.copy_(yb)
    return y
