"""Plain 64-bit statements of the positioned append, tree attention, kept tokens, forks and page copies, on the caches
of paged_reference.  Nothing here uses the library."""
from __future__ import annotations

import math

import torch

from tests import paged_reference as R


def tree_rows(parents):
    """Sets of drafted tokens that each token of a tree sees (itself and what is above it), and depths."""
    rows, depths = [], []
    for t, p in enumerate(parents):
        rows.append({t} | (rows[p] if p >= 0 else set()))
        depths.append(depths[p] + 1 if p >= 0 else 0)
    return rows, depths


def words(rows, tokens):
    """Mask words [tokens, ceil(tokens / 32)] of one sequence's rows."""
    out = torch.zeros((tokens, -(-tokens // 32)), dtype=torch.int64)
    for t, row in enumerate(rows):
        for j in row:
            out[t, j // 32] |= 1 << (j % 32)
    return torch.where(out >= 1 << 31, out - (1 << 32), out).to(torch.int32)


def random_parents(tokens, g):
    u = torch.rand(tokens, generator=g)
    return [max(-1, t - 1 - int(u[t] * u[t] * (t + 1))) for t in range(tokens)]


def attention(cache, q, b, length, n, rows, window, sinks, scale=None):
    """(out, sum_j p_j |v_j|, largest sum_c |q_c k_jc|) of the n drafted tokens of sequence b, as
    paged_reference.attention gives them for a window.  rows[t]: the drafted tokens that query t sees."""
    hq, d = q.shape[1:]
    G = hq // cache.hkv
    scale = scale or 1.0 / math.sqrt(d)
    dev = q.device
    if n == 0 or length == 0:
        z = torch.zeros((n, hq, d), dtype=torch.float64, device=dev)
        return z, z, z[..., 0]
    ctx = length - n
    seen = torch.zeros((n, length), dtype=torch.bool)
    for t in range(n):
        mine = [j for j in rows[t] if j < n]
        depth = max(len(mine) - 1, 0)
        j = torch.arange(length)
        seen[t] = j < ctx
        if window is not None:
            seen[t] &= (j < sinks) | (j > ctx + depth - window)
        for x in mine:
            if ctx + x >= 0:
                seen[t, ctx + x] = True
    seen = seen.to(dev) & cache.good_tokens(b, length)[None]
    anybody = seen.any(0)
    zero = torch.zeros((), dtype=torch.float64, device=dev)
    k = torch.where(anybody[None, :, None], cache.wide(0, b, length), zero).repeat_interleave(G, 0)
    v = torch.where(anybody[None, :, None], cache.wide(1, b, length), zero).repeat_interleave(G, 0)
    x = q[:n].double().transpose(0, 1)
    s = (x @ k.transpose(1, 2) * scale).masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top.isinf(), torch.zeros_like(top), top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-300)
    size = (x.abs() @ k.abs().transpose(1, 2)).masked_fill(~seen, 0.0).amax(-1)
    return (p @ v).transpose(0, 1), (p @ v.abs()).transpose(0, 1), size.transpose(0, 1)


def rotate(x, table, positions, axes, interleaved):
    """x [n, H, d]; positions [axes][n]; axes[i]: the axis of pair i.  In 64 bits."""
    y = x.double().clone()
    half = table.shape[2]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        at = positions[axes[i]].long()
        cos, sin = table[at, 0, i].double()[:, None], table[at, 1, i].double()[:, None]
        y[..., a], y[..., b] = x[..., a].double() * cos - x[..., b].double() * sin, x[..., b].double() * cos + x[..., a].double() * sin
    return y


def e4m3(y):
    """Nearest E4M3 value of 64-bit numbers, ties to even, saturating."""
    mag = y.abs()
    exponent = torch.frexp(mag.clamp(min=1e-300)).exponent - 1
    step = torch.ldexp(torch.ones_like(mag), (exponent - 3).clamp(min=-9))
    return torch.copysign((torch.round(mag / step) * step).clamp(max=448.0), y) + 0.0


def stored(cache):
    """Pools and boxes in 64 bits as stored (E4M3: code values without the scale), scales."""
    r = {}
    for name, x in (("k", cache.k_pool), ("v", cache.v_pool), ("box", cache.bounds)):
        r[name] = (x.view(R.F8) if cache.dtype == "e4m3" else x).double()
    if cache.dtype == "e4m3":
        r["scales"] = cache.scales.double().clone()
    return r


def same(a, b):
    """Equal numbers, NaN where NaN."""
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def keep(cache, b, length, start, kept, r):
    """What r (as `stored` gives it) becomes when of sequence b's tokens those at start + kept move behind start.
    r["quotients"]: the same code values before their last rounding; r["touched"]: (page, its tokens) of the boxes."""
    P, table = cache.page, cache.table[b].tolist()
    touched = r.pop("touched", [])
    quotients = r.pop("quotients", {name: r[name].clone() for name in "kv"})
    before = {k: v.clone() for k, v in r.items()}
    end = start + len(kept)
    good = lambda page: 0 <= page < cache.count  # noqa: E731
    for page in range(start // P, -(-end // P)):
        at = table[page]
        if not good(at):
            continue
        lo, hi = page * P, min(end, page * P + P)
        for w, name in enumerate("kv"):
            old = before["scales"][at, :, w] if "scales" in r else None
            new, source = [], []
            for pos in range(lo, hi):
                src = pos if pos < start else start + kept[pos - start]
                sp = table[src // P]
                src_page = sp if good(sp) else at
                src_slot = src % P if good(sp) else pos % P
                new.append(before[name][src_page, :, src_slot])
                source.append(src_page)
            new = torch.stack(new, 1)                                # [hkv, rows, d]
            if "scales" in r:
                step = torch.stack([before["scales"][s, :, w] for s in source], 1)
                other = torch.tensor([s != at for s in source], device=new.device)
                top = torch.where(other, (new * step[..., None] / 448.0).abs().amax(-1), torch.zeros_like(step)).amax(1)
                amax = torch.maximum(old, top)
                ratio = (torch.where(other, step, old[:, None]) / amax.clamp(min=1e-300)[:, None])[..., None]
                quotients[name][at, :, :hi - lo] = new * ratio
                new = torch.where(ratio == 1, new, e4m3(new * ratio))
                r["scales"][at, :, w] = amax
            r[name][at, :, :hi - lo] = new
            if w == 0:
                r["box"][at, :, 0], r["box"][at, :, 1] = new.amin(1), new.amax(1)
                touched.append((at, hi - lo))
    r["touched"], r["quotients"] = touched, quotients
    return r
