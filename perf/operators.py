"""Cases, plain forms and exact values of two operators on the paged KV cache.

append   new keys and values go into their pages with the position rotation applied on the way, the page
         boxes (and, for E4M3 pages, the scales) kept current, and the new queries are rotated by the same call
attend   attention of the newest tokens of every sequence over the paged cache with a sliding window and a few
         first tokens that stay visible

Every case is a dict of plain values.  Sequence lengths come from the case alone, values from the seed.
"""
import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
# type of q, the outputs and the appended values; E4M3 caches take and give f16
VALUE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float16}
POOL = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.uint8}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
NO_WINDOW = 0      # a case's window of 0: every earlier token is visible


def listed():
    return [
        # One decode step's append of the library's smallest workload (one sequence, one token): call latency.
        dict(name="append 1x1 f32", op="append", dtype="f32", batch=1, tokens=1, min_tokens=1, hq=4, hkv=4, d=64,
             page=16, ctx_min=2047, ctx_max=2047, rot=64, interleaved=False),
        # The append of one decode step of a full serving batch, lengths all over the page.
        dict(name="append 128x1 f16", op="append", dtype="f16", batch=128, tokens=1, min_tokens=1, hq=32, hkv=4, d=128,
             page=16, ctx_min=15, ctx_max=500, rot=128, interleaved=False),
        # Long prompt chunks of two sequences that continue in the middle of a page; pairs of neighbouring channels.
        dict(name="append 2x4096 bf16", op="append", dtype="bf16", batch=2, tokens=4096, min_tokens=4096, hq=32, hkv=8,
             d=128, page=32, ctx_min=37, ctx_max=4101, rot=128, interleaved=True),
        # Ragged prompts into an E4M3 cache, part of them continuing pages that have to be requantised.
        dict(name="append 16x1024 e4m3", op="append", dtype="e4m3", batch=16, tokens=1024, min_tokens=1, hq=32, hkv=4,
             d=128, page=16, ctx_min=0, ctx_max=700, rot=64, interleaved=False),
        # Decode step of the smallest workload with a window: one sequence, latency.
        dict(name="decode 1 f32", op="attend", dtype="f32", batch=1, tokens=1, min_tokens=1, hq=4, hkv=4, d=64, page=16,
             ctx_min=2048, ctx_max=2048, window=512, sinks=4),
        # Decode step of a ragged serving batch on a windowed layer: lengths below and far above the window.
        dict(name="decode 128 f16 window", op="attend", dtype="f16", batch=128, tokens=1, min_tokens=1, hq=32, hkv=4,
             d=128, page=16, ctx_min=512, ctx_max=16384, window=1024, sinks=4),
        # Decode step over long contexts with every token visible.
        dict(name="decode 8x32k bf16", op="attend", dtype="bf16", batch=8, tokens=1, min_tokens=1, hq=32, hkv=8, d=128,
             page=32, ctx_min=32768, ctx_max=32768, window=NO_WINDOW, sinks=0),
        # Decode step over an E4M3 cache with a wide window and a page of sinks.
        dict(name="decode 128 e4m3 window", op="attend", dtype="e4m3", batch=128, tokens=1, min_tokens=1, hq=32, hkv=4,
             d=128, page=16, ctx_min=8192, ctx_max=8192, window=4096, sinks=16),
        # Five drafted tokens of each sequence verified in one call.
        dict(name="verify 16x5 f16", op="attend", dtype="f16", batch=16, tokens=5, min_tokens=5, hq=32, hkv=4, d=64,
             page=16, ctx_min=3900, ctx_max=4101, window=1024, sinks=4),
        # A long prompt in one piece on a windowed layer.
        dict(name="prompt 1x8192 bf16", op="attend", dtype="bf16", batch=1, tokens=8192, min_tokens=8192, hq=32, hkv=8,
             d=128, page=32, ctx_min=8192, ctx_max=8192, window=4096, sinks=4),
        # Ragged prompts of a batch, every earlier token visible, as many KV heads as query heads.
        dict(name="prompts 16x1024 f16", op="attend", dtype="f16", batch=16, tokens=1024, min_tokens=256, hq=16, hkv=16,
             d=64, page=16, ctx_min=0, ctx_max=0, window=NO_WINDOW, sinks=0),
        # A prompt chunk that continues a long E4M3 cache on a windowed layer.
        dict(name="chunk 2x2048 e4m3", op="attend", dtype="e4m3", batch=2, tokens=2048, min_tokens=2048, hq=32, hkv=4,
             d=128, page=16, ctx_min=8000, ctx_max=8192, window=1024, sinks=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["f32", "f16", "f16", "bf16", "bf16", "e4m3"])
    hkv = rng.choice([1, 2, 4, 8, 16])
    group = rng.choice([1, 2, 3, 4, 6, 8]) if hkv <= 8 else rng.choice([1, 2])
    d, page = rng.choice([64, 128]), rng.choice([16, 32])
    c = dict(dtype=dtype, hq=hkv * group, hkv=hkv, d=d, page=page)
    if rng.random() < 0.35:
        tokens = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4096)
        # no more values than the largest listed case moves
        most = (8192 * 48 * 128) // (tokens * (hkv * group + 2 * hkv) * d * (2 if dtype == "f32" else 1))
        batch = _log_int(rng, 1, max(1, min(160, most)))
        ctx = _log_int(rng, 1, 2000)
        return dict(op="append", batch=batch, tokens=tokens, min_tokens=rng.choice([1, tokens]),
                    ctx_min=rng.choice([0, ctx]), ctx_max=ctx, rot=rng.choice([16, 32, 64, d]),
                    interleaved=rng.random() < 0.4, **c)
    form = rng.choice(["decode", "verify", "prompt"])
    tokens = 1 if form == "decode" else rng.randint(2, 16) if form == "verify" else _log_int(rng, 17, 4096)
    if dtype == "f32":
        tokens = min(tokens, 512)
    ctx = tokens + (0 if form == "prompt" and rng.random() < 0.5 else _log_int(rng, 1, 16384))
    # no more work than the largest listed case has, and K and V below 2 GiB in all
    most = 8192 * 4096 * 32 * 128 // (tokens * hkv * group * d)
    ctx = max(tokens, min(ctx, most))
    batch = max(1, min(_log_int(rng, 1, 128), most // ctx, (1 << 30) // (ctx * hkv * d * 2)))
    window = NO_WINDOW if rng.random() < 0.3 else _log_int(rng, 16, 8192)
    return dict(op="attend", batch=batch, tokens=tokens, min_tokens=rng.choice([1, tokens]) if tokens > 1 else 1,
                ctx_min=rng.choice([tokens, ctx]), ctx_max=ctx, window=window,
                sinks=rng.choice([0, 1, 4, 16, 100]) if window else 0, **c)


def _spread(lo, hi, n, step):
    """n whole numbers spread over lo .. hi, the last of them hi."""
    x = np.mod(np.arange(1, n + 1) * step, 1.0)
    v = lo + np.floor(x * (hi - lo + 1)).astype(np.int64)
    v[-1] = hi
    return v


def _lengths(case):
    """(tokens in the cache before the call, new tokens) of every sequence; an attend case's lengths include the
    new tokens, a context of 0 standing for prompts that are all there is."""
    n = _spread(case["min_tokens"], case["tokens"], case["batch"], 0.7548776662466927)
    ctx = _spread(case["ctx_min"], case["ctx_max"], case["batch"], 0.6180339887498949)
    if case["op"] == "attend":
        ctx = np.maximum(ctx, n)
    return ctx, n


def _first_visible(case, lens, n):
    """First position in the window of the oldest query."""
    if case["window"] == NO_WINDOW:
        return np.zeros_like(lens)
    return np.maximum(lens - n - case["window"] + 1, 0)


def work(case):
    ctx, n = _lengths(case)
    es = SIZE[case["dtype"]]
    ev = 2 if case["dtype"] == "e4m3" else es
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    if case["op"] == "append":
        rows = int(n.sum())
        touched = int(((ctx + n - 1) // page - ctx // page + 1).sum())
        kept = int((ctx % page != 0).sum())           # pages whose box (and scale) is read back too
        moved = rows * ((hq + 2 * hkv) * d * ev + hq * d * ev + 2 * hkv * d * es)
        boxes = (touched + kept) * hkv * (2 * d * es + (8 if case["dtype"] == "e4m3" else 0))
        positions = len(np.unique(np.concatenate([np.arange(a, a + m) for a, m in zip(ctx, n)])))
        return {"bytes": moved + boxes + positions * case["rot"] * 4 + touched * 4 + 4 * len(n),
                "flops": rows * (hq + hkv) * case["rot"] * 3}
    first = ctx - n
    pairs = keys = pages = 0
    for L, m, a in zip(ctx.tolist(), n.tolist(), first.tolist()):
        i = np.arange(a, a + m)
        w = case["window"] if case["window"] else L + 1
        start = np.maximum(i - w + 1, 0)
        s = np.minimum(case["sinks"], i + 1)
        pairs += int((i + 1 - start + np.minimum(s, start)).sum())
        lo = int(start[0])
        head = min(case["sinks"], lo)
        keys += L - lo + head
        pages += (L - 1) // page - lo // page + 1 + -(-head // page)
    scales = pages * hkv * 8 if case["dtype"] == "e4m3" else 0
    return {"bytes": 2 * int(n.sum()) * hq * d * ev + 2 * keys * hkv * d * es + scales + pages * 4,
            "flops": 4 * d * hq * pairs}


def _table(case, positions, device):
    """cos and sin of every position's angles, [positions, 2, rot / 2] in 32 bits, from angles in 64 bits."""
    half = case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], dim=1).float().contiguous()


def _quantise(x):
    """E4M3 codes and amax of each tile x [..., page, d], as an append into an empty page stores it."""
    amax = x.abs().amax(dim=(-2, -1))
    s = amax / 448.0
    y = torch.where(s[..., None, None] > 0, x / s[..., None, None], torch.zeros_like(x))
    code = y.to(F8).view(torch.uint8)
    return torch.where(code == 0x80, torch.zeros_like(code), code), amax


def _boxes(pool, valid):
    """Boxes of pages with the given numbers of valid slots (an empty page's is 0)."""
    page = pool.shape[2]
    keys = (pool.view(F8) if pool.dtype == torch.uint8 else pool).float()
    inside = (torch.arange(page, device=pool.device) < valid[:, None])[:, None, :, None]
    lo = keys.masked_fill(~inside, math.inf).amin(2)
    hi = keys.masked_fill(~inside, -math.inf).amax(2)
    box = torch.stack([lo, hi], 2)
    box = torch.where(box.isinf(), torch.zeros_like(box), box)
    return box.to(F8).view(torch.uint8) if pool.dtype == torch.uint8 else box.to(pool.dtype)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    ctx, n = _lengths(case)
    B, T, hq, hkv, d, P = (case[k] for k in ("batch", "tokens", "hq", "hkv", "d", "page"))
    value, pool_type = VALUE[case["dtype"]], POOL[case["dtype"]]
    end = ctx + n if case["op"] == "append" else ctx
    width = max(1, int(-(-end.max() // P)))
    page_ids = np.arange(width)[None, :]
    used = page_ids < -(-end // P)[:, None]
    if case["op"] == "attend":     # pages that no query can see any more have been given back
        seen = page_ids >= (_first_visible(case, ctx, n) // P)[:, None]
        used &= seen | (page_ids < -(-case["sinks"] // P))
    count = int(used.sum()) + 1    # one page belongs to nobody
    order = torch.randperm(count - 1, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    table[torch.from_numpy(used).to(dev)] = order

    # K and V in one allocation; stale values in the slots that no token has
    pools = []
    scales = torch.zeros((count, hkv, 4), dtype=torch.float32, device=dev) if case["dtype"] == "e4m3" else None
    kv = torch.empty((2, count, hkv, P, d), dtype=pool_type, device=dev)
    for i in range(2):
        if case["dtype"] == "e4m3":
            step = 1 << 12
            for a in range(0, count, step):
                x = torch.randn((min(step, count - a), hkv, P, d), generator=g, device=dev)
                kv[i, a:a + step], scales[a:a + step, :, i] = _quantise(x)
        else:
            kv[i].normal_(generator=g)
        pools.append(kv[i])
    s = {"case": case, "k_pool": pools[0], "v_pool": pools[1], "scales": scales, "block_table": table,
         "seq_lens": torch.from_numpy(ctx.astype(np.int32)).to(dev),
         "new_lens": torch.from_numpy(n.astype(np.int32)).to(dev)}
    if case["op"] == "append":
        filled = np.clip(ctx[:, None] - page_ids * P, 0, P)
        valid = torch.zeros(count, dtype=torch.int64, device=dev)
        valid[order.long()] = torch.from_numpy(filled[used]).to(dev)
        s["bounds"] = _boxes(pools[0], valid)
        # one projection's output holds the queries, keys and values of every new token
        qkv = torch.randn((B, T, (hq + 2 * hkv) * d), generator=g, device=dev).to(value)
        heads = qkv.view(B, T, hq + 2 * hkv, d)
        s["q"], s["k_new"], s["v_new"] = heads[:, :, :hq], heads[:, :, hq:hq + hkv], heads[:, :, hq + hkv:]
        s["q_out"] = torch.zeros((B, T, hq, d), dtype=value, device=dev)
        s["table"] = _table(case, width * P, dev)
        s["lens"] = s["new_lens"] if case["min_tokens"] < T else None
    else:
        s["bounds"] = torch.zeros((count, hkv, 2, d), dtype=pool_type, device=dev)
        s["q"] = torch.randn((B, T, hq, d), generator=g, device=dev).to(value)
        s["out"] = torch.zeros((B, T, hq, d), dtype=value, device=dev)
        s["lens"] = s["new_lens"] if case["min_tokens"] < T else None
    if own:
        from query_aware_sparse_append_gb300 import binding as qasa
        s["qasa"] = qasa
        s["cache"] = qasa.PagedKVCache(s["k_pool"], s["v_pool"], s["bounds"], scales)
        if case["op"] == "attend":
            s["window"] = case["window"] or None
            s["workspace"] = qasa.alloc_window_workspace(s["cache"], B, hq, T, width, window=s["window"],
                                                         sink_tokens=case["sinks"])
    return s


def run(s):
    if s["case"]["op"] == "append":
        if own:
            s["qasa"].kv_append_rotated(s["cache"], s["block_table"], s["seq_lens"], s["k_new"], s["v_new"], s["table"],
                                        q=s["q"], q_out=s["q_out"], append_lens=s["lens"],
                                        interleaved=s["case"]["interleaved"])
        else:
            _append_plain(s)
        eight = s["scales"] is not None
        r = {"q": s["q_out"]}
        for name in ("k_pool", "v_pool", "bounds"):
            r[name] = s[name].view(F8) if eight else s[name]
        if eight:
            r["scales"] = s["scales"]
        return r
    if own:
        return s["qasa"].window_attention(s["cache"], s["q"], s["block_table"], s["seq_lens"], window=s["window"],
                                          sink_tokens=s["case"]["sinks"], q_lens=s["lens"], out=s["out"],
                                          workspace=s["workspace"])
    return _attend_plain(s)


# ---------------------------------------------------------------- plain forms

def _rotate_plain(x, table, pos, interleaved):
    """x [B, T, H, d] rotated, in 64 bits, rounded to 32."""
    half = table.shape[2]
    cs = table[pos].double()
    cos, sin = cs[:, :, None, 0], cs[:, :, None, 1]
    rot, rest = x[..., :2 * half].double(), x[..., 2 * half:].double()
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rot[..., :half], rot[..., half:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1).float()


def _append_plain(s):
    case = s["case"]
    P, d = case["page"], case["d"]
    B, T, hkv = s["k_new"].shape[:3]
    dev = s["q"].device
    L, n = s["seq_lens"].long(), s["new_lens"].long()
    t = torch.arange(T, device=dev)
    live = t < n[:, None]
    pos = torch.where(live, L[:, None] + t, torch.zeros_like(live, dtype=torch.int64))
    value = s["q"].dtype
    q = _rotate_plain(s["q"], s["table"], pos, case["interleaved"]).to(value)
    s["q_out"].copy_(torch.where(live[:, :, None, None], q, s["q_out"]))

    # the touched pages of every sequence as tiles [B, pages, hkv, P, d]; what no token goes to is put back as it was,
    # pages that a sequence does not touch stand for the page that belongs to nobody
    pages = (T + P - 1) // P + 1
    first = L // P
    logical = first[:, None] + torch.arange(pages, device=dev)
    touched = logical <= ((L + n - 1) // P)[:, None]
    width = s["block_table"].shape[1]
    phys = s["block_table"].long().gather(1, logical.clamp(max=width - 1))
    phys = torch.where(touched, phys, torch.full_like(phys, s["k_pool"].shape[0] - 1))
    slot_pos = logical[:, :, None] * P + torch.arange(P, device=dev)
    index = slot_pos - L[:, None, None]
    new = (index >= 0) & (index < n[:, None, None])
    fresh = (logical * P >= L[:, None])[:, :, None]                        # slot 0 is written by this call
    mask = new[:, :, None, :, None]
    at = index.clamp(0, T - 1).flatten(1)[:, :, None, None].expand(-1, -1, hkv, d)
    rows = {"k_pool": _rotate_plain(s["k_new"], s["table"], pos, case["interleaved"]), "v_pool": s["v_new"].float()}
    for which, name in enumerate(("k_pool", "v_pool")):
        x = rows[name].gather(1, at).view(B, pages, P, hkv, d).transpose(2, 3)
        old = s[name][phys]
        box = s["bounds"][phys]
        if s["scales"] is None:
            x = x.to(value)
            lo_hi = box.float()
        else:
            before = torch.where(fresh, torch.zeros((), device=dev), s["scales"][phys][..., which])
            top = x.abs().masked_fill(~mask, 0).amax(dim=(-2, -1))
            amax = torch.maximum(before, top)
            s_old, s_new = before / 448.0, amax / 448.0
            grown = (amax > before) & ~fresh

            def code(v, s_new=s_new):
                sc = s_new[..., None, None]
                c = torch.where(sc > 0, v / sc, torch.zeros_like(v)).to(F8).view(torch.uint8)
                return torch.where(c == 0x80, torch.zeros_like(c), c)

            def again(c, s_old=s_old, grown=grown):
                return torch.where(grown[..., None, None], code(c.view(F8).float() * s_old[..., None, None]), c)

            kept = slot_pos[:, :, None, :, None] < L[:, None, None, None, None]
            old = torch.where(kept, again(old), old)
            x = code(x)
            if which == 0:
                lo_hi = again(box).view(F8).float()
            s["scales"][phys.flatten(), :, which] = torch.where(touched[:, :, None], amax,
                                                                s["scales"][phys][..., which]).flatten(0, 1)
        s[name][phys.flatten()] = torch.where(mask, x, old).flatten(0, 1)
        if which == 0:
            keys = (x.view(F8) if s["scales"] is not None else x).float()
            none = fresh[..., None]
            lo = torch.minimum(keys.masked_fill(~mask, math.inf).amin(3), lo_hi[..., 0, :].masked_fill(none, math.inf))
            hi = torch.maximum(keys.masked_fill(~mask, -math.inf).amax(3), lo_hi[..., 1, :].masked_fill(none, -math.inf))
            folded = torch.stack([lo, hi], 3)
            folded = folded.to(F8).view(torch.uint8) if s["scales"] is not None else folded.to(value)
            s["bounds"][phys.flatten()] = torch.where(touched[:, :, None, None, None], folded, box).flatten(0, 1)


def _attend_plain(s):
    case = s["case"]
    P, d, hkv = case["page"], case["d"], case["hkv"]
    B, T, hq = s["q"].shape[:3]
    G, dev = hq // hkv, s["q"].device
    L, n = s["seq_lens"].long(), s["new_lens"].long()
    longest = s["block_table"].shape[1] * P
    window = min(case["window"] or longest, longest)
    # the columns that some query of the sequence can see: the window of all its queries, and the sinks before that
    span = min(window + T - 1, longest)
    start = (L - n - window + 1).clamp(min=0)
    sink = torch.arange(case["sinks"], device=dev).expand(B, -1)
    pos = torch.cat([sink, start[:, None] + torch.arange(span, device=dev)], 1)
    inside = pos < L[:, None]
    inside[:, :case["sinks"]] &= sink < start[:, None]
    pos = torch.where(inside, pos, torch.zeros_like(pos))
    phys = s["block_table"].long().gather(1, pos // P).clamp(min=0)
    slot = pos % P

    def rows(pool, which):
        x = pool[phys, :, slot]                                             # [B, M, hkv, d]
        if s["scales"] is not None:
            x = x.view(F8).float() * (s["scales"][phys][..., which] / 448.0)[..., None]
        x = x.float().masked_fill(~inside[:, :, None, None], 0)
        return x.transpose(1, 2)                                            # [B, hkv, M, d]

    q = s["q"].float().view(B, T, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, T * G, d)
    scores = torch.matmul(q, rows(s["k_pool"], 0).transpose(2, 3)) / math.sqrt(d)
    i = (L - n)[:, None] + torch.arange(T, device=dev)
    j = pos[:, None, :]
    seen = inside[:, None, :] & (j <= i[:, :, None]) & ((j < case["sinks"]) | (j > i[:, :, None] - window))
    hidden = ~seen[:, None, :, None, :].expand(-1, -1, -1, G, -1).reshape(B, 1, T * G, -1)
    scores = scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top.isinf(), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows(s["v_pool"], 1)) / torch.where(total > 0, total, torch.ones_like(total))
    out = out.view(B, hkv, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, hq, d).to(s["q"].dtype)
    live = torch.arange(T, device=dev) < n[:, None]
    s["out"].copy_(torch.where(live[:, :, None, None], out, s["out"]))
    return s["out"]


# ---------------------------------------------------------------- exact values

def _e4m3_exact(y):
    """Nearest E4M3 value of 64-bit numbers, ties to even, saturating."""
    mag = y.abs()
    exponent = torch.frexp(mag.clamp(min=1e-300)).exponent - 1
    quantum = torch.ldexp(torch.ones_like(mag), (exponent - 3).clamp(min=-9))
    return torch.copysign((torch.round(mag / quantum) * quantum).clamp(max=448.0), y) + 0.0


def _append_exact(s):
    case = s["case"]
    P = case["page"]
    eight = s["scales"] is not None
    wide = lambda x: (x.view(F8).float() if eight else x).double()  # noqa: E731
    q, k, v, box = s["q_out"].double(), wide(s["k_pool"]), wide(s["v_pool"]), wide(s["bounds"])
    scales = s["scales"].double() if eight else None
    for b, (L, n) in enumerate(zip(s["seq_lens"].tolist(), s["new_lens"].tolist())):
        cs = s["table"][L:L + n].double()
        cos, sin = cs[:, None, 0], cs[:, None, 1]
        if case["interleaved"]:
            rot = lambda x: torch.cat([_pairs_exact(x, cos, sin), x[..., 2 * cos.shape[-1]:]], -1)  # noqa: E731
        else:
            rot = lambda x: _halves_exact(x, cos, sin)  # noqa: E731
        q[b, :n] = rot(s["q"][b, :n].double())
        kn, vn = rot(s["k_new"][b, :n].double()), s["v_new"][b, :n].double()
        for page in range(L // P, (L + n - 1) // P + 1):
            at = int(s["block_table"][b, page])
            lo, hi = max(L, page * P), min(L + n, page * P + P)
            a, e = lo - page * P, hi - page * P
            for which, (pool, x) in enumerate(((k, kn), (v, vn))):
                rows = x[lo - L:hi - L].transpose(0, 1)                     # [hkv, new, d]
                if eight:
                    before = scales[at, :, which].clone() if a else torch.zeros_like(scales[at, :, which])
                    amax = torch.maximum(before, rows.abs().amax(dim=(1, 2)))
                    step = (amax / 448.0)[:, None, None]
                    change = torch.where(amax > before, before / amax.clamp(min=1e-300), torch.ones_like(amax))
                    change = change[:, None, None]
                    if a:
                        pool[at, :, :a] = torch.where(change < 1, _e4m3_exact(pool[at, :, :a] * change), pool[at, :, :a])
                        if which == 0:
                            box[at] = torch.where(change < 1, _e4m3_exact(box[at] * change), box[at])
                    rows = _e4m3_exact(rows / step.clamp(min=1e-300)) * (step > 0)
                    scales[at, :, which] = amax
                pool[at, :, a:e] = rows
                if which == 0:
                    low, high = rows.amin(1), rows.amax(1)
                    box[at, :, 0] = torch.minimum(low, box[at, :, 0]) if a else low
                    box[at, :, 1] = torch.maximum(high, box[at, :, 1]) if a else high
    r = {"q": q, "k_pool": k, "v_pool": v, "bounds": box}
    if eight:
        r["scales"] = scales
    return r


def _pairs_exact(x, cos, sin):
    z = torch.view_as_complex(x[..., :2 * cos.shape[-1]].reshape(x.shape[:-1] + (-1, 2)).contiguous())
    return torch.view_as_real(z * torch.complex(cos, sin)).flatten(-2)


def _halves_exact(x, cos, sin):
    h = cos.shape[-1]
    z = torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous()) * torch.complex(cos, sin)
    return torch.cat([z.real, z.imag, x[..., 2 * h:]], -1)


def _attend_exact(s):
    case = s["case"]
    P, d, hkv = case["page"], case["d"], case["hkv"]
    G = case["hq"] // hkv
    out = s["out"].double()
    for b, (L, n) in enumerate(zip(s["seq_lens"].tolist(), s["new_lens"].tolist())):
        ids = s["block_table"][b, :-(-L // P)].long().clamp(min=0)
        i = torch.arange(L - n, L, device=out.device)[:, None]
        j = torch.arange(L, device=out.device)[None, :]
        seen = j <= i
        if case["window"]:
            seen &= (j < case["sinks"]) | (i - j < case["window"])
        for h in range(hkv):
            k, v = s["k_pool"][ids, h], s["v_pool"][ids, h]
            if s["scales"] is not None:
                step = s["scales"][ids, h].double() / 448.0
                k = k.view(F8).double() * step[:, 0, None, None]
                v = v.view(F8).double() * step[:, 1, None, None]
            k, v = (x.double().reshape(-1, d)[:L] for x in (k, v))
            for g in range(h * G, h * G + G):
                w = (s["q"][b, :n, g].double() @ k.T) * d ** -0.5
                w = torch.softmax(w.masked_fill_(~seen, -math.inf), -1)
                out[b, :n, g] = w @ v
    return out


def exact(case, seed):
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    return _append_exact(s) if case["op"] == "append" else _attend_exact(s)
