"""Cases, plain forms and exact values of the operators that serve trees of drafted tokens and forked sequences.

tree     attention of a tree of drafted tokens over the paged cache: the cached context as in windowed attention, the
         drafted tokens by a mask (with `from_parents`, made from the tree's parents by the same pass)
append   the rotating append with the positions of the new tokens given: a tree's depths, or the time, height and width
         of image tokens
keep     tokens that stay (an accepted path, a subset of a long cache) move together behind a start; boxes and scales follow
fork     new sequences share their parent's full pages and get a copy of the part-filled one
copy     whole pages copied inside the pools

Every case is a dict of plain values.  Lengths come from the case alone, values, trees and page orders from the seed.
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
NO_WINDOW = 0      # a case's window of 0: all of the context is visible


def listed():
    return [
        # One sequence with a short context verifies a small tree whose shape is new: call latency.
        dict(name="tree 1x8 f16", op="tree", dtype="f16", batch=1, tokens=8, min_tokens=8, hq=32, hkv=4, d=64, page=16,
             ctx_min=504, ctx_max=504, window=NO_WINDOW, sinks=0, from_parents=True, shared=False, pruned=False),
        # A ragged serving batch verifies trees of up to 24 tokens, some of them cut short.
        dict(name="tree 16x24 f16", op="tree", dtype="f16", batch=16, tokens=24, min_tokens=1, hq=32, hkv=4, d=128,
             page=16, ctx_min=500, ctx_max=4000, window=NO_WINDOW, sinks=0, from_parents=False, shared=False, pruned=True),
        # A tree of fixed shape over one long context: few sequences, many keys.
        dict(name="tree 1x64 32k bf16", op="tree", dtype="bf16", batch=1, tokens=64, min_tokens=64, hq=32, hkv=8, d=128,
             page=32, ctx_min=32704, ctx_max=32704, window=NO_WINDOW, sinks=0, from_parents=False, shared=True,
             pruned=False),
        # A full serving batch of an E4M3 cache verifies trees over contexts of 8K.
        dict(name="tree 64x32 8k e4m3", op="tree", dtype="e4m3", batch=64, tokens=32, min_tokens=32, hq=32, hkv=4, d=128,
             page=16, ctx_min=8160, ctx_max=8160, window=NO_WINDOW, sinks=0, from_parents=False, shared=False,
             pruned=False),
        # The append of a small tree's tokens, siblings at one position: call latency.
        dict(name="append tree 1x8 f32", op="append", dtype="f32", batch=1, tokens=8, min_tokens=8, hq=4, hkv=4, d=64,
             page=16, ctx_min=2047, ctx_max=2047, rot=64, interleaved=False, axes=1, alternate=False),
        # Prompt chunks of image and text tokens with positions in time, height and width.
        dict(name="append image 2x4096 bf16", op="append", dtype="bf16", batch=2, tokens=4096, min_tokens=4096, hq=32,
             hkv=8, d=128, page=32, ctx_min=37, ctx_max=4101, rot=128, interleaved=False, axes=3, alternate=False),
        # Accepted paths of a batch's trees move together in an E4M3 cache.
        dict(name="keep 64x6 of 32 e4m3", op="keep", dtype="e4m3", batch=64, tokens=32, kept=6, min_kept=1, hkv=4, d=128,
             page=16, ctx_min=500, ctx_max=4000),
        # A quarter of the tokens of long sequences stays, the rest is given up.
        dict(name="keep 8x4096 of 16384 bf16", op="keep", dtype="bf16", batch=8, tokens=16384, kept=4096, min_kept=4096,
             hkv=8, d=128, page=32, ctx_min=0, ctx_max=0),
        # One prompt answered four times: its part-filled page copied three times.
        dict(name="fork 1x4 e4m3", op="fork", dtype="e4m3", batch=1, children=4, hkv=4, d=128, page=16, ctx_min=1003,
             ctx_max=1003),
        # A batch of beams that all go on from other beams.
        dict(name="fork 64x256 bf16", op="fork", dtype="bf16", batch=64, children=256, hkv=8, d=128, page=32, ctx_min=500,
             ctx_max=4000),
        # A few pages made a sequence's own before they are written.
        dict(name="copy 6 f32", op="copy", dtype="f32", pages=6, hkv=4, d=64, page=16),
        # A pool put in order: half a GiB of pages moved.
        dict(name="copy 16384 f16", op="copy", dtype="f16", pages=16384, hkv=4, d=128, page=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["f32", "f16", "f16", "bf16", "bf16", "e4m3", "e4m3"])
    hkv = rng.choice([1, 2, 3, 4, 8, 16])
    d, page = rng.choice([64, 128]), rng.choice([16, 32])
    c = dict(dtype=dtype, hkv=hkv, d=d, page=page)
    op = rng.choice(["tree", "tree", "tree", "append", "append", "keep", "keep", "fork", "copy"])
    if op == "tree":
        hq = hkv * (rng.choice([1, 2, 3, 4, 6, 8]) if hkv <= 8 else rng.choice([1, 2]))
        tokens = rng.choice([1, rng.randint(2, 16), _log_int(rng, 8, 256)])
        if dtype == "f32":
            tokens = min(tokens, 64)
        ctx = _log_int(rng, 1, 32768)
        # no more work than the largest listed case has, and K and V below 2 GiB in all
        most = 64 * 8192 * 32 * 32 * 128 // (tokens * hq * d * (16 if dtype == "f32" else 1))
        ctx = max(1, min(ctx, most - tokens))
        batch = max(1, min(_log_int(rng, 1, 128), most // (ctx + tokens), (1 << 30) // ((ctx + tokens) * hkv * d * 2)))
        window = NO_WINDOW if rng.random() < 0.6 else _log_int(rng, 16, 8192)
        return dict(op=op, batch=batch, tokens=tokens, min_tokens=rng.choice([1, tokens]), hq=hq,
                    ctx_min=rng.choice([0, ctx]), ctx_max=ctx, window=window,
                    sinks=rng.choice([0, 1, 4, 16, 100]) if window else 0, from_parents=rng.random() < 0.3,
                    shared=rng.random() < 0.3, pruned=rng.random() < 0.3, **c)
    if op == "append":
        hq = hkv * (rng.choice([1, 2, 3, 4, 6, 8]) if hkv <= 8 else rng.choice([1, 2]))
        tokens = _log_int(rng, 1, 4096)
        most = (8192 * 48 * 128) // (tokens * (hq + 2 * hkv) * d * (2 if dtype == "f32" else 1))
        ctx = _log_int(rng, 1, 2000)
        return dict(op=op, batch=_log_int(rng, 1, max(1, min(160, most))), tokens=tokens,
                    min_tokens=rng.choice([1, tokens]), hq=hq, ctx_min=rng.choice([0, ctx]), ctx_max=ctx,
                    rot=rng.choice([16, 32, 64, d]), interleaved=rng.random() < 0.4, axes=rng.choice([1, 2, 3, 3]),
                    alternate=rng.random() < 0.4, **c)
    # no more bytes than the largest listed case moves
    if op == "keep":
        tokens = rng.choice([_log_int(rng, 2, 256), _log_int(rng, 256, 16384)])
        kept = _log_int(rng, 1, tokens)
        ctx = _log_int(rng, 1, 2000)
        most = 8 * 16384 * 8 * 128 * 2 // ((tokens + ctx) * hkv * d * SIZE[dtype])
        return dict(op=op, batch=_log_int(rng, 1, max(1, min(128, most))), tokens=tokens, kept=kept,
                    min_kept=rng.choice([0, 1, kept]), ctx_min=rng.choice([0, ctx]), ctx_max=ctx, **c)
    if op == "fork":
        ctx = _log_int(rng, 1, 4000)
        most = (1 << 29) // ((ctx + page) * hkv * d * SIZE[dtype])
        batch = _log_int(rng, 1, max(1, min(128, most)))
        return dict(op=op, batch=batch, children=batch * rng.choice([1, 2, 3, 4, 8]), ctx_min=rng.choice([0, ctx]),
                    ctx_max=ctx, **c)
    tile = hkv * d * page * SIZE[dtype]
    return dict(op=op, pages=_log_int(rng, 1, (1 << 28) // tile), **c)


def _spread(lo, hi, n, step):
    """n whole numbers spread over lo .. hi, the last of them hi."""
    x = np.mod(np.arange(1, n + 1) * step, 1.0)
    v = lo + np.floor(x * (hi - lo + 1)).astype(np.int64)
    v[-1] = hi
    return v


def _lengths(case):
    """(tokens before the new, drafted or candidate ones; count of new, drafted or kept ones) of every sequence."""
    n = np.zeros(case["batch"], dtype=np.int64)
    if case["op"] in ("tree", "append"):
        n = _spread(case["min_tokens"], case["tokens"], case["batch"], 0.7548776662466927)
    elif case["op"] == "keep":
        n = _spread(case["min_kept"], case["kept"], case["batch"], 0.7548776662466927)
    return _spread(case["ctx_min"], case["ctx_max"], case["batch"], 0.6180339887498949), n


def _parents_and_new(case):
    """Parent of every child, and whether it needs a page of its own: the first child of a parent takes its over."""
    B, C = case["batch"], case["children"]
    parent = (np.arange(C) * 7919 + 5) % B
    first = np.zeros(C, dtype=bool)
    first[np.unique(parent, return_index=True)[1]] = True
    return parent, ~first


def work(case):
    es = SIZE[case["dtype"]]
    ev = 2 if case["dtype"] == "e4m3" else es
    hkv, d, page = case["hkv"], case["d"], case["page"]
    scale = 8 if case["dtype"] == "e4m3" else 0
    row = hkv * d
    box = hkv * (2 * d * es + scale)
    if case["op"] == "copy":
        return {"bytes": 2 * case["pages"] * (2 * row * page * es + box) + 8 * case["pages"], "flops": 0}
    ctx, n = _lengths(case)
    if case["op"] == "fork":
        parent, new = _parents_and_new(case)
        part = ctx[parent] % page
        rows, copies = int(part[new].sum()), int((new & (part > 0)).sum())
        entries = int((-(-ctx[parent] // page)).sum())
        return {"bytes": 4 * rows * row * es + 2 * copies * box + 8 * entries + 16 * len(parent), "flops": 0}
    if case["op"] == "keep":
        # boxes: the keys of the touched pages that do not move are read too
        old = int(np.where((n > 0) | (ctx % page > 0), ctx % page, 0).sum())
        touched = int(np.maximum((ctx + n - 1) // page - ctx // page + 1, 0)[n > 0].sum())
        return {"bytes": int(n.sum()) * (4 * row * es + 4) + old * row * es + touched * box + 12 * len(n), "flops": 0}
    hq, pos_bytes = case["hq"], 4
    if case["op"] == "append":
        rows = int(n.sum())
        touched = int(((ctx + n - 1) // page - ctx // page + 1).sum())
        kept = int((ctx % page != 0).sum())           # pages whose box (and scale) is read back too
        moved = rows * ((hq + 2 * hkv) * d * ev + hq * d * ev + 2 * row * es)
        angles = min(rows, int((ctx + n).max())) * case["rot"] * 4
        return {"bytes": moved + (touched + kept) * box + angles + rows * case["axes"] * pos_bytes + touched * 4 + 4 * len(n),
                "flops": rows * (hq + hkv) * case["rot"] * 3}
    w = case["window"] or 1 << 40
    lo = np.maximum(ctx - w + 1, 0)
    head = np.minimum(case["sinks"], lo)
    keys = ctx - lo + head + n
    pages = (ctx + n - 1) // page - lo // page + 1 + -(-head // page)
    mask = int((n * -(-n // 32) * 4).sum())
    return {"bytes": 2 * int(n.sum()) * hq * d * ev + 2 * int(keys.sum()) * row * es + int(pages.sum()) * (hkv * scale + 4) + mask,
            "flops": 4 * d * hq * int((n * (ctx - lo + head + 1)).sum())}


def _table(case, positions, device):
    """cos and sin of every position's angles, [positions, 2, rot / 2] in 32 bits, from angles in 64 bits."""
    half = case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=device) / half)
    angle = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * freq
    return torch.stack([angle.cos(), angle.sin()], dim=1).float().contiguous()


def _pair_axes(case):
    """Axis of every channel pair: spans of a quarter and of the rest, or the axes in turn."""
    half, axes = case["rot"] // 2, case["axes"]
    if case["alternate"]:
        return [i % axes for i in range(half)]
    cut = [half] if axes == 1 else [half // 4, half] if axes == 2 else [half // 4, half // 4 + 3 * half // 8, half]
    return [next(a for a, end in enumerate(cut) if i < end) for i in range(half)]


def _code(y):
    c = y.to(F8).view(torch.uint8)
    return torch.where(c == 0x80, torch.zeros_like(c), c)


def _quantise(x):
    """E4M3 codes and amax of each tile x [..., page, d], as an append into an empty page stores it."""
    amax = x.abs().amax(dim=(-2, -1))
    s = amax / 448.0
    return _code(torch.where(s[..., None, None] > 0, x / s[..., None, None], torch.zeros_like(x))), amax


def _boxes(pool, valid):
    """Boxes of pages with the given numbers of valid slots (an empty page's is 0)."""
    page = pool.shape[2]
    inside = (torch.arange(page, device=pool.device) < valid[:, None])[:, None, :, None]
    box = torch.empty((pool.shape[0], pool.shape[1], 2, pool.shape[3]), dtype=pool.dtype, device=pool.device)
    for a in range(0, pool.shape[0], 4096):
        part = slice(a, a + 4096)
        keys = (pool[part].view(F8) if pool.dtype == torch.uint8 else pool[part]).float()
        lo = keys.masked_fill(~inside[part], math.inf).amin(2)
        hi = keys.masked_fill(~inside[part], -math.inf).amax(2)
        b = torch.stack([lo, hi], 2)
        b = torch.where(b.isinf(), torch.zeros_like(b), b)
        box[part] = b.to(F8).view(torch.uint8) if pool.dtype == torch.uint8 else b.to(pool.dtype)
    return box


def _masks_plain(parents):
    """Mask bits [B, T, T] and depths [B, T] of trees: every token sees itself and the tokens above it."""
    B, T = parents.shape
    sees = torch.zeros((B, T, T), dtype=torch.bool, device=parents.device)
    depths = torch.zeros((B, T), dtype=torch.int32, device=parents.device)
    at = torch.arange(T, device=parents.device).expand(B, T)
    # from every token up to the top at once, a step at a time
    here = torch.ones((B, T), dtype=torch.bool, device=parents.device)
    for _ in range(T):
        sees |= (torch.arange(T, device=parents.device) == at[:, :, None]) & here[:, :, None]
        up = parents.long().gather(1, at.clamp(min=0))
        here = here & (up >= 0)
        depths += here.int()
        at = torch.where(here, up, at)
    return sees, depths


def _words(sees):
    """Rows of bits as 32-bit words, bit j % 32 of word j / 32 for column j."""
    B, T, n = sees.shape
    wide = torch.nn.functional.pad(sees, (0, -n % 32)).view(B, T, -1, 32).long()
    words = (wide << torch.arange(32, device=sees.device)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _bits(words, n):
    return (words[..., None].long() >> torch.arange(32, device=words.device) & 1).bool().flatten(-2)[..., :n]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    hkv, d, P = case["hkv"], case["d"], case["page"]
    value, pool_type = VALUE[case["dtype"]], POOL[case["dtype"]]
    op, eight = case["op"], case["dtype"] == "e4m3"
    if op == "copy":
        count, used, filled = 2 * case["pages"], None, None
        order = torch.randperm(count, generator=g, device=dev).to(torch.int32)
    else:
        B = case["batch"]
        ctx, n = _lengths(case)
        end = ctx + (case["tokens"] if op == "keep" else n)
        width = max(1, int(-(-end.max() // P))) + (1 if op == "fork" else 0)
        page_ids = np.arange(width)[None, :]
        used = page_ids < -(-end // P)[:, None]
        filled = np.clip((ctx if op == "append" else end)[:, None] - page_ids * P, 0, P)
        if op == "tree":     # pages that no query can see any more have been given back
            lo = np.maximum(ctx - (case["window"] or 1 << 40) + 1, 0)
            used &= (page_ids >= (lo // P)[:, None]) | (page_ids < -(-case["sinks"] // P))
        spare = case["children"] if op == "fork" else 1           # pages that belong to nobody yet
        count = int(used.sum()) + spare
        order = torch.randperm(count - spare, generator=g, device=dev).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
        table[torch.from_numpy(used).to(dev)] = order

    # K and V in one allocation; stale values in the slots that no token has
    scales = torch.zeros((count, hkv, 4), dtype=torch.float32, device=dev) if eight else None
    kv = torch.empty((2, count, hkv, P, d), dtype=pool_type, device=dev)
    for i in range(2):
        for a in range(0, count, 1 << 12):
            if eight:
                x = torch.randn((min(1 << 12, count - a), hkv, P, d), generator=g, device=dev)
                kv[i, a:a + (1 << 12)], scales[a:a + (1 << 12), :, i] = _quantise(x)
            else:
                kv[i, a:a + (1 << 12)].normal_(generator=g)
    valid = torch.full((count,), P, dtype=torch.int64, device=dev)
    if filled is not None:
        valid.zero_()
        valid[order.long()] = torch.from_numpy(filled[used]).to(dev)
    bounds = _boxes(kv[0], valid) if op != "tree" else torch.zeros((count, hkv, 2, d), dtype=pool_type, device=dev)
    s = {"case": case, "k_pool": kv[0], "v_pool": kv[1], "scales": scales, "bounds": bounds}
    if op == "copy":
        s["src"], s["dst"] = order[:case["pages"]].contiguous(), order[case["pages"]:].contiguous()
    else:
        s["block_table"] = table
        ints = lambda x: torch.from_numpy(np.ascontiguousarray(x).astype(np.int32)).to(dev)  # noqa: E731
        s["ctx"], s["new_lens"] = ints(ctx), ints(n)
    if op == "tree":
        T, hq = case["tokens"], case["hq"]
        s["seq_lens"] = ints(end)
        s["lens"] = s["new_lens"] if case["min_tokens"] < T else None
        s["q"] = torch.randn((B, T, hq, d), generator=g, device=dev).to(value)
        s["out"] = torch.zeros((B, T, hq, d), dtype=value, device=dev)
        trees = 1 if case["shared"] else B
        u = torch.rand((trees, T), generator=g, device=dev)
        t = torch.arange(T, device=dev)
        s["parents"] = (t - 1 - (u * u * (t + 1)).floor().long().clamp(max=T)).clamp(min=-1).to(torch.int32)
        sees = _masks_plain(s["parents"])[0]
        if case["pruned"] and not case["from_parents"]:    # tokens that were given up see the context alone
            sees[torch.rand((trees, T), generator=g, device=dev) < 0.2] = False
        s["mask"] = _words(sees)
        s["depths"] = torch.zeros((trees, T), dtype=torch.int32, device=dev)
    elif op == "append":
        T, hq = case["tokens"], case["hq"]
        s["seq_lens"], s["lens"] = s["ctx"], s["new_lens"] if case["min_tokens"] < T else None
        # one projection's output holds the queries, keys and values of every new token
        heads = torch.randn((B, T, (hq + 2 * hkv) * d), generator=g, device=dev).to(value).view(B, T, hq + 2 * hkv, d)
        s["q"], s["k_new"], s["v_new"] = heads[:, :, :hq], heads[:, :, hq:hq + hkv], heads[:, :, hq + hkv:]
        s["q_out"] = torch.zeros((B, T, hq, d), dtype=value, device=dev)
        limit = width * P
        s["table"] = _table(case, limit, dev)
        t = torch.arange(T, device=dev)
        if case["axes"] == 1:      # a tree's depths behind the context
            u = torch.rand((B, T), generator=g, device=dev)
            deep = (u * torch.sqrt(t + 1.0)).floor().long()
            pos = (s["ctx"].long()[:, None] + deep)[None]
        else:                      # rows of an image: time stands still, height and width count
            side = max(1, math.isqrt(T))
            first = s["ctx"].long()[:, None]
            pos = torch.stack([first + 0 * t, first + t // side, first + t % side][:case["axes"]])
        s["positions"] = pos.clamp(max=limit - 1).to(torch.int32).contiguous()
        s["pair_axes"] = _pair_axes(case)
    elif op == "keep":
        s["seq_lens"] = ints(end)
        rank = torch.rand((B, case["tokens"]), generator=g, device=dev).argsort(1)[:, :case["kept"]]
        late = torch.arange(case["kept"], device=dev) >= s["new_lens"][:, None]
        s["keep"] = rank.masked_fill(late, 1 << 24).sort(1).values.masked_fill(late, -1).to(torch.int32).contiguous()
        s["lens"] = s["new_lens"] if case["min_kept"] < case["kept"] else None
        s["lens_out"] = torch.zeros(B, dtype=torch.int32, device=dev)
    elif op == "fork":
        C = case["children"]
        parent, new = _parents_and_new(case)
        s["seq_lens"] = s["ctx"]
        s["parents"] = ints(parent)
        own_page = torch.arange(count - spare, count, device=dev, dtype=torch.int32)
        s["new_pages"] = torch.where(torch.from_numpy(new).to(dev), own_page, torch.full_like(own_page, -1))
        s["table_out"] = torch.full((C, width), -1, dtype=torch.int32, device=dev)
        s["lens_out"] = torch.zeros(C, dtype=torch.int32, device=dev)
    if own:
        from query_aware_sparse_append_gb300 import binding as qasa
        s["qasa"] = qasa
        s["cache"] = qasa.PagedKVCache(s["k_pool"], s["v_pool"], bounds, scales)
        if op == "tree":
            s["workspace"] = qasa.alloc_tree_workspace(s["cache"], B, hq, T, width)
    return s


def run(s):
    op = s["case"]["op"]
    if op == "tree":
        if not own:
            return _tree_plain(s)
        case, mask, r = s["case"], s["mask"], {}
        if case["from_parents"]:
            mask, depths = s["qasa"].tree_masks(s["parents"], mask=mask, depths=s["depths"])
            r = {"mask": mask, "depths": depths}
        r["out"] = s["qasa"].tree_attention(s["cache"], s["q"], s["block_table"], s["seq_lens"], mask, q_lens=s["lens"],
                                            window=case["window"] or None, sink_tokens=case["sinks"], out=s["out"],
                                            workspace=s["workspace"])
        return r
    if op == "append":
        if own:
            s["qasa"].kv_append_positioned(s["cache"], s["block_table"], s["seq_lens"], s["k_new"], s["v_new"], s["table"],
                                           s["positions"], q=s["q"], q_out=s["q_out"], append_lens=s["lens"],
                                           pair_axes=s["pair_axes"], interleaved=s["case"]["interleaved"])
        else:
            _append_plain(s)
        return dict(_pools(s), q=s["q_out"])
    if op == "keep":
        if own:
            s["qasa"].kv_keep_tokens(s["cache"], s["block_table"], s["seq_lens"], s["ctx"], s["keep"], keep_lens=s["lens"],
                                     lens_out=s["lens_out"])
        else:
            _keep_plain(s)
        return dict(_pools(s), lens=s["lens_out"])
    if op == "fork":
        if own:
            s["qasa"].kv_fork(s["cache"], s["block_table"], s["seq_lens"], s["parents"], s["new_pages"],
                              table_out=s["table_out"], lens_out=s["lens_out"])
        else:
            _fork_plain(s)
        return dict(_pools(s), table=s["table_out"], lens=s["lens_out"])
    if own:
        s["qasa"].kv_copy_pages(s["cache"], s["src"], s["dst"])
    else:
        src, dst = s["src"].long(), s["dst"].long()
        for x in (s["k_pool"], s["v_pool"], s["bounds"], s["scales"]):
            if x is not None:
                x[dst] = x[src]
    return _pools(s)


def _pools(s):
    """The cache as it now is, E4M3 codes as the values they stand for."""
    eight = s["scales"] is not None
    r = {name: s[name].view(F8) if eight else s[name] for name in ("k_pool", "v_pool", "bounds")}
    if eight:
        r["scales"] = s["scales"]
    return r


# ---------------------------------------------------------------- plain forms

def _tree_plain(s):
    case = s["case"]
    P, d, hkv = case["page"], case["d"], case["hkv"]
    B, T, hq = s["q"].shape[:3]
    G, dev = hq // hkv, s["q"].device
    r = {}
    if case["from_parents"]:
        tree, depths = _masks_plain(s["parents"])
        s["mask"].copy_(_words(tree))
        s["depths"].copy_(depths)
        r = {"mask": s["mask"], "depths": s["depths"]}
    L, n = s["seq_lens"].long(), s["new_lens"].long()
    ctx = L - n
    longest = s["block_table"].shape[1] * P
    window = min(case["window"] or longest, longest)
    # the columns that some query of the sequence can see: the sinks, the window of depth 0, the drafted tokens
    span = min(window + T - 1, longest)
    start = (ctx - window + 1).clamp(min=0)
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
    live = torch.arange(T, device=dev) < n[:, None]
    sees = _bits(s["mask"], T) & live[:, None, :]                           # [B, T, T]
    depth = (sees.sum(-1) - 1).clamp(min=0)
    j = pos[:, None, :]
    before = (j < ctx[:, None, None]) & ((j < case["sinks"]) | (j > (ctx[:, None] + depth)[:, :, None] - window))
    drafted = (pos - ctx[:, None]).clamp(0, T - 1)[:, None, :].expand(-1, T, -1)
    seen = inside[:, None, :] & (before | ((j >= ctx[:, None, None]) & sees.gather(2, drafted)))
    hidden = ~seen[:, None, :, None, :].expand(-1, -1, -1, G, -1).reshape(B, 1, T * G, -1)
    scores = scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top.isinf(), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows(s["v_pool"], 1)) / torch.where(total > 0, total, torch.ones_like(total))
    out = out.view(B, hkv, T, G, d).permute(0, 2, 1, 3, 4).reshape(B, T, hq, d).to(s["q"].dtype)
    s["out"].copy_(torch.where(live[:, :, None, None], out, s["out"]))
    r["out"] = s["out"]
    return r


def _rotate_plain(x, s, live):
    """x [B, T, H, d] rotated, in 64 bits, rounded to 32."""
    half = s["table"].shape[2]
    pos = s["positions"].long().masked_fill(~live, 0)                       # [axes, B, T]
    axis = torch.tensor(s["pair_axes"], device=x.device)
    rows = pos[axis].permute(1, 2, 0)                                       # [B, T, half]: a row for every pair
    pair = torch.arange(half, device=x.device)
    cos, sin = (s["table"][rows, i, pair].double()[:, :, None] for i in range(2))
    rot, rest = x[..., :2 * half].double(), x[..., 2 * half:].double()
    if s["case"]["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rot[..., :half], rot[..., half:]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, rest], -1).float()


def _touched(s, first, n, most):
    """The pages that hold tokens [first, first + n) of every sequence, `most` at most, as [B, pages]: logical number,
    physical page (-1 for none), and [B, pages, P] tokens counted from `first`.  The page of `first` is among them if
    it holds earlier tokens, whatever n."""
    P = s["case"]["page"]
    logical = (first // P)[:, None] + torch.arange((most + P - 1) // P + 1, device=first.device)
    width = s["block_table"].shape[1]
    phys = s["block_table"].long().gather(1, logical.clamp(max=width - 1))
    phys = torch.where((logical * P < (first + n)[:, None]) & (logical < width), phys, torch.full_like(phys, -1))
    slot = logical[:, :, None] * P + torch.arange(P, device=first.device)
    return logical, phys, slot - first[:, None, None]


def _fold(s, phys, keys, inside):
    """lo and hi [B, pages, hkv, 2, d] of the tiles' keys [B, pages, hkv, P, d] that are inside."""
    keys = (keys.view(F8) if s["scales"] is not None else keys).float()
    return torch.stack([keys.masked_fill(~inside, math.inf).amin(3), keys.masked_fill(~inside, -math.inf).amax(3)], 3)


def _put(s, name, phys, tiles):
    there = phys >= 0
    s[name][phys[there]] = tiles[there]


def _append_plain(s):
    B, T, hkv, d = s["k_new"].shape
    L, n = s["ctx"].long(), s["new_lens"].long()
    live = torch.arange(T, device=L.device) < n[:, None]
    q = _rotate_plain(s["q"], s, live).to(s["q"].dtype)
    s["q_out"].copy_(torch.where(live[:, :, None, None], q, s["q_out"]))
    logical, phys, index = _touched(s, L, n, T)
    phys = torch.where((n > 0)[:, None], phys, torch.full_like(phys, -1))
    P, pages, safe = s["case"]["page"], phys.shape[1], phys.clamp(min=0)
    fresh = index[:, :, 0] >= 0                                             # slot 0 is written by this call
    mask = ((index >= 0) & (index < n[:, None, None]))[:, :, None, :, None]
    at = index.clamp(0, T - 1).flatten(1)[:, :, None, None].expand(-1, -1, hkv, d)
    rows = {"k_pool": _rotate_plain(s["k_new"], s, live), "v_pool": s["v_new"].float()}
    for which, name in enumerate(("k_pool", "v_pool")):
        x = rows[name].gather(1, at).view(B, pages, P, hkv, d).transpose(2, 3)
        old, box = s[name][safe], s["bounds"][safe]
        if s["scales"] is None:
            x = x.to(s[name].dtype)
        else:
            before = torch.where(fresh[:, :, None], torch.zeros((), device=L.device), s["scales"][safe][..., which])
            amax = torch.maximum(before, x.abs().masked_fill(~mask, 0).amax(dim=(-2, -1)))
            old = torch.where((index < 0)[:, :, None, :, None], _rescaled(old, before, amax), old)
            box, x = _rescaled(box, before, amax), _coded(x, amax)
            new_scales = s["scales"][safe]
            new_scales[..., which] = amax
            _put(s, "scales", phys, new_scales)
        _put(s, name, phys, torch.where(mask, x, old))
        if which == 0:
            new = _fold(s, phys, x, mask)
            kept = (box.view(F8) if s["scales"] is not None else box).float()
            none = fresh[:, :, None, None]
            lo = torch.minimum(new[..., 0, :], kept[..., 0, :].masked_fill(none, math.inf))
            hi = torch.maximum(new[..., 1, :], kept[..., 1, :].masked_fill(none, -math.inf))
            folded = torch.stack([lo, hi], 3)
            _put(s, "bounds", phys, folded.to(F8).view(torch.uint8) if s["scales"] is not None else folded.to(box.dtype))


def _coded(x, amax):
    """Codes of values x [..., rows, d] under the scales of amax [...]."""
    sc = (amax / 448.0)[..., None, None]
    return _code(torch.where(sc > 0, x / sc, torch.zeros_like(x)))


def _rescaled(c, before, amax):
    """Codes [..., rows, d] under the scale of `before` as codes under that of `amax`."""
    again = _coded(c.view(F8).float() * (before / 448.0)[..., None, None], amax)
    return torch.where((amax > before)[..., None, None], again, c)


def _keep_plain(s):
    P, B = s["case"]["page"], s["case"]["batch"]
    start, n = s["ctx"].long(), s["new_lens"].long()
    logical, phys, index = _touched(s, start, n, s["case"]["kept"])
    pages, safe = phys.shape[1], phys.clamp(min=0)
    moved = (index >= 0) & (index < n[:, None, None])
    kept = s["keep"].long().gather(1, index.clamp(0, s["keep"].shape[1] - 1).flatten(1)).view(index.shape)
    source = torch.where(moved, start[:, None, None] + kept, torch.zeros_like(kept))
    from_page = s["block_table"].long().gather(1, (source // P).flatten(1)).view(source.shape).clamp(min=0)
    mask = moved[:, :, None, :, None]
    inside = ((logical[:, :, None] * P + torch.arange(P, device=start.device)) < (start + n)[:, None, None])[:, :, None, :, None]
    tiles = {}
    for which, name in enumerate(("k_pool", "v_pool")):
        old = s[name][safe]                                                 # [B, pages, hkv, P, d]
        x = s[name][from_page, :, source % P].transpose(2, 3)
        if s["scales"] is not None:
            before = s["scales"][safe][..., which]                          # [B, pages, hkv]
            of_row = s["scales"][from_page][..., which].transpose(2, 3)     # [B, pages, hkv, P]
            other = (moved & (source // P != logical[:, :, None]))[:, :, None, :]
            value = x.view(F8).float() * (of_row / 448.0)[..., None]
            amax = torch.maximum(before, value.abs().amax(-1).masked_fill(~other, 0).amax(-1))
            x = torch.where(other[..., None], _coded(value, amax), _rescaled(x, before, amax))
            old = _rescaled(old, before, amax)
            new_scales = tiles.setdefault("scales", s["scales"][safe])
            new_scales[..., which] = amax
        tiles[name] = torch.where(mask, x, old)
        if which == 0:
            box = _fold(s, phys, tiles[name], inside)
            tiles["bounds"] = box.to(F8).view(torch.uint8) if s["scales"] is not None else box.to(old.dtype)
    for name, t in tiles.items():
        if name in ("k_pool", "v_pool"):      # slots behind the last token stay as they were
            t = torch.where(inside, t, s[name][safe])
        _put(s, name, phys, t)
    s["lens_out"].copy_(start + n)


def _fork_plain(s):
    P = s["case"]["page"]
    parent, new = s["parents"].long(), s["new_pages"].long()
    L = s["seq_lens"].long()[parent]
    width = s["block_table"].shape[1]
    ids = torch.arange(width, device=L.device)
    rows = s["block_table"][parent]
    last = (L // P)[:, None]
    part = (L % P > 0)[:, None]
    takes = part & (ids == last) & (new >= 0)[:, None]
    rows = torch.where(takes, new[:, None].to(torch.int32), rows)
    s["table_out"].copy_(torch.where(ids < last + part, rows, s["table_out"]))
    s["lens_out"].copy_(L)
    copies = part[:, 0] & (new >= 0)
    src, dst = s["block_table"].long()[parent, (L // P).clamp(max=width - 1)][copies], new[copies]
    inside = (torch.arange(P, device=L.device) < (L % P)[copies][:, None])[:, None, :, None]
    for name in ("k_pool", "v_pool"):
        s[name][dst] = torch.where(inside, s[name][src], s[name][dst])
    for name in ("bounds", "scales"):
        if s[name] is not None:
            s[name][dst] = s[name][src]


# ---------------------------------------------------------------- exact values

def _e4m3_exact(y):
    """Nearest E4M3 value of 64-bit numbers, ties to even, saturating."""
    mag = y.abs()
    exponent = torch.frexp(mag.clamp(min=1e-300)).exponent - 1
    quantum = torch.ldexp(torch.ones_like(mag), (exponent - 3).clamp(min=-9))
    return torch.copysign((torch.round(mag / quantum) * quantum).clamp(max=448.0), y) + 0.0


def _wide(s):
    """The cache in 64 bits: codes as the values they stand for (without their scale), boxes, scales."""
    eight = s["scales"] is not None
    r = {k: (s[k].view(F8).float() if eight else s[k]).double() for k in ("k_pool", "v_pool", "bounds")}
    if eight:
        r["scales"] = s["scales"].double()
    return r


def _tree_exact(s):
    case = s["case"]
    P, d, hkv, T = case["page"], case["d"], case["hkv"], case["tokens"]
    G = case["hq"] // hkv
    out = s["out"].double()
    words = s["mask"].cpu().numpy().view(np.uint32)
    r = {}
    if case["from_parents"]:
        parents = s["parents"].cpu().numpy()
        rows = np.zeros((parents.shape[0], T), dtype=object)
        depths = np.zeros(parents.shape, dtype=np.int32)
        for b in range(parents.shape[0]):
            for t in range(T):
                p = parents[b, t]
                rows[b, t] = (1 << t) | (rows[b, p] if p >= 0 else 0)
                depths[b, t] = depths[b, p] + 1 if p >= 0 else 0
        words = np.array([[[m >> 32 * w & 0xffffffff for w in range(-(-T // 32))] for m in row] for row in rows],
                         dtype=np.uint32)
        r = {"mask": torch.from_numpy(words.view(np.int32)), "depths": torch.from_numpy(depths)}
    for b, (L, n) in enumerate(zip(s["seq_lens"].tolist(), s["new_lens"].tolist())):
        ctx = L - n
        tree = np.unpackbits(words[0 if case["shared"] else b].view(np.uint8), axis=-1, bitorder="little")[:n, :n] > 0
        depth = np.maximum(tree.sum(1) - 1, 0)
        j = np.arange(ctx)
        seen = np.ones((n, ctx), dtype=bool)
        if case["window"]:
            seen = (j < case["sinks"]) | (ctx + depth[:, None] - j < case["window"])
        hidden = torch.from_numpy(~np.concatenate([seen, tree], 1)).to(out.device)
        empty = hidden.all(1)[:, None]
        ids = s["block_table"][b, :-(-L // P)].long().clamp(min=0)
        for h in range(hkv):
            k, v = s["k_pool"][ids, h], s["v_pool"][ids, h]
            if s["scales"] is not None:
                step = s["scales"][ids, h].double() / 448.0
                k = k.view(F8).double() * step[:, 0, None, None]
                v = v.view(F8).double() * step[:, 1, None, None]
            k, v = (x.double().reshape(-1, d)[:L] for x in (k, v))
            for g in range(h * G, h * G + G):
                w = ((s["q"][b, :n, g].double() @ k.T) * d ** -0.5).masked_fill_(hidden, -math.inf)
                out[b, :n, g] = (torch.softmax(w, -1) @ v).masked_fill(empty, 0.0)
    return dict(r, out=out)


def _append_exact(s):
    case = s["case"]
    P, half = case["page"], case["rot"] // 2
    r = _wide(s)
    eight = "scales" in r
    q = s["q_out"].double()
    axis = np.array(_pair_axes(case))
    positions = s["positions"].cpu().numpy()
    a_of = np.arange(half) * 2 if case["interleaved"] else np.arange(half)
    b_of = a_of + (1 if case["interleaved"] else half)
    for b, (L, n) in enumerate(zip(s["ctx"].tolist(), s["new_lens"].tolist())):
        rows = torch.from_numpy(positions[axis, b, :n].T.astype(np.int64)).to(q.device)
        turn = s["table"].double()[rows, :, torch.arange(half, device=q.device)]          # [n, half, 2]
        turn = torch.complex(turn[..., 0].contiguous(), turn[..., 1].contiguous())[:, None]

        def rot(x):
            x = x.double().clone()
            z = torch.complex(x[..., a_of].contiguous(), x[..., b_of].contiguous()) * turn
            x[..., a_of], x[..., b_of] = z.real, z.imag
            return x

        q[b, :n] = rot(s["q"][b, :n])
        kn, vn = rot(s["k_new"][b, :n]), s["v_new"][b, :n].double()
        for page in range(L // P, (L + n - 1) // P + 1 if n else 0):
            at = int(s["block_table"][b, page])
            lo, hi = max(L, page * P), min(L + n, page * P + P)
            a, e = lo - page * P, hi - page * P
            for which, (name, x) in enumerate((("k_pool", kn), ("v_pool", vn))):
                new = x[lo - L:hi - L].transpose(0, 1)                      # [hkv, new, d]
                if eight:
                    amax = new.abs().amax(dim=(1, 2))
                    if a:
                        amax = _grow_exact(r, at, which, name, a, torch.maximum(r["scales"][at, :, which], amax))
                    r["scales"][at, :, which] = amax
                    step = (amax / 448.0)[:, None, None]
                    new = _e4m3_exact(new / step.clamp(min=1e-300)) * (step > 0)
                r[name][at, :, a:e] = new
                if which == 0:
                    low, high = new.amin(1), new.amax(1)
                    r["bounds"][at, :, 0] = torch.minimum(low, r["bounds"][at, :, 0]) if a else low
                    r["bounds"][at, :, 1] = torch.maximum(high, r["bounds"][at, :, 1]) if a else high
    return dict(r, q=q)


def _grow_exact(r, at, which, name, rows, amax):
    """The first rows of a page (and its box) under the scale of amax; amax."""
    change = (r["scales"][at, :, which] / amax.clamp(min=1e-300))[:, None, None]
    again = lambda x: torch.where(change < 1, _e4m3_exact(x * change), x)  # noqa: E731
    r[name][at, :, :rows] = again(r[name][at, :, :rows])
    if which == 0:
        r["bounds"][at] = again(r["bounds"][at])
    return amax


def _keep_exact(s):
    P = s["case"]["page"]
    r = _wide(s)
    before = {k: v.clone() for k, v in r.items()}
    table = s["block_table"].cpu().numpy()
    ends = []
    for b, (start, n) in enumerate(zip(s["ctx"].tolist(), s["new_lens"].tolist())):
        source = start + s["keep"][b, :n].cpu().numpy().astype(np.int64)
        ends.append(start + n)
        for page in range(start // P, -(-(start + n) // P)):
            at, a = table[b, page], max(start - page * P, 0)
            rows = source[max(page * P - start, 0):(page + 1) * P - start]
            pages, slots = torch.from_numpy(table[b, rows // P].astype(np.int64)), torch.from_numpy(rows % P)
            other = torch.from_numpy(rows // P != page).to(r["k_pool"].device)
            for which, name in enumerate(("k_pool", "v_pool")):
                x = before[name][pages, :, slots].transpose(0, 1)           # [hkv, rows, d]
                if "scales" in r and len(rows):
                    old = before["scales"][at, :, which]
                    step = before["scales"][pages, :, which].T[:, :, None]
                    largest = torch.where(other, (x * step / 448.0).abs().amax(-1), torch.zeros((), device=x.device).double())
                    amax = torch.maximum(old, largest.amax(1))
                    ratio = torch.where(other[:, None], step, old[:, None, None]) / amax.clamp(min=1e-300)[:, None, None]
                    x = torch.where(ratio == 1, x, _e4m3_exact(x * ratio))
                    r[name][at, :, :a] = torch.where((amax > old)[:, None, None], _e4m3_exact(
                        r[name][at, :, :a] * (old / amax.clamp(min=1e-300))[:, None, None]), r[name][at, :, :a])
                    r["scales"][at, :, which] = amax
                r[name][at, :, a:a + len(rows)] = x
                if which == 0:
                    now = r[name][at, :, :a + len(rows)]
                    r["bounds"][at, :, 0], r["bounds"][at, :, 1] = now.amin(1), now.amax(1)
    return dict(r, lens=torch.tensor(ends, dtype=torch.int32))


def _fork_exact(s):
    P = s["case"]["page"]
    r = _wide(s)
    table, out = s["block_table"].cpu().numpy(), s["table_out"].cpu().numpy().copy()
    lens = s["seq_lens"].tolist()
    parents, new = s["parents"].tolist(), s["new_pages"].tolist()
    for c, parent in enumerate(parents):
        full, part = divmod(lens[parent], P)
        out[c, :full] = table[parent, :full]
        if part:
            at = table[parent, full]
            out[c, full] = at if new[c] < 0 else new[c]
            if new[c] >= 0:
                r["k_pool"][new[c], :, :part], r["v_pool"][new[c], :, :part] = r["k_pool"][at, :, :part], r["v_pool"][at, :, :part]
                for name in ("bounds", "scales"):
                    if name in r:
                        r[name][new[c]] = r[name][at]
    return dict(r, table=torch.from_numpy(out), lens=torch.tensor([lens[p] for p in parents], dtype=torch.int32))


def _copy_exact(s):
    r = _wide(s)
    src, dst = s["src"].long(), s["dst"].long()
    for x in r.values():
        x.index_copy_(0, dst, x.index_select(0, src))
    return r


def exact(case, seed):
    global own
    mine, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = mine
    return {"tree": _tree_exact, "append": _append_exact, "keep": _keep_exact, "fork": _fork_exact,
            "copy": _copy_exact}[case["op"]](s)
