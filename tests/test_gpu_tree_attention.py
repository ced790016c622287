"""tree_attention and tree_masks against 64-bit attention over the tokens that a tree's queries see."""
import pytest
import torch

from tests import paged_reference as R
from tests import tree_reference as X

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from query_aware_sparse_append_gb300 import build
    build.build()


@pytest.fixture(params=["rule", "whole", "cut"], autouse=True)
def _form(request, monkeypatch):
    """The form that the sizes choose, and the two of the tree kernel, which small calls would not reach."""
    if request.param == "rule":
        monkeypatch.delenv("QASA_TREE_FORM", raising=False)
    elif "f32" in request.node.name or "mask" in request.node.name or "parents" in request.node.name:
        pytest.skip("has one form")
    else:
        monkeypatch.setenv("QASA_TREE_FORM", request.param)


def _qasa():
    from query_aware_sparse_append_gb300 import binding
    return binding


def _queries(c, T, hq, seed=1, scale=1.0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randn((len(c.lens), T, hq, c.d), generator=g) * scale).to(R.VALUE[c.dtype]).to(c.device)


def _trees(c, T, n, seed=5, pruned=False):
    """Rows of every sequence's tree, and the mask; rows and bits behind n[b] hold anything."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    rows = []
    for b in range(len(c.lens)):
        r = X.tree_rows(X.random_parents(T, g))[0]
        if pruned:
            r = [set() if t % 3 == 1 else s for t, s in enumerate(r)]
        rows.append([r[t] if t < n[b] else set(range(T)) for t in range(T)])
        rows[b] = [s | {j for j in range(n[b], T) if (j + t) % 2} for t, s in enumerate(rows[b])]
    return rows, torch.stack([X.words(r, T) for r in rows]).cuda()


def _run(c, q, n, rows, mask, window, sinks, T, scale=None, bits=0, workspace=None):
    qasa = _qasa()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 9.0)
    lens = None if n == [T] * len(c.lens) else torch.tensor(n, dtype=torch.int32, device="cuda")
    got = qasa.tree_attention(c.library(), q, c.table, c.seq_lens, mask, q_lens=lens, window=window, sink_tokens=sinks,
                              scale=scale, out=out, status=status, workspace=workspace)
    assert got is out
    torch.cuda.synchronize()
    assert int(status) == bits, hex(int(status))
    for b in range(len(c.lens)):
        assert bool((out[b, n[b]:] == 9.0).all()), "rows behind the last query were written"
    return out


def _check(c, q, out, n, rows, window, sinks, scale=None):
    for b, L in enumerate(c.lens):
        ref, weighed, size = X.attention(c, q[b], b, L, n[b], rows[b], window, sinks, scale)
        tol = R.attention_tolerance(ref, weighed, size, c.d, R.VALUE[c.dtype], scale)
        err = (out[b, :n[b]].double() - ref).abs()
        assert bool((err <= tol).all()), (b, L, n[b], err.max().item(), (err - tol).max().item())


def _free(c, n, rows, window, sinks):
    """Tokens that no query sees become NaN; pages of such context tokens are given back: their entries go bad."""
    nan = 0x7F if c.dtype == "e4m3" else float("nan")
    for b, L in enumerate(c.lens):
        ctx = L - n[b]
        for j in range(n[b]):
            if ctx + j >= 0 and not any(j in rows[b][t] for t in range(n[b])):
                at = int(c.table[b, (ctx + j) // c.page])
                c.k_pool[at, :, (ctx + j) % c.page] = nan
                c.v_pool[at, :, (ctx + j) % c.page] = nan
        if window is None:
            continue
        lo = max(0, ctx - window + 1)
        for j in range(min(sinks, lo), lo):
            at = int(c.table[b, j // c.page])
            c.k_pool[at, :, j % c.page] = nan
            c.v_pool[at, :, j % c.page] = nan
        for i in range(-(-min(sinks, lo) // c.page), lo // c.page):
            c.table[b, i] = R.BAD_PAGE


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "e4m3"])
@pytest.mark.parametrize("hkv,group,d,page,T", [(4, 1, 64, 16, 1), (2, 8, 128, 16, 1), (1, 3, 128, 32, 2), (2, 4, 64, 32, 4),
                                                (3, 2, 64, 16, 7), (2, 8, 64, 16, 5), (1, 8, 128, 16, 16), (2, 5, 128, 32, 12),
                                                (1, 1, 64, 32, 33), (2, 8, 128, 32, 24), (1, 7, 64, 16, 70),
                                                (1, 2, 128, 16, 130)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (40, 5)])
def test_trees(dtype, hkv, group, d, page, T, window, sinks):
    lens = [T, T + 1, T + 15, T + 130, 400 + T, T // 2, T + 90, T + 127]
    n = [T, T, max(1, T // 3), T, T, T // 2, 0, max(1, T - 1)]
    c = R.Paged(dtype, lens, hkv, d, page, seed=41, amax_spread=1.0)
    q = _queries(c, T, hkv * group, scale=1.5)
    rows, mask = _trees(c, T, n)
    _free(c, n, rows, window, sinks)
    out = _run(c, q, n, rows, mask, window, sinks, T)
    _check(c, q, out, n, rows, window, sinks)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "e4m3"])
@pytest.mark.parametrize("T,group", [(3, 2), (20, 8), (64, 4)])
def test_rows_that_see_little_or_nothing(dtype, T, group):
    # a third of the rows sees the context alone, which two of the sequences do not have; unseen tokens hold NaN
    lens = [T, T + 200, T, T + 17]
    n = [T, T, max(1, T // 2), T]
    lens[2] = n[2]
    c = R.Paged(dtype, lens, 2, 64, 16, seed=42)
    q = _queries(c, T, 2 * group)
    rows, mask = _trees(c, T, n, pruned=True)
    _free(c, n, rows, None, 0)
    out = _run(c, q, n, rows, mask, None, 0, T)
    _check(c, q, out, n, rows, None, 0)
    for t in range(1, T, 3):
        assert bool((out[0, t] == 0).all()), "a query that sees nothing gives zeros"
    # nobody sees anything
    empty = torch.zeros_like(mask)
    c2 = R.Paged(dtype, [T, 0], 2, 64, 16, seed=43)
    out = _run(c2, q[:2].contiguous(), [T, 0], None, empty[:2].contiguous(), None, 0, T)
    assert bool((out[0] == 0).all())


@pytest.mark.parametrize("dtype", ["f16", "bf16", "e4m3", "f32"])
@pytest.mark.parametrize("hkv,group,d,page,T,L", [(1, 8, 128, 16, 16, 3000), (2, 4, 128, 32, 64, 1500), (1, 8, 64, 32, 40, 2500),
                                                  (1, 1, 128, 16, 300, 900), (4, 8, 128, 16, 20, 700), (1, 6, 64, 16, 43, 4000)])
def test_long_contexts(dtype, hkv, group, d, page, T, L):
    lens, n = [L, 150 + T, T, T + 1000], [T, T, min(3, T), T]
    lens[2] = 3 + 129
    c = R.Paged(dtype, lens, hkv, d, page, seed=44, amax_spread=1.0)
    q = _queries(c, T, hkv * group, seed=6, scale=1.5)
    rows, mask = _trees(c, T, n)
    for window, sinks in ((None, 0), (400, 70)):
        out = _run(c, q, n, rows, mask, window, sinks, T)
        _check(c, q, out, n, rows, window, sinks)


@pytest.mark.parametrize("dtype", ["f16", "e4m3", "f32"])
def test_sharp_scores_and_scale(dtype):
    c = R.Paged(dtype, [700, 64], 2, 128, 16, seed=45, amax_spread=2.0)
    for T, scale in ((1, 1.0), (24, 0.5), (60, 1.0)):
        q = _queries(c, T, 8, seed=4, scale=2.0)
        n = [T, T]
        rows, mask = _trees(c, T, n)
        out = _run(c, q, n, rows, mask, None, 0, T, scale=scale)
        _check(c, q, out, n, rows, None, 0, scale=scale)


@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
@pytest.mark.parametrize("T", [5, 40])
def test_a_chain_is_windowed_attention(dtype, T):
    # a tree without branches sees what the newest tokens of windowed attention see
    qasa = _qasa()
    c = R.Paged(dtype, [300 + T, 77 + T, T], 2, 128, 16, seed=46)
    q = _queries(c, T, 8)
    n = [T] * 3
    chain = [[set(range(t + 1)) for t in range(T)]] * 3
    mask = X.words(chain[0], T)[None].cuda()                   # one mask for all sequences
    out = _run(c, q, n, chain, mask, None, 0, T)
    other = qasa.window_attention(c.library(), q, c.table, c.seq_lens)
    for b, L in enumerate(c.lens):
        ref, weighed, size = R.attention(c, q[b], b, L, T, None, 0)
        tol = R.attention_tolerance(ref, weighed, size, c.d, R.VALUE[c.dtype])
        assert bool(((out[b].double() - ref).abs() <= tol).all())
        assert bool(((out[b].double() - other[b].double()).abs() <= 2 * tol).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "e4m3"])
@pytest.mark.parametrize("T", [1, 12, 70])
def test_bad_pages_are_skipped_and_reported(dtype, T):
    c = R.Paged(dtype, [200, 300], 2, 64, 16, seed=47)
    c.table[0, 3] = -1
    c.table[1, 0] = c.count + 7
    c.table[1, 18] = -5                                        # the last tokens, drafted ones
    q = _queries(c, T, 8)
    rows, mask = _trees(c, T, [T, T])
    out = _run(c, q, [T, T], rows, mask, None, 0, T, bits=0x1)
    _check(c, q, out, [T, T], rows, None, 0)
    c.table[1] = -1
    out = _run(c, q, [T, T], rows, mask, None, 0, T, bits=0x1)
    assert bool((out[1] == 0).all())


@pytest.mark.parametrize("T", [1, 40])
def test_bad_lengths_are_clamped_and_reported(T):
    qasa = _qasa()
    c = R.Paged("f16", [64, 50], 2, 64, 32, seed=48)
    q = _queries(c, T, 8)
    rows, mask = _trees(c, T, [T, T])
    table = c.table[:, :2].contiguous()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = qasa.tree_attention(c.library(), q, table, torch.tensor([90, -4], dtype=torch.int32, device="cuda"), mask,
                              status=status)
    torch.cuda.synchronize()
    assert int(status) == 0x2
    ref, weighed, size = X.attention(c, q[0], 0, 64, T, rows[0], None, 0)
    tol = R.attention_tolerance(ref, weighed, size, 64, torch.float16)
    assert bool(((out[0].double() - ref).abs() <= tol).all())
    assert bool((out[1] == 0).all())
    status.zero_()
    out = torch.full_like(q, 9.0)
    qasa.tree_attention(c.library(), q, table, c.seq_lens, mask, out=out, status=status,
                        q_lens=torch.tensor([T + 5, -1], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert int(status) == 0x10
    assert bool(((out[0].double() - ref).abs() <= tol).all())
    assert bool((out[1] == 9).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "e4m3"])
@pytest.mark.parametrize("T", [6, 40, 150])
def test_more_drafted_tokens_than_the_sequence_has(dtype, T):
    # those before position 0 do not exist: nobody sees them, and their own queries see what their rows show
    c = R.Paged(dtype, [3, T + 20, T - 1], 2, 64, 16, seed=55)
    q = _queries(c, T, 8)
    rows, mask = _trees(c, T, [T] * 3)
    out = _run(c, q, [T] * 3, rows, mask, None, 0, T)
    _check(c, q, out, [T] * 3, rows, None, 0)


@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
def test_more_sequences_than_threads(dtype):
    B, T = 900, 3
    lens = [T + 7 * (b % 13) + (90 if b % 97 == 5 else 0) for b in range(B)]
    n = [b % (T + 1) for b in range(B)]
    c = R.Paged(dtype, lens, 1, 64, 16, seed=56)
    q = _queries(c, T, 2)
    rows, mask = _trees(c, T, n)
    out = _run(c, q, n, rows, mask, 30, 2, T)
    _check(c, q, out, n, rows, 30, 2)


@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
@pytest.mark.parametrize("T,group", [(10, 8), (60, 4)])
def test_waits_with_a_short_limit_end_and_leave_rows_right_or_as_they_were(dtype, T, group, monkeypatch):
    qasa = _qasa()
    c = R.Paged(dtype, [1600, 300, T], 2, 128, 16, seed=57)
    q = _queries(c, T, 2 * group)
    n = [T] * 3
    rows, mask = _trees(c, T, n)
    clean = _run(c, q, n, rows, mask, None, 0, T)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setenv("QASA_WAIT_LIMIT_NS", "1000")
    out = torch.full_like(q, 9.0)
    qasa.tree_attention(c.library(), q, c.table, c.seq_lens, mask, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status) in (0, 0x8), hex(int(status))
    same = (out == clean).all(-1) | (out == 9.0).all(-1)
    assert bool(same.all())
    if int(status) == 0:
        assert torch.equal(out, clean)
    monkeypatch.delenv("QASA_WAIT_LIMIT_NS")
    out = _run(c, q, n, rows, mask, None, 0, T)
    assert torch.equal(out, clean)


def test_empty_calls():
    qasa = _qasa()
    c = R.Paged("f16", [40], 2, 64, 16, seed=58)
    q = _queries(c, 4, 8)
    mask = torch.zeros((1, 4, 1), dtype=torch.int32, device="cuda")
    got = qasa.tree_attention(c.library(), q[:, :0], c.table, c.seq_lens, mask[:, :0, :0])
    assert got.shape == (1, 0, 8, 64)
    got = qasa.tree_attention(c.library(), q[:0], c.table[:0], c.seq_lens[:0], mask)
    assert got.shape == (0, 4, 8, 64)
    m, d = qasa.tree_masks(torch.zeros((2, 0), dtype=torch.int32, device="cuda"))
    assert m.shape == (2, 0, 0) and d.shape == (2, 0)


@pytest.mark.parametrize("dtype,T,group", [("f16", 2, 4), ("f16", 24, 8), ("f16", 64, 8), ("e4m3", 24, 8), ("f32", 6, 2)])
def test_nan_and_infinite_queries_reach_their_own_rows_alone(dtype, T, group):
    c = R.Paged(dtype, [500 + T, T + 33], 2, 128, 16, seed=49)
    q = _queries(c, T, 2 * group)
    n = [T, T]
    rows, mask = _trees(c, T, n)
    clean = _run(c, q, n, rows, mask, None, 0, T)
    bad = q.clone()
    bad[0, T - 1, 1, 5] = float("nan")
    bad[1, 0, 0, 0] = float("inf")
    out = _run(c, bad, n, rows, mask, None, 0, T)
    assert bool(out[0, T - 1, 1].isnan().all())
    assert bool((out[1, 0, 0].isnan() | (out[1, 0, 0] == 0)).all())
    out[0, T - 1, 1], out[1, 0, 0] = clean[0, T - 1, 1], clean[1, 0, 0]
    _check(c, q, out, n, rows, None, 0)


@pytest.mark.parametrize("dtype,T,group", [("f16", 1, 4), ("f16", 6, 4), ("f16", 64, 4), ("e4m3", 24, 8), ("f32", 6, 4)])
def test_repeats_bit_for_bit_and_replays_from_graphs_that_share_a_workspace(dtype, T, group):
    qasa = _qasa()
    c = R.Paged(dtype, [900 + T, 70 + T, T], 2, 128, 16, seed=50)
    hq = 2 * group
    q = _queries(c, T, hq)
    rows, mask = _trees(c, T, [T] * 3)
    cache = c.library()
    ws = [qasa.alloc_tree_workspace(cache, 3, hq, T, c.table.shape[1]) for _ in range(2)]
    for w in ws:
        w.fill_(0xA5)
    a = qasa.tree_attention(cache, q, c.table, c.seq_lens, mask, workspace=ws[0])
    b = qasa.tree_attention(cache, q, c.table, c.seq_lens, mask, workspace=ws[0])
    assert torch.equal(a, b)
    q2 = _queries(c, T, hq, seed=8)
    a2 = qasa.tree_attention(cache, q2, c.table, c.seq_lens, mask, window=300, sink_tokens=4, workspace=ws[0])
    outs = [torch.zeros_like(q) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.graph(graphs[0], stream=side):
        qasa.tree_attention(cache, q, c.table, c.seq_lens, mask, out=outs[0], workspace=ws[1])
    with torch.cuda.graph(graphs[1], stream=side):
        qasa.tree_attention(cache, q2, c.table, c.seq_lens, mask, window=300, sink_tokens=4, out=outs[1], workspace=ws[1])
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()                            # the same stream: one after the other in one workspace
        b = qasa.tree_attention(cache, q, c.table, c.seq_lens, mask, workspace=ws[0])
    torch.cuda.synchronize()
    assert torch.equal(a, outs[0]) and torch.equal(a2, outs[1]) and torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
def test_two_calls_at_once_on_two_streams(dtype):
    qasa = _qasa()
    c = R.Paged(dtype, [600, 300], 2, 128, 16, seed=51)
    cache = c.library()
    qs = [_queries(c, T, 8, seed=T) for T in (1, 50, 2, 90)]
    masks = [_trees(c, q.shape[1], [q.shape[1]] * 2)[1] for q in qs]
    alone = [qasa.tree_attention(cache, q, c.table, c.seq_lens, m) for q, m in zip(qs, masks)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [torch.zeros_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(3):
        for q, m, out, s in zip(qs, masks, outs, streams):
            with torch.cuda.stream(s):
                qasa.tree_attention(cache, q, c.table, c.seq_lens, m, out=out)
        for q, m, out, s in zip(qs, masks, outs, streams):      # the stream named in the call
            qasa.tree_attention(cache, q, c.table, c.seq_lens, m, out=out, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(alone, outs):
        assert torch.equal(a, b)


def test_a_workspace_of_a_larger_call_serves_smaller_ones():
    qasa = _qasa()
    c = R.Paged("bf16", [1900, 40, 900, 256], 2, 128, 32, seed=52)
    cache = c.library()
    size = lambda B, hq, T, maxp: qasa.alloc_tree_workspace(cache, B, hq, T, maxp).numel()  # noqa: E731
    for small, large in (((1, 2, 1, 1), (4, 16, 60, 64)), ((4, 16, 16, 64), (4, 16, 17, 64)), ((1, 16, 60, 64), (2, 16, 60, 64)),
                         ((3, 16, 60, 20), (4, 16, 60, 64)), ((2, 16, 60, 300), (9, 16, 61, 4000))):
        assert size(*small) <= size(*large)
    ws = torch.full((size(4, 16, 60, 64),), 0xA5, dtype=torch.uint8, device="cuda")
    for T, B in ((60, 4), (33, 3), (17, 1), (2, 4)):
        q = _queries(c, T, 16)[:B].contiguous()
        sub = R.Paged("bf16", c.lens[:B], 2, 128, 32, seed=52)
        n = [min(T, L) for L in sub.lens]
        rows, mask = _trees(sub, T, n)
        out = _run(sub, q, n, rows, mask, None, 0, T, workspace=ws)
        _check(sub, q, out, n, rows, None, 0)


@pytest.mark.parametrize("dtype,T", [("f16", 1), ("f16", 40), ("e4m3", 40), ("f32", 3)])
def test_pages_beyond_four_gib(dtype, T):
    qasa = _qasa()
    c = R.Paged(dtype, [300 + T], 1, 128, 16, seed=53)
    es = c.k_pool.element_size()
    far = (5 << 30) // (16 * 128 * es)
    kv = torch.empty((2, far, 1, 16, 128), dtype=c.k_pool.dtype, device="cuda")
    kv[0, far - c.count:], kv[1, far - c.count:] = c.k_pool, c.v_pool
    bounds = torch.empty((far, 1, 2, 128), dtype=c.k_pool.dtype, device="cuda")
    scales = torch.empty((far, 1, 4), device="cuda") if dtype == "e4m3" else None
    if scales is not None:
        scales[far - c.count:] = c.scales
    table = torch.where(c.table < c.count, c.table + (far - c.count), c.table)
    q = _queries(c, T, 4)
    rows, mask = _trees(c, T, [T])
    near = qasa.tree_attention(c.library(), q, c.table, c.seq_lens, mask, window=250, sink_tokens=4)
    there = qasa.tree_attention(qasa.PagedKVCache(kv[0], kv[1], bounds, scales), q, table, c.seq_lens, mask, window=250,
                                sink_tokens=4)
    assert torch.equal(near, there)
    _check(c, q, there, [T], rows, 250, 4)


@pytest.mark.parametrize("T", [1, 31, 32, 33, 64, 200, 1024])
def test_tree_masks(T):
    qasa = _qasa()
    g = torch.Generator(device="cpu").manual_seed(54)
    n = [T, 1, max(1, T // 2), 0]
    parents = [X.random_parents(T, g) for _ in n]
    parents[2] = list(range(-1, T - 1))                        # a chain
    dev = torch.tensor(parents, dtype=torch.int32, device="cuda")
    mask = torch.full((4, T, -(-T // 32)), 7, dtype=torch.int32, device="cuda")
    depths = torch.full((4, T), 7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = qasa.tree_masks(dev, torch.tensor(n, dtype=torch.int32, device="cuda"), mask, depths, status=status)
    torch.cuda.synchronize()
    assert got[0] is mask and got[1] is depths and int(status) == 0
    for b in range(4):
        rows, deep = X.tree_rows(parents[b][:n[b]])
        assert torch.equal(mask[b, :n[b]].cpu(), X.words(rows, T)[:n[b]])
        assert depths[b, :n[b]].tolist() == deep
        assert bool((mask[b, n[b]:] == 7).all()) and bool((depths[b, n[b]:] == 7).all())


def test_bad_parents_are_reported_and_counted_as_none():
    qasa = _qasa()
    dev = torch.tensor([[-1, 0, 2, 1, -7, 99, 4]], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mask, depths = qasa.tree_masks(dev, status=status)
    torch.cuda.synchronize()
    rows, deep = X.tree_rows([-1, 0, -1, 1, -1, -1, 4])
    assert int(status) == 0x80
    assert torch.equal(mask[0].cpu(), X.words(rows, 7)) and depths[0].tolist() == deep
