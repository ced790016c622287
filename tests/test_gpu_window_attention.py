"""window_attention against 64-bit attention over the visible tokens."""
import pytest
import torch

from tests import paged_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from query_aware_sparse_append_gb300 import build
    build.build()


def _qasa():
    from query_aware_sparse_append_gb300 import binding
    return binding


def _queries(c, T, hq, seed=1, scale=1.0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    return (torch.randn((len(c.lens), T, hq, c.d), generator=g) * scale).to(R.VALUE[c.dtype]).to(c.device)


def _check(c, q, out, n, window, sinks, scale=None, skip=()):
    for b, L in enumerate(c.lens):
        if b in skip:
            continue
        ref, weighed, size = R.attention(c, q[b], b, L, n[b], window, sinks, scale)
        tol = R.attention_tolerance(ref, weighed, size, c.d, R.VALUE[c.dtype], scale)
        err = (out[b, :n[b]].double() - ref).abs()
        worst = (err - tol).max().item() if n[b] else 0.0
        assert bool((err <= tol).all()), (b, L, n[b], err.max().item(), worst)


def _run(c, q, n, window, sinks, T, scale=None, bits=0):
    qasa = _qasa()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 9.0)
    lens = None if n == [T] * len(c.lens) else torch.tensor(n, dtype=torch.int32, device="cuda")
    got = qasa.window_attention(c.library(), q, c.table, c.seq_lens, window=window, sink_tokens=sinks, q_lens=lens,
                                scale=scale, out=out, status=status)
    assert got is out
    torch.cuda.synchronize()
    assert int(status) == bits, hex(int(status))
    for b in range(len(c.lens)):
        assert bool((out[b, n[b]:] == 9.0).all()), "rows behind the last query were written"
    return out


def _free(c, n, window, sinks):
    """Tokens that no query sees become NaN; pages of such tokens are given back: their table entries go bad."""
    if window is None:
        return
    nan = 0x7F if c.dtype == "e4m3" else float("nan")
    for b, L in enumerate(c.lens):
        lo = max(0, L - n[b] - window + 1)
        for j in range(min(sinks, lo), lo):
            at = int(c.table[b, j // c.page])
            c.k_pool[at, :, j % c.page] = nan
            c.v_pool[at, :, j % c.page] = nan
        for i in range(-(-min(sinks, lo) // c.page), lo // c.page):
            c.table[b, i] = R.BAD_PAGE


HEADS = [(4, 1), (2, 8), (1, 3), (3, 2), (2, 5)]        # KV heads, group


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "e4m3"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (64, 32), (128, 32)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (1, 0), (1, 1), (16, 4), (33, 16), (100, 40), (1000, 3)])
def test_one_query_each(dtype, d, page, window, sinks):
    hkv, group = HEADS[(d + page + (window or 0)) % len(HEADS)]
    lens = [1, 15, 16, 17, 100, 33, 530, 0, 333]
    c = R.Paged(dtype, lens, hkv, d, page, seed=11, amax_spread=1.0)
    q = _queries(c, 1, hkv * group, scale=1.5)
    n = [1] * len(lens)
    _free(c, n, window, sinks)
    out = _run(c, q, n, window, sinks, 1)
    _check(c, q, out, n, window, sinks, skip=(7,))
    assert bool((out[7] == 0).all()), "an empty sequence gives zeros"


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "e4m3"])
@pytest.mark.parametrize("hkv,group,d,page,T", [(2, 8, 64, 16, 5), (1, 3, 128, 32, 9), (4, 1, 128, 16, 16), (3, 2, 64, 32, 2),
                                                (2, 4, 128, 16, 33), (1, 7, 64, 16, 70), (2, 1, 128, 32, 200)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (7, 2), (64, 20)])
def test_several_queries(dtype, hkv, group, d, page, T, window, sinks):
    lens = [T, T + 1, T + 15, 3, 400 + T, 0, T + 90]
    n = [T, T, 1, min(3, T), T, 0, max(1, T // 2)]
    c = R.Paged(dtype, lens, hkv, d, page, seed=12, amax_spread=1.0)
    q = _queries(c, T, hkv * group, seed=2)
    _free(c, n, window, sinks)
    out = _run(c, q, n, window, sinks, T)
    _check(c, q, out, n, window, sinks)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "e4m3", "f32"])
@pytest.mark.parametrize("T,prefix,window,sinks", [(384, 0, None, 0), (300, 517, 200, 5), (257, 1000, None, 0), (513, 40, 128, 16)])
def test_prompts(dtype, T, prefix, window, sinks):
    lens = [prefix + T, prefix + T // 3]
    n = [T, T // 3]
    for hkv, group, d, page in ((2, 4, 128, 16), (1, 8, 64, 32), (2, 1, 64, 16)):
        c = R.Paged(dtype, lens, hkv, d, page, seed=13)
        q = _queries(c, T, hkv * group, seed=3)
        _free(c, n, window, sinks)
        out = _run(c, q, n, window, sinks, T)
        _check(c, q, out, n, window, sinks)


@pytest.mark.parametrize("dtype", ["f16", "e4m3", "f32"])
def test_sharp_scores_and_scale(dtype):
    # scores far apart: one token takes nearly all the weight, later maxima rescale what came before
    c = R.Paged(dtype, [700, 64], 2, 128, 16, seed=14)
    for T, scale in ((1, 1.0), (24, 0.5), (90, 1.0)):
        q = _queries(c, T, 8, seed=4, scale=2.0)
        n = [T, min(T, 64)]
        q2 = q.clone()
        out = _run(c, q2, n, None, 0, T, scale=scale)
        _check(c, q2, out, n, None, 0, scale=scale)


def test_more_queries_than_tokens_gives_zeros_before_position_zero():
    c = R.Paged("f16", [3, 40], 2, 64, 16, seed=15)
    for T in (6, 40):
        q = _queries(c, T, 4)
        out = _run(c, q, [T, T], 8, 2, T)
        assert bool((out[0, :T - 3] == 0).all())
        ref, weighed, size = R.attention(c, q[0, T - 3:], 0, 3, 3, 8, 2)
        tol = R.attention_tolerance(ref, weighed, size, 64, torch.float16)
        assert bool(((out[0, T - 3:].double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "e4m3"])
@pytest.mark.parametrize("T", [1, 12, 130])
def test_bad_pages_are_skipped_and_reported(dtype, T):
    c = R.Paged(dtype, [200, 300], 2, 64, 16, seed=16)
    c.table[0, 3] = -1
    c.table[1, 0] = c.count + 7
    q = _queries(c, T, 4)
    out = _run(c, q, [T, T], None, 0, T, bits=0x1)
    _check(c, q, out, [T, T], None, 0)
    # every page of a sequence bad: zeros
    c.table[1] = -1
    out = _run(c, q, [T, T], None, 0, T, bits=0x1)
    assert bool((out[1] == 0).all())


@pytest.mark.parametrize("T", [1, 40])
def test_bad_lengths_are_clamped_and_reported(T):
    qasa = _qasa()
    c = R.Paged("f16", [64, 50], 2, 64, 32, seed=17)
    q = _queries(c, T, 4)
    maxp = 2
    table = c.table[:, :maxp].contiguous()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = qasa.window_attention(c.library(), q, table, torch.tensor([90, -4], dtype=torch.int32, device="cuda"), window=20,
                                status=status)
    torch.cuda.synchronize()
    assert int(status) == 0x2
    ref, weighed, size = R.attention(c, q[0], 0, 64, T, 20, 0)
    assert bool(((out[0].double() - ref).abs() <= R.attention_tolerance(ref, weighed, size, 64, torch.float16)).all())
    assert bool((out[1] == 0).all())
    status.zero_()
    out = torch.full_like(q, 9.0)
    qasa.window_attention(c.library(), q, table, c.seq_lens, window=20, out=out, status=status,
                          q_lens=torch.tensor([T + 5, -1], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert int(status) == 0x10
    assert bool(((out[0].double() - ref).abs() <= R.attention_tolerance(ref, weighed, size, 64, torch.float16)).all())
    assert bool((out[1] == 9).all())


def test_agrees_with_dense_decode_attention():
    qasa = _qasa()
    lens = [700, 33, 1, 256]
    c = R.Paged("bf16", lens, 2, 128, 16, seed=18)
    q = _queries(c, 1, 16)
    dense = qasa.dense_decode_attention(c.library(), q[:, 0].contiguous(), c.table, c.seq_lens)
    mine = qasa.window_attention(c.library(), q[:, 0].contiguous(), c.table, c.seq_lens)
    assert mine.shape == dense.shape
    for b, L in enumerate(lens):
        ref, weighed, size = R.attention(c, q[b], b, L, 1, None, 0)
        tol = R.attention_tolerance(ref, weighed, size, 128, torch.bfloat16)[0]
        assert bool(((mine[b].double() - dense[b].double()).abs() <= 2 * tol).all())


@pytest.mark.parametrize("T", [1, 6, 140])
def test_repeats_bit_for_bit_and_replays_from_a_graph_on_another_stream(T):
    qasa = _qasa()
    lens = [900 + T, 70 + T, T]
    c = R.Paged("f16", lens, 2, 128, 16, seed=19)
    q = _queries(c, T, 8)
    cache = c.library()
    ws = [qasa.alloc_window_workspace(cache, 3, 8, T, c.table.shape[1], 300, 4) for _ in range(2)]
    for w in ws:
        w.fill_(0xA5)
    a = qasa.window_attention(cache, q, c.table, c.seq_lens, 300, 4, workspace=ws[0])
    b = qasa.window_attention(cache, q, c.table, c.seq_lens, 300, 4, workspace=ws[0])
    assert torch.equal(a, b)
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        qasa.window_attention(cache, q, c.table, c.seq_lens, 300, 4, out=out, workspace=ws[1])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        qasa.window_attention(cache, q, c.table, c.seq_lens, 300, 4, out=out, workspace=ws[1])
    out.zero_()
    for _ in range(3):
        graph.replay()
        # an eager call with its own workspace may run at the same time
        b = qasa.window_attention(cache, q, c.table, c.seq_lens, 300, 4, workspace=ws[0])
    torch.cuda.synchronize()
    assert torch.equal(a, out) and torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
def test_prompt_waits_with_a_short_limit_end_or_are_reported(dtype, monkeypatch):
    # with a limit of 1 us a wait may give up (the hardware's own wait inside one attempt
    # may also outlast it): the call ends by itself, right or reported, and the next one is right
    qasa = _qasa()
    c = R.Paged(dtype, [600, 300], 2, 128, 16, seed=20)
    q = _queries(c, 300, 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    monkeypatch.setenv("QASA_WAIT_LIMIT_NS", "1000")
    out = qasa.window_attention(c.library(), q, c.table, c.seq_lens, 200, 4, status=status)
    torch.cuda.synchronize()
    assert int(status) in (0, 0x8), hex(int(status))
    if int(status) == 0:
        _check(c, q, out, [300, 300], 200, 4)
    monkeypatch.delenv("QASA_WAIT_LIMIT_NS")
    out = _run(c, q, [300, 300], 200, 4, 300)
    _check(c, q, out, [300, 300], 200, 4)


@pytest.mark.parametrize("dtype", ["f16", "e4m3", "f32"])
@pytest.mark.parametrize("tiles", [3, 9, 17, 25, 33, 41, 49, 57, 65, 130])
def test_every_number_of_ctas_to_a_unit(dtype, tiles):
    # one KV head, one sequence: the number of CTAs follows the visible tiles of 16 tokens
    L = 16 * tiles - 5
    c = R.Paged(dtype, [L], 1, 64, 16, seed=21)
    c.table = c.table[:, :-(-L // 16)].contiguous()
    q = _queries(c, 1, 4)
    out = _run(c, q, [1], None, 0, 1)
    _check(c, q, out, [1], None, 0)


@pytest.mark.parametrize("T,group", [(70, 2), (33, 4), (128, 1), (65, 2)])
def test_prompt_kernel_and_few_rows_kernel_meet_on_e4m3(T, group):
    # up to 128 query rows the pages are read as they are, from there on unpacked first
    c = R.Paged("e4m3", [T + 300, T], 2, 128, 32, seed=22, amax_spread=2.0)
    q = _queries(c, T, 2 * group)
    for window, sinks in ((None, 0), (100, 35)):
        out = _run(c, q, [T, T], window, sinks, T)
        _check(c, q, out, [T, T], window, sinks)


def test_e4m3_prompts_in_several_groups_of_sequences():
    # a table of 16384 pages: half a GiB holds the pages of eight sequences, nine are asked for
    qasa = _qasa()
    lens = [200 + 17 * b for b in range(9)]
    c = R.Paged("e4m3", lens, 1, 64, 16, seed=23)
    wide = torch.full((9, 16384), R.BAD_PAGE, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    n = [200 - b for b in range(9)]
    q = _queries(c, 200, 1)
    cache = c.library()
    bytes_ = qasa.alloc_window_workspace(cache, 9, 1, 200, 16384).numel()
    assert bytes_ == 8 * 16384 * 16 * 64 * 4
    out = _run(c, q, n, None, 0, 200)
    for b, L in enumerate(lens):
        ref, weighed, size = R.attention(c, q[b], b, L, n[b], None, 0)
        assert bool(((out[b, :n[b]].double() - ref).abs() <= R.attention_tolerance(ref, weighed, size, 64, torch.float16)).all()), b


def test_too_small_a_workspace_is_refused():
    qasa = _qasa()
    c = R.Paged("e4m3", [400], 1, 64, 16, seed=24)
    q = _queries(c, 200, 1)
    with pytest.raises(qasa.QasaError, match="workspace"):
        qasa.window_attention(c.library(), q, c.table, c.seq_lens, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype,T", [("f16", 1), ("f16", 40), ("e4m3", 1), ("e4m3", 200), ("f32", 3)])
def test_pages_beyond_four_gib(dtype, T):
    # the same pages at the far end of pools whose last byte is beyond 2^32
    qasa = _qasa()
    c = R.Paged(dtype, [300 + T], 1, 128, 16, seed=25)
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
    near = qasa.window_attention(c.library(), q, c.table, c.seq_lens, 250, 4)
    there = qasa.window_attention(qasa.PagedKVCache(kv[0], kv[1], bounds, scales), q, table, c.seq_lens, 250, 4)
    assert torch.equal(near, there)
    _check(c, q, there, [T], 250, 4)


@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
def test_two_calls_at_once_on_two_streams(dtype):
    qasa = _qasa()
    c = R.Paged(dtype, [600, 300], 2, 128, 16, seed=26)
    cache = c.library()
    qs = [_queries(c, T, 8, seed=T) for T in (1, 150, 1, 150)]
    alone = [qasa.window_attention(cache, q, c.table, c.seq_lens, 200, 4) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [torch.zeros_like(q) for q in qs]
    for _ in range(3):
        for q, out, s in zip(qs, outs, streams):
            with torch.cuda.stream(s):
                qasa.window_attention(cache, q, c.table, c.seq_lens, 200, 4, out=out)
        for q, out, s in zip(qs, outs, streams):      # the stream named in the call
            qasa.window_attention(cache, q, c.table, c.seq_lens, 200, 4, out=out, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(alone, outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("hkv,group,d,T,L", [(1, 8, 128, 20, 2500), (2, 4, 64, 40, 1300), (1, 1, 64, 300, 900), (4, 8, 128, 17, 700),
                                             (1, 6, 128, 43, 4000)])
def test_few_prompt_rows_over_many_keys(dtype, hkv, group, d, T, L):
    # clusters that share the key tiles, of every size that these lengths give, some CTAs without any
    lens, n = [L, 150 + T, T], [T, T, 3]
    c = R.Paged(dtype, lens, hkv, d, 32, seed=27, amax_spread=1.0)
    q = _queries(c, T, hkv * group, seed=5, scale=1.5)
    for window, sinks in ((None, 0), (400, 70)):
        out = _run(c, q, n, window, sinks, T)
        _check(c, q, out, n, window, sinks)
