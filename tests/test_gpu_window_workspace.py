"""Workspaces of E4M3 prompts: one made for a larger call serves every smaller one, whatever number of
sequences goes at once."""
import ctypes

import pytest
import torch

from tests import paged_reference as R


def _qasa():
    from query_aware_sparse_append_gb300 import build
    build.build()
    from query_aware_sparse_append_gb300 import binding
    return binding


def _size(qasa, cache, batch, hq, T, pages, window, sinks):
    return int(qasa._lib.qasa_window_workspace_size(batch, hq, cache.c_ref, T, pages, window, sinks))


def _host_cache(qasa, hkv, d, page):
    kv = torch.zeros((2, 4, hkv, page, d), dtype=torch.uint8)
    return qasa.PagedKVCache(kv[0], kv[1], torch.zeros((4, hkv, 2, d), dtype=torch.uint8), torch.zeros((4, hkv, 4)))


@pytest.mark.parametrize("batch,hkv,d,page", [(1, 8, 128, 16), (4, 8, 128, 16), (16, 8, 128, 16), (64, 8, 128, 32),
                                              (9, 1, 64, 16)])
def test_a_call_needs_its_longest_sequence_alone(batch, hkv, d, page):
    # what a call asks for at the least is one sequence's pages, which grow with each of tokens, pages, window and
    # sinks: so the size of any larger call covers it
    qasa = _qasa()
    cache = _host_cache(qasa, hkv, d, page)
    calls = [(T, pages, window, sinks) for T in (200, 512, 3000, 4096, 8192) for pages in (300, 4000, 5000, 16384)
             for window in (64, 8192, 61500, 1 << 30) for sinks in (0, 100)]
    least = {c: _size(qasa, cache, 1, hkv, *c) for c in calls}
    full = {c: _size(qasa, cache, batch, hkv, *c) for c in calls}
    for large in calls:
        for small in calls:
            if all(s <= x for s, x in zip(small, large)):
                assert 0 < least[small] <= full[large], (small, large)
    # one byte less than that is refused before any launch
    for T, pages, window, sinks in calls[::7]:
        code = qasa._lib.qasa_window_attention(cache.c_ref, 0x40000, hkv, T, None, 0x50000, pages, 0x60000, window, sinks,
                                               0.0, 0x80000, 0x90000, least[T, pages, window, sinks] - 1, batch, None, None)
        assert code == 6


@pytest.mark.gpu
def test_a_workspace_of_a_larger_call_serves_smaller_ones():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    qasa = _qasa()
    lens = [200 + 17 * b for b in range(9)]
    c = R.Paged("e4m3", lens, 1, 64, 16, seed=51)
    cache = c.library()
    g = torch.Generator(device="cpu").manual_seed(52)

    def run(T, pages, window, ws):
        q = torch.randn((9, T, 1, 64), generator=g).half().cuda()
        table = torch.full((9, pages), R.BAD_PAGE, dtype=torch.int32, device="cuda")
        table[:, :c.table.shape[1]] = c.table
        out = qasa.window_attention(cache, q, table, c.seq_lens, window, 4, workspace=ws)
        torch.cuda.synchronize()
        for b, L in enumerate(lens):
            ref, weighed, size = R.attention(c, q[b], b, L, T, window, 4)
            tol = R.attention_tolerance(ref, weighed, size, 64, torch.float16)
            assert bool(((out[b].double() - ref).abs() <= tol).all()), (T, pages, window, b)
        return q, table, out

    # half a GiB holds 8 sequences of 15000 pages (469 MiB), and 9 of 14000 (492 MiB) or of fewer visible ones
    ws = qasa.alloc_window_workspace(cache, 9, 1, 200, 15000, None, 4)
    run(200, 15000, None, ws)
    run(200, 14000, None, ws)
    run(150, 14000, None, ws)
    run(200, 15000, 14000 * 16, ws)
    # down to one sequence at a time, with the same bits
    one = _size(qasa, cache, 1, 1, 200, 15000, 300, 4)
    q, table, out = run(200, 15000, 300, ws[:one])
    more = qasa.window_attention(cache, q, table, c.seq_lens, 300, 4, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, more)
    with pytest.raises(qasa.QasaError, match="workspace"):
        qasa.window_attention(cache, q, table, c.seq_lens, 300, 4, workspace=ws[:one - 16])
