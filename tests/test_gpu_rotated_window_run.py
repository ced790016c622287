"""Both operators as a model's layer uses them: prompt chunks, a verification of drafted tokens and
decode steps, each an append of raw q, k and v with rotation followed by windowed attention, the
tokens of a sequence checked against 64-bit attention over its rotated keys, with the page selection
of the library working on the same cache."""
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


def _layer(dtype, hkv, group, d, page, rot, interleaved, window, sinks, chunks, graph_steps):
    from query_aware_sparse_append_gb300 import binding as qasa
    B, hq = 2, hkv * group
    total = max(sum(c[b] for c in chunks) for b in range(B)) + graph_steps
    value = R.VALUE[dtype]
    g = torch.Generator(device="cpu").manual_seed(31)
    raw = torch.randn((B, total, (hq + 2 * hkv) * d), generator=g).to(value).cuda()
    heads = raw.view(B, total, hq + 2 * hkv, d)
    c = R.Paged(dtype, [0] * B, hkv, d, page, seed=31, reserve=total)
    cache = c.library()
    table = qasa.rotation_table(total, rot, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    done = [0] * B
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [[] for _ in range(B)]
    u = R.half_step(value)

    def rows(n):
        T = max(n)
        x = torch.zeros((B, T, hq + 2 * hkv, d), dtype=value, device="cuda")
        for b in range(B):
            x[b, :n[b]] = heads[b, done[b]:done[b] + n[b]]
        return x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]

    for n in chunks:
        q, k, v = rows(n)
        counts = torch.tensor(n, dtype=torch.int32, device="cuda")
        turned = qasa.kv_append_rotated(cache, c.table, lens, k, v, table, q=q, append_lens=counts,
                                        interleaved=interleaved, status=status)
        lens = lens + counts
        out = qasa.window_attention(cache, turned, c.table, lens, window, sinks, q_lens=counts, status=status)
        for b in range(B):
            outs[b].append(out[b, :n[b]])
            done[b] += n[b]
    # the last steps from one graph: append, attend, advance
    if graph_steps:
        q, k, v = (x.contiguous() for x in rows([1] * B))
        turned = torch.zeros_like(q)
        out = torch.zeros_like(q)
        ws = qasa.alloc_window_workspace(cache, B, hq, 1, c.table.shape[1], window, sinks)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            qasa.kv_append_rotated(cache, c.table, lens, k, v, table, q=q, q_out=turned, interleaved=interleaved, status=status)
            lens.add_(1)
            qasa.window_attention(cache, turned, c.table, lens, window, sinks, out=out, workspace=ws, status=status)
        for _ in range(graph_steps):
            for t, s in zip((q, k, v), rows([1] * B)):
                t.copy_(s)
            graph.replay()
            torch.cuda.synchronize()
            for b in range(B):
                outs[b].append(out[b].clone())
                done[b] += 1
    torch.cuda.synchronize()
    assert int(status) == 0
    assert lens.tolist() == done
    for b in range(B):
        got = torch.cat(outs[b])
        c.seq_lens = lens
        turned = R.rotate(heads[b, :done[b], :hq], table, 0, interleaved).to(value)
        ref, weighed, size = R.attention(c, turned, b, done[b], done[b], window, sinks)
        # the queries' own rounding may fall either way where fp32 and 64-bit rotation differ: one more step in the scores
        tol = R.attention_tolerance(ref, weighed, size, d, value) + 2 * 2 * u * size[..., None] / d ** 0.5 * weighed
        err = (got.double() - ref).abs()
        assert bool((err <= tol).all()), (b, (err - tol).max().item())
    return qasa, c, cache, lens, heads, done, table


@pytest.mark.parametrize("dtype,hkv,group,d,page,rot,interleaved,window,sinks", [
    ("f32", 2, 2, 64, 16, 64, False, 50, 4),
    ("f16", 2, 8, 128, 16, 128, False, 100, 20),
    ("bf16", 3, 1, 64, 32, 32, True, None, 0),
    ("bf16", 1, 4, 128, 32, 128, False, 64, 1),
])
def test_prompt_chunks_verification_and_decode(dtype, hkv, group, d, page, rot, interleaved, window, sinks):
    chunks = [[150, 33], [70, 129], [4, 4], [1, 1], [1, 1]]
    qasa, c, cache, lens, heads, done, table = _layer(dtype, hkv, group, d, page, rot, interleaved, window, sinks, chunks, 3)
    # the boxes that the rotating append keeps serve the page selection: with every page kept it is dense attention
    q = R.rotate(torch.stack([heads[b, done[b] - 1:done[b], :hkv * group] for b in range(2)]).flatten(0, 1), table, 0, False)
    q = q.to(R.VALUE[dtype]).view(2, hkv * group, d).contiguous()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, kept = qasa.sparse_decode_attention(cache, q, c.table, lens, c.table.shape[1], status=status)
    mine = qasa.window_attention(cache, q, c.table, lens, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for b in range(2):
        ref, weighed, size = R.attention(c, q[b:b + 1], b, done[b], 1, None, 0)
        tol = R.attention_tolerance(ref, weighed, size, d, R.VALUE[dtype])[0]
        assert bool(((out[b].double() - ref[0]).abs() <= 2e-3 + 1e-2 * ref[0].abs()).all())
        assert bool(((mine[b].double() - ref[0]).abs() <= tol).all())


def test_e4m3_decode_follows_the_cache():
    # codes are re-quantised as pages fill, so each step is checked against the cache as it then is
    from query_aware_sparse_append_gb300 import binding as qasa
    hkv, hq, d, page, T = 2, 8, 128, 16, 70
    c = R.Paged("e4m3", [0, 0], hkv, d, page, seed=33, reserve=T + 20)
    cache = c.library()
    table = qasa.rotation_table(T + 20, 64, device="cuda")
    g = torch.Generator(device="cpu").manual_seed(34)
    lens, done = torch.zeros(2, dtype=torch.int32, device="cuda"), [0, 0]
    for n in ([T, 40], [1, 1], [5, 5], [1, 1], [1, 1]):
        x = (torch.randn((2, max(n), hq + 2 * hkv, d), generator=g) * 2).half().cuda()
        counts = torch.tensor(n, dtype=torch.int32, device="cuda")
        q = qasa.kv_append_rotated(cache, c.table, lens, x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], table, q=x[:, :, :hq],
                                   append_lens=counts)
        lens = lens + counts
        out = qasa.window_attention(cache, q, c.table, lens, 30, 3, q_lens=counts)
        torch.cuda.synchronize()
        for b in range(2):
            done[b] += n[b]
            ref, weighed, size = R.attention(c, q[b], b, done[b], n[b], 30, 3)
            tol = R.attention_tolerance(ref, weighed, size, d, torch.float16)
            assert bool(((out[b, :n[b]].double() - ref).abs() <= tol).all()), (n, b)
