"""Outputs and workspaces that a call makes itself belong to the stream that the call runs on: what the current
stream still has to do with memory it gave back may not meet them."""
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


def _leave_a_late_write(like):
    """Give back a block of this size that the current stream is still to write, tens of milliseconds from now."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = torch.empty_like(like)
    torch.cuda._sleep(100_000_000)
    x.fill_(9.0)


@pytest.mark.parametrize("dtype,T", [("f16", 1), ("bf16", 40), ("e4m3", 200), ("f32", 4)])
def test_window_attention_makes_its_output_on_the_call_s_stream(dtype, T):
    qasa = _qasa()
    c = R.Paged(dtype, [600 + T, T], 2, 128, 16, seed=61)
    cache = c.library()
    g = torch.Generator(device="cpu").manual_seed(62)
    q = torch.randn((2, T, 8, 128), generator=g).to(R.VALUE[dtype]).cuda()
    expected = qasa.window_attention(cache, q, c.table, c.seq_lens, 200, 4)
    side = torch.cuda.Stream()
    _leave_a_late_write(expected)
    out = qasa.window_attention(cache, q, c.table, c.seq_lens, 200, 4, stream=side)
    torch.cuda.synchronize()
    assert bool((out == expected).all())


@pytest.mark.parametrize("dtype,T", [("f16", 1), ("e4m3", 70)])
def test_rotating_append_makes_its_queries_on_the_call_s_stream(dtype, T):
    qasa = _qasa()
    lens = [5, 30]
    c = R.Paged(dtype, lens, 2, 64, 16, seed=63, reserve=T)
    g = torch.Generator(device="cpu").manual_seed(64)
    x = torch.randn((2, T, 4 + 4, 64), generator=g).to(R.VALUE[dtype]).cuda()
    q, k, v = x[:, :, :4], x[:, :, 4:6], x[:, :, 6:]
    table = qasa.rotation_table(T + 30, 64)
    expected = qasa.kv_append_rotated(c.library(), c.table, c.seq_lens, k, v, table, q=q)
    side = torch.cuda.Stream()
    _leave_a_late_write(expected)
    out = qasa.kv_append_rotated(c.library(), c.table, c.seq_lens, k, v, table, q=q, stream=side)
    torch.cuda.synchronize()
    assert bool((out == expected).all())


def test_the_workspace_comes_from_the_call_s_stream(monkeypatch):
    qasa = _qasa()
    c = R.Paged("e4m3", [600, 300], 2, 128, 16, seed=65)
    q = torch.randn((2, 200, 8, 128), generator=torch.Generator(device="cpu").manual_seed(66)).half().cuda()
    made_on = []
    alloc = qasa.alloc_window_workspace

    def spy(*a, **kw):
        made_on.append(torch.cuda.current_stream())
        return alloc(*a, **kw)

    monkeypatch.setattr(qasa, "alloc_window_workspace", spy)
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    first = qasa.window_attention(c.library(), q, c.table, c.seq_lens, 200, 4)
    second = qasa.window_attention(c.library(), q, c.table, c.seq_lens, 200, 4, stream=side)
    assert made_on == [here, side] and torch.cuda.current_stream() == here
    torch.cuda.synchronize()
    assert bool((first == second).all())


def test_a_layer_on_another_stream_that_lets_its_queries_go():
    # append, attend, drop the rotated queries, while the current stream allocates and writes blocks of their size
    qasa = _qasa()
    T, lens = 64, [100, 40]
    c = R.Paged("bf16", lens, 2, 128, 16, seed=67, reserve=T)
    cache = c.library()
    g = torch.Generator(device="cpu").manual_seed(68)
    x = torch.randn((2, T, 12, 128), generator=g).bfloat16().cuda()
    q, k, v = x[:, :, :8], x[:, :, 8:10], x[:, :, 10:]
    table = qasa.rotation_table(T + 100, 128)
    after = c.seq_lens + T

    def layer(stream):
        turned = qasa.kv_append_rotated(cache, c.table, c.seq_lens, k, v, table, q=q, stream=stream)
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(20_000_000)         # the queries are there; who attends with them comes late
        return qasa.window_attention(cache, turned, c.table, after, 50, 2, stream=stream)

    expected = layer(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(2):
        out = layer(side)
        held = [torch.empty_like(expected) for _ in range(4)]
        torch.cuda._sleep(5_000_000)                  # past the append
        for x in held:
            x.fill_(9.0)
        torch.cuda.synchronize()
        assert bool((out == expected).all())
