"""Tree attention of as many drafted tokens as a call takes: all words of a mask row, blocks of every group size."""
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


@pytest.mark.parametrize("form", ["rule", "whole", "cut"])
@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
@pytest.mark.parametrize("T,group,d,page", [(1024, 3, 64, 16), (1024, 8, 128, 16), (1023, 1, 128, 32), (993, 7, 64, 32)])
@pytest.mark.parametrize("window,sinks", [(None, 0), (100, 1 << 30), (1, 0)])
def test_most_drafted_tokens(form, dtype, T, group, d, page, window, sinks, monkeypatch):
    from query_aware_sparse_append_gb300 import binding as qasa
    if form == "rule":
        monkeypatch.delenv("QASA_TREE_FORM", raising=False)
    else:
        monkeypatch.setenv("QASA_TREE_FORM", form)
    lens, n = [T, T + 500, T + 77], [T, T, T - 31]
    c = R.Paged(dtype, lens, 1, d, page, seed=151, amax_spread=0.5)
    g = torch.Generator(device="cpu").manual_seed(152)
    q = torch.randn((3, T, group, d), generator=g).to(R.VALUE[dtype]).cuda()
    rows = [X.tree_rows(X.random_parents(T, g))[0] for _ in lens]
    mask = torch.stack([X.words(r, T) for r in rows]).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 9.0)
    qasa.tree_attention(c.library(), q, c.table, c.seq_lens, mask, q_lens=torch.tensor(n, dtype=torch.int32, device="cuda"),
                        window=window, sink_tokens=sinks, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for b, L in enumerate(lens):
        ref, weighed, size = X.attention(c, q[b], b, L, n[b], rows[b], window, sinks)
        tol = R.attention_tolerance(ref, weighed, size, d, R.VALUE[dtype])
        err = (out[b, :n[b]].double() - ref).abs()
        assert bool((err <= tol).all()), (b, (err - tol).max().item())
        assert bool((out[b, n[b]:] == 9.0).all())
