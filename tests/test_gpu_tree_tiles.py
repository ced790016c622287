"""Tree attention over many key tiles per CTA with 64 channels and one row tile, every page of an E4M3 cache with
scales of its own: against 64-bit attention, and the same bits in every run."""
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
@pytest.mark.parametrize("dtype,spread", [("e4m3", 2.0), ("f16", 0.0), ("bf16", 0.0)])
@pytest.mark.parametrize("T,group", [(16, 8), (5, 6), (1, 8)])
@pytest.mark.parametrize("page", [16, 32])
def test_many_tiles_of_one_row_tile(form, dtype, spread, T, group, page, monkeypatch):
    # 160 units of 20 and 21 tiles: as many for each CTA, whole or cut
    from query_aware_sparse_append_gb300 import binding as qasa
    if form == "rule":
        monkeypatch.delenv("QASA_TREE_FORM", raising=False)
    else:
        monkeypatch.setenv("QASA_TREE_FORM", form)
    hkv, lens = 8, [2560 + T + 7 * b for b in range(19)] + [2560]
    c = R.Paged(dtype, lens, hkv, 64, page, seed=101, amax_spread=spread)
    g = torch.Generator(device="cpu").manual_seed(102)
    q = (torch.randn((len(lens), T, hkv * group, 64), generator=g) * 1.5).to(R.VALUE[dtype]).cuda()
    rows = [X.tree_rows(X.random_parents(T, g))[0] for _ in lens]
    mask = torch.stack([X.words(r, T) for r in rows]).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = [qasa.tree_attention(c.library(), q, c.table, c.seq_lens, mask, status=status) for _ in range(6)]
    torch.cuda.synchronize()
    assert int(status) == 0
    for other in out[1:]:
        assert torch.equal(out[0], other)
    for b, L in enumerate(lens):
        ref, weighed, size = X.attention(c, q[b], b, L, T, rows[b], None, 0)
        tol = R.attention_tolerance(ref, weighed, size, c.d, R.VALUE[dtype])
        err = (out[0][b].double() - ref).abs()
        assert bool((err <= tol).all()), (b, L, err.max().item(), (err - tol).max().item())
