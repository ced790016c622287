"""The tree kernel's bounded waits, made to run out: a limit of 1 us is over before the first keys are there.  The call
returns and reports it, every row of out is right or as it was, and the next call is right."""
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


@pytest.mark.parametrize("form", ["whole", "cut"])
@pytest.mark.parametrize("dtype", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("T,group", [(10, 8), (60, 4)])
@pytest.mark.parametrize("d", [64, 128])
def test_waits_that_run_out_are_reported_and_leave_rows_right_or_alone(form, dtype, T, group, d, monkeypatch):
    from query_aware_sparse_append_gb300 import binding as qasa
    monkeypatch.setenv("QASA_TREE_FORM", form)
    lens, hq = [4000, 3000, T], 2 * group
    c = R.Paged(dtype, lens, 2, d, 16, seed=121)
    g = torch.Generator(device="cpu").manual_seed(122)
    q = torch.randn((3, T, hq, d), generator=g).to(R.VALUE[dtype]).cuda()
    rows = [X.tree_rows(X.random_parents(T, g))[0] for _ in lens]
    mask = torch.stack([X.words(r, T) for r in rows]).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def right(out, b):
        ref, weighed, size = X.attention(c, q[b], b, lens[b], T, rows[b], None, 0)
        tol = R.attention_tolerance(ref, weighed, size, d, R.VALUE[dtype])
        return ((out[b].double() - ref).abs() <= tol).all(-1)

    away = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 9.0)
    monkeypatch.setenv("QASA_WAIT_LIMIT_NS", "1000")
    away.zero_()                                                # more than L2 holds: the keys come from memory
    qasa.tree_attention(c.library(), q, c.table, c.seq_lens, mask, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0x8, hex(int(status))
    left = 0
    for b in range(3):
        alone = (out[b] == 9.0).all(-1)
        left += int(alone.sum())
        assert bool((alone | right(out, b)).all()), (b, int(alone.sum()), alone.numel())
    assert left > 0
    monkeypatch.delenv("QASA_WAIT_LIMIT_NS")
    status.zero_()
    qasa.tree_attention(c.library(), q, c.table, c.seq_lens, mask, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert all(bool(right(out, b).all()) for b in range(3))
