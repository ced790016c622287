"""The prompt kernel's bounded waits, made to run out: a limit of 1 us is over before the first keys are there.
The call returns and reports it, every row of out is right or as it was, and the next call is right."""
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


def _right(c, q, out, b, L, n):
    ref, weighed, size = R.attention(c, q[b], b, L, n, None, 0)
    tol = R.attention_tolerance(ref, weighed, size, c.d, R.VALUE[c.dtype])
    return ((out[b].double() - ref).abs() <= tol).all(-1)


SINGLE = [400, 330]          # few keys: a CTA goes through all of its rows' keys itself
SHARED = [1200, 900]        # clusters of four share a row's keys


@pytest.mark.parametrize("dtype", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("d,lens", [(128, SINGLE), (64, SINGLE), (128, SHARED), (64, SHARED)])
def test_waits_that_run_out_are_reported_and_leave_rows_right_or_alone(dtype, d, lens, monkeypatch):
    from query_aware_sparse_append_gb300 import binding as qasa
    T = 300
    c = R.Paged(dtype, lens, 2, d, 16, seed=81)
    q = torch.randn((2, T, 8, d), generator=torch.Generator(device="cpu").manual_seed(82)).to(R.VALUE[dtype]).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 9.0)
    monkeypatch.setenv("QASA_WAIT_LIMIT_NS", "1000")
    qasa.window_attention(c.library(), q, c.table, c.seq_lens, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0x8, hex(int(status))
    for b, L in enumerate(lens):
        alone = (out[b] == 9.0).all(-1)
        assert bool((alone | _right(c, q, out, b, L, T)).all()), (b, int(alone.sum()), alone.numel())
    monkeypatch.delenv("QASA_WAIT_LIMIT_NS")
    status.zero_()
    qasa.window_attention(c.library(), q, c.table, c.seq_lens, out=out, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for b, L in enumerate(lens):
        assert bool(_right(c, q, out, b, L, T).all())
