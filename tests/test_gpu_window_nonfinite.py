"""A query with a NaN or an infinity gives a row of NaN, in every form of windowed attention, and leaves
the other rows alone."""
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


# One token, a few, a part of a row tile, several row tiles; alone (the prompt kernel in single CTAs, decode in
# clusters of two) and behind enough keys that clusters share them.
@pytest.mark.parametrize("value,prefix", [(float("nan"), 0), (float("nan"), 900), (float("inf"), 900)])
@pytest.mark.parametrize("T", [1, 6, 40, 200])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "e4m3"])
def test_a_query_that_is_not_finite(dtype, d, page, T, value, prefix):
    from query_aware_sparse_append_gb300 import binding as qasa
    hkv, group = 2, 4
    lens = [T + prefix, T + 30, T]
    c = R.Paged(dtype, lens, hkv, d, page, seed=41)
    g = torch.Generator(device="cpu").manual_seed(42)
    q = torch.randn((3, T, hkv * group, d), generator=g).to(R.VALUE[dtype]).cuda()
    broken = q.clone()
    at = [(0, T // 2, 1), (1, T - 1, hkv * group - 1)]
    for b, t, h in at:
        broken[b, t, h, d // 2 + 3] = value
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = qasa.window_attention(c.library(), broken, c.table, c.seq_lens, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    bad = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    for i in at:
        # of an infinity the few keys of the second sequence might all be on one side
        if value != value or i[0] == 0:
            assert bool(out[i].isnan().all()), i
        bad[i] = True
    for b, L in enumerate(lens):
        ref, weighed, size = R.attention(c, q[b], b, L, T, None, 0)
        tol = R.attention_tolerance(ref, weighed, size, d, R.VALUE[dtype])
        err = (out[b].double() - ref).abs()
        assert bool((err <= tol)[~bad[b]].all()), (b, (err - tol)[~bad[b]].max().item())


@pytest.mark.parametrize("dtype", ["f32", "f16", "e4m3"])
@pytest.mark.parametrize("T", [3, 200])
def test_a_query_that_sees_nothing_gives_zeros_whatever_it_holds(dtype, T):
    from query_aware_sparse_append_gb300 import binding as qasa
    c = R.Paged(dtype, [T - 2], 2, 64, 16, seed=43)
    q = torch.full((1, T, 4, 64), float("nan"), dtype=R.VALUE[dtype], device="cuda")
    out = qasa.window_attention(c.library(), q, c.table, c.seq_lens)
    torch.cuda.synchronize()
    assert bool((out[0, :2] == 0).all()) and bool(out[0, 2:].isnan().all())
