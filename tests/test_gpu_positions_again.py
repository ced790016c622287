"""A positioned append that skips tokens for positions outside the table, made again with good ones: the cache is then
that of one good call, whatever the pages held before."""
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


# E4M3 only from page borders: codes that are in a page already may be rounded twice where its scale grows twice
@pytest.mark.parametrize("dtype,lens", [("f32", [16, 0, 7]), ("f16", [16, 0, 7]), ("bf16", [5, 31, 32]), ("e4m3", [16, 0, 32])])
def test_a_call_made_again_with_good_positions(dtype, lens):
    from query_aware_sparse_append_gb300 import binding as qasa
    T, hkv, d = 40, 2, 64
    g = torch.Generator(device="cpu").manual_seed(141)
    x = torch.randn((3, T, 8, d), generator=g).to(R.VALUE[dtype]).cuda()
    table = qasa.rotation_table(100, 64, device="cuda")
    good = torch.arange(T, dtype=torch.int32, device="cuda").repeat(2, 3, 1)
    bad = good.clone()
    bad[0, 0, 3], bad[1, 1, 20] = -1, 100
    bad[1, 0, 16:32] = -5                                       # a page of sequence 0 gets no token at all
    bad[0, 2, :20] = 1 << 30                                    # nor do the first ones of sequence 2
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = []
    for calls in ([bad, good], [good]):
        c = R.Paged(dtype, lens, hkv, d, 16, seed=142, reserve=T)
        empty = torch.ones(c.count, dtype=torch.bool)           # pages of some earlier owner, with boxes and scales of its own
        for b, L in enumerate(lens):
            empty[c.table[b, :-(-L // 16)].long().cpu()] = False
        empty = empty.to("cuda")
        if dtype == "e4m3":
            c.scales[empty] = 1e4
            c.bounds[empty] = 0x7E
        else:
            c.bounds[empty] = 5e4
        for positions in calls:
            status.zero_()
            q = qasa.kv_append_positioned(c.library(), c.table, c.seq_lens, x[:, :, 4:6], x[:, :, 6:], table, positions,
                                          q=x[:, :, :4], pair_axes=[0, 1] * 16, status=status)
            torch.cuda.synchronize()
            assert int(status) == (0x40 if positions is bad else 0)
        got.append((q, X.stored(c)))
    assert torch.equal(got[0][0], got[1][0])
    for name in got[0][1]:
        assert X.same(got[0][1][name], got[1][1][name]), name
