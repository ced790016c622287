"""Kept tokens of an E4M3 cache whose rows hold a NaN next to their largest value, coming from pages of a larger scale:
the NaN counts for nothing, the finite values beside it for what they are."""
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


@pytest.mark.parametrize("hkv,d,page", [(2, 64, 16), (1, 128, 32)])
@pytest.mark.parametrize("code", [0x7F, 0xFF])
@pytest.mark.parametrize("whole_row", [False, True])
def test_a_nan_takes_no_finite_value_out_of_the_scale(hkv, d, page, code, whole_row):
    from query_aware_sparse_append_gb300 import binding as qasa
    L, start = 6 * page, 5
    keep = [page + 1, 2 * page + 3, 2 * page + 9, 4 * page, 4 * page + 7]      # all to the first page's end and beyond
    keep += list(range(4 * page + 8, 4 * page + 8 + page))
    c = R.Paged("e4m3", [L], hkv, d, page, seed=111)
    c.scales[c.table[0, 2:6].long()] *= 40.0                    # the tokens that come outgrow the pages that they come to
    was = X.stored(c)
    ids = c.table[0, :6].long()
    tokens = [start + k for k in keep]
    for pool in (c.k_pool, c.v_pool):
        for t in tokens[::2]:
            row = pool[ids[t // page], :, t % page]             # [hkv, d]
            if whole_row:
                row[:] = code
            else:
                at = (row.view(R.F8).float().abs().argmax(-1, keepdim=True)) ^ 1     # the largest one's neighbour
                row.scatter_(-1, at, code)
            pool[ids[t // page], :, t % page] = row
    holes = X.stored(c)
    out = qasa.kv_keep_tokens(c.library(), c.table, c.seq_lens, torch.tensor([start], dtype=torch.int32, device="cuda"),
                              torch.tensor([keep], dtype=torch.int32, device="cuda"))
    assert out.tolist() == [start + len(keep)]
    now = X.stored(c)
    for w, name in enumerate("kv"):
        for p in range(-(-(start + len(keep)) // page)):
            at, lo, hi = int(ids[p]), p * page, min(p * page + page, start + len(keep))
            amax = was["scales"][at, :, w].clone()
            src = [pos if pos < start else tokens[pos - start] for pos in range(lo, hi)]
            values = torch.stack([holes[name][ids[s // page], :, s % page] * (was["scales"][ids[s // page], :, w] / 448)[:, None]
                                  for s in src], 1)             # [hkv, rows, d]
            for i, s in enumerate(src):
                if s // page != p:
                    amax = torch.maximum(amax, values[:, i].abs().nan_to_num(0.0).amax(-1))
            got = now["scales"][at, :, w]
            # amax is a code times a scale: two fp32 roundings
            assert bool(((got - amax).abs() <= 2.0 ** -22 * amax).all()), (name, p, (got / amax).tolist())
            step = (got / 448)[:, None, None]
            there = now[name][at, :, :hi - lo] * step
            assert torch.equal(there.isnan(), values.isnan())
            # half a code's step: 2^-4 of the value, 2^-10 of the scale where codes are subnormal; 2^-20 for quotients on a border
            off = (there - values).abs().nan_to_num(0.0)
            assert bool((off <= (2.0 ** -4 + 2.0 ** -20) * values.abs().nan_to_num(0.0) + 2.0 ** -10 * step).all()), (name, p)
            if w == 0:
                keys = now["k"][at, :, :hi - lo]
                low, high = keys.nan_to_num(nan=float("inf")).amin(1), keys.nan_to_num(nan=-float("inf")).amax(1)
                some = ~keys.isnan().all(1)
                assert bool((now["box"][at, :, 0] == low)[some].all()) and bool((now["box"][at, :, 1] == high)[some].all())
