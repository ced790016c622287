"""A sequence with a bad length, count, position or page leaves the others of a rotating append untouched: what is
stored of them, their boxes, scales and queries, are those of a call of their own."""
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


LENS, COUNTS, T, D, PAGE, HQ, HKV = [37, 13, 0], [9, 20, 11], 20, 64, 16, 6, 2


def _negative_length(c, lens, n):
    lens[1] = -7


def _negative_count(c, lens, n):
    n[1] = -1


def _beyond_the_table(c, lens, n):
    lens[1] = 5000


def _bad_page(c, lens, n):
    c.table[1, 0] = c.count


def _past_the_block_table(c, lens, n):
    lens[1] = 100 * PAGE


@pytest.mark.parametrize("break_,bits", [(_negative_length, 0x2), (_negative_count, 0x10), (_beyond_the_table, 0x40),
                                         (_bad_page, 0x1), (_past_the_block_table, 0x2)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "e4m3"])
def test_the_others_are_as_in_a_call_of_their_own(dtype, break_, bits):
    from query_aware_sparse_append_gb300 import binding as qasa
    g = torch.Generator(device="cpu").manual_seed(92)
    x = torch.randn((3, T, HQ + 2 * HKV, D), generator=g).to(R.VALUE[dtype]).cuda()
    table = qasa.rotation_table(2048, D)

    def call(rows, spoil):
        c = R.Paged(dtype, LENS, HKV, D, PAGE, seed=91, reserve=T)
        lens, n = list(LENS), list(COUNTS)
        if spoil:
            break_(c, lens, n)
        lens, n = (torch.tensor([v[b] for b in rows], dtype=torch.int32, device="cuda") for v in (lens, n))
        y = x[rows]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((len(rows), T, HQ, D), 7.0, dtype=R.VALUE[dtype], device="cuda")
        qasa.kv_append_rotated(c.library(), c.table[rows].contiguous(), lens, y[:, :, HQ:HQ + HKV], y[:, :, HQ + HKV:], table,
                               q=y[:, :, :HQ], q_out=out, append_lens=n, status=status)
        torch.cuda.synchronize()
        return c, out, int(status)

    mine, out, st = call([0, 1, 2], True)
    assert st == bits, hex(st)
    for b in (0, 2):
        own, q, st = call([b], False)
        assert st == 0
        assert bool((q[0, :COUNTS[b]] != 7.0).any(-1).all())
        assert bool((out[b] == q[0]).all())
        at = own.table[b, :-(-(LENS[b] + COUNTS[b]) // PAGE)].long()
        for name in ("k_pool", "v_pool", "bounds", "scales"):
            a, e = getattr(mine, name), getattr(own, name)
            if a is not None:
                assert bool((a[at].view(torch.uint8) == e[at].view(torch.uint8)).all()), name
    # the bad sequence stored nothing (beside a bad page, its other page takes its rows)
    pages = mine.table[1, :3].long()
    pages = pages[(pages >= 0) & (pages < mine.count)]
    fresh = R.Paged(dtype, LENS, HKV, D, PAGE, seed=91, reserve=T)
    if break_ is not _bad_page:
        assert bool((mine.k_pool[pages].view(torch.uint8) == fresh.k_pool[pages].view(torch.uint8)).all())
        assert bool((mine.v_pool[pages].view(torch.uint8) == fresh.v_pool[pages].view(torch.uint8)).all())


def test_the_largest_number_of_tokens():
    # rows of one token repeated (a stride of 0): the call has room for 2^31 - 1 tokens and appends 40
    from query_aware_sparse_append_gb300 import binding as qasa
    most = 2 ** 31 - 1
    c = R.Paged("f16", [5], 1, D, PAGE, seed=93, reserve=40)
    e = R.Paged("f16", [5], 1, D, PAGE, seed=93, reserve=40)
    row = torch.randn((1, 1, 1, D), generator=torch.Generator(device="cpu").manual_seed(94)).half().cuda()
    table = qasa.rotation_table(64, D)
    n = torch.tensor([40], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for x, tokens in ((c, most), (e, 40)):
        rows = row.expand(1, tokens, 1, D)
        qasa.kv_append_rotated(x.library(), x.table, x.seq_lens, rows, rows, table, append_lens=n, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    for name in ("k_pool", "v_pool", "bounds"):
        assert bool((getattr(c, name).view(torch.uint8) == getattr(e, name).view(torch.uint8)).all()), name
