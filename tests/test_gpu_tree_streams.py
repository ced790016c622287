"""A call given a stream makes its outputs and workspace there: the current stream, tens of milliseconds
behind, neither fills nor overwrites them."""
import pytest
import torch

from tests import paged_reference as R

pytestmark = pytest.mark.gpu

LENS = [90, 200, 33]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from query_aware_sparse_append_gb300 import build
    build.build()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _case(dtype):
    """A call of each kind that returns what it makes and changes nothing that another reads."""
    from query_aware_sparse_append_gb300 import binding as qasa
    c = R.Paged(dtype, LENS, 2, 64, 16, seed=91, reserve=40)
    lib, value = c.library(), R.VALUE[dtype]
    g = torch.Generator(device="cpu").manual_seed(92)
    x = torch.randn((3, 24, 12, 64), generator=g).to(value).cuda()
    q, k, v = x[:, :, :8], x[:, :, 8:10], x[:, :, 10:]
    parents = _ints([[i // 2 - 1 for i in range(24)]] * 3)
    mask, _ = qasa.tree_masks(parents)
    table, positions = qasa.rotation_table(300, 64, device="cuda"), _ints([list(range(24))] * 3)
    dense, lens = q.contiguous(), c.seq_lens
    starts, keep = _ints(LENS), torch.empty((3, 0), dtype=torch.int32, device="cuda")
    of, new = _ints([0, 1, 2]), _ints([int(c.table[1, 14]), -1, -1])
    return {
        "masks": lambda s: qasa.tree_masks(parents, stream=s),
        "tree": lambda s: (qasa.tree_attention(lib, dense, c.table, lens, mask, stream=s),),
        "append": lambda s: (qasa.kv_append_positioned(lib, c.table, lens, k, v, table, positions, q=q, stream=s),),
        "keep": lambda s: (qasa.kv_keep_tokens(lib, c.table, lens, starts, keep, stream=s),),
        "fork": lambda s: qasa.kv_fork(lib, c.table, lens, of, new, stream=s),
    }


@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
@pytest.mark.parametrize("name", ["masks", "tree", "append", "keep", "fork"])
def test_what_a_call_makes_is_made_on_its_stream(dtype, name):
    calls = _case(dtype)
    call = calls[name]
    expected = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    late = [torch.empty_like(x) for x in expected]
    torch.cuda._sleep(100_000_000)
    for x in late:
        x.fill_(1)
    del late, x
    got = call(side)
    torch.cuda.synchronize()
    for a, b in zip(got, expected):
        assert torch.equal(a, b)
