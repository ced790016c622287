"""A call given a stream makes its outputs, workspace and budget there: the current stream, tens of milliseconds
behind, neither fills nor overwrites them."""
import pytest
import torch

from query_aware_sparse_append_gb300 import workloads as W
from tests import harness as H

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from query_aware_sparse_append_gb300 import build
    build.build()


@pytest.fixture(scope="module")
def case():
    return H.make_case(W.CONFIGS["tinyllama"].with_batch(4), seed=71)


def _calls(case):
    from query_aware_sparse_append_gb300 import binding as qasa
    c, q, bt, lens = case.cache, case.q_dev, case.bt, case.lens_dev
    k = 8
    kept = qasa.select_pages(c, q, bt, lens, k, k)
    budget = torch.full((q.shape[0],), k, dtype=torch.int32, device="cuda")
    mass = qasa.page_attention_mass(c, q, bt, lens)
    return {
        "select": lambda s: (qasa.select_pages(c, q, bt, lens, k, k, stream=s),),
        "sparse": lambda s: (qasa.sparse_attention(c, q, bt, lens, k, kept, stream=s),),
        "decode": lambda s: qasa.sparse_decode_attention(c, q, bt, lens, k, k, stream=s),
        "dense": lambda s: (qasa.dense_decode_attention(c, q, bt, lens, stream=s),),
        "mass": lambda s: (qasa.page_attention_mass(c, q, bt, lens, stream=s),),
        "hits": lambda s: qasa.page_hit_rate(c, mass, lens, budget, kept, stream=s),
    }


@pytest.mark.parametrize("name", ["select", "sparse", "decode", "dense", "mass", "hits"])
def test_what_a_call_makes_is_made_on_its_stream(case, name):
    call = _calls(case)[name]
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
        assert bool((a == b).all())
