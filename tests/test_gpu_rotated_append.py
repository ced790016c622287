"""kv_append_rotated against 64-bit rotation, against kv_append and against boxes rebuilt from the pool."""
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


def _qasa():
    from query_aware_sparse_append_gb300 import binding
    return binding


def _bits(t):
    return t.contiguous().view(torch.uint8)


def _new_rows(c, T, hq, seed=1, fused=True):
    g = torch.Generator(device="cpu").manual_seed(seed)
    B, H = len(c.lens), hq + 2 * c.hkv
    x = torch.randn((B, T, H, c.d), generator=g).to(R.VALUE[c.dtype]).to(c.device)
    parts = x[:, :, :hq], x[:, :, hq:hq + c.hkv], x[:, :, hq + c.hkv:]
    return parts if fused else tuple(p.contiguous() for p in parts)


def _slots(c, b, first, n):
    pos = torch.arange(first, first + n, device=c.device)
    return c.table[b].long()[pos // c.page], pos % c.page


CASES = [
    # dtype, d, page, hkv, hq, rot, interleaved, lengths before, tokens, counts
    ("f32", 64, 16, 4, 4, 64, False, [2047], 1, None),
    ("f32", 128, 32, 2, 6, 32, True, [0, 31, 33], 40, [40, 1, 0]),
    ("f16", 128, 16, 4, 32, 128, False, [0, 15, 16, 17, 300], 1, None),
    ("f16", 128, 16, 1, 8, 64, True, [5, 0, 48], 37, [37, 16, 20]),
    ("f16", 64, 32, 3, 3, 16, False, [100, 7], 70, None),
    ("bf16", 128, 32, 8, 32, 128, True, [37, 64], 65, [65, 33]),
    ("bf16", 64, 16, 5, 35, 48, False, [1, 2, 3], 19, [0, 19, 7]),
    ("e4m3", 128, 16, 4, 32, 128, False, [0, 9, 16, 40], 1, None),
    ("e4m3", 128, 32, 2, 2, 64, True, [20, 0, 64], 50, [50, 3, 0]),
    ("e4m3", 64, 16, 3, 9, 16, False, [14, 31], 33, [33, 2]),
]


@pytest.mark.parametrize("dtype,d,page,hkv,hq,rot,interleaved,lens,T,counts", CASES)
def test_rows_boxes_and_queries(dtype, d, page, hkv, hq, rot, interleaved, lens, T, counts):
    qasa = _qasa()
    c = R.Paged(dtype, lens, hkv, d, page, seed=3, reserve=T)
    q, k, v = _new_rows(c, T, hq)
    table = qasa.rotation_table(max(lens) + T, rot, device="cuda")
    n = counts or [T] * len(lens)
    cache = c.library()
    before = [t.clone() for t in (c.k_pool, c.v_pool, c.bounds)] + ([c.scales.clone()] if c.scales is not None else [])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.full((len(lens), T, hq, d), 7.0, dtype=R.VALUE[dtype], device="cuda")
    got = qasa.kv_append_rotated(cache, c.table, c.seq_lens, k, v, table, q=q, q_out=q_out, interleaved=interleaved,
                                 append_lens=torch.tensor(counts, dtype=torch.int32, device="cuda") if counts else None,
                                 status=status)
    assert got is q_out
    torch.cuda.synchronize()
    assert int(status) == 0
    u = R.half_step(R.VALUE[dtype])
    touched = torch.zeros(c.count, dtype=torch.bool, device="cuda")
    written = torch.zeros((c.count, page), dtype=torch.bool, device="cuda")
    for b, L in enumerate(lens):
        # queries: one rounding of the fp32 rotation, whose two products and sum are each half a step off
        ref = R.rotate(q[b, :n[b]], table, L, interleaved)
        slack = 3 * 2.0 ** -24 * 2 * q[b, :n[b]].double().abs().amax() if n[b] else 0.0
        err = (q_out[b, :n[b]].double() - ref).abs()
        assert bool((err <= u * ref.abs() + slack + 1e-7).all())
        assert bool((q_out[b, n[b]:] == 7.0).all()), "rows behind the last token were written"
        if n[b] == 0:
            continue
        at, slot = _slots(c, b, L, n[b])
        touched[at] = True
        written[at, slot] = True
        rk = R.rotate(k[b, :n[b]], table, L, interleaved)
        for w, (pool, x) in enumerate(((c.k_pool, rk), (c.v_pool, v[b, :n[b]].double()))):
            stored = pool[at, :, slot]
            if dtype == "e4m3":
                s = (c.scales[at][:, :, w].double() / 448.0)[..., None]
                val = stored.view(R.F8).double() * s
                # half a step of three mantissa bits, or of the smallest exponent's 2^-9; 2^-20 for the fp32 steps
                tol = torch.maximum(x.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20) + 2.0 ** -20
                assert bool(((val - x).abs() <= tol).all())
            elif w == 0:
                assert bool(((stored.double() - x).abs() <= u * x.abs() + 6 * 2.0 ** -24 * x.abs().amax() + 1e-7).all())
            else:
                assert torch.equal(stored.double(), x)
    # what the call does not own stays as it was
    for t, old in zip((c.k_pool, c.v_pool, c.bounds), before):
        assert torch.equal(_bits(t[~touched]), _bits(old[~touched]))
    if dtype != "e4m3":
        keep = ~written[:, None, :, None].expand_as(c.k_pool)
        for t, old in zip((c.k_pool, c.v_pool), before):
            assert torch.equal(_bits(t[keep]), _bits(old[keep]))
    else:
        assert torch.equal(_bits(c.scales[~touched]), _bits(before[3][~touched]))
    # the boxes are those of the stored keys
    mine = c.bounds.clone()
    after = torch.tensor([L + m for L, m in zip(lens, n)], dtype=torch.int32, device="cuda")
    qasa.rebuild_page_bounds(cache, c.table, after, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert torch.equal(_bits(mine[touched]), _bits(c.bounds[touched]))


@pytest.mark.parametrize("dtype,interleaved", [("f32", True), ("f16", False), ("bf16", True), ("e4m3", False), ("e4m3", True)])
def test_angles_of_zero_are_kv_append(dtype, interleaved):
    # cos 1, sin 0: the stored bits, boxes, scales and re-quantised codes are kv_append's
    qasa = _qasa()
    lens, T, counts = [0, 13, 32, 47], 21, [21, 5, 0, 17]
    pools = []
    for rotated in (False, True):
        c = R.Paged(dtype, lens, 3, 128, 16, seed=5, reserve=T)
        q, k, v = _new_rows(c, T, 3, fused=rotated)
        n = torch.tensor(counts, dtype=torch.int32, device="cuda")
        k, v = k * 3, v * 3           # the scales of half-filled E4M3 pages grow
        if rotated:
            table = torch.zeros((128, 2, 32), device="cuda")
            table[:, 0] = 1.0
            out = qasa.kv_append_rotated(c.library(), c.table, c.seq_lens, k, v, table, q=q, append_lens=n,
                                         interleaved=interleaved)
            for b in range(4):
                assert torch.equal(out[b, :counts[b]], q[b, :counts[b]])
        else:
            qasa.kv_append(c.library(), c.table, c.seq_lens, k.contiguous(), v.contiguous(), append_lens=n)
        torch.cuda.synchronize()
        pools.append([c.k_pool, c.v_pool, c.bounds] + ([c.scales] if c.scales is not None else []))
    for a, b in zip(*pools):
        assert torch.equal(_bits(a), _bits(b))


def test_strides_without_queries_and_in_place():
    qasa = _qasa()
    c = R.Paged("f16", [3, 20], 2, 64, 16, seed=8, reserve=8)
    d = R.Paged("f16", [3, 20], 2, 64, 16, seed=8, reserve=8)
    q, k, v = _new_rows(c, 8, 4)
    table = qasa.rotation_table(64, 64, device="cuda")
    first = qasa.kv_append_rotated(c.library(), c.table, c.seq_lens, k, v, table, q=q)
    # tokens before sequences in memory, keys alone, the queries rotated in their own place
    flip = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in (k, v)]
    assert qasa.kv_append_rotated(d.library(), d.table, d.seq_lens, flip[0], flip[1], table) is None
    own = q.contiguous()
    assert qasa.kv_append_rotated(d.library(), d.table, d.seq_lens, k, v, table, q=own, q_out=own) is own
    torch.cuda.synchronize()
    assert torch.equal(first, own)
    for a, b in ((c.k_pool, d.k_pool), (c.v_pool, d.v_pool), (c.bounds, d.bounds)):
        assert torch.equal(_bits(a), _bits(b))


def test_bad_lengths_pages_and_positions_are_reported():
    qasa = _qasa()
    T = 4
    table = qasa.rotation_table(40, 64, device="cuda")

    def run(lens, counts=None, edit=None, tab=table):
        c = R.Paged("f16", [max(0, min(x, 60)) for x in lens], 2, 64, 16, seed=9, reserve=T)
        c.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if edit:
            edit(c)
        q, k, v = _new_rows(c, T, 2)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        old = c.k_pool.clone()
        out = torch.full((len(lens), T, 2, 64), 7.0, dtype=torch.float16, device="cuda")
        n = None if counts is None else torch.tensor(counts, dtype=torch.int32, device="cuda")
        qasa.kv_append_rotated(c.library(), c.table, c.seq_lens, k, v, tab, q=q, q_out=out, append_lens=n, status=status)
        torch.cuda.synchronize()
        return int(status), c, old, out

    st, c, old, out = run([-1, 5])
    assert st == 0x2 and bool((out[0] == 7).all()) and not bool((out[1] == 7).any(-1).all())
    st, c, old, out = run([5, 5], counts=[-3, 9])
    assert st == 0x10 and bool((out[0] == 7).all()) and not bool((out[1] == 7).all(-1).any())
    # positions 38 .. 41 of a table of 40: two tokens go in, two are left out
    st, c, old, out = run([38, 50])
    assert st == 0x40
    assert not bool((out[0, :2] == 7).all(-1).any()) and bool((out[0, 2:] == 7).all()) and bool((out[1] == 7).all())
    at = int(c.table[0, 2])
    assert bool(c.k_pool[at, :, 6:8].isfinite().all())
    assert torch.equal(_bits(c.k_pool[at, :, 8:]), _bits(old[at, :, 8:]))
    # a bad page: nothing stored, the query rotated all the same
    def bad(c):
        c.table[1, 0] = c.count
    st, c, old, out = run([2, 3], edit=bad)
    assert st == 0x1 and not bool((out[1] == 7).all(-1).any())
    # past the block table
    def short(c):
        c.table = c.table[:, :1].contiguous()
    st, c, old, out = run([15, 0], edit=short)
    assert st == 0x2 and not bool((out[0] == 7).all(-1).any())
    # nothing to do
    st, c, old, out = run([2, 3], counts=[0, 0])
    assert st == 0 and torch.equal(_bits(c.k_pool), _bits(old)) and bool((out == 7).all())
