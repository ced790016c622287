"""The positioned append, kept tokens, forks and page copies against plain statements, and a run of them together."""
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


def _qasa():
    from query_aware_sparse_append_gb300 import binding
    return binding


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ positioned append

def _axes(half, num, how):
    if how == "turns":
        return [i % num for i in range(half)]
    if how == "spans":
        return [min(num - 1, i * (num + 1) // half) for i in range(half)]
    return [(i * 7 + i // 3) % num for i in range(half)]        # no order


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "e4m3"])
@pytest.mark.parametrize("hkv,group,d,page,rot,interleaved", [(2, 4, 64, 16, 64, False), (1, 8, 128, 32, 128, True),
                                                              (3, 1, 128, 16, 32, False), (2, 2, 64, 32, 16, True)])
@pytest.mark.parametrize("num,how", [(1, "spans"), (2, "turns"), (3, "spans"), (3, "turns"), (3, "mixed")])
def test_positioned_append(dtype, hkv, group, d, page, rot, interleaved, num, how):
    qasa = _qasa()
    lens, n, T = [0, 5, 16, 33, 70], [21, 40, 0, 1, 40], 40
    c = R.Paged(dtype, lens, hkv, d, page, seed=61, reserve=T)
    B, hq, value = len(lens), hkv * group, R.VALUE[dtype]
    g = torch.Generator(device="cpu").manual_seed(62)
    x = torch.randn((B, T, hq + 2 * hkv, d), generator=g).to(value).cuda()
    q, k, v = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
    table = qasa.rotation_table(500, rot, device="cuda")
    positions = torch.randint(0, 500, (num, B, T), generator=g).to(torch.int32).cuda()
    axes = _axes(rot // 2, num, how)
    # the same keys rotated beforehand, through the plain append
    plain = R.Paged(dtype, lens, hkv, d, page, seed=61, reserve=T)
    status = _status()
    cache = c.library()
    out = torch.full((B, T, hq, d), 9.0, dtype=value, device="cuda")
    got = qasa.kv_append_positioned(cache, c.table, c.seq_lens, k, v, table, positions, q=q, q_out=out, append_lens=_ints(n),
                                    pair_axes=axes, interleaved=interleaved, status=status)
    torch.cuda.synchronize()
    assert got is out and int(status) == 0
    u = R.half_step(value)
    turned = torch.zeros((B, T, hkv, d), dtype=torch.float64, device="cuda")
    for b in range(B):
        turned[b] = X.rotate(k[b], table, positions[:, b], axes, interleaved)
        ref = X.rotate(q[b, :n[b]], table, positions[:, b, :n[b]], axes, interleaved)
        # one rounding to the type, after two products and a sum in fp32
        tol = u * ref.abs() + 3 * 2.0 ** -24 * 2 * q[b, :n[b]].double().abs().amax(-1, keepdim=True)
        assert bool(((out[b, :n[b]].double() - ref).abs() <= tol).all())
        assert bool((out[b, n[b]:] == 9.0).all())
    # what the cache then holds, in 64 bits from what it held
    was, now = X.stored(plain), X.stored(c)
    touched = torch.zeros(c.count, dtype=torch.bool)
    for b, L in enumerate(lens):
        for page_no in range(L // page, -(-(L + n[b]) // page) if n[b] else 0):
            at = int(c.table[b, page_no])
            touched[at] = True
            lo, hi = max(L, page_no * page), min(L + n[b], page_no * page + page)
            a, e = lo - page_no * page, hi - page_no * page
            for w, (name, new) in enumerate((("k", turned[b]), ("v", v[b].double()))):
                rows = new[lo - L:hi - L].transpose(0, 1)
                size = v.double().abs().max() if w else k[b].double().abs().max()
                if dtype == "e4m3":
                    amax = rows.abs().amax(dim=(1, 2))
                    if a:
                        amax = torch.maximum(amax, was["scales"][at, :, w])
                    assert bool(((now["scales"][at, :, w] - amax).abs() <= 2.0 ** -21 * amax).all())
                    step = amax / 448
                    ref = rows / step[:, None, None]
                    tol = 2.0 ** -4 * ref.abs() + 2.0 ** -10 + 1e-4     # half a code's step, subnormals, near borders
                else:
                    ref = rows
                    tol = (u if w == 0 else 0) * ref.abs() + (3 * 2.0 ** -23 * size if w == 0 else 0)
                assert bool(((now[name][at, :, a:e] - ref).abs() <= tol).all()), (b, page_no, name)
                assert X.same(now[name][at, :, e:], was[name][at, :, e:])
                if a and dtype != "e4m3":
                    assert X.same(now[name][at, :, :a], was[name][at, :, :a])
            keys = now["k"][at, :, :e]
            assert X.same(now["box"][at, :, 0], keys.amin(1)) and X.same(now["box"][at, :, 1], keys.amax(1))
    for name in now:
        assert X.same(now[name][~touched], was[name][~touched])


@pytest.mark.parametrize("dtype", ["f32", "f16", "e4m3"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_slot_positions_give_the_rotating_append(dtype, interleaved):
    qasa = _qasa()
    lens, T = [3, 40, 0], 50
    B = len(lens)
    g = torch.Generator(device="cpu").manual_seed(63)
    x = torch.randn((B, T, 12, 128), generator=g).to(R.VALUE[dtype]).cuda()
    table = qasa.rotation_table(200, 64, device="cuda")
    caches = [R.Paged(dtype, lens, 2, 128, 16, seed=64, reserve=T) for _ in range(3)]
    qs = []
    for i, c in enumerate(caches):
        args = (c.library(), c.table, c.seq_lens, x[:, :, 8:10], x[:, :, 10:], table)
        pos = (c.seq_lens[:, None] + torch.arange(T, device="cuda", dtype=torch.int32)).contiguous()
        if i == 0:
            qs.append(qasa.kv_append_rotated(*args, q=x[:, :, :8], interleaved=interleaved))
        else:
            both = torch.stack([pos, pos, pos]) if i == 2 else pos
            qs.append(qasa.kv_append_positioned(*args, both, q=x[:, :, :8], interleaved=interleaved,
                                                pair_axes=[j % 3 for j in range(32)] if i == 2 else None))
    torch.cuda.synchronize()
    for i in (1, 2):
        assert torch.equal(qs[0], qs[i])
        for a, b in zip(X.stored(caches[0]).values(), X.stored(caches[i]).values()):
            assert X.same(a, b)


@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
def test_tokens_without_a_position_are_skipped_and_reported(dtype):
    qasa = _qasa()
    T, hkv, d = 40, 2, 64
    c = R.Paged(dtype, [16, 0, 7], hkv, d, 16, seed=65, reserve=T)
    was = X.stored(c)
    x = torch.randn((3, T, 8, d), generator=torch.Generator().manual_seed(66)).half().cuda()
    positions = torch.arange(T, dtype=torch.int32, device="cuda").repeat(2, 3, 1)
    positions[0, 0, 3], positions[1, 1, 20], positions[0, 2, 0] = -1, 100, 1 << 30
    positions[1, 0, 16:32] = -5                                # a page of sequence 0 gets no token at all
    out = torch.full((3, T, 4, d), 9.0, dtype=torch.float16, device="cuda")
    status = _status()
    qasa.kv_append_positioned(c.library(), c.table, c.seq_lens, x[:, :, 4:6], x[:, :, 6:], qasa.rotation_table(100, 64, device="cuda"),
                              positions, q=x[:, :, :4], q_out=out, pair_axes=[0, 1] * 16, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0x40
    now = X.stored(c)
    skipped = [{3, *range(16, 32)}, {20}, {0}]
    for b, L in enumerate(c.lens):
        for t in range(T):
            at, slot = int(c.table[b, (L + t) // 16]), (L + t) % 16
            if t in skipped[b]:
                assert bool((out[b, t] == 9.0).all())
                assert X.same(now["k"][at, :, slot], was["k"][at, :, slot])
                assert X.same(now["v"][at, :, slot], was["v"][at, :, slot])
            else:
                assert bool((out[b, t] != 9.0).any())
                if dtype == "f16":
                    assert X.same(now["v"][at, :, slot], x[b, t, 6:].double())
    at = int(c.table[0, 2])                                    # no token: nothing of the page changes
    for name in now:
        assert X.same(now[name][at], was[name][at])
    at = int(c.table[1, 1])                                    # the box has the page's other tokens alone
    keys = now["k"][at][:, [s for s in range(16) if 16 + s != 20]]
    assert X.same(now["box"][at, :, 0], keys.amin(1)) and X.same(now["box"][at, :, 1], keys.amax(1))


def test_positions_shared_by_sequences_and_axes():
    qasa = _qasa()
    T = 20
    x = torch.randn((3, T, 8, 64), generator=torch.Generator().manual_seed(67)).bfloat16().cuda()
    table = qasa.rotation_table(100, 64, device="cuda")
    one = torch.randint(0, 100, (1, T), generator=torch.Generator().manual_seed(68)).to(torch.int32).cuda()
    forms = [one, one.expand(3, T), one[None].expand(3, 3, T), one.repeat(2, 3, 1)]
    got = []
    for pos in forms:
        c = R.Paged("bf16", [5, 0, 31], 2, 64, 32, seed=69, reserve=T)
        q = qasa.kv_append_positioned(c.library(), c.table, c.seq_lens, x[:, :, 4:6], x[:, :, 6:], table, pos, q=x[:, :, :4],
                                      pair_axes=[i % 2 for i in range(32)] if pos.dim() == 3 else None)
        got.append((q, X.stored(c)))
    torch.cuda.synchronize()
    for q, r in got[1:]:
        assert torch.equal(q, got[0][0])
        assert all(X.same(r[name], got[0][1][name]) for name in r)


# ------------------------------------------------------------------------- kept tokens

def _random_kept(total, n, g):
    return sorted(torch.randperm(total, generator=g)[:n].tolist())


def _compare(now, want, dtype):
    """Everything equal, but that an E4M3 code may be the neighbouring one where both are nearly as far from the quotient.

    The library takes the even code where its quotient code * amax_src / amax lies within 2^-22 of a border between two
    codes, else the nearest.  Its amax has two fp32 roundings that the 64-bit one has not (the scale and a product), 2^-24
    each, the quotient's ends are rounded to fp32, 2^-24.  So a code other than the nearest one of the 64-bit quotient y
    lies on the other side of a border that is within (2^-22 + 2^-23 + 2^-24) y of y, less than 2^-21 y, and its distance
    from y exceeds the nearest one's by less than twice that.
    That is no rare event: amax is itself some code * s_src, so that quotients are 448 x / c of two codes x and c, which
    fall on borders exactly for some x, and then for every x of the page."""
    touched, quotients = want.pop("touched"), want.pop("quotients")
    if dtype != "e4m3":
        assert all(X.same(now[name], want[name]) for name in want)
        return
    for name in "kv":
        a, b, y = now[name], want[name], quotients[name]
        level = ((a - y).abs() - (b - y).abs()).abs() <= 2.0 ** -20 * y.abs()
        assert bool(((a == b) | (a.isnan() & b.isnan()) | level).all()), name
    assert bool((((now["scales"] - want["scales"]).abs() <= 2.0 ** -22 * want["scales"]) | want["scales"].isnan()).all())
    for at, rows in touched:                                   # the box of what is stored
        keys = now["k"][at, :, :rows]
        want["box"][at, :, 0], want["box"][at, :, 1] = keys.amin(1), keys.amax(1)
    assert X.same(now["box"], want["box"])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "e4m3"])
@pytest.mark.parametrize("hkv,d,page", [(1, 64, 16), (3, 128, 16), (2, 64, 32), (2, 128, 32)])
@pytest.mark.parametrize("M", [0, 1, 6, 40, 700])
def test_kept_tokens(dtype, hkv, d, page, M):
    qasa = _qasa()
    g = torch.Generator(device="cpu").manual_seed(71)
    starts = [0, 5, 16, 33, 100, 0, 64]
    extra = [M + 3, M + 40, M, 2 * M + 1, 0, 5 * M + 9, M + 1]
    lens = [s + e for s, e in zip(starts, extra)]
    n = [min(M, e) for e in extra]
    n[3], n[6] = n[3] // 2, 0
    kept = [_random_kept(e, k, g) for e, k in zip(extra, n)]
    kept[2] = list(range(n[2]))                                # nobody moves
    c = R.Paged(dtype, lens, hkv, d, page, seed=72, amax_spread=1.0)
    want = X.stored(c)
    for b in range(len(lens)):
        X.keep(c, b, lens[b], starts[b], kept[b], want)
    keep = torch.full((len(lens), M), -9, dtype=torch.int32)
    for b, k in enumerate(kept):
        keep[b, :len(k)] = torch.tensor(k, dtype=torch.int32)
    status, out = _status(), torch.full((len(lens),), -1, dtype=torch.int32, device="cuda")
    got = qasa.kv_keep_tokens(c.library(), c.table, c.seq_lens, _ints(starts), keep.cuda(), keep_lens=_ints(n), lens_out=out,
                              status=status)
    torch.cuda.synchronize()
    assert got is out and int(status) == 0
    assert out.tolist() == [s + k for s, k in zip(starts, n)]
    _compare(X.stored(c), want, dtype)


@pytest.mark.parametrize("dtype", ["f16", "e4m3", "f32"])
def test_long_lists_in_several_rounds(dtype):
    # more pages than a cluster of CTAs holds at once
    qasa = _qasa()
    g = torch.Generator(device="cpu").manual_seed(73)
    lens, starts, n = [5000, 4000], [17, 0], [2900, 3990]
    c = R.Paged(dtype, lens, 1, 128 if dtype == "f32" else 64, 16, seed=74, amax_spread=0.5)
    kept = [_random_kept(L - s, k, g) for L, s, k in zip(lens, starts, n)]
    want = X.stored(c)
    for b in range(2):
        X.keep(c, b, lens[b], starts[b], kept[b], want)
    keep = torch.zeros((2, max(n)), dtype=torch.int32)
    for b, k in enumerate(kept):
        keep[b, :len(k)] = torch.tensor(k, dtype=torch.int32)
    got = qasa.kv_keep_tokens(c.library(), c.table, c.seq_lens, _ints(starts), keep.cuda(), keep_lens=_ints(n))
    assert got.tolist() == [s + k for s, k in zip(starts, n)]
    _compare(X.stored(c), want, dtype)


def test_bad_lists_lengths_and_pages():
    qasa = _qasa()
    lens = [60, 60, 60, 60, 60, 60]
    starts = [10, 20, -3, 99, 0, 30]
    keep = [[0, 3, 3, 7], [1, 2, 40, 41], [0, 1, 2, 5], [0, 1, 2, 3], [-1, 2, 3, 4], [2, 9, 11, 29]]
    n = [4, 4, 7, -1, 4, 4]
    c = R.Paged("f16", lens, 2, 64, 16, seed=75)
    c.table[5, 2] = -1                                          # tokens 32 .. 47 of the last sequence have no page
    want = X.stored(c)
    good = [[0, 3], [1, 2], [0, 1, 2, 5], [], [], [2, 9, 11, 29]]
    at = [10, 20, 0, 60, 0, 30]
    for b in range(6):
        X.keep(c, b, 60, at[b], good[b], want)
    status = _status()
    out = qasa.kv_keep_tokens(c.library(), c.table, c.seq_lens, _ints(starts), _ints(keep), keep_lens=_ints(n), status=status)
    torch.cuda.synchronize()
    assert int(status) == 0x1 | 0x2 | 0x10 | 0x100
    assert out.tolist() == [a + len(k) for a, k in zip(at, good)]
    _compare(X.stored(c), want, "f16")


@pytest.mark.parametrize("dtype", ["f16", "e4m3"])
def test_keep_repeats_and_replays_on_another_stream(dtype):
    qasa = _qasa()
    g = torch.Generator(device="cpu").manual_seed(76)
    lens, starts = [90, 200], [70, 11]
    keep = _ints([_random_kept(L - s, 9, g) for L, s in zip(lens, starts)])
    caches = [R.Paged(dtype, lens, 2, 128, 16, seed=77, amax_spread=1.0) for _ in range(3)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    qasa.kv_keep_tokens(caches[0].library(), caches[0].table, caches[0].seq_lens, _ints(starts), keep)
    qasa.kv_keep_tokens(caches[1].library(), caches[1].table, caches[1].seq_lens, _ints(starts), keep, stream=side)
    lib, st, out = caches[2].library(), _ints(starts), torch.zeros(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        qasa.kv_keep_tokens(lib, caches[2].table, caches[2].seq_lens, st, keep, lens_out=out)
    assert out.tolist() == [0, 0]
    graph.replay()
    torch.cuda.synchronize()
    assert out.tolist() == [79, 20]
    a = X.stored(caches[0])
    for c in caches[1:]:
        b = X.stored(c)
        assert all(X.same(a[name], b[name]) for name in a)


@pytest.mark.parametrize("power", [-90, 90])
def test_codes_do_not_depend_on_the_size_of_the_scales(power):
    # scales times a power of two change no quotient and round alike: the same codes
    qasa = _qasa()
    g = torch.Generator(device="cpu").manual_seed(78)
    lens, starts = [300, 800, 90], [3, 160, 0]
    keep = _ints([_random_kept(L - s, 80, g) for L, s in zip(lens, starts)])
    a, b = (R.Paged("e4m3", lens, 3, 128, 16, seed=79, amax_spread=1.0) for _ in range(2))
    b.scales *= 2.0 ** power
    for c in (a, b):
        qasa.kv_keep_tokens(c.library(), c.table, c.seq_lens, _ints(starts), keep)
    torch.cuda.synchronize()
    x, y = X.stored(a), X.stored(b)
    y["scales"] *= 2.0 ** -power
    assert all(X.same(x[name], y[name]) for name in x)


# -------------------------------------------------------------------- copies and forks

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "e4m3"])
@pytest.mark.parametrize("hkv,d,page", [(1, 64, 16), (3, 128, 32), (16, 128, 16)])
def test_copied_pages(dtype, hkv, d, page):
    qasa = _qasa()
    c = R.Paged(dtype, [300, 200], hkv, d, page, seed=81)
    want = X.stored(c)
    order = torch.randperm(c.count, generator=torch.Generator().manual_seed(82)).tolist()
    half = c.count // 2
    src, dst = order[:half], order[half:2 * half]
    src[1] = src[0]                                             # read twice
    dst[2] = src[2]                                             # its own copy
    bad = [(-1, order[0]), (c.count, dst[0]), (src[0], -4), (src[0], 1 << 30)]
    for name in want:
        x = want[name].clone()
        for s, t in zip(src, dst):
            want[name][t] = x[s]
    pairs = [*zip(src, dst), *bad]
    status = _status()
    qasa.kv_copy_pages(c.library(), _ints([p[0] for p in pairs]), _ints([p[1] for p in pairs]), status=status)
    torch.cuda.synchronize()
    assert int(status) == 0x1
    now = X.stored(c)
    assert all(X.same(now[name], want[name]) for name in want)
    qasa.kv_copy_pages(c.library(), _ints([]), _ints([]))


@pytest.mark.parametrize("dtype", ["f32", "f16", "e4m3"])
@pytest.mark.parametrize("hkv,d,page", [(2, 64, 16), (5, 128, 32)])
def test_forks(dtype, hkv, d, page):
    qasa = _qasa()
    lens = [100, 64, 0, 1, 333, 47]
    c = R.Paged(dtype, lens, hkv, d, page, seed=83, reserve=100)
    free = sorted(set(range(c.count)) - set(c.table.flatten().tolist()))
    spare = [int(c.table[b, -3]) for b in range(6) if 0 <= int(c.table[b, -3]) < c.count] + free
    spare += [int(c.table[4, (lens[4] + 100) // page - i]) for i in range(2)]
    spare = list(dict.fromkeys(spare))
    parents = [0, 0, 1, 2, 3, 4, 5, 6, -1, 4, 0]
    new = [-1, spare[0], spare[1], -1, spare[2], spare[3], c.count, spare[4], spare[4], -1, int(c.table[0, 100 // page])]
    want = X.stored(c)
    rows = torch.full((len(parents), c.table.shape[1]), 77, dtype=torch.int32)
    out_lens = [9] * len(parents)
    table = c.table.cpu()
    bits = 0
    for i, (r, fresh) in enumerate(zip(parents, new)):
        if not 0 <= r < len(lens):
            bits |= 0x80
            continue
        full, part = divmod(lens[r], page)
        if part and fresh >= c.count:
            bits |= 0x1
            continue
        rows[i, :full] = table[r, :full]
        out_lens[i] = lens[r]
        if part:
            at = int(table[r, full])
            rows[i, full] = at if fresh < 0 else fresh
            if fresh >= 0 and fresh != at:
                for name in "kv":
                    want[name][fresh, :, :part] = want[name][at, :, :part]
                for name in set(want) - {"k", "v"}:
                    want[name][fresh] = want[name][at]
    status = _status()
    got, n = torch.full_like(rows, 77).cuda(), torch.full((len(parents),), 9, dtype=torch.int32, device="cuda")
    a, b = qasa.kv_fork(c.library(), c.table, c.seq_lens, _ints(parents), _ints(new), table_out=got, lens_out=n, status=status)
    torch.cuda.synchronize()
    assert a is got and b is n and int(status) == bits
    assert torch.equal(got.cpu(), rows) and n.tolist() == out_lens
    now = X.stored(c)
    assert all(X.same(now[name], want[name]) for name in want)


def test_forks_of_a_bad_page_and_of_a_bad_length():
    qasa = _qasa()
    c = R.Paged("f16", [40, 40, 40], 2, 64, 16, seed=84, reserve=40)
    was = X.stored(c)
    c.table[0, 2] = -1
    lens = _ints([40, -2, 1 << 30])
    status = _status()
    rows, n = qasa.kv_fork(c.library(), c.table, lens, _ints([0, 1, 2]), _ints([int(c.table[1, 4]), 0, 0]), status=status)
    torch.cuda.synchronize()
    assert int(status) == 0x1 | 0x2
    assert n.tolist() == [0, 0, c.table.shape[1] * 16]
    assert bool((rows[:2] == -1).all()) and torch.equal(rows[2], c.table[2])
    now = X.stored(c)
    assert all(X.same(now[name], was[name]) for name in was)


# --------------------------------------------------------------------- a run together

@pytest.mark.parametrize("dtype,hkv,group,d,page,window,sinks", [
    ("f32", 2, 2, 64, 16, None, 0), ("f16", 2, 8, 128, 16, 60, 5), ("bf16", 1, 4, 128, 32, None, 0), ("f16", 4, 1, 64, 32, 33, 1)])
def test_speculation_over_forked_sequences(dtype, hkv, group, d, page, window, sinks):
    """A prompt, forked, then steps of a drafted tree each: append at its depths, attention by its mask, the accepted
    path kept.  Every step's attention is checked against 64-bit attention over the rotated tokens of the path."""
    qasa = _qasa()
    hq, value, u = hkv * group, R.VALUE[dtype], R.half_step(R.VALUE[dtype])
    prompt, T, steps, B = 75, 13, 4, 3
    c = R.Paged(dtype, [0] + [0] * (B - 1), hkv, d, page, seed=91, reserve=prompt + steps * T)
    cache, g = c.library(), torch.Generator(device="cpu").manual_seed(92)
    table = qasa.rotation_table(prompt + steps * T, d, device="cuda")
    raw = lambda n, b: torch.randn((b, n, hq + 2 * hkv, d), generator=g).to(value).cuda()  # noqa: E731
    status = _status()
    x = raw(prompt, 1)
    qasa.kv_append_rotated(cache, c.table[:1].contiguous(), _ints([0]), x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], table,
                           status=status)
    # all go on from the first: the first keeps its page, the others' rows get the shared pages and one of their own
    rows = c.table.clone()
    rows, lens = qasa.kv_fork(cache, c.table, _ints([prompt] + [0] * (B - 1)), _ints([0] * B),
                              _ints([-1] + [int(c.table[b, prompt // page]) for b in range(1, B)]), table_out=rows, status=status)
    path = [x[0].clone() for _ in range(B)]                     # raw rows of every token of the path
    for step in range(steps):
        x = raw(T, B)
        parents = [X.random_parents(T, g) for _ in range(B)]
        mask, depths = qasa.tree_masks(_ints(parents), status=status)
        q = qasa.kv_append_positioned(cache, rows, lens, x[:, :, hq:hq + hkv], x[:, :, hq + hkv:], table,
                                      lens[:, None] + depths, q=x[:, :, :hq], status=status)
        out = qasa.tree_attention(cache, q, rows, lens + T, mask, window=window, sink_tokens=sinks, status=status)
        accepted = []
        for b in range(B):
            tree, deep = X.tree_rows(parents[b])
            best = max(range(T), key=lambda t: (deep[t], t))
            accepted.append(sorted(tree[best]))
            for t in range(T):                                  # every query as the end of a chain of its own
                above = sorted(tree[t])
                chain = torch.cat([path[b], x[b, above]])
                L, n = chain.shape[0], len(above)
                pos = [torch.arange(L, device="cuda")]
                k = X.rotate(chain[:, hq:hq + hkv], table, pos, [0] * (d // 2), False).to(value).double()
                qt = X.rotate(chain[-1:, :hq], table, [pos[0][-1:]], [0] * (d // 2), False).to(value).double()[0]
                v = chain[:, hq + hkv:].double()
                j, i = torch.arange(L, device="cuda"), L - 1
                seen = (j >= L - n) | (j < sinks) | (j > i - (window or 1 << 30))
                k, v = (z.repeat_interleave(group, 1) for z in (k, v))
                s = torch.einsum("hd,lhd->hl", qt, k) / d ** 0.5
                p = torch.softmax(s.masked_fill(~seen, float("-inf")), -1)
                ref = torch.einsum("hl,lhd->hd", p, v)
                weighed = torch.einsum("hl,lhd->hd", p, v.abs())
                size = torch.einsum("hd,lhd->hl", qt.abs(), k.abs()).masked_fill(~seen, 0).amax(-1)
                # keys and queries may be rounded the other way than here, a step of either in the scores
                tol = R.attention_tolerance(ref, weighed, size, d, value) + 4 * 2 * u * size[:, None] / d ** 0.5 * weighed
                err = (out[b, t].double() - ref).abs()
                assert bool((err <= tol).all()), (step, b, t, (err - tol).max().item())
            path[b] = torch.cat([path[b], x[b, accepted[b]]])
        most = max(map(len, accepted))
        keep = _ints([a + [-1] * (most - len(a)) for a in accepted])
        lens = qasa.kv_keep_tokens(cache, rows, lens + T, lens, keep, keep_lens=_ints([len(a) for a in accepted]), status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert lens.tolist() == [p.shape[0] for p in path]
    # the boxes are those of the tokens that are left
    boxes = cache.page_bounds.clone()
    qasa.rebuild_page_bounds(cache, rows, lens)
    for b in range(B):
        for i in range(-(-int(lens[b]) // page)):
            assert torch.equal(boxes[int(rows[b, i])], cache.page_bounds[int(rows[b, i])])
    # and the page selection works on them
    q = torch.randn((B, hq, d), generator=g).to(value).cuda()
    a, _ = qasa.sparse_decode_attention(cache, q, rows, lens, rows.shape[1])
    b = qasa.window_attention(cache, q, rows, lens)
    assert bool(((a.double() - b.double()).abs() <= 2e-3 + 1e-2 * b.double().abs()).all())
