"""Tree attention, the positioned append, kept tokens, forks and page copies reject bad arguments on the host."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from query_aware_sparse_append_gb300 import build
    build.build()
    from query_aware_sparse_append_gb300 import binding
    return binding


def _cache(lib, **kw):
    f = dict(k_pool=0x10000, v_pool=0x20000, page_bounds=0x30000, num_phys_pages=64, num_kv_heads=4, page_size=16,
             head_dim=128, dtype=1, page_scales=None)
    f.update(kw)
    return lib._Cache(*f.values())


def _tree(lib, cache=None, **kw):
    a = dict(q=0x40000, hq=32, T=40, q_lens=None, mask=0x41000, mb=80, bt=0x50000, maxp=64, lens=0x60000, window=128, sinks=4,
             out=0x80000, ws=None, wsb=0, batch=2, status=None)
    a.update(kw)
    return lib._lib.qasa_tree_attention(ctypes.byref(cache or _cache(lib)), a["q"], a["hq"], a["T"], a["q_lens"], a["mask"],
                                        a["mb"], a["bt"], a["maxp"], a["lens"], a["window"], a["sinks"], 0.0, a["out"],
                                        a["ws"], a["wsb"], a["batch"], a["status"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(window=0), 3), (dict(window=-5), 3), (dict(sinks=-1), 3), (dict(T=-1), 3), (dict(T=1025), 3), (dict(q=None), 1),
    (dict(out=None), 1), (dict(bt=None), 1), (dict(lens=None), 1), (dict(mask=None), 1), (dict(hq=30), 3), (dict(hq=36), 3),
    (dict(maxp=0), 3), (dict(maxp=16385), 3), (dict(batch=-1), 3), (dict(batch=8193), 3), (dict(q=0x40008), 4),
    (dict(out=0x80004), 4), (dict(mask=0x41002), 4), (dict(q_lens=0x60002), 4), (dict(status=0x60001), 4),
    (dict(lens=0x60003), 4), (dict(mb=79), 3), (dict(mb=-80), 3),
])
def test_tree_refusals(lib, kw, code):
    assert _tree(lib, **kw) == code


def test_tree_without_work_needs_no_pointers(lib):
    assert _tree(lib, batch=0, q=None, out=None, bt=None, lens=None, mask=None) == 0
    assert _tree(lib, T=0, q=None, out=None, bt=None, lens=None, mask=None) == 0
    assert _tree(lib, cache=_cache(lib, page_size=8), batch=0) == 3
    assert _tree(lib, cache=_cache(lib, dtype=3)) == 1          # E4M3 pages without scales


@pytest.mark.parametrize("args,code", [
    ((0x100, 2, 1025, None, 0x200, None, None), 3), ((0x100, -1, 8, None, 0x200, None, None), 3),
    ((0x100, 8193, 8, None, 0x200, None, None), 3), ((None, 2, 8, None, 0x200, None, None), 1),
    ((0x100, 2, 8, None, None, None, None), 1), ((0x102, 2, 8, None, 0x200, None, None), 4),
    ((0x100, 2, 8, 0x101, 0x200, None, None), 4), ((0x100, 2, 8, None, 0x200, 0x303, None), 4),
    ((None, 0, 8, None, None, None, None), 0), ((None, 3, 0, None, None, None, None), 0),
])
def test_mask_refusals(lib, args, code):
    assert lib._lib.qasa_tree_masks(*args, None) == code


def _append(lib, cache=None, **kw):
    a = dict(table=0x40000, positions=4096, rot=128, inter=0, at=0x42000, sa=8, sb=2, axes=3, pair=bytes([0, 1, 2, 0] * 16),
             bt=0x50000, maxp=8, lens=0x60000, q=0x70000, q_out=0x80000, k=0x90000, v=0xA0000, batch=2, T=2, given=True)
    a.update(kw)
    rot = lib._Rotation(a["table"], a["positions"], a["rot"], a["inter"])
    pos = lib._Positions(a["at"], a["sa"], a["sb"], a["axes"], a["pair"])
    row = lambda x: ctypes.byref(lib._TokenRows(x, 4096, 4096))  # noqa: E731
    return lib._lib.qasa_kv_append_positioned(
        ctypes.byref(cache or _cache(lib)), ctypes.byref(rot), ctypes.byref(pos) if a["given"] else None, a["bt"], a["maxp"],
        a["lens"], None, row(a["q"]), 32, a["q_out"], row(a["k"]), row(a["v"]), a["batch"], a["T"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(given=False), 1), (dict(at=None), 1), (dict(at=0x42002), 4), (dict(sa=-1), 3), (dict(sb=-2), 3), (dict(axes=0), 3),
    (dict(axes=4), 3), (dict(axes=2), 3), (dict(pair=bytes([0] * 63 + [3])), 3), (dict(rot=24), 3), (dict(table=None), 1),
    (dict(bt=None), 1), (dict(q_out=None), 1), (dict(k=0x90008), 4), (dict(batch=65536), 3), (dict(T=-1), 3),
    (dict(batch=0, at=None), 0), (dict(T=0, at=None), 0),
])
def test_positioned_append_refusals(lib, kw, code):
    assert _append(lib, **kw) == code


def _keep(lib, cache=None, **kw):
    a = dict(bt=0x50000, maxp=8, lens=0x60000, starts=0x61000, keep=0x62000, M=6, counts=0x63000, out=0x64000, batch=2,
             status=None)
    a.update(kw)
    return lib._lib.qasa_kv_keep_tokens(ctypes.byref(cache or _cache(lib)), a["bt"], a["maxp"], a["lens"], a["starts"],
                                        a["keep"], a["M"], a["counts"], a["out"], a["batch"], a["status"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(bt=None), 1), (dict(lens=None), 1), (dict(starts=None), 1), (dict(keep=None), 1), (dict(M=-1), 3), (dict(M=129), 3),
    (dict(batch=-1), 3), (dict(batch=8193), 3), (dict(maxp=0), 3), (dict(maxp=16385), 3), (dict(keep=0x62002), 4),
    (dict(out=0x64001), 4), (dict(starts=0x61003), 4), (dict(status=0x100001), 4), (dict(out=0x60000), 3), (dict(out=0x61004), 3),
    (dict(out=0x62010), 3), (dict(out=0x63004), 3), (dict(out=0x50020), 3), (dict(batch=0, bt=None, lens=None, keep=None), 0),
])
def test_keep_refusals(lib, kw, code):
    assert _keep(lib, **kw) == code


def test_page_refusals(lib):
    c = ctypes.byref(_cache(lib))
    copy = lib._lib.qasa_kv_copy_pages
    for args, code in (((None, 0x100, 1), 1), ((0x100, None, 1), 1), ((0x100, 0x200, -1), 3), ((0x102, 0x200, 1), 4),
                       ((0x100, 0x201, 1), 4), ((None, None, 0), 0), ((0x100, 0x200, 0x7fffffff), 3)):
        assert copy(c, *args, None, None) == code, args
    assert copy(ctypes.byref(_cache(lib, page_size=8)), None, None, 0, None, None) == 3

    def fork(**kw):
        a = dict(bt=0x50000, maxp=8, lens=0x60000, batch=2, parents=0x61000, new=0x62000, n=3, out=0x70000, lo=0x71000)
        a.update(kw)
        return lib._lib.qasa_kv_fork(c, a["bt"], a["maxp"], a["lens"], a["batch"], a["parents"], a["new"], a["n"], a["out"],
                                     a["lo"], None, None)

    for kw, code in ((dict(bt=None), 1), (dict(lens=None), 1), (dict(parents=None), 1), (dict(new=None), 1), (dict(out=None), 1),
                     (dict(maxp=0), 3), (dict(batch=-1), 3), (dict(n=-1), 3), (dict(parents=0x61002), 4), (dict(lo=0x71001), 4),
                     (dict(out=0x50000), 3), (dict(out=0x50020), 3), (dict(out=0x4ffc0), 3), (dict(lo=0x60004), 3),
                     (dict(lo=0x70004), 3), (dict(out=0x61008), 3), (dict(n=0, bt=None, out=None), 0),
                     (dict(n=0x7fffffff, out=0x10000000, lo=None), 3)):
        assert fork(**kw) == code, kw


def test_binding_checks_tensors(lib):
    kv = torch.zeros((2, 4, 2, 16, 64), dtype=torch.float16)
    cache = lib.PagedKVCache(kv[0], kv[1], torch.zeros((4, 2, 2, 64), dtype=torch.float16))
    bt, lens = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros((1, 2, 4, 64), dtype=torch.float16)
    k = torch.zeros((1, 2, 2, 64), dtype=torch.float16)
    mask = torch.zeros((1, 2, 1), dtype=torch.int32)
    table = lib.rotation_table(64, 64, device="cpu")
    pos = torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        lib.tree_attention(cache, q, bt, lens, mask)
    with pytest.raises(ValueError, match="CUDA"):
        lib.kv_append_positioned(cache, bt, lens, k, k, table, pos)
    with pytest.raises(ValueError, match="CUDA"):
        lib.kv_keep_tokens(cache, bt, lens, lens, pos)
    with pytest.raises(ValueError, match="CUDA"):
        lib.kv_copy_pages(cache, lens, lens)
    with pytest.raises(ValueError, match="CUDA"):
        lib.kv_fork(cache, bt, lens, lens, lens)
    with pytest.raises(ValueError, match="CUDA"):
        lib.tree_masks(pos)
    with pytest.raises(ValueError, match="mask"):
        lib.tree_attention(cache, q, bt, lens, mask[0])
    with pytest.raises(ValueError, match="heads"):
        lib.tree_attention(cache, q[0], bt, lens, mask)
    with pytest.raises(ValueError, match="head_dim"):
        lib.tree_attention(cache, q[..., :32], bt, lens, mask)
    with pytest.raises(ValueError, match="keep"):
        lib.kv_keep_tokens(cache, bt, lens, lens, lens)
    with pytest.raises(ValueError, match="parents"):
        lib.kv_fork(cache, bt, lens, pos, lens)
    for bad in (pos.long(), pos[:, :1], pos.expand(2, 2), pos.view(1, 1, 1, 2)):
        with pytest.raises(ValueError, match="positions"):
            lib._positions(bad, None, 1, 2, 32, -1)
    with pytest.raises(ValueError, match="axes"):
        lib._positions(pos.expand(4, 1, 2), None, 1, 2, 32, -1)
    for axes in ([0] * 31, [0] * 31 + [1], [-1] + [0] * 31):
        with pytest.raises(ValueError, match="pair_axes"):
            lib._positions(pos, axes, 1, 2, 32, -1)
    got = lib._positions(pos.view(1, 1, 2).expand(3, 1, 2), lib.pair_sections([8, 12, 12]), 5, 2, 32, -1)
    assert (got.axis_stride, got.batch_stride, got.num_axes) == (0, 0, 3)
    assert list(lib.pair_sections([1, 2, 1])) == [0, 1, 1, 2]
