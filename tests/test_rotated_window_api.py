"""The rotating append and windowed attention reject bad arguments on the host, before any launch."""
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


def _append(lib, cache=None, **kw):
    a = dict(table=0x40000, positions=4096, rot=128, inter=0, bt=0x50000, maxp=8, lens=0x60000, counts=None, q=0x70000,
             hq=32, q_out=0x80000, k=0x90000, v=0xA0000, qs=(4096, 4096), ks=(512, 512), vs=(512, 512), batch=2, T=2,
             status=None)
    a.update(kw)
    rot = lib._Rotation(a["table"], a["positions"], a["rot"], a["inter"])
    q = None if a["q"] is None else ctypes.byref(lib._TokenRows(a["q"], *a["qs"]))
    return lib._lib.qasa_kv_append_rotated(
        ctypes.byref(cache or _cache(lib)), ctypes.byref(rot), a["bt"], a["maxp"], a["lens"], a["counts"], q, a["hq"],
        a["q_out"], ctypes.byref(lib._TokenRows(a["k"], *a["ks"])), ctypes.byref(lib._TokenRows(a["v"], *a["vs"])),
        a["batch"], a["T"], a["status"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(rot=0), 3), (dict(rot=24), 3), (dict(rot=144), 3), (dict(positions=0), 3), (dict(inter=2), 3), (dict(inter=-1), 3),
    (dict(table=None), 1), (dict(table=0x40008), 4), (dict(bt=None), 1), (dict(lens=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(q_out=None), 1), (dict(hq=0), 3), (dict(maxp=0), 3), (dict(maxp=16385), 3), (dict(batch=-1), 3),
    (dict(batch=65536), 3), (dict(T=-1), 3), (dict(k=0x90008), 4), (dict(q=0x70004), 4), (dict(q_out=0x80002), 4),
    (dict(ks=(512, 508)), 4), (dict(vs=(511, 512)), 4), (dict(qs=(-4096, 4096)), 3), (dict(ks=(512, -512)), 3),
    (dict(lens=0x60002), 4), (dict(counts=0x60001), 4), (dict(bt=0x50003), 4), (dict(status=0x60002), 4),
])
def test_append_refusals(lib, kw, code):
    assert _append(lib, **kw) == code


def test_append_without_work_needs_no_pointers(lib):
    assert _append(lib, batch=0, bt=None, k=None, v=None, q=None) == 0
    assert _append(lib, T=0, bt=None, k=None, v=None, q=None) == 0
    assert _append(lib, cache=_cache(lib, head_dim=96)) == 3
    assert _append(lib, cache=_cache(lib, dtype=3)) == 1          # E4M3 pages without scales
    assert lib._lib.qasa_kv_append_rotated(ctypes.byref(_cache(lib)), None, 0x100, 8, 0x100, None, None, 0, None, None, None,
                                           1, 1, None, None) == 1


def _attend(lib, cache=None, **kw):
    a = dict(q=0x40000, hq=32, T=4, q_lens=None, bt=0x50000, maxp=64, lens=0x60000, window=128, sinks=4, out=0x80000,
             ws=None, wsb=0, batch=2, status=None)
    a.update(kw)
    return lib._lib.qasa_window_attention(ctypes.byref(cache or _cache(lib)), a["q"], a["hq"], a["T"], a["q_lens"], a["bt"],
                                          a["maxp"], a["lens"], a["window"], a["sinks"], 0.0, a["out"], a["ws"], a["wsb"],
                                          a["batch"], a["status"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(window=0), 3), (dict(window=-5), 3), (dict(sinks=-1), 3), (dict(T=-1), 3), (dict(T=65537), 3), (dict(q=None), 1),
    (dict(out=None), 1), (dict(bt=None), 1), (dict(lens=None), 1), (dict(hq=30), 3), (dict(hq=36), 3), (dict(maxp=0), 3),
    (dict(maxp=16385), 3), (dict(batch=-1), 3), (dict(batch=8193), 3), (dict(q=0x40008), 4), (dict(out=0x80004), 4),
    (dict(q_lens=0x60002), 4), (dict(status=0x60001), 4), (dict(lens=0x60003), 4),
])
def test_attention_refusals(lib, kw, code):
    assert _attend(lib, **kw) == code


def test_attention_without_work_needs_no_pointers(lib):
    assert _attend(lib, batch=0, q=None, out=None, bt=None, lens=None) == 0
    assert _attend(lib, T=0, q=None, out=None, bt=None, lens=None) == 0
    assert _attend(lib, cache=_cache(lib, page_size=8)) == 3
    assert _attend(lib, cache=_cache(lib, page_size=8), batch=0) == 3


def test_binding_checks_tensors(lib):
    kv = torch.zeros((2, 4, 2, 16, 64), dtype=torch.float16)
    cache = lib.PagedKVCache(kv[0], kv[1], torch.zeros((4, 2, 2, 64), dtype=torch.float16))
    bt, lens = torch.zeros((1, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros((1, 2, 4, 64), dtype=torch.float16)
    k = torch.zeros((1, 2, 2, 64), dtype=torch.float16)
    table = lib.rotation_table(64, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        lib.window_attention(cache, q, bt, lens, workspace=torch.empty(16, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        lib.kv_append_rotated(cache, bt, lens, k, k, table)
    for bad in (q.float(), q[..., :32], q[:, :, :, None]):
        with pytest.raises(ValueError):
            lib.window_attention(cache, bad, bt, lens)
    with pytest.raises(ValueError, match="k_new"):
        lib.kv_append_rotated(cache, bt, lens, k.float(), k, table)
    with pytest.raises(ValueError, match="contiguous"):
        lib.kv_append_rotated(cache, bt, lens, k.transpose(2, 3).contiguous().transpose(2, 3), k, table)
    with pytest.raises(ValueError, match="num_kv_heads"):
        lib.kv_append_rotated(cache, bt, lens, q, q, table)
    with pytest.raises(ValueError, match="table"):
        lib.kv_append_rotated(cache, bt, lens, k, k, table[:, 0])
    with pytest.raises(ValueError, match="batch and tokens"):
        lib.kv_append_rotated(cache, bt, lens, k, k, table, q=q[:, :1])
    with pytest.raises(ValueError, match="q_out"):
        lib.kv_append_rotated(cache, bt, lens, k, k, table, q_out=q)


def test_rotation_table_keeps_far_angles(lib):
    t = lib.rotation_table(100_000, 64, device="cpu")
    assert t.shape == (100_000, 2, 32) and t.dtype == torch.float32
    angle = 99_999.0 * 10000.0 ** (-2 * 3 / 64)
    import math
    assert abs(float(t[99_999, 0, 3]) - math.cos(angle)) <= 2.0 ** -24
    assert abs(float(t[99_999, 1, 3]) - math.sin(angle)) <= 2.0 ** -24


def test_unpacked_e4m3_pages_beyond_32_bit_rows_are_refused(lib):
    # 16384 visible pages x 16 slots x 8192 heads are 2^31 rows of the workspace; few rows need none
    many = _cache(lib, dtype=3, page_scales=0x90000, num_phys_pages=1, num_kv_heads=8192)
    kw = dict(hq=8192, maxp=16384, window=1 << 30, batch=1, ws=0xA0000, wsb=1 << 40)
    assert _attend(lib, cache=many, T=200, **kw) == 3
    assert lib._lib.qasa_window_workspace_size(1, 8192, ctypes.byref(many), 128, 16384, 1 << 30, 0) == 0


def test_workspace_sizes(lib):
    f = lib._lib.qasa_window_workspace_size
    e4m3, f16 = _cache(lib, dtype=3, page_scales=0x90000), _cache(lib)
    assert f(2, 32, ctypes.byref(f16), 4096, 512, 1024, 16) == 0
    assert f(2, 32, ctypes.byref(e4m3), 16, 512, 1024, 16) == 0           # 128 rows: read as they are
    # 17 tokens of 8 heads: the pages of 1024 + 16 tokens, not aligned, and one of sinks
    pages = (1024 + 17 + 14) // 16 + 1 + 1
    assert f(2, 32, ctypes.byref(e4m3), 17, 512, 1024, 16) == 2 * pages * 4 * 16 * 128 * 4
    assert f(2, 32, ctypes.byref(e4m3), 17, 20, 1024, 16) == 2 * 20 * 4 * 16 * 128 * 4
    for bad in ((0, 32, 17, 512, 1024, 16), (2, 3, 17, 512, 1024, 16), (2, 32, 0, 512, 1024, 16), (2, 32, 17, 0, 1024, 16),
                (2, 32, 17, 512, 0, 16), (2, 32, 17, 512, 1024, -1)):
        assert f(bad[0], bad[1], ctypes.byref(e4m3), *bad[2:]) == 0
    assert f(2, 32, None, 17, 512, 1024, 16) == 0
