"""The 8-bit cache on the CPU: what the host refuses before any GPU work, and
the tests' own definitions against hand-worked values."""
import ctypes

import numpy as np
import pytest

import cache_helpers as ch
import graph_transformer_sparse_gb300 as gt

INV, UNS, OK = gt.GTATTN_ERR_INVALID_ARG, gt.GTATTN_ERR_UNSUPPORTED, gt.GTATTN_OK


@pytest.fixture(scope="module")
def lib():
    gt.build()
    return gt.load()


def struct(k8=16, v8=16, ks=16, vs=16, km=16, pages=4, page=16, Hkv=2, D=8):
    return gt._CacheStruct(k8, v8, ks, vs, km, pages, page, Hkv, D)


BAD_CACHES = [dict(page=8), dict(page=48), dict(page=128), dict(page=0), dict(pages=-1), dict(pages=1 << 27), dict(Hkv=0),
              dict(Hkv=1025), dict(D=0), dict(D=257), dict(k8=8), dict(v8=24), dict(km=2), dict(ks=18), dict(vs=17)]


def test_slots_refusals(lib):
    f = lib.gtattn_cache_slots   # length add table free new_length tok_off slots counts S max_pages n_free T page stream
    ok = [16, 16, 16, 16, 64, 16, 16, 16, 4, 4, 4, 4, 16, None]
    for at, bad in [(4, 16), (4, 28), (4, 4), (0, None), (1, None), (2, None), (3, None), (4, None), (5, None), (6, None), (7, None), (0, 18), (2, 17),
                    (3, 18), (4, 18), (5, 18), (6, 18), (7, 18), (8, -1), (9, -1), (10, -1), (11, -1), (8, 1 << 31),
                    (10, 1 << 31), (11, 1 << 31), (9, 1 << 27), (9, 1 << 62), (12, 0), (12, 8), (12, 128), (12, -16)]:
        a = list(ok)
        a[at] = bad
        assert f(*a) == INV, (at, bad)


def test_append_refusals(lib):
    f = lib.gtattn_cache_append   # cache K V slots T dtype stream
    c = ctypes.byref(struct())
    assert f(None, 16, 16, 16, 4, 0, None) == INV
    for a in ((None, 16, 16, 4, 0), (16, None, 16, 4, 0), (16, 16, None, 4, 0), (18, 16, 16, 4, 0), (16, 17, 16, 4, 1),
              (16, 16, 18, 4, 0), (16, 16, 16, -1, 0), (16, 16, 16, 1 << 31, 0), (16, 16, 16, 4, 7), (16, 16, 16, 4, -1)):
        assert f(c, *a, None) == INV, a
    for bad in BAD_CACHES + [dict(k8=None), dict(v8=None), dict(ks=None), dict(vs=None)]:
        assert f(ctypes.byref(struct(**bad)), 16, 16, 16, 4, 0, None) == INV, bad
    assert f(c, None, None, None, 0, 0, None) == OK                                   # no tokens
    assert f(ctypes.byref(struct(None, None, None, None, None, pages=0)), 16, 16, 16, 4, 0, None) == OK   # no pages


def test_select_refusals(lib):
    f = lib.gtattn_cache_select   # cache Q table length tok_off sel S T max_pages H n_sel dtype stream
    c = ctypes.byref(struct())
    ok = [16, 16, 16, 16, 16, 4, 4, 4, 4, 3, 0]
    assert f(None, *ok, None) == INV
    for at, bad in [(0, None), (1, None), (2, None), (3, None), (4, None), (0, 18), (1, 18), (2, 18), (3, 18), (4, 18),
                    (5, -1), (6, -1), (7, -1), (5, 1 << 31), (6, 1 << 31), (7, 1 << 27), (7, 1 << 62), (8, 0), (8, 3),
                    (8, 2048), (9, 0), (9, -1), (9, (1 << 20) + 1), (10, 3)]:
        a = list(ok)
        a[at] = bad
        assert f(c, *a, None) == INV, (at, bad)
    for bad in BAD_CACHES + [dict(km=None)]:
        assert f(ctypes.byref(struct(**bad)), *ok, None) == INV, bad
    a = list(ok)
    a[6] = 1 << 30
    assert f(c, *a, None) == UNS                                                      # T * Hkv
    a[6] = 0
    assert f(c, *a, None) == OK


def test_attention_refusals(lib):
    f = lib.gtattn_fwd_cache   # cache Q table length tok_off sel out S T max_pages H n_sel scale dtype stream
    c = ctypes.byref(struct())
    ok = [16, 16, 16, 16, None, 16, 4, 4, 4, 4, 0, 1.0, 0]
    assert f(None, *ok, None) == INV
    for at, bad in [(0, None), (1, None), (2, None), (3, None), (5, None), (0, 18), (1, 18), (2, 18), (3, 18), (4, 18),
                    (4, 16), (5, 18), (6, -1), (7, -1), (8, -1), (6, 1 << 31), (7, 1 << 31), (8, 1 << 27), (9, 0), (9, 3),
                    (9, 2048), (10, 1), (10, -1), (12, 5)]:
        a = list(ok)
        a[at] = bad
        assert f(c, *a, None) == INV, (at, bad)
    for bad in BAD_CACHES + [dict(k8=None), dict(v8=None), dict(ks=None), dict(vs=None)]:
        assert f(ctypes.byref(struct(**bad)), *ok, None) == INV, bad
    a = list(ok)
    a[7] = 1 << 30
    assert f(c, *a, None) == UNS                                                      # T * H
    a[7] = 0
    assert f(c, *a, None) == OK
    a[7], a[6] = 4, 0
    a[1] = a[2] = a[3] = None
    assert f(c, *a, None) == OK                                                       # no requests


def test_cache_object_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    tile = torch.zeros(3, 2, 16, 8, dtype=torch.uint8)
    scale, mean = torch.zeros(3, 2), torch.zeros(3, 2, 8, dtype=torch.bfloat16)
    for bad in ((None, tile, scale, scale, None), (tile[:2], tile, scale, scale, mean), (tile.float(), tile, scale, scale, None),
                (tile, tile, scale.double(), scale, None), (tile, tile, scale, scale, mean.float()),
                (tile, tile, scale, scale, mean[:, :1])):
        with pytest.raises(ValueError):
            gt.Cache(*bad)
    with pytest.raises(ValueError):
        gt.Cache(tile, tile, scale, scale, mean, page=32)
    with pytest.raises(ValueError):        # tensors of the CPU
        gt.Cache(tile, tile, scale, scale, mean)


def test_helpers_e4m3():
    assert ch.VALUES[0x7e] == 448 and ch.VALUES[0x08] == 2.0 ** -6 and ch.VALUES[0x01] == 2.0 ** -9 and ch.VALUES[0xb8] == -1
    x = np.array([0, 1, -1, 448, 500, 17, 19, 2.0 ** -10, 3 * 2.0 ** -10, -2.0 ** -11, np.inf, np.nan, 16.99])
    #                                   ties: 17 -> 16 (even), 19 -> 20, 2^-10 -> 0, 3 * 2^-10 -> 2^-8
    y = ch.VALUES[ch.encode(x)]
    assert np.array_equal(y[:10], [0, 1, -1, 448, 448, 16, 20, 0, 2.0 ** -8, 0]) and np.isnan(y[10:12]).all() and y[12] == 16
    codes = np.arange(256)
    fine = (codes & 0x7f) != 0x7f
    assert np.array_equal(ch.encode(ch.VALUES[fine]), codes[fine])
    assert [ch.scale_of(a) for a in (0, 448, 449, 224, 1.0)] == [2.0 ** -64, 1, 2, 0.5, 2.0 ** -8]
    assert ch.scale_of(3.4e38) == 2.0 ** 120 and ch.scale_of(1e-300) == 2.0 ** -64


def test_helpers_slots_and_select():
    r = ch.slots([15, 0, 5], [2, 0, 20], np.array([[7, -1], [-1, -1], [3, -1]]), np.array([9, 1]), 2, 2, 30, 16)
    assert r["slots"].tolist()[:2] == [7 * 16 + 15, 9 * 16] and r["slots"][2] == 3 * 16 + 5 and r["slots"][13] == 16
    assert r["counts"].tolist() == [2, 22, 0] and r["tok_off"].tolist() == [0, 2, 2, 22] and r["slots"][22] == -1
    r = ch.slots([15, 5], [2, 20], np.array([[7, -1], [3, -1]]), np.array([9]), 2, 1, 30, 16)
    assert r["counts"].tolist() == [1, 22, 1] and (r["slots"][2:] == -1).all() and r["new_length"].tolist() == [17, 5]
    km = np.array([[[1.0]], [[3.0]], [[3.0]], [[2.0]]])
    sel = ch.select(np.ones((1, 1, 1)), km, np.arange(4)[None], [64], [0, 1], 2, 16)
    assert sel.tolist() == [[[1, 3]]]        # the own page, and of the two of score 3 the earlier
