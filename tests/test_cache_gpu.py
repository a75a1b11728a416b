"""The 8-bit K/V cache operators on the GPU against their definitions in 64 bits."""
import numpy as np
import pytest

import cache_helpers as ch

torch = pytest.importorskip("torch")
import graph_transformer_sparse_gb300 as gt   # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f32": (gt.GTATTN_F32, "float32", "float32"), "bf16": (gt.GTATTN_BF16, "bfloat16", "bfloat16"),
      "bf16_out_f32": (gt.GTATTN_BF16_OUT_F32, "bfloat16", "float32")}


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def ints(x):
    return dev(np.asarray(x).astype(np.int32))


def f64(t):
    return t.detach().double().cpu().numpy()


def typed(rng, shape, dtype, spread=1.0):
    """(tensor of the input type, its values in fp64)"""
    x = (spread * rng.standard_normal(shape)).astype(np.float32)
    t = torch.from_numpy(x).to(getattr(torch, DT[dtype][1]))
    return t.cuda(), f64(t)


class Store:
    """A cache and its table with requests of the given lengths: random codes
    in use, NaN codes and NaN scales wherever nothing is stored."""

    def __init__(self, rng, lengths, Hkv, D, page, max_pages=None, spare=3):
        self.page, self.lengths = page, list(lengths)
        S = len(lengths)
        have = [-(-n // page) for n in lengths]
        self.max_pages = max(have + [1]) if max_pages is None else max_pages
        pages = sum(have) + spare
        ids = rng.permutation(pages)
        self.table = np.full((S, self.max_pages), -1, dtype=np.int32)
        self.k8 = np.full((pages, Hkv, page, D), 0x7f, dtype=np.uint8)
        self.v8 = np.full((pages, Hkv, page, D), 0x7f, dtype=np.uint8)
        self.ks = np.full((pages, Hkv), np.nan, dtype=np.float32)
        self.vs = np.full((pages, Hkv), np.nan, dtype=np.float32)
        self.km = np.full((pages, Hkv, D), np.nan)
        at = 0
        for s, n in enumerate(lengths):
            for p in range(have[s]):
                pg = ids[at]
                at += 1
                self.table[s, p] = pg
                m = min(page, n - p * page)
                for c8, sc in ((self.k8, self.ks), (self.v8, self.vs)):
                    c8[pg, :, :m] = ch.encode(np.clip(100.0 * rng.standard_normal((Hkv, m, D)), -448, 448))
                    sc[pg] = 2.0 ** rng.integers(-9, -5, Hkv)
                self.km[pg] = ch.bf16((ch.VALUES[self.k8[pg, :, :m]].mean(1) * self.ks[pg][:, None]).astype(np.float32))
        self.free = ids[at:].astype(np.int32)

    def cache(self):
        return gt.Cache(dev(self.k8), dev(self.v8), dev(self.ks), dev(self.vs),
                        dev(self.km.astype(np.float32)).to(torch.bfloat16))


def offsets(adds):
    return np.concatenate([[0], np.cumsum(adds)]).astype(np.int32)


# ---------------------------------------------------------------------------
# slots
# ---------------------------------------------------------------------------
def run_slots(length, add, table, free, T, page, extra=0):
    S, max_pages = table.shape
    d = dict(length=ints(length), add=ints(add), table=ints(table), free=ints(free),
             new=torch.full((S,), -7, dtype=torch.int32, device="cuda"),
             off=torch.full((S + 1,), -7, dtype=torch.int32, device="cuda"),
             slots=torch.full((T + extra,), -7, dtype=torch.int32, device="cuda"),
             counts=torch.full((3,), -7, dtype=torch.int32, device="cuda"))
    gt.gtattn_cache_slots(d["length"], d["add"], d["table"], d["free"], d["new"], d["off"], d["slots"], d["counts"], S,
                          max_pages, len(free), T, page)
    torch.cuda.synchronize()
    return d


def check_slots(length, add, table, free, T, page):
    d = run_slots(length, add, table, free, T, page, extra=4)
    ref = ch.slots(length, add, table, free, table.shape[1], len(free), T, page)
    for k, g in (("new_length", "new"), ("tok_off", "off"), ("counts", "counts"), ("table", "table")):
        assert np.array_equal(d[g].cpu().numpy(), ref[k]), k
    got = d["slots"].cpu().numpy()
    assert np.array_equal(got[:T], ref["slots"]) and (got[T:] == -7).all()
    return ref


@pytest.mark.parametrize("S,page,lo,hi,add,T_over", [
    (1, 16, 0, 0, 1, 0), (1, 64, 63, 65, 1, 3), (7, 32, 0, 100, 40, 0), (64, 64, 1, 5000, 1, 5), (300, 16, 0, 400, 90, 17),
    (1025, 32, 0, 70, 3, 0), (5000, 64, 0, 300, 2, 1), (2, 16, 0, 10, 70000, 0), (33, 64, 0, 9, 4000, 100000)])
def test_slots(S, page, lo, hi, add, T_over):
    rng = np.random.default_rng(S + page)
    length = rng.integers(lo, hi + 1, S)
    adds = rng.integers(0 if S > 1 else 1, add + 1, S)
    max_pages = int((length + adds).max() // page + 2)
    have = -(-length // page)
    need = int((-(-(length + adds) // page) - have).sum())
    ids = rng.permutation(int(have.sum()) + need + 5).astype(np.int32)
    table = np.full((S, max_pages), -1, dtype=np.int32)
    at = 0
    for s in range(S):
        table[s, :have[s]] = ids[at:at + have[s]]
        at += have[s]
    ref = check_slots(length, adds, table, ids[at:], int(adds.sum()) + T_over, page)
    assert ref["counts"][2] == 0 and ref["counts"][0] == need


@pytest.mark.parametrize("n_free,T", [(0, 500), (1, 500), (4, 500), (9, 500), (40, 500), (40, 60), (40, 0), (3, 37)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("times", [1, 300])
def test_slots_refusals(n_free, T, page, times):
    # negative sizes, requests past the table, a free list and a row list that end early
    length = np.tile([5, -1, 16, 0, 60, 3, 2000000000, 15, 64, 10], times)
    add = np.tile([11, 3, 1, 70, -2, 0, 2000000000, 1, 2, 17], times)
    n_free, T = n_free * times // 2 + n_free % 2, T * times // 2
    rng = np.random.default_rng(4)
    max_pages = 6
    table = rng.permutation(10 * times * max_pages).reshape(10 * times, max_pages).astype(np.int32)
    free = (100 + np.arange(n_free)).astype(np.int32)
    ref = check_slots(length, add, table, free, T, page)
    assert ref["counts"][2] >= 3 * times


def test_slots_without_requests():
    d = run_slots(np.zeros(0), np.zeros(0), np.zeros((0, 4)), np.arange(3), 5, 16)
    assert d["off"].tolist() == [0] and d["slots"].tolist() == [-1] * 5 and d["counts"].tolist() == [0, 0, 0]


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def check_append(st, x, v, slot_list, dtype, tensors, means=True):
    """Appends to the store on both sides; everything equal bit for bit."""
    cache = st.cache()
    if not means:
        cache = gt.Cache(cache.k8, cache.v8, cache.kscale, cache.vscale, None)
    gt.gtattn_cache_append(cache, tensors[0], tensors[1], ints(slot_list), len(slot_list), DT[dtype][0])
    torch.cuda.synchronize()
    ch.append(st.k8, st.ks, x, slot_list, st.page, st.km if means else None)
    ch.append(st.v8, st.vs, v, slot_list, st.page)
    for name, mine, ref in (("k8", cache.k8, st.k8), ("v8", cache.v8, st.v8)):
        assert ch.same_codes(mine.view(torch.uint8).cpu().numpy(), ref).all(), name
    for name, mine, ref in (("kscale", cache.kscale, st.ks), ("vscale", cache.vscale, st.vs)):
        assert np.array_equal(f64(mine), ref.astype(np.float64), equal_nan=True), name
    if means:
        assert np.array_equal(f64(cache.kmean), st.km, equal_nan=True)
    return cache


def slots_for(st, adds):
    """Slots of `adds` new tokens per request, pages taken from the free list."""
    ref = ch.slots(np.array(st.lengths), np.array(adds), st.table, st.free, st.max_pages, len(st.free), int(sum(adds)),
                   st.page)
    assert ref["counts"][2] == 0
    st.table, st.free = ref["table"].astype(np.int32), st.free[ref["counts"][0]:]
    st.lengths = ref["new_length"].tolist()
    return ref["slots"].astype(np.int32)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("Hkv,D,page", [(1, 1, 16), (4, 32, 16), (8, 64, 32), (2, 128, 64), (3, 80, 32), (2, 256, 64),
                                        (5, 33, 64)])
def test_append(dtype, Hkv, D, page):
    rng = np.random.default_rng(D + page)
    lens = [0, 1, page - 1, page, page + 1, 3 * page - 2, 7, 0]
    adds = [1, 1, 1, 1, page, 2 * page + 3, 0, 3 * page]
    st = Store(rng, lens, Hkv, D, page, max_pages=8, spare=20)
    sl = slots_for(st, adds)
    T = len(sl)
    (tk, k), (tv, v) = typed(rng, (T, Hkv, D), dtype, 2.0), typed(rng, (T, Hkv, D), dtype, 0.02)
    check_append(st, k, v, sl, dtype, (tk, tv))


@pytest.mark.parametrize("page", [16, 64])
def test_append_ranges(page):
    # tiny, huge, zero and mixed tokens: scales clamp at both ends, grow by many powers, old codes become subnormal
    rng = np.random.default_rng(2)
    Hkv, D = 2, 64
    st = Store(rng, [3, 3, 3, 0, 0, 0, 5, 5], Hkv, D, page, max_pages=4, spare=9)
    sl = slots_for(st, [2] * 8)
    x = rng.standard_normal((16, Hkv, D)).astype(np.float32)
    x[0:2] *= np.float32(1e-30)
    x[2:4] *= np.float32(1e30)
    x[4:6] = 0
    x[6:8] = 0
    x[8:10] = np.float32(3.4e38) * np.sign(x[8:10])
    x[10:12] *= np.float32(1e-42)
    x[12] = 448 * 2.0 ** -7
    x[13] = -448 * 2.0 ** -7
    x[14, :, ::2] = 2.0 ** -8
    x[15] = np.nextafter(np.float32(448 * 2.0 ** -3), np.float32(1e9))
    t = dev(x)
    check_append(st, x.astype(np.float64), x.astype(np.float64), sl, "f32", (t, t.clone()))


def test_append_not_finite():
    rng = np.random.default_rng(3)
    st = Store(rng, [3, 0, 31], 2, 32, 32, max_pages=4, spare=9)
    sl = slots_for(st, [2, 2, 3])
    x = rng.standard_normal((7, 2, 32)).astype(np.float32)
    x[0, 0, 3], x[1, 1, 4], x[2, 0], x[3, 1, 7] = np.nan, np.inf, -np.inf, np.nan
    check_append(st, x.astype(np.float64), x.astype(np.float64), sl, "f32", (dev(x), dev(x)))


def test_append_skips_and_rewinds():
    # slots outside the cache are skipped; a request cut back to 2 tokens is written over from there
    rng = np.random.default_rng(5)
    st = Store(rng, [40, 40], 2, 32, 16, max_pages=4, spare=2)
    pages = st.k8.shape[0]
    a, b = int(st.table[0, 0]) * 16, int(st.table[1, 2]) * 16
    sl = np.array([-1, a + 2, a + 3, a + 4, pages * 16, b + 8, -5, 2 ** 31 - 1, -2 ** 31], dtype=np.int64)
    x = rng.standard_normal((9, 2, 32)).astype(np.float32)
    check_append(st, x.astype(np.float64), x.astype(np.float64), sl.astype(np.int32), "f32", (dev(x), dev(x)))


def test_append_without_means():
    rng = np.random.default_rng(6)
    st = Store(rng, [10, 33], 2, 64, 32, max_pages=4)
    sl = slots_for(st, [1, 4])
    (tk, k), (tv, v) = typed(rng, (5, 2, 64), "bf16"), typed(rng, (5, 2, 64), "bf16")
    check_append(st, k, v, sl, "bf16", (tk, tv), means=False)


@pytest.mark.parametrize("D", [64, 96])
def test_append_unaligned_rows(D):
    # K and V one element off any 16-byte boundary
    rng = np.random.default_rng(7)
    for dtype in ("f32", "bf16"):
        st = Store(rng, [10, 33, 0], 2, D, 32, max_pages=4)
        sl = slots_for(st, [1, 4, 40])
        T = len(sl)
        flat = [typed(rng, (T * 2 * D + 1,), dtype) for _ in range(2)]
        (tk, k), (tv, v) = ((t[1:].view(T, 2, D), x[1:].reshape(T, 2, D)) for t, x in flat)
        check_append(st, k, v, sl, dtype, (tk, tv))


# ---------------------------------------------------------------------------
# select
# ---------------------------------------------------------------------------
def check_select(Q, tQ, km, table, length, off, n_sel, page, dtype):
    T = Q.shape[0]
    pages, Hkv, D = km.shape
    tkm = dev(km.astype(np.float32)).to(torch.bfloat16)
    cache = gt.Cache(None, None, None, None, tkm, page)
    sel = torch.full((T, Hkv, n_sel), -9, dtype=torch.int32, device="cuda")
    S, max_pages = table.shape
    gt.gtattn_cache_select(cache, tQ, ints(table), ints(length), ints(off), sel, S, T, max_pages, Q.shape[1], n_sel,
                           DT[dtype][0])
    torch.cuda.synchronize()
    ref = ch.select(Q[:off[-1]], f64(tkm), table, length, off, n_sel, page)
    got = sel.cpu().numpy()
    assert np.array_equal(got[:off[-1]], ref), np.argwhere(got[:off[-1]] != ref)[:5]
    assert (got[off[-1]:] == -9).all()
    return got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H,Hkv,D,page,n_sel", [(1, 1, 1, 16, 1), (4, 4, 32, 16, 4), (8, 2, 64, 32, 7), (16, 2, 128, 64, 33),
                                                (12, 4, 80, 16, 200), (6, 3, 256, 32, 2), (32, 1, 128, 16, 16),
                                                (9, 3, 33, 16, 12)])
def test_select(dtype, H, Hkv, D, page, n_sel):
    rng = np.random.default_rng(H + D + n_sel)
    lens = [1, page, page + 1, 40 * page + 3, 0, 7 * page, 333 * page - 1, 2]
    adds = [1, 2, 1, 5, 0, 3, 2, 2]
    max_pages = 340
    pages = 700
    table = rng.integers(0, pages, (8, max_pages)).astype(np.int32)
    km = ch.bf16(rng.standard_normal((pages, Hkv, D)))
    off = offsets(adds)
    tQ, Q = typed(rng, (off[-1] + 3, H, D), dtype)
    check_select(Q, tQ, km, table, lens, off, n_sel, page, dtype)


@pytest.mark.parametrize("n_pages,n_sel", [(9000, 50), (20000, 3), (5000, 4990), (5000, 6000)])
def test_select_many_pages(n_pages, n_sel):
    rng = np.random.default_rng(n_pages)
    pages, Hkv, D, page = 500, 2, 32, 16
    km = ch.bf16(rng.standard_normal((pages, Hkv, D)))      # (each page many times in the table: ties)
    table = rng.integers(0, pages, (1, n_pages)).astype(np.int32)
    tQ, Q = typed(rng, (2, 4, D), "bf16")
    check_select(Q, tQ, km, table, [n_pages * page - 5], offsets([2]), n_sel, page, "bf16")


@pytest.mark.parametrize("n_sel", [2, 9, 64, 150])
def test_select_ties(n_sel):
    # equal pages: the earlier ones; zero queries and queries that cancel: all tie
    rng = np.random.default_rng(n_sel)
    pages, Hkv, D, page = 40, 2, 64, 16
    km = ch.bf16(rng.standard_normal((pages, Hkv, D)))
    km[::4] = km[0]
    km[1::4] = 0
    table = rng.integers(0, pages, (3, 130)).astype(np.int32)
    off = offsets([1, 2, 1])
    tQ, _ = typed(rng, (4, 4, D), "bf16")
    tQ[1] = 0
    tQ[2, 1] = -tQ[2, 0]
    tQ[3, 2:] = -0.0
    check_select(f64(tQ), tQ, km, table, [130 * 16, 100 * 16, 128 * 16 + 1], off, n_sel, page, "bf16")


def test_select_close_scores():
    # scores that differ far below fp32's rounding of their terms: large terms cancel, the order lies in small ones
    rng = np.random.default_rng(8)
    pages, Hkv, D, page, n_sel = 300, 2, 64, 16, 20
    km = ch.bf16(rng.integers(-3, 4, (pages, Hkv, D)).astype(np.float64))
    km[:, :, 0] = km[:, :, 1] = 256.0 * rng.integers(1, 4, (pages, Hkv))
    table = rng.permutation(pages)[None].astype(np.int32)
    q = rng.integers(-2, 3, (1, 4, D)).astype(np.float64)
    q[..., 0], q[..., 1] = 2.0 ** 23, -2.0 ** 23
    t = dev(q.astype(np.float32))
    check_select(q, t, km, table, [pages * page], offsets([1]), n_sel, page, "f32")
    check_select(q, t.to(torch.bfloat16), km, table, [pages * page], offsets([1]), n_sel, page, "bf16")


def test_select_not_finite_and_bad_pages():
    rng = np.random.default_rng(9)
    pages, Hkv, D, page = 50, 2, 32, 16
    km = ch.bf16(rng.standard_normal((pages, Hkv, D)))
    km[3, 0, 5] = np.nan
    km[4, 1, 5], km[5, 1, 2] = np.inf, -np.inf
    table = rng.permutation(pages)[None].astype(np.int32)
    table = np.concatenate([table, table])
    table[1, 7], table[1, 9], table[1, 11] = -1, pages, 2 ** 31 - 1
    tq = dev(np.abs(rng.standard_normal((2, 4, D))).astype(np.float32))
    for n_sel in (4, 30, 49):
        check_select(f64(tq), tq, km, table, [pages * page] * 2, offsets([1, 1]), n_sel, page, "f32")


def test_select_ranges():
    # scores past fp32's range, and far below it; a query of NaN: every score NaN, the earliest pages
    rng = np.random.default_rng(15)
    pages, Hkv, D, page = 60, 2, 32, 16
    table = rng.permutation(pages)[None].repeat(4, 0).astype(np.int32)
    for s in (2.0 ** 100, 2.0 ** -100):
        km = ch.bf16(s * rng.standard_normal((pages, Hkv, D)))
        q = rng.standard_normal((4, 4, D)).astype(np.float32)
        q[1] *= np.float32(2.0 ** 100)
        q[2] *= np.float32(2.0 ** -100)
        q[3, 0, 3], q[3, 2, 4] = np.nan, np.inf
        t = dev(q)
        check_select(f64(t), t, km, table, [pages * page - 20] * 4, offsets([1] * 4), 9, page, "f32")


def test_select_length_past_the_table():
    rng = np.random.default_rng(10)
    km = ch.bf16(rng.standard_normal((30, 2, 32)))
    table = rng.integers(0, 30, (3, 10)).astype(np.int32)
    tQ, Q = typed(rng, (6, 4, 32), "f32")
    check_select(Q, tQ, km, table, [1000, 1, -4], offsets([2, 3, 1]), 5, 16, "f32")


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def run_attend(st, tQ, off, H, dtype, scale, sel=None, lengths=None, cache=None):
    T, _, D = tQ.shape
    out = torch.full((T, H, D), 77.0, dtype=getattr(torch, DT[dtype][2]), device="cuda")
    S, max_pages = st.table.shape
    gt.gtattn_fwd_cache(st.cache() if cache is None else cache, tQ, ints(st.table),
                        ints(st.lengths if lengths is None else lengths), ints(off), out, S, T, max_pages, H, scale,
                        DT[dtype][0], sel=None if sel is None else ints(sel), n_sel=0 if sel is None else sel.shape[2])
    torch.cuda.synchronize()
    return out


def attend_tol(dtype, ref, mag, big, count, D):
    # p is held in 16-bit floats (11 bits) where the output is bf16, in 21 bits or more where it is fp32
    return ch.attend_bound(ref, mag, big, count, D, 11 if dtype == "bf16" else 21, 8 if dtype == "bf16" else 24)


def check_attend(st, Q, tQ, off, H, dtype, scale, sel=None, lengths=None):
    out = run_attend(st, tQ, off, H, dtype, scale, sel, lengths=lengths)
    n = off[-1]
    ref, mag, big, count = ch.attend(Q[:n], st.k8, st.ks, st.v8, st.vs, st.table, st.lengths if lengths is None else lengths,
                                     off, scale, st.page, sel)
    got = f64(out)
    tol = attend_tol(dtype, ref, mag, big, count, Q.shape[2])
    err = np.abs(got[:n] - ref)
    assert np.array_equal(np.isnan(got[:n]), np.isnan(ref))
    bad = err > tol
    assert not bad.any(), (np.argwhere(bad)[:4], err[bad][:4], tol[bad][:4], ref[bad][:4])
    assert (got[n:] == 77.0).all()
    return got


SHAPES = [(1, 1, 32, 16), (4, 4, 32, 16), (8, 8, 64, 32), (8, 2, 64, 16), (16, 2, 128, 64), (32, 4, 128, 32), (20, 1, 64, 64),
          (3, 3, 128, 16), (40, 1, 32, 32), (6, 2, 1, 16), (4, 2, 80, 32), (4, 2, 256, 64), (5, 5, 33, 16), (6, 3, 16, 16), (4, 1, 48, 64), (8, 2, 112, 32)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("H,Hkv,D,page", SHAPES)
def test_attend(dtype, H, Hkv, D, page):
    rng = np.random.default_rng(H * 7 + D + page)
    lens = [1, 2, page, 5 * page + 3, 0, 17 * page - 1, 2, 64]
    adds = [1, 2, 1, 7, 0, 1, 1, 33]
    st = Store(rng, lens, Hkv, D, page)
    off = offsets(adds)
    tQ, Q = typed(rng, (off[-1] + 2, H, D), dtype)
    check_attend(st, Q, tQ, off, H, dtype, D ** -0.5)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("H,Hkv,D,page", SHAPES)
def test_attend_selected(dtype, H, Hkv, D, page):
    rng = np.random.default_rng(H * 5 + D + page)
    lens = [1, page + 2, 0, 9 * page + 3, 30 * page]
    adds = [1, 3, 0, 5, 2]
    st = Store(rng, lens, Hkv, D, page)
    off = offsets(adds)
    tQ, Q = typed(rng, (off[-1] + 2, H, D), dtype)
    n_sel = 7
    sel = ch.select(Q[:off[-1]], np.nan_to_num(st.km), st.table, st.lengths, off, n_sel, page)
    sel = np.concatenate([sel, np.full((2, Hkv, n_sel), 3)]).astype(np.int32)
    check_attend(st, Q, tQ, off, H, dtype, D ** -0.5, sel)
    # any order, pages twice, none at all, entries outside
    sel = rng.permuted(sel, axis=-1)
    sel[0] = -1
    sel[1, :, 0] = 2 ** 31 - 1
    sel[2, :, 1] = -7
    sel[4, :, :3] = 4
    check_attend(st, Q, tQ, off, H, dtype, D ** -0.5, sel)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hkv,D", [(4, 4, 32), (8, 2, 64), (8, 1, 128), (4, 2, 48), (4, 2, 96), (2, 1, 256), (3, 3, 7)])
def test_attend_long_requests(dtype, H, Hkv, D):
    rng = np.random.default_rng(D)
    st = Store(rng, [7001, 3, 2600], Hkv, D, 32)
    off = offsets([1, 1, 2])
    tQ, Q = typed(rng, (4, H, D), dtype, 2.0)
    check_attend(st, Q, tQ, off, H, dtype, D ** -0.5)
    sel = ch.select(Q, np.nan_to_num(st.km), st.table, st.lengths, off, 100, 32).astype(np.int32)
    check_attend(st, Q, tQ, off, H, dtype, D ** -0.5, sel)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("H,Hkv,D,page", [(8, 8, 64, 32), (8, 2, 32, 16), (4, 2, 128, 64), (16, 1, 64, 16)])
def test_attend_a_piece_of_a_prompt(dtype, H, Hkv, D, page):
    rng = np.random.default_rng(D + page)
    st = Store(rng, [300, 170, 5], Hkv, D, page)
    off = offsets([133, 170, 4])
    tQ, Q = typed(rng, (off[-1], H, D), dtype)
    check_attend(st, Q, tQ, off, H, dtype, D ** -0.5)


@pytest.mark.parametrize("D", [32, 64, 128, 40, 96])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_nan_reaches_only_its_rows(D, dtype):
    # a NaN in key or value of a late token: rows before it do not see it, rows from it on do
    rng = np.random.default_rng(D)
    H, Hkv, page = 4, 2, 16
    for which in ("k8", "v8"):
        st = Store(rng, [60, 41], Hkv, D, page)
        off = offsets([20, 3])
        pg, at = st.table[0, 50 // page], 50 % page
        getattr(st, which)[pg, 1, at, D // 2] = 0x7f
        tQ, Q = typed(rng, (23, H, D), dtype)
        got = check_attend(st, Q, tQ, off, H, dtype, D ** -0.5)
        seen = np.isnan(got).any((1, 2))
        assert seen[10:20].all() and not seen[:10].any() and not seen[20:].any()


@pytest.mark.parametrize("D", [32, 64, 128, 40, 96])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_extremes(D, dtype):
    # scales of pages far apart, large logits of either sign, equal keys, queries of very unlike sizes
    rng = np.random.default_rng(D)
    H, Hkv, page = 8, 2, 16
    st = Store(rng, [200, 90, 33], Hkv, D, page)
    st.vs[st.table[0, :8]] = 2.0 ** rng.integers(-40, 20, (8, Hkv))
    st.ks[st.table[0, :8]] = 2.0 ** rng.integers(-20, -4, (8, Hkv))
    st.k8[st.table[1, :6]] = 0x30
    off = offsets([3, 2, 1])
    tQ, Q = typed(rng, (6, H, D), dtype)
    tQ[1] *= 64
    tQ[2] *= 2.0 ** -30
    tQ[3] = 0
    tQ[4, ::2] *= 2.0 ** -25
    check_attend(st, f64(tQ), tQ, off, H, dtype, D ** -0.5)
    check_attend(st, f64(tQ), tQ, off, H, dtype, -0.25)
    check_attend(st, f64(tQ), tQ, off, H, dtype, 0.0)


@pytest.mark.parametrize("dtype", ["bf16", "bf16_out_f32"])
@pytest.mark.parametrize("H,Hkv,D,page", [(4, 4, 64, 16), (4, 2, 128, 32), (6, 2, 64, 64), (3, 1, 128, 16)])
def test_attend_many_rows(dtype, H, Hkv, D, page):
    # tiles of 128 rows: lengths around the tiles' and pages' ends, requests of a few rows and of none among them
    rng = np.random.default_rng(H + D + page)
    adds = [257, 1, 0, 128, 300, 40]
    st = Store(rng, [257, 500, 3, 128, 700, 129], Hkv, D, page)
    off = offsets(adds)
    tQ, Q = typed(rng, (off[-1] + 5, H, D), dtype)
    got = check_attend(st, Q, tQ, off, H, dtype, D ** -0.5)
    cache = st.cache()
    for _ in range(3):
        again = run_attend(st, tQ, off, H, dtype, D ** -0.5, cache=cache)
        assert np.array_equal(f64(again), got)
    assert gt.gtattn_device_errors() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "bf16_out_f32"])
def test_attend_many_rows_odd_values(D, dtype):
    # NaN in keys and values of tokens that some rows do not see, scales far apart, bad pages, unlike queries
    rng = np.random.default_rng(D)
    H, Hkv, page = 4, 2, 16
    for which in ("k8", "v8"):
        st = Store(rng, [400, 330], Hkv, D, page)
        off = offsets([200, 150])
        for at, g, d in ((250, 1, 3), (250, 1, D - 1), (399, 0, 0), (290, 0, D // 2)):
            getattr(st, which)[st.table[0, at // page], g, at % page, d] = 0x7f
        st.vs[st.table[1]] = 2.0 ** rng.integers(-30, 20, (len(st.table[1]), Hkv))
        st.ks[st.table[1]] = 2.0 ** rng.integers(-20, -4, (len(st.table[1]), Hkv))
        st.table[1, 3], st.table[1, 8] = -1, st.k8.shape[0]
        tQ, Q = typed(rng, (350, H, D), dtype)
        tQ[210] *= 64
        tQ[211] *= 2.0 ** -30
        tQ[212] = 0
        got = check_attend(st, f64(tQ), tQ, off, H, dtype, D ** -0.5)
        seen = np.isnan(got[:200]).any(2)
        assert not seen[:50].any() and seen[50:, 2:].all() and not seen[:90, :2].any() and seen[90:, :2].all()
        assert not np.isnan(got[200:]).any()
    # rows of requests that hold fewer tokens than they have rows
    tQ, Q = typed(rng, (350, H, D), dtype)
    st = Store(rng, [400, 330], Hkv, D, page)
    check_attend(st, Q, tQ, off, H, dtype, -0.3, lengths=[120, -9])


@pytest.mark.parametrize("D", [64, 40, 48])
def test_attend_bad_pages_and_lengths(D):
    rng = np.random.default_rng(11)
    H, Hkv, page = 4, 2, 16
    st = Store(rng, [100, 100, 100, 64, 100], Hkv, D, page)
    pages = st.k8.shape[0]
    st.table[0, 2], st.table[0, 6], st.table[1, 0], st.table[1, 3] = -1, pages, 2 ** 31 - 1, -2 ** 31
    st.table[2, :] = -1                       # no page at all: zeros
    off = offsets([2, 1, 1, 5, 4])
    tQ, Q = typed(rng, (13, H, D), "f32")
    # lengths: past the table, below the rows that a request has, negative
    got = check_attend(st, Q, tQ, off, H, "f32", 0.2, lengths=[100, 99, 100, 3, -5])
    assert (got[3] == 0).all() and (got[4:6] == 0).all() and (got[9:13] == 0).all()
    st.table = st.table[:, :4].copy()
    check_attend(st, Q, tQ, off, H, "f32", 0.2, lengths=[100, 2 ** 31 - 1, 64, 64, 65])


@pytest.mark.parametrize("H,D,T", [(4, 64, 3), (4, 64, 300), (4, 128, 200), (4, 40, 5)])
def test_attend_rows_past_the_batch_and_empty_tables(H, D, T):
    # offsets that pass T: only rows below T are written; a table without pages, a cache without pages: zeros
    rng = np.random.default_rng(17)
    st = Store(rng, [400, 60], 2, D, 16)
    off = offsets([T, 9])
    tQ, Q = typed(rng, (T, H, D), "bf16")
    flat = torch.full((T + 20, H, D), 77.0, dtype=torch.bfloat16, device="cuda")
    gt.gtattn_fwd_cache(st.cache(), tQ, ints(st.table), ints(st.lengths), ints(off), flat[:T], 2, T, st.max_pages, H, 0.1,
                        gt.GTATTN_BF16)
    torch.cuda.synchronize()
    assert (flat[T:] == 77).all()
    assert torch.equal(flat[:T], run_attend(st, tQ, offsets([T, 0]), H, "bf16", 0.1))
    out = torch.full((T, H, D), 77.0, dtype=torch.bfloat16, device="cuda")
    empty = torch.zeros(2, 0, dtype=torch.int32, device="cuda")
    gt.gtattn_fwd_cache(st.cache(), tQ, empty, ints(st.lengths), ints(offsets([T, 0])), out, 2, T, 0, H, 0.1, gt.GTATTN_BF16)
    assert (out == 0).all()
    out.fill_(77)
    gt.gtattn_fwd_cache(gt.Cache.empty(0, 2, D, 16), tQ, ints(st.table), ints(st.lengths), ints(offsets([T, 0])), out, 2, T,
                        st.max_pages, H, 0.1, gt.GTATTN_BF16)
    assert (out == 0).all()


def test_attend_tail_of_a_page_is_not_read():
    # what lies behind a request's last token in its page is NaN in a Store: it changes nothing
    rng = np.random.default_rng(12)
    for n in range(1, 67, 5):
        st = Store(rng, [n], 1, 64, 64)
        tQ, Q = typed(rng, (1, 3, 64), "bf16")
        check_attend(st, Q, tQ, offsets([1]), 3, "bf16", 0.125)


@pytest.mark.parametrize("D", [64, 96])
def test_attend_unaligned_rows(D):
    # Q and out one element off any 16-byte boundary
    rng = np.random.default_rng(13)
    st = Store(rng, [130, 7], 2, D, 32)
    off = offsets([2, 1])
    for dtype in DT:
        tQ, Q = typed(rng, (3, 4, D), dtype)
        flat = torch.empty(tQ.numel() + 1, dtype=tQ.dtype, device="cuda")
        flat[1:] = tQ.reshape(-1)
        ofl = torch.empty(tQ.numel() + 1, dtype=getattr(torch, DT[dtype][2]), device="cuda")
        args = (ints(st.table), ints(st.lengths), ints(off))
        aligned = run_attend(st, tQ, off, 4, dtype, 0.1)
        gt.gtattn_fwd_cache(st.cache(), flat[1:].view(3, 4, D), *args, ofl[1:].view(3, 4, D), 2, 3, st.max_pages, 4, 0.1,
                            DT[dtype][0])
        torch.cuda.synchronize()
        assert torch.equal(ofl[1:].view(3, 4, D), aligned)


def test_attend_same_bits_every_run():
    rng = np.random.default_rng(14)
    st = Store(rng, [3000, 10, 700], 2, 64, 32)
    off = offsets([1, 2, 40])
    cache = st.cache()
    tQ, Q = typed(rng, (43, 8, 64), "bf16_out_f32")
    first = run_attend(st, tQ, off, 8, "bf16_out_f32", 0.125, cache=cache)
    for _ in range(5):
        assert torch.equal(first, run_attend(st, tQ, off, 8, "bf16_out_f32", 0.125, cache=cache))


def test_attend_past_4_gib():
    # pages whose offsets in the cache pass 32 bits: the same answer as from a small cache
    rng = np.random.default_rng(16)
    Hkv, D, page, H = 8, 64, 64, 8
    st = Store(rng, [500, 90], Hkv, D, page)
    off = offsets([1, 2])
    tQ, Q = typed(rng, (3, H, D), "bf16")
    small = run_attend(st, tQ, off, H, "bf16", 0.125)
    pages = (5 << 30) // (Hkv * page * D)
    k8, v8 = (torch.empty(pages, Hkv, page, D, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(pages, Hkv, device="cuda") for _ in range(2))
    n = st.k8.shape[0]
    for big, own in ((k8, st.k8), (v8, st.v8), (ks, st.ks), (vs, st.vs)):
        big[pages - n:] = dev(own)
    st.table = np.where(st.table >= 0, st.table + pages - n, -1).astype(np.int32)
    cache = gt.Cache(k8, v8, ks, vs)
    assert torch.equal(small, run_attend(st, tQ, off, H, "bf16", 0.125, cache=cache))
    # and appended there: the last page of request 0 gets three tokens more
    sl = int(st.table[0, 7]) * page + 52 + np.arange(3)
    (tk, k), (tv, v) = typed(rng, (3, Hkv, D), "bf16"), typed(rng, (3, Hkv, D), "bf16")
    gt.gtattn_cache_append(cache, tk, tv, ints(sl), 3, gt.GTATTN_BF16)
    torch.cuda.synchronize()
    at = int(st.table[0, 7]) - (pages - n)
    ch.append(st.k8, st.ks, k, sl - (pages - n) * page, page)
    assert ch.same_codes(k8[pages - n + at].cpu().numpy()[:, :55], st.k8[at][:, :55]).all()


# ---------------------------------------------------------------------------
# the calls together
# ---------------------------------------------------------------------------
class Batch:
    """Requests on the GPU, stepped through slots, append, select and attend."""

    def __init__(self, S, Hkv, D, page, max_pages, pages, H, dtype, n_sel, T):
        self.sizes = S, Hkv, D, page, max_pages, H, n_sel, T
        self.dtype = dtype
        self.cache = gt.Cache.empty(pages, Hkv, D, page)
        z = dict(dtype=torch.int32, device="cuda")
        self.length, self.new_length, self.add = (torch.zeros(S, **z) for _ in range(3))
        self.table = torch.full((S, max_pages), -1, **z)
        self.free = torch.arange(pages - 1, -1, -1, **z)
        self.off, self.slots, self.counts = torch.zeros(S + 1, **z), torch.zeros(T, **z), torch.zeros(3, **z)
        self.sel = torch.full((T, Hkv, n_sel), -1, **z)
        t = getattr(torch, DT[dtype][1])
        self.Q = torch.zeros(T, H, D, dtype=t, device="cuda")
        self.K, self.V = (torch.zeros(T, Hkv, D, dtype=t, device="cuda") for _ in range(2))
        self.out, self.full = (torch.zeros(T, H, D, dtype=getattr(torch, DT[dtype][2]), device="cuda") for _ in range(2))

    def step(self, stream=None):
        S, Hkv, D, page, max_pages, H, n_sel, T = self.sizes
        d = DT[self.dtype][0]
        gt.gtattn_cache_slots(self.length, self.add, self.table, self.free, self.new_length, self.off, self.slots, self.counts,
                              S, max_pages, self.free.numel(), T, page, stream=stream)
        gt.gtattn_cache_append(self.cache, self.K, self.V, self.slots, T, d, stream=stream)
        gt.gtattn_cache_select(self.cache, self.Q, self.table, self.new_length, self.off, self.sel, S, T, max_pages, H, n_sel,
                               d, stream=stream)
        gt.gtattn_fwd_cache(self.cache, self.Q, self.table, self.new_length, self.off, self.out, S, T, max_pages, H, 0.125, d,
                            sel=self.sel, n_sel=n_sel, stream=stream)
        gt.gtattn_fwd_cache(self.cache, self.Q, self.table, self.new_length, self.off, self.full, S, T, max_pages, H, 0.125,
                            d, stream=stream)

    def fill(self, rng, adds):
        self.add.copy_(ints(adds))
        for x in (self.Q, self.K, self.V):
            x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape)).astype(np.float32)))

    def after(self):
        """What a program does between steps: the lengths move on, and the
        pages left move to the front of the free list (which keeps its place)."""
        self.length.copy_(self.new_length)
        used = int(self.counts[0])
        left = self.free[used:].clone()
        self.free[:left.numel()] = left


class Model:
    """The same batch in numpy."""

    def __init__(self, b):
        S, Hkv, D, page, max_pages, H, n_sel, T = b.sizes
        pages = b.cache.pages
        self.b = b
        self.k8, self.v8 = (np.zeros((pages, Hkv, page, D), dtype=np.uint8) for _ in range(2))
        self.ks, self.vs = (np.zeros((pages, Hkv), dtype=np.float32) for _ in range(2))
        self.km = np.zeros((pages, Hkv, D))
        self.length = np.zeros(S, dtype=np.int64)
        self.table = np.full((S, max_pages), -1)
        self.free = np.arange(pages - 1, -1, -1)

    def step_and_check(self, adds):
        S, Hkv, D, page, max_pages, H, n_sel, T = self.b.sizes
        r = ch.slots(self.length, adds, self.table, self.free, max_pages, len(self.free), T, page)
        assert r["counts"][2] == 0
        for name, mine in (("table", self.b.table), ("new_length", self.b.new_length), ("tok_off", self.b.off),
                           ("slots", self.b.slots), ("counts", self.b.counts)):
            assert np.array_equal(mine.cpu().numpy(), r[name]), name
        used = r["counts"][0]
        self.table, self.length = r["table"], r["new_length"]
        self.free[:len(self.free) - used] = self.free[used:].copy()
        ch.append(self.k8, self.ks, f64(self.b.K), r["slots"], page, self.km)
        ch.append(self.v8, self.vs, f64(self.b.V), r["slots"], page)
        c = self.b.cache
        assert ch.same_codes(c.k8.view(torch.uint8).cpu().numpy(), self.k8).all()
        assert ch.same_codes(c.v8.view(torch.uint8).cpu().numpy(), self.v8).all()
        n = r["tok_off"][-1]
        Q = f64(self.b.Q)[:n]
        sel = ch.select(Q, self.km, self.table, self.length, r["tok_off"], n_sel, page)
        assert np.array_equal(self.b.sel.cpu().numpy()[:n], sel)
        for got, s in ((self.b.out, sel), (self.b.full, None)):
            ref, mag, big, count = ch.attend(Q, self.k8, self.ks, self.v8, self.vs, self.table, self.length, r["tok_off"],
                                             0.125, page, s)
            tol = attend_tol(self.b.dtype, ref, mag, big, count, D)
            assert (np.abs(f64(got)[:n] - ref) <= tol).all()


@pytest.mark.parametrize("dtype,H,Hkv,D,page", [("bf16", 8, 8, 64, 16), ("f32", 8, 2, 32, 32), ("bf16_out_f32", 4, 2, 128, 16),
                                                ("bf16", 4, 4, 24, 64)])
def test_steps(dtype, H, Hkv, D, page):
    rng = np.random.default_rng(D)
    b = Batch(4, Hkv, D, page, 12, 40, H, dtype, 3, 60)
    m = Model(b)
    for adds in ([17, 0, 33, 5], [1, 1, 1, 1], [1, 16, 0, 40], [min(page, 50), 1, 1, 0], [1, 1, 1, 1], [0, 0, 0, 0],
                 [2, 1, 3, 1]):
        b.fill(rng, adds)
        b.step()
        torch.cuda.synchronize()
        m.step_and_check(np.array(adds))
        b.after()


def test_steps_captured_and_replayed():
    # two batches' steps captured once each, replayed in turn with new inputs
    rng = np.random.default_rng(21)
    batches = [Batch(5, 2, 64, 16, 8, 60, 8, "bf16", 3, 8), Batch(3, 4, 32, 32, 8, 40, 8, "f32", 2, 5)]
    models, graphs = [Model(b) for b in batches], []
    for b, m in zip(batches, models):
        adds = np.ones(b.sizes[0], dtype=np.int64)
        b.fill(rng, adds)
        b.step()
        torch.cuda.synchronize()
        m.step_and_check(adds)
        b.after()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.step()
        graphs.append(g)
    for i in range(20):
        adds = [np.array([(i + s) % 3 > 0 for s in range(b.sizes[0])], dtype=np.int64) for b in batches]
        for b, a in zip(batches, adds):
            b.fill(rng, a)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for b, m, a in zip(batches, models, adds):
            m.step_and_check(a)
            b.after()


def test_two_streams_at_once():
    rng = np.random.default_rng(22)
    batches = [Batch(6, 2, 64, 16, 8, 60, 8, "bf16", 3, 6) for _ in range(2)]
    models = [Model(b) for b in batches]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(8):
        adds = np.ones(6, dtype=np.int64)
        for b in batches:
            b.fill(rng, adds)
        torch.cuda.synchronize()
        for b, s in zip(batches, streams):
            b.step(stream=s)
        torch.cuda.synchronize()
        for b, m in zip(batches, models):
            m.step_and_check(adds)
            b.after()


def test_projected_nodes_through_the_cache():
    # q, k, v of the attention block with its projections, stored and attended
    # over: the last row of a complete graph's attention, up to the cache's 8 bits
    rng = np.random.default_rng(23)
    N, H, D, F = 48, 4, 32, 64
    X = dev(rng.standard_normal((N, F)).astype(np.float32))
    W, Wo = (dev((rng.standard_normal(s) / 8).astype(np.float32)) for s in ((3 * H * D, F), (F, H * D)))
    indptr = ints(np.arange(N + 1) * N)
    indices = ints(np.tile(np.arange(N), N))
    qkv, o, Y = (torch.empty(s, device="cuda") for s in ((3, N, H, D), (N, H, D), (N, F)))
    gt.gtattn_fwd_proj(indptr, indices, X, W, None, Wo, None, Y, N, N * N, F, H, D, F, D ** -0.5, gt.GTATTN_F32, qkv=qkv,
                       attn=o)
    b = Batch(1, H, D, 16, 4, 4, H, "f32", 2, N)
    b.add.fill_(N)
    for x, y in zip((b.Q, b.K, b.V), qkv):
        x.copy_(y)
    gt.gtattn_cache_slots(b.length, b.add, b.table, b.free, b.new_length, b.off, b.slots, b.counts, 1, 4, 4, N, 16)
    gt.gtattn_cache_append(b.cache, b.K, b.V, b.slots, N, gt.GTATTN_F32)
    gt.gtattn_fwd_cache(b.cache, b.Q, b.table, b.new_length, b.off, b.full, 1, N, 4, H, D ** -0.5, gt.GTATTN_F32)
    torch.cuda.synchronize()
    k, v = (f64(x) for x in qkv[1:])
    # a stored value is off by half a step of 3 bits (2^-4 of itself), or by half a step of the
    # subnormal codes (2^-10 of a scale that is below 2 amax / 448)
    dv = np.abs(v) * 2.0 ** -4 + 2.0 ** -10 * 2 * np.abs(v).max() / 448
    dk = np.abs(k) * 2.0 ** -4 + 2.0 ** -10 * 2 * np.abs(k).max() / 448
    q = f64(qkv[0])[-1]
    dl = (D ** -0.5) * np.einsum("hd,nhd->nh", np.abs(q), dk).max(0)      # largest change of a logit, per head
    lg = (D ** -0.5) * np.einsum("hd,nhd->nh", q, k)
    p = np.exp(lg - lg.max(0))
    p /= p.sum(0)
    mag = np.einsum("nh,nhd->hd", p, np.abs(v) + dv)
    tol = np.expm1(2 * dl)[:, None] * mag + np.einsum("nh,nhd->hd", p, dv) + 1e-5
    assert (np.abs(f64(b.full)[-1] - f64(o)[-1]) <= tol).all()
