"""The 8-bit cache operators in 64 bits, straight from their definitions
(numpy, request by request), and the error bounds of their tests."""
import numpy as np


# ---- e4m3 ------------------------------------------------------------------
def _values():
    v = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        v[c] = s * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    v[0x7f] = v[0xff] = np.nan
    return v


VALUES = _values()
_POS = VALUES[:0x7f]            # 0 .. 448, rising with the code


def encode(x):
    """Nearest e4m3 code, ties to the even code; values past 448 give 448, what is not finite NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(_POS, a), 1, 0x7e)      # _POS[hi-1] < a <= _POS[hi] (or a = 0)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a > _POS[0x7e], 0x7e, code)
    code = np.where(np.isfinite(x), code, 0x7f)
    return (code | np.where(np.signbit(x) & np.isfinite(x), 0x80, 0)).astype(np.uint8)


def same_codes(a, b):
    """Equal codes, NaN of either sign alike."""
    a, b = np.asarray(a), np.asarray(b)
    return (a == b) | (((a & 0x7f) == 0x7f) & ((b & 0x7f) == 0x7f))


def scale_of(amax):
    if amax == 0:
        return 2.0 ** -64
    e = int(np.ceil(np.log2(amax / 448.0)))
    while 448.0 * 2.0 ** e < amax:      # (log2's rounding)
        e += 1
    while 448.0 * 2.0 ** (e - 1) >= amax:
        e -= 1
    return 2.0 ** min(max(e, -64), 120)


def bf16(x):
    """fp32 nearest even, then bf16 nearest even, as float64."""
    u = np.ascontiguousarray(np.asarray(x, dtype=np.float32)).view(np.uint32)
    r = (u.astype(np.uint64) + 0x7fff + ((u >> 16) & 1)).astype(np.uint64) >> 16 << 16
    f = r.astype(np.uint32).view(np.float32).astype(np.float64)
    return np.where(np.isnan(x), np.nan, f)


# ---- the operators ---------------------------------------------------------
def slots(length, add, table, free, max_pages, n_free, T, page):
    table = table.copy()
    S = len(length)
    tok, pages, taken, refused = 0, 0, 0, 0
    new, off, out = [], [], np.full(T, -1, dtype=np.int64)
    for s in range(S):
        n, a = int(length[s]), int(add[s])
        bad = n < 0 or a < 0 or n + a > max_pages * page
        have = -(-max(n, 0) // page)
        need = 0 if bad else -(-(n + a) // page) - have
        a = 0 if bad else a
        ok = not bad and (a == 0 or tok + a <= T) and (need == 0 or pages + need <= n_free)
        off.append(min(tok, T))
        new.append(n + a if ok else n)
        refused += not ok
        if ok:
            if need:
                taken = pages + need
                table[s, have:have + need] = free[pages:pages + need]
            for i in range(a):
                out[tok + i] = table[s, (n + i) // page] * page + (n + i) % page
        tok += a
        pages += need
    off.append(min(tok, T))
    return dict(table=table, new_length=np.array(new, dtype=np.int64), tok_off=np.array(off), slots=out,
                counts=np.array([taken, off[-1], refused]))


def append(k8, scale, x, slot_list, page, mean=None):
    """One of K and V: codes [pages, Hkv, page, D] and scale [pages, Hkv] in place; x [T, Hkv, D] fp64."""
    total = k8.shape[0] * page
    t, T = 0, len(slot_list)
    while t < T:
        s = int(slot_list[t])
        if s < 0 or s >= total:
            t += 1
            continue
        n = 1
        while t + n < T and slot_list[t + n] == s + n and (s + n) % page:
            n += 1
        pg, f = s // page, s % page
        for h in range(k8.shape[1]):
            new = x[t:t + n, h]
            fin = np.abs(new[np.isfinite(new)])
            now = scale_of(fin.max() if fin.size else 0.0)
            if f:
                now = max(now, float(scale[pg, h]))
                k8[pg, h, :f] = encode(VALUES[k8[pg, h, :f]] * (float(scale[pg, h]) / now))
            k8[pg, h, f:f + n] = encode(new / now)
            scale[pg, h] = now
            if mean is not None:
                with np.errstate(over="ignore"):
                    total32 = (VALUES[k8[pg, h, :f + n]].sum(0) * now).astype(np.float32)   # exact in fp32
                mean[pg, h] = bf16(total32 / np.float32(f + n))
        t += n


def rows(length, tok_off):
    """(row, request, position) of every row."""
    for s in range(len(length)):
        for t in range(tok_off[s], tok_off[s + 1]):
            yield t, s, int(length[s]) - int(tok_off[s + 1]) + t


def select(Q, kmean, table, length, tok_off, n_sel, page):
    """Q [T, H, D], kmean [pages, Hkv, D] in fp64."""
    T, H, D = Q.shape
    pages, Hkv = kmean.shape[:2]
    sel = np.full((T, Hkv, n_sel), -1)
    for t, s, pos in rows(length, tok_off):
        pos = min(pos, table.shape[1] * page - 1)
        if pos < 0:
            continue
        own = pos // page
        for g in range(Hkv):
            q = Q[t].reshape(Hkv, H // Hkv, D)[g].sum(0)
            ids = table[s, :own]
            ok = (ids >= 0) & (ids < pages)
            with np.errstate(invalid="ignore"):
                sc = np.where(ok, (kmean[np.where(ok, ids, 0), g] * q).sum(-1), 0.0)
            sc = np.where(np.isnan(sc), -np.inf, sc)
            best = np.argsort(-sc, kind="stable")[:n_sel - 1]
            mine = np.sort(np.append(best, own))
            sel[t, g, :len(mine)] = mine
    return sel


def attend(Q, k8, kscale, v8, vscale, table, length, tok_off, scale, page, sel=None):
    """out, and for the bounds, per element, sum p|v|, and per row the largest |scale| sum|q||k| and the keys read."""
    T, H, D = Q.shape
    pages, Hkv = k8.shape[:2]
    out, mag = np.zeros((T, H, D)), np.zeros((T, H, D))
    big, count = np.zeros((T, H, 1)), np.zeros((T, H, 1))
    for t, s, pos in rows(length, tok_off):
        pos = min(pos, table.shape[1] * page - 1)
        if pos < 0:
            continue
        for g in range(Hkv):
            listed = range(pos // page + 1) if sel is None else [p for p in sel[t, g] if 0 <= p <= pos // page]
            k, v = [], []
            for p in listed:
                pg = table[s, p]
                if not 0 <= pg < pages:
                    continue
                n = min(page, pos - p * page + 1)
                k.append(VALUES[k8[pg, g, :n]] * float(kscale[pg, g]))
                v.append(VALUES[v8[pg, g, :n]] * float(vscale[pg, g]))
            if not k:
                continue
            k, v = np.concatenate(k), np.concatenate(v)
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                lg = scale * (k @ Q[t, h])
                p = np.exp(lg - lg.max())
                p /= p.sum()
                out[t, h], mag[t, h] = p @ v, p @ np.abs(v)
                big[t, h] = np.abs(scale) * (np.abs(k) @ np.abs(Q[t, h])).max()
                count[t, h] = len(k)
    return out, mag, big, count


def attend_bound(out, mag, big, count, D, p_bits, out_bits):
    """Largest error of an fp32-accumulating form, per element.

    logit: its D products are summed in fp32 (D/8 + 8 sequential roundings of
    2^-23 at most, those of a truncating adder, relative to sum |q||k|), q and
    the scale's factors rounded to 22 bits or better (2^-22), and its size in
    the exponent rounded twice (2^-24): dl; a logit off by dl changes every p
    by a factor within e^(2 dl).  exp2 is good to 2^-22 above and below the
    fraction line.  p rounded to p_bits bits (2^-p_bits), the sums over count
    keys in fp32 (count + 64 roundings of 2^-23), division 2^-22; at the end
    the output's own rounding."""
    dl = big * ((D / 8 + 8) * 2.0 ** -23 + 2.0 ** -22 + 2 * 2.0 ** -24)
    rel = np.expm1(2 * dl) + 2 * 2.0 ** -22 + 2.0 ** -p_bits + 2 * (count + 64) * 2.0 ** -23 + 2.0 ** -22
    return mag * rel + np.abs(out) * 2.0 ** -out_bits + 1e-35
