"""Plain reference of the 8-bit operators (E4M3 codes, one FP32 scale per block of
128; paged K/V cache), in numpy: binary64 throughout, binary32 where the format
itself is (scales, the quotients that are rounded to codes).

TEST INFRASTRUCTURE ONLY, like the rest of this package.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def bf16_values(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32)


def encode(v: np.ndarray) -> np.ndarray:
    """E4M3 codes: nearest value, ties to even, saturating at 448, sign kept, NaN -> 0x7f."""
    v = np.asarray(v)
    mag = np.minimum(np.where(np.isnan(v), 0, np.abs(v)).astype(np.float64), 448.0)
    _, e = np.frexp(mag)  # mag in [2^(e-1), 2^e)
    e = np.maximum(np.where(mag == 0, -6, e - 1), -6)
    n = np.rint(np.ldexp(mag, 3 - e)).astype(np.int64)  # multiples of the step 2^(e-3), 0..16
    # n < 8 only at e = -6 (subnormals); n = 16 is the next binade's 8
    code = np.where(n < 8, n, ((e + 7) << 3) + (n - 8)).astype(np.int64)
    code = np.where(np.isnan(v), 0x7F, np.minimum(code, 0x7E) | np.where(np.signbit(v), 0x80, 0))
    return code.astype(np.uint8)


def decode(codes: np.ndarray) -> np.ndarray:
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


def _amax(v, axis):
    return np.max(np.where(np.isnan(v), 0, np.abs(v)), axis=axis, initial=0).astype(np.float32)


def _quot(x, s):
    """x / s in binary32; where s is 0, x holds zeros and NaN alone: 0 and NaN."""
    with np.errstate(all="ignore"):
        none = np.where(np.isnan(x), np.float32(np.nan), np.float32(0))
        return np.where(s == 0, none, x / np.where(s == 0, np.float32(1), s)).astype(np.float32)


def quantize(x: np.ndarray, tile: bool):
    """codes [M, K], scales [ceil(K/128), M or ceil(M/128)] of float32 x."""
    M, K = x.shape
    kb, mb = -(-K // BLOCK), -(-M // BLOCK)
    codes = np.empty((M, K), np.uint8)
    scales = np.empty((kb, mb if tile else M), np.float32)
    for b in range(kb):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        if tile:
            top = np.array([_amax(v[r * BLOCK:(r + 1) * BLOCK], None) for r in range(mb)], np.float32)
        else:
            top = _amax(v, 1)
        scales[b] = top / np.float32(448)
        s = np.repeat(scales[b], BLOCK)[:M] if tile else scales[b]
        codes[:, b * BLOCK:(b + 1) * BLOCK] = encode(_quot(v, s[:, None]))
    return codes, scales


def values(codes, scales, tile: bool):
    """Dequantized float64 [M, K]."""
    M, K = codes.shape
    s = np.repeat(scales.astype(np.float64), BLOCK, axis=0)[:K].T
    if tile:
        s = np.repeat(s, BLOCK, axis=0)[:M]
    return decode(codes) * s


def gemm(a, b):
    """(D, sum of |products|) of dequantized operands."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def page_scale(amax: np.float32) -> np.float32:
    """Smallest power of two s >= amax/448, at least 2^-126; 0 for 0."""
    if amax == 0:
        return np.float32(0)
    if np.isinf(amax):
        return np.float32(2.0 ** 120)
    f, e = np.frexp(np.float64(amax))  # amax = f 2^e, f in [1/2, 1); 448 = 0.875 * 2^9
    return np.float32(2.0 ** max(-126, int(e) - 9 + (f > 0.875)))


def kv_append(k, v, cache, table, cu, lens):
    """The cache [k codes, v codes, k scales, v scales] (numpy copies, changed in place)."""
    page = cache[0].shape[2]
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        begin = int(lens[b]) - n
        for p in range(begin // page, -(-int(lens[b]) // page) if n else 0):
            lo, hi = max(begin, p * page), min(int(lens[b]), (p + 1) * page)
            where, kept = int(table[b, p]), lo - p * page
            for x, codes, scales in ((k, cache[0], cache[2]), (v, cache[1], cache[3])):
                for h in range(codes.shape[1]):
                    new = x[cu[b] + lo - begin:cu[b] + hi - begin, h]
                    old = scales[where, h] if kept else np.float32(0)
                    s = max(old, page_scale(_amax(new, None)))
                    if kept and s > old:
                        x0 = decode(codes[where, h, :kept])
                        codes[where, h, :kept] = encode(x0 * float(old) / float(s)) if old else encode(_quot(x0, old))
                    scales[where, h] = s
                    codes[where, h, kept:kept + hi - lo] = encode(_quot(new, np.float32(s)))
    return cache


def attention(q, cache, table, cu, lens, causal, scale):
    """o, lse, and what their tolerances need, per query and head: sum p |v| [.., D], the largest
    sum |q| |k| * scale over its keys, and the largest |v|."""
    kc, vc, ks, vs = cache
    page, D = kc.shape[2], kc.shape[3]
    T, Hq = q.shape[:2]
    G = Hq // kc.shape[1]
    o, pv = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, reach, vmax = np.full((T, Hq), -np.inf), np.zeros((T, Hq)), np.zeros((T, Hq))
    for b in range(len(lens)):
        lo, n, L = int(cu[b]), int(cu[b + 1] - cu[b]), int(lens[b])
        if n == 0 or L == 0:
            continue
        pages = table[b, :-(-L // page)]
        for h in range(kc.shape[1]):
            k = (decode(kc[pages, h]) * ks[pages, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:L]
            v = (decode(vc[pages, h]) * vs[pages, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:L]
            for i in range(n):
                seen = L if not causal else L - n + i + 1
                if seen <= 0:
                    continue
                for g in range(h * G, (h + 1) * G):
                    x = q[lo + i, g].astype(np.float64)
                    with np.errstate(invalid="ignore"):
                        s = k[:seen] @ x * scale
                        top = s.max()
                        e = np.exp(s - top)
                        o[lo + i, g] = (e / e.sum()) @ v[:seen]
                        pv[lo + i, g] = (e / e.sum()) @ np.abs(v[:seen])
                        lse[lo + i, g] = top + np.log(e.sum())
                    reach[lo + i, g] = (np.abs(k[:seen]) @ np.abs(x)).max() * abs(scale)
                    vmax[lo + i, g] = np.abs(v[:seen]).max()
    return o, lse, pv, reach, vmax
