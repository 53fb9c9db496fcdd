"""The 8-bit paged cache in fp64: e4m3 codes with one power-of-two scale per (page, KV head).

Caches are arrays of bytes [pages][heads][16][d] and of scales [pages][heads]; written from the definition,
token by token, apart from the library and from every other form of it.
"""

import numpy as np

PAGE = 16
E_MIN, E_MAX = -100, 119


def _e4m3_values():
    """Value of every byte: sign, four exponent bits (bias 7), three fraction bits; 0x7F and 0xFF are NaN."""
    v = np.empty(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[b] = -x if s else x
    v[0x7F] = v[0xFF] = np.nan
    return v


VALUES = _e4m3_values()
_POS = VALUES[:127]


def e4m3_encode(x):
    """Nearest code (ties to the even one, beyond 448 saturated) of fp64 values; NaN becomes zero."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=np.inf, neginf=-np.inf)), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (code + 128 * (np.signbit(x) & ~np.isnan(x))).astype(np.uint8)


def block_exponent(amax):
    """Smallest e in range with amax <= 448 * 2^e."""
    for e in range(E_MIN, E_MAX + 1):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return E_MAX


def rotate(x, cos, sin, interleaved):
    """x [.., d] with its first 2 * len(cos) channels' pairs turned."""
    y = np.array(x, np.float64)
    n = len(cos)
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    with np.errstate(invalid="ignore", over="ignore"):
        y1 = x[..., a] * cos - x[..., b] * sin
        y2 = x[..., b] * cos + x[..., a] * sin
    y[..., a], y[..., b] = y1, y2
    return y


def append_token(codes, scales, page, slot, x, amax_of=None):
    """Write one token's heads x [h][d] at (page, slot) of one cache, in place.  A block that starts (slot 0) takes
    its own scale; amax_of, if given, the largest finite value per head that the scale has to hold."""
    for h in range(x.shape[0]):
        fin = np.abs(x[h][np.isfinite(x[h])])
        amax = (fin.max() if fin.size else 0.0) if amax_of is None else amax_of[h]
        e = block_exponent(amax)
        if slot > 0:
            e_old = int(np.log2(scales[page, h]))
            if e > e_old:
                codes[page, h, :slot] = e4m3_encode(VALUES[codes[page, h, :slot]] * 2.0 ** (e_old - e))
            e = max(e, e_old)
        scales[page, h] = 2.0 ** e
        codes[page, h, slot] = e4m3_encode(x[h] * 2.0 ** -e)


def append(codes, scales, row, start, x):
    """Tokens x [n][h][d] of one call at positions start .. of the sequence whose pages are `row`: a page's tokens of
    the call share the scale they need together."""
    n = x.shape[0]
    t = 0
    while t < n:
        pos = start + t
        m = min(n - t, PAGE - pos % PAGE)
        y = np.abs(np.where(np.isfinite(x[t:t + m]), x[t:t + m], 0.0))
        amax = y.max(axis=(0, 2))
        for i in range(m):
            append_token(codes, scales, row[(pos + i) // PAGE], (pos + i) % PAGE, x[t + i], amax)
        t += m


def visible(p, j, window, sinks):
    return (j <= p) & ((window == 0) | (j > p - window) | (j < sinks))


def attention(q, codes_k, scale_k, codes_v, scale_v, row, p, window, sinks, softmax_scale, hidden=()):
    """q [hq][d] of one query at position p: (out, sum of weight * |value|, and over the seen keys the largest sum |q k|,
    the largest sum |k|, and their number).
    `hidden`: positions that are not there."""
    hq, d = q.shape
    h = codes_k.shape[1]
    g = hq // h
    j = np.arange(p + 1)
    seen = visible(p, j, window, sinks) & ~np.isin(j, list(hidden))
    j = j[seen]
    out, mag, dots, ksum = np.zeros((hq, d)), np.zeros((hq, d)), np.zeros(hq), np.zeros(hq)
    if j.size == 0:
        return out, mag, dots, ksum, 0
    pg, sl = np.asarray(row)[j // PAGE], j % PAGE
    for kv in range(h):
        k = VALUES[codes_k[pg, kv, sl]] * scale_k[pg, kv].astype(np.float64)[:, None]
        v = VALUES[codes_v[pg, kv, sl]] * scale_v[pg, kv].astype(np.float64)[:, None]
        for a in range(kv * g, (kv + 1) * g):
            s = (k @ q[a].astype(np.float64)) * softmax_scale
            w = np.exp(s - s.max())
            w /= w.sum()
            out[a], mag[a] = w @ v, w @ np.abs(v)
            dots[a] = (np.abs(k) @ np.abs(q[a].astype(np.float64))).max()
            ksum[a] = np.abs(k).sum(axis=1).max()
    return out, mag, dots, ksum, j.size
