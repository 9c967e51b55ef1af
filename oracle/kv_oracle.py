"""Paged key/value cache (oracle side): appending with rotation, attention.

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).  float64, plain loops over
sequences and tokens; e4m3 numbers are found in a table of all of them.

A cache is a dict: "k", "v" float64 [blocks, heads, block, d] of the stored
numbers, "ks", "vs" float64 [blocks, heads] (ones for an unquantised cache).
A stored number times its scale is the value.
"""
import numpy as np


def e4m3_table():
    """The 256 e4m3 numbers by code: sign, 4 exponent bits (bias 7), 3 mantissa
    bits; exponent 0 is subnormal, 0x7f and 0xff are NaN, there is no infinity."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            out[c] = np.nan
        elif e == 0:
            out[c] = s * m / 8 * 2.0 ** -6
        else:
            out[c] = s * (1 + m / 8) * 2.0 ** (e - 7)
    return out


_POS = e4m3_table()[:127]            # 0 .. 448, ascending; index = code


def e4m3_round(x):
    """Nearest e4m3 number (ties to the even code), saturating at +-448."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=1e300, neginf=-1e300)), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 1, 126)
    lo = hi - 1
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    r = np.copysign(_POS[pick], x)
    return np.where(np.isnan(x), np.nan, r)


def e4m3_scale(amax):
    """Smallest power of two s >= 2^-64 with amax <= 448 s."""
    s = 2.0 ** -64
    while s * 448.0 < amax:
        s *= 2.0
    return s


def rotate(x, pos, table, interleaved):
    """x [d] at position pos; table float [positions, d]: cosines, then sines."""
    d = x.shape[-1]
    cos, sin = table[pos, :d // 2].astype(np.float64), table[pos, d // 2:].astype(np.float64)
    y = np.empty(x.shape)
    ia = np.arange(0, d, 2) if interleaved else np.arange(d // 2)
    ib = ia + 1 if interleaved else ia + d // 2
    y[..., ia] = x[..., ia] * cos - x[..., ib] * sin
    y[..., ib] = x[..., ib] * cos + x[..., ia] * sin
    return y


def positions(seq_lens, new_lens, S):
    """[(b, s, position)] of the valid new tokens that have a place."""
    out = []
    for b, n in enumerate(seq_lens):
        f = S if new_lens is None else new_lens[b]
        out += [(b, s, n - f + s) for s in range(f) if n - f + s >= 0]
    return out


def append(cache, k, v, block_table, seq_lens, new_lens, table, interleaved, quantised,
           round_k=True):
    """Stores k, v [B, heads, S, d] into `cache`, in place.  round_k False leaves
    the keys' quotients unrounded (the values that rounding starts from)."""
    B, H, S, d = k.shape
    bs = cache["k"].shape[2]
    places = {}
    for b, s, p in positions(seq_lens, new_lens, S):
        places.setdefault((b, p // bs), []).append((s, p))
    for (b, i), toks in places.items():
        blk = block_table[b][i]
        slots = np.array([p % bs for _, p in toks])
        for h in range(H):
            kk = np.stack([k[b, h, s] if table is None else
                           rotate(k[b, h, s], p, table, interleaved) for s, p in toks])
            vv = np.stack([v[b, h, s] for s, _ in toks])
            for name, sc, x, rnd in (("k", "ks", kk, round_k), ("v", "vs", vv, True)):
                if not quantised:
                    cache[name][blk, h, slots] = x
                    continue
                fin = np.abs(x[np.isfinite(x)])
                scale = e4m3_scale(fin.max() if fin.size else 0.0)
                if slots[0] > 0:
                    was = cache[sc][blk, h]
                    scale = max(scale, was)
                    if was < scale:
                        old = cache[name][blk, h, :slots[0]]
                        cache[name][blk, h, :slots[0]] = e4m3_round(old * (was / scale))
                cache[sc][blk, h] = scale
                cache[name][blk, h, slots] = e4m3_round(x / scale) if rnd else x / scale


def attention(q, cache, block_table, seq_lens, new_lens, window):
    """q [B, hq, S, d] -> (out, lse, spread): spread[b, h, s, :] is
    sum_j w_j |v_j| / sum_j w_j, what a relative error of the weights acts on.
    Padded rows are NaN in all three."""
    B, hq, S, d = q.shape
    H, bs = cache["k"].shape[1], cache["k"].shape[2]
    out = np.full(q.shape, np.nan)
    spread = np.full(q.shape, np.nan)
    lse = np.full((B, hq, S), np.nan)
    for b, n in enumerate(seq_lens):
        f = S if new_lens is None else new_lens[b]
        blocks = [block_table[b][i] if block_table[b][i] >= 0 else 0
                  for i in range(-(-n // bs))]
        for h in range(H):
            K = np.concatenate([cache["k"][i, h] * cache["ks"][i, h] for i in blocks] or
                               [np.zeros((0, d))])
            V = np.concatenate([cache["v"][i, h] * cache["vs"][i, h] for i in blocks] or
                               [np.zeros((0, d))])
            for g in range(h * (hq // H), (h + 1) * (hq // H)):
                for s in range(f):
                    p = n - f + s
                    lo = max(0, p - window + 1) if window else 0
                    if p < lo or p < 0:
                        out[b, g, s], spread[b, g, s], lse[b, g, s] = 0.0, 0.0, -np.inf
                        continue
                    x = K[lo:p + 1] @ q[b, g, s] / np.sqrt(d)
                    m = x.max()
                    w = np.exp(x - m)
                    out[b, g, s] = w @ V[lo:p + 1] / w.sum()
                    spread[b, g, s] = w @ np.abs(V[lo:p + 1]) / w.sum()
                    lse[b, g, s] = m + np.log(w.sum())
    return out, lse, spread
