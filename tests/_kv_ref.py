"""The 8-bit key/value cache from its definition, in 64 bits and on the CPU: what the GPU tests compare with.

A cache is a dict of numpy arrays: the value of each code over its scale (``k``, ``v``) and the scale exponents (``kx``,
``vx``); FP8 rounding is done on the sorted table of a format's values."""

import numpy as np

from _gpu import fp8_table

FMAX = (448.0, 57344.0)


def exponent(amax: float, fmt: int) -> int:
    """The smallest X in [-127, 127] with amax <= fmax 2^X; -127 for 0."""
    if amax == 0:
        return -127
    x = int(np.ceil(np.log2(amax / FMAX[fmt]))) + 2
    while x > -127 and amax <= FMAX[fmt] * 2.0 ** (x - 1):
        x -= 1
    return max(-127, min(127, x))


def fp8_round(v: np.ndarray, fmt: int) -> np.ndarray:
    """Nearest value of the format, ties to the even code, saturating; not finite: NaN."""
    t = fp8_table(fmt)[:128]
    t = t[np.isfinite(t)]
    a = np.minimum(np.abs(v), FMAX[fmt])
    with np.errstate(invalid="ignore"):
        hi = np.clip(np.searchsorted(t, np.nan_to_num(a)), 0, len(t) - 1)
        lo = np.maximum(hi - 1, 0)
        below, above = a - t[lo], t[hi] - a
        up = (above < below) | ((above == below) & (hi % 2 == 0))
        r = np.where(up, t[hi], t[lo])
    return np.where(np.isfinite(v), np.copysign(r, v), np.nan)


def rows_of(n_seqs, T, row_start):
    """[(first row, rows)] of each sequence."""
    if row_start is None:
        return [(s * (T // n_seqs), T // n_seqs) for s in range(n_seqs)]
    return [(row_start[s], row_start[s + 1] - row_start[s]) for s in range(n_seqs)]


def append(cache, fmt, P, pages, lens, rows, kv):
    """kv [T, 2, heads, dh] float64 into the cache, in place."""
    for s, (first, n) in enumerate(rows):
        at = lens[s] - n
        j = max(0, -at)
        while j < n:
            slot, page = (at + j) % P, pages[s][(at + j) // P]
            m = min(P - slot, n - j)
            if 0 <= page < len(cache["k"]):
                for part, name in enumerate("kv"):
                    x = kv[first + j:first + j + m, part]
                    for h in range(x.shape[1]):
                        fine = np.abs(x[:, h][np.isfinite(x[:, h])])
                        X = exponent(float(fine.max()) if fine.size else 0.0, fmt)
                        was = cache[name + "x"][page, h]
                        if slot:
                            X = max(X, was)
                            old = cache[name][page, h, :slot]
                            if X > was:
                                cache[name][page, h, :slot] = fp8_round(old * 2.0 ** (int(was) - X), fmt)
                        cache[name][page, h, slot:slot + m] = fp8_round(x[:, h] * 2.0 ** -X, fmt)
                        cache[name + "x"][page, h] = X
            j += m


def held(cache, P, pages, s, upto, name):
    """Tokens 0 .. upto - 1 of sequence s as [upto, heads, dh], and which of them have a page."""
    heads, dh = cache[name].shape[1], cache[name].shape[3]
    out, ok = np.zeros((upto, heads, dh)), np.zeros(upto, bool)
    for t in range(0, upto, P):
        page, m = pages[s][t // P], min(P, upto - t)
        if 0 <= page < len(cache[name]):
            out[t:t + m] = (cache[name][page] * 2.0 ** cache[name + "x"][page].astype(float)[:, None, None]).transpose(1, 0, 2)[:m]
            ok[t:t + m] = True
    return out, ok


def read(cache, P, pages, lens, rows, T):
    """[T, 2 heads dh]; rows that no sequence owns are NaN."""
    heads, dh = cache["k"].shape[1], cache["k"].shape[3]
    out = np.full((T, 2, heads, dh), np.nan)
    for s, (first, n) in enumerate(rows):
        for part, name in enumerate("kv"):
            x, _ = held(cache, P, pages, s, max(0, lens[s]), name)
            pad = max(0, n - lens[s])
            out[first:first + pad, part] = 0
            out[first + pad:first + n, part] = x[len(x) - (n - pad):]
    return out.reshape(T, -1)


def attend(cache, P, pages, lens, rows, q):
    """q [T, hq, dh] -> att [T, hq, dh], its terms' magnitudes sum p |v| / sum p, lse [hq, T], the largest
    sum |q| |k| / sqrt(dh) of a score [hq, T]; NaN where no sequence owns a row."""
    T, hq, dh = q.shape
    att, size, lse = np.full((T, hq, dh), np.nan), np.full((T, hq, dh), np.nan), np.full((hq, T), np.nan)
    mag = np.zeros((hq, T))
    group = hq // cache["k"].shape[1]
    for s, (first, n) in enumerate(rows):
        K, ok = held(cache, P, pages, s, max(0, lens[s]), "k")
        V, _ = held(cache, P, pages, s, max(0, lens[s]), "v")
        for j in range(n):
            upto = max(0, lens[s] - n + j + 1)
            see = ok[:upto]
            att[first + j], size[first + j], lse[:, first + j] = 0, 0, -np.inf
            if not see.any():
                continue
            for h in range(hq):
                k, v = K[:upto][see][:, h // group], V[:upto][see][:, h // group]
                z = k @ q[first + j, h] / np.sqrt(dh)
                m = z.max()
                mag[h, first + j] = (np.abs(k) @ np.abs(q[first + j, h])).max() / np.sqrt(dh)
                p = np.exp(z - m)
                att[first + j, h] = p @ v / p.sum()
                size[first + j, h] = p @ np.abs(v) / p.sum()
                lse[h, first + j] = m + np.log(p.sum())
    return att, size, lse, mag
