"""Plain 64-bit forms of the paged-cache operators, in numpy, a sequence at a time.  Test
infrastructure: shares no code with the library."""
import numpy as np

E4M3_MAX = 448.0
TINY = 1e-30


def e4m3_values():
    """The value of each of the 256 e4m3 codes (sign, 4 exponent bits with bias 7, 3 mantissa bits)."""
    out = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            v = np.nan
        out[code] = -v if code & 128 else v
    return out


def round_e4m3(y):
    """The nearest e4m3 value within +-448, ties to even."""
    y = np.clip(y, -E4M3_MAX, E4M3_MAX)
    _, e = np.frexp(y)
    step = np.exp2(np.maximum(e - 4, -9).astype(np.float64))
    return np.rint(y / step) * step


def quantise32(x):
    """The library's definition of a written row, each step rounded to 32 bits: (values, scale)."""
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        amax = np.maximum(np.abs(x).max(-1), np.float32(TINY))
        y = x * (np.float32(E4M3_MAX) / amax)[..., None]
        return round_e4m3(y.astype(np.float64)), amax * np.float32(1.0 / E4M3_MAX)


def rows(data, table, n, pages, page):
    """(there, page, row) of a sequence's positions 0 .. n-1, given as an array of positions."""
    n = np.asarray(n, np.int64)
    there = (n >= 0) & (n < len(table) * page)
    ids = np.where(there, table[np.where(there, n // page, 0)], -1) if len(table) else np.full(n.shape, -1)
    there &= (ids >= 0) & (ids < pages)
    return there, np.where(there, ids, 0), np.where(there, n % page, 0)


def logits(q, w, k, scale, table, lens, N):
    """(out [B*T, N] with -inf outside, the sum of absolute terms): q [B, T, H, D], k [pages, page, D]."""
    B, T = q.shape[:2]
    pages, page = k.shape[:2]
    out, size = np.full((B, T, N), -np.inf), np.zeros((B, T, N))
    for b in range(B):
        for t in range(T):
            n = np.arange(max(0, min(N, int(lens[b]) - (T - 1 - t))))
            there, ids, row = rows(k, table[b], n, pages, page)
            n, ids, row = n[there], ids[there], row[there]
            keys, by = k[ids, row], scale[ids, row]
            dots = keys @ q[b, t].T
            out[b, t, n] = (np.maximum(dots, 0) * w[b, t]).sum(1) * by
            size[b, t, n] = ((np.abs(keys) @ np.abs(q[b, t]).T) * np.abs(w[b, t])).sum(1) * np.abs(by)
    return out.reshape(B * T, N), size.reshape(B * T, N)


def attention(q, k, v, table, lens, sm_scale, indices=None):
    """(out, lse, sum of p |v|, largest |x| term sum): q [B, Hq, D], k and v [pages, page, Hk, D]."""
    B, Hq, D = q.shape
    pages, page, Hk, _ = k.shape
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    size, dots = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    for b in range(B):
        n = np.arange(max(0, int(lens[b])))
        if indices is not None:
            n = indices[b][(indices[b] >= 0) & (indices[b] < lens[b])]
        there, ids, row = rows(k, table[b], n, pages, page)
        ids, row = ids[there], row[there]
        if len(ids) == 0:
            continue
        for h in range(Hq):
            g = h // (Hq // Hk)
            x = sm_scale * (k[ids, row, g] @ q[b, h])
            p = np.exp(x - x.max())
            out[b, h] = p @ v[ids, row, g] / p.sum()
            size[b, h] = p @ np.abs(v[ids, row, g]) / p.sum()
            lse[b, h] = x.max() + np.log(p.sum())
            dots[b, h] = (abs(sm_scale) * (np.abs(k[ids, row, g]) @ np.abs(q[b, h]))).max()
    return out, lse, size, dots
