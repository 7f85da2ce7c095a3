"""Plain forms of a serving step's other operators, in numpy: page tables (a request at a time), norms with
rotation (64 bits), and rows in 4 bits (each step as defined).  Test infrastructure: shares no code with the
library."""
import numpy as np

from .paged import E4M3_MAX, TINY, round_e4m3

GROUP = 16
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def pages(table, lens, change, free, n_free, page, total):
    """Updates table, lens and free in place; returns (n_free, slots, positions, rows, starts, changed)."""
    B, cols = table.shape
    count = lambda n: -(-n // page)  # noqa: E731
    n0 = min(max(int(n_free), 0), len(free))
    len0 = [min(max(int(n), 0), cols * page) for n in lens]
    to = [max(0, n + int(c)) for n, c in zip(len0, change)]
    stack = [int(x) for x in free[:n0]]
    for b in range(B):
        if change[b] < 0:
            stack += [int(x) for x in table[b, count(to[b]):count(len0[b])]]
    stack = stack[:len(free)]
    short, fits = False, [True] * B
    for b in range(B):
        want = count(to[b]) - count(len0[b])
        if change[b] <= 0:
            continue
        if to[b] > cols * page:
            fits[b] = False
        elif want:
            short |= want > len(stack)
            fits[b] = not short
            for c in range(count(len0[b]), count(to[b]) if fits[b] else 0):
                table[b, c] = stack.pop()
    free[n0:len(stack)] = stack[n0:]
    starts = np.minimum(np.concatenate([[0], np.cumsum([max(0, t - n) for t, n in zip(to, len0)])]), 2 ** 31 - 1)
    slots, positions, rows = np.full(total, -1, np.int32), np.zeros(total, np.int32), np.zeros(total, np.int32)
    for b in range(B):
        for i in range(int(starts[b]), min(int(starts[b + 1]), total)):
            at = len0[b] + i - int(starts[b])
            rows[i], positions[i] = b, min(at, 2 ** 31 - 1)
            if fits[b] and table[b, at // page] >= 0:
                slots[i] = table[b, at // page] * page + at % page
    changed = np.array([t - n if f else 0 for t, n, f in zip(to, len0, fits)], np.int32)
    lens[:] = [t if f else n for t, n, f in zip(to, len0, fits)]
    return len(stack), slots, positions, rows, starts.astype(np.int32), changed


def norm_rotate(x, weight, positions, inv_freq, eps, interleaved):
    """(out, the sum of absolute terms): x [T, H, D] in 64 bits."""
    T, _, D = x.shape
    by = np.ones(x.shape[:2] + (1,))
    w = np.ones(D)
    if weight is not None:
        by, w = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps), weight
    y = x * by * w
    out, size = y.copy(), np.abs(y)
    n = len(inv_freq)
    # (the product of a 32-bit position and a 24-bit frequency is rounded to 64 bits at most once)
    angle = (positions.astype(np.longdouble)[:, None] * inv_freq.astype(np.longdouble)) % (2 * PI)
    cos, sin = np.cos(angle).astype(np.float64)[:, None], np.sin(angle).astype(np.float64)[:, None]
    i = np.arange(n)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    out[..., a] = y[..., a] * cos - y[..., b] * sin
    out[..., b] = y[..., b] * cos + y[..., a] * sin
    size[..., a] = size[..., b] = np.abs(y[..., a]) + np.abs(y[..., b])
    return out, size


PI = np.longdouble("3.14159265358979323846264338327950288")


def round_e2m1(y):
    """The nearest e2m1 value within +-6, ties to even."""
    y = np.clip(y, -6, 6)
    _, e = np.frexp(y)
    step = np.exp2(np.maximum(e - 2, -1).astype(np.float64))
    return np.rint(y / step) * step


def quantise4(x):
    """The library's definition of a row in 4 bits, products and quotients rounded to 32 bits: (values, groups, scale)."""
    x = x.astype(np.float32)
    f = np.float32
    with np.errstate(all="ignore"):
        a = np.maximum(np.abs(x).max(-1), f(TINY))
        parts = x.reshape(x.shape[:-1] + (-1, GROUP))
        m = np.abs(parts).max(-1)
        # (7/8 and 2^-9, 21/32 and 2^-12 stand for 448 and 2688: no overflow)
        groups = round_e4m3(((m * f(0.875)) / (a * f(2.0 ** -9))[..., None]).astype(np.float64))
        by = groups.astype(f) * (a * f(2.0 ** -12))[..., None]
        y = np.where(by[..., None] > 0, (parts * f(21 / 32)) / by[..., None], f(0))
        return round_e2m1(y.astype(np.float64)).reshape(x.shape), groups, a * f(1 / 2688)


def unpack(codes):
    """The values of e2m1 codes, two a byte, the first one low."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
