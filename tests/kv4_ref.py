"""Plain restatements of kv4_attn.h in float64, for the tests: the cache format byte by byte, the
step tables, the query/key norm with rotation, attention over a cache."""
import math

import numpy as np

GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])


def bf16_to_f64(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def f32_to_bf16(x):
    """Round to nearest even (finite values)."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


# ------------------------------------------------------------------------ cache format ----

def quantize(bits):
    """bf16 bits [..., D] -> (codes [..., D], scale bytes [..., D/32])."""
    x = bf16_to_f64(bits)
    b = x.reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 1.0, np.abs(np.where(np.isfinite(b), b, 0)).max(-1))
    e = np.full(amax.shape, -126)
    for k in range(-125, 126):  # the smallest that holds amax, if one does
        e = np.where(6.0 * 2.0 ** (k - 1) < amax, k, e)
    y = np.where(bad[..., None], 0.0, b / np.exp2(e)[..., None])
    a = np.abs(y)
    lo = np.clip(np.searchsorted(GRID, a, side="right") - 1, 0, 7)
    hi = np.minimum(lo + 1, 7)
    up = (a - GRID[lo] > GRID[hi] - a) | ((a - GRID[lo] == GRID[hi] - a) & (lo % 2 == 1))
    code = np.where(up, hi, lo) + 8 * np.signbit(y)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scales):
    mag = GRID[codes & 7]
    v = np.where(codes & 8, -mag, mag)
    f = np.where(scales == 255, np.nan, np.where(scales == 0, 0.0, np.exp2(scales.astype(float) - 127)))
    return v * np.repeat(f, 32, -1)


def offsets(D):
    """For a tile: byte offsets of key codes, value codes [16, D] and scales [16, D/32]."""
    t, d = np.arange(16)[:, None], np.arange(D)[None]
    n = t // 8 * (D // 8) + d // 32 * 4 + d % 8 // 2
    kc = n // 16 * 512 + (t % 8 * 4 + d % 32 // 8) * 16 + n % 16
    n = (t // 8 * 2 + t % 2) * (D // 16) + d // 32 * 2 + d % 4 // 2
    vc = 8 * D + n // 16 * 512 + (d % 32 // 4 * 4 + t % 8 // 2) * 16 + n % 16
    b = np.arange(D // 32)[None]
    ks = 16 * D + t % 8 * (D // 16) + t // 8 * (D // 32) + b
    vs = 16 * D + D // 2 + t % 8 // 2 * (D // 8) + 4 * b + t // 8 * 2 + t % 2
    return kc, vc, ks, vs


def write_row(cache, slot, k, v):
    """bf16 bits k, v [heads, D] into `slot` of cache [pages, heads, tiles, 17 D] (uint8)."""
    D = cache.shape[3] // 17
    page, off = divmod(int(slot), cache.shape[2] * 16)
    tile, t = divmod(off, 16)
    kc, vc, ks, vs = offsets(D)
    for at, sat, x in ((kc, ks, k), (vc, vs, v)):
        codes, scales = quantize(x)
        row = cache[page, :, tile]
        row[:, at[t, ::2]] = codes[:, ::2] | codes[:, 1::2] << 4
        row[:, sat[t]] = scales


def fill(cache, k, v):
    """bf16 bits [pages, heads, page_size, D] into the whole cache."""
    P, H, tiles, B = cache.shape
    D = B // 17
    kc, vc, ks, vs = offsets(D)
    for at, sat, x in ((kc, ks, k), (vc, vs, v)):
        codes, scales = quantize(x.reshape(P, H, tiles, 16, D))
        cache[..., at[:, ::2]] = codes[..., ::2] | codes[..., 1::2] << 4
        cache[..., sat] = scales


def decode(cache):
    """The whole cache as float64 keys, values [pages, heads, page_size, D]."""
    P, H, tiles, B = cache.shape
    D = B // 17
    kc, vc, ks, vs = offsets(D)
    up = 4 * (np.arange(D) % 2)
    out = []
    for at, sat in ((kc, ks), (vc, vs)):
        out.append(values((cache[..., at] >> up) & 15, cache[..., sat]).reshape(P, H, tiles * 16, D))
    return out


# ------------------------------------------------------------------------- step tables ----

def step_tables(cached, new, free, table, page, max_rows):
    table = table.copy()
    starts, lens, pos, slots, used, bits = [0], [], [], [], 0, 0
    for r, (c, n) in enumerate(zip(cached.tolist(), new.tolist())):
        if c < 0 or n < 0 or c + n > table.shape[1] * page:
            bits |= 16
            c = n = 0
        have, want = -(-c // page), -(-(c + n) // page) if n else -(-c // page)
        for e in range(have, want):
            if used < len(free):
                table[r, e] = free[used]
            else:
                table[r, e] = -1
                bits |= 32
            used += 1
        lens.append(c + n)
        for i in range(n):
            p = c + i
            pos.append(p)
            slots.append(table[r, p // page] * page + p % page if table[r, p // page] >= 0 else -1)
        starts.append(starts[-1] + n)
    if starts[-1] > max_rows:
        bits |= 64
    starts = [min(s, max_rows) for s in starts]
    pos = (pos + [0] * max_rows)[:max(max_rows, 0)] if len(pos) < max_rows else pos[:max_rows]
    slots = (slots + [-1] * max_rows)[:max_rows]
    return table, np.array(starts), np.array(lens), np.array(pos), np.array(slots), min(used, len(free)), bits


# ---------------------------------------------------------------------- norm + rotation ----

def norm_rope(x, gamma, pos, freq, eps, interleaved):
    """float64 x [T, heads, D] -> the unrounded result and, for the tolerance, each element's
    pair magnitude |a| + |b| before the rotation."""
    n = x.copy()
    if gamma is not None:
        n = n / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * gamma
    half = len(freq)
    ang = (pos.astype(np.longdouble)[:, None] * freq.astype(np.longdouble)[None]) % (2 * np.longdouble(math.pi))
    # (2 pi to 64 bits: over 2^31 radians that is 2^-31 off at most)
    c, s = np.cos(ang).astype(float)[:, None], np.sin(ang).astype(float)[:, None]
    y, mag = n.copy(), np.abs(n)
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = n[..., ia], n[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = np.abs(a) + np.abs(b)
    return y, mag


# --------------------------------------------------------------------------- attention ----

def attention(q, K, V, table, starts, lens, page, scale, window=0, sinks=0):
    """q float64 [T, Hq, D], K, V [pages, heads, page, D] -> {row: (out [Hq, D], avg [Hq, D] =
    sum p |v| / sum p, spread [Hq] = scale * max_j sum_d |q_d k_jd|, total [Hq, D] = sum |v|)}."""
    T, Hq, D = q.shape
    H = K.shape[1]
    G = Hq // H
    res = {}
    for r, L in enumerate(lens.tolist()):
        n = starts[r + 1] - starts[r]
        for i in range(starts[r], starts[r + 1]):
            p = L - (starts[r + 1] - i)
            j = np.arange(0, max(p + 1, 0))
            if window:
                j = j[(j > p - window) | (j < sinks)]
            out, avg, spread, total = np.zeros((Hq, D)), np.zeros((Hq, D)), np.zeros(Hq), np.zeros((Hq, D))
            j = j[(table[r, j // page] >= 0) & (table[r, j // page] < K.shape[0])]
            if len(j):
                pg, off = table[r, j // page], j % page
                for h in range(H):
                    k, v = K[pg, h, off], V[pg, h, off]
                    qq = q[i, h * G:(h + 1) * G]
                    s = qq @ k.T * scale
                    with np.errstate(invalid="ignore"):
                        w = np.exp(s - s.max(-1, keepdims=True))
                        w /= w.sum(-1, keepdims=True)
                        out[h * G:(h + 1) * G] = w @ v
                        avg[h * G:(h + 1) * G] = w @ np.abs(v)
                    spread[h * G:(h + 1) * G] = (np.abs(qq) @ np.abs(k).T).max(-1) * scale
                    total[h * G:(h + 1) * G] = np.abs(v).sum(0)
            res[i] = (out, avg, spread, total)
    return res


def attention_tolerance(out, avg, spread, total, D):
    """|kernel - out| at most: the result's own rounding to bf16 (half a step: 2^-8 of the value);
    the numerators' rounding to tf32 (half a step, 2^-11 of each term, so 2^-11 of sum p |v| /
    sum p; the sum of the numerators takes them unrounded); queries and keys enter the score's
    product exactly (8 and 2 significant bits), its fp32 sums are D / 8 additions of 8 products,
    each off by at most 2^-22 of the terms' magnitudes (2^-23 for each of alignment and cut), and
    the scale one more, in the exponent of numerator and denominator alike (twice); the output
    sums are fp32 additions of 8 tokens each, at most 128 of them in one range here (1024 tokens),
    2^-23 each: 2^-16 with the exponentials' 2^-22 and the join's few.  Numerators and the join's
    weights below 2^-126 are flushed to zero, against a sum of 1 at least (a row's reference is at
    most its maximum): 2 2^-126 |v| of each token; a subnormal result is off by its half step,
    2^-134."""
    d = (D / 8 + 1) * 2.0 ** -22 * spread[:, None]
    return (2.0 ** -8 * np.abs(out) + avg * (2.0 ** -11 + 2 * d + 2.0 ** -16) + 2.0 ** -125 * total
            + 2.0 ** -134)
