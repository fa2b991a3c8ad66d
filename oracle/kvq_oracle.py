"""Plain fp64 oracle of the 8-bit K/V cache.  Test infrastructure only.

An element of the cache stands for code * scale: one 8-bit code per element
(e4m3 or int8), one scale per block of 64 tokens and KV head.  Codes are kept here
as the numbers they are, in float64, and every rounding is done on real quotients
(exact for the scales that a write makes: powers of two for e4m3, eight
significant bits for int8, so that float64's own rounding never reaches a tie).
"""

import math

import numpy as np

BLOCK = 64
SCALE_MIN = 2.0 ** -100
TOP = {"e4m3": 448.0, "int8": 127.0}


def e4m3_numbers():
    """The non-negative e4m3 numbers in the order of their codes 0 .. 126."""
    sub = [m * 2.0 ** -9 for m in range(8)]
    return np.array(sub + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def e4m3_from_bits(bits):
    """Values of e4m3 codes (uint8)."""
    b = np.asarray(bits, dtype=np.uint8)
    mag = np.append(e4m3_numbers(), np.nan)[b & 0x7F]
    return np.where(b & 0x80, -mag, mag)


def nearest(y, fmt):
    """y rounded to the format: nearest, ties to even, saturating; NaN to NaN (e4m3) or 0 (int8)."""
    y = np.asarray(y, dtype=np.float64)
    if fmt == "int8":
        return np.clip(np.rint(np.nan_to_num(y, nan=0.0, posinf=127.0, neginf=-127.0)), -127, 127)
    tab = e4m3_numbers()
    a = np.minimum(np.abs(y), 448.0)
    i = np.clip(np.searchsorted(tab, np.nan_to_num(a, nan=0.0), side="right") - 1, 0, len(tab) - 2)
    lo, hi = tab[i], tab[i + 1]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 1))
    return np.where(np.isnan(y), np.nan, np.copysign(np.where(up, hi, lo), y))


def scale_for(amax, fmt):
    """The smallest power of two s with amax <= 448 s, or bf16 number s with amax <= 127 s; at least 2^-100."""
    if amax == 0:
        return SCALE_MIN
    m, e = math.frexp(amax)
    if fmt == "e4m3":
        s = math.ldexp(1.0, e - 9 if m <= 0.875 else e - 8)  # 448 = 0.875 * 2^9
    else:
        _, e = math.frexp(amax / 127)
        unit = math.ldexp(1.0, e - 8)  # eight significant bits
        n = math.floor(amax / 127 / unit) - 1
        while n * unit * 127 < amax:
            n += 1
        s = n * unit
    return max(s, SCALE_MIN)


def write(codes, scales, x, first, fmt):
    """Write x [n, H, d] as rows [first, first + n) of codes [H, rows, d] and scales [H, blocks], in place."""
    n = x.shape[0]
    x = np.asarray(x, dtype=np.float64)
    for blk in range(first // BLOCK, (first + n + BLOCK - 1) // BLOCK):
        lo, r0, r1 = blk * BLOCK, max(first, blk * BLOCK), min(first + n, (blk + 1) * BLOCK)
        if r0 >= r1:
            continue
        for h in range(codes.shape[0]):
            new = x[r0 - first:r1 - first, h]
            fine = np.abs(new[np.isfinite(new)])
            s = scale_for(float(fine.max()) if fine.size else 0.0, fmt)
            if r0 > lo:
                old = scales[h, blk]
                s = max(s, old)
                codes[h, lo:r0] = nearest(codes[h, lo:r0] * old / s, fmt)
            codes[h, r0:r1] = nearest(new / s, fmt)
            scales[h, blk] = s


def values(codes, scales):
    """What codes [..., rows, d] with scales [..., blocks] stand for."""
    s = np.repeat(np.asarray(scales, dtype=np.float64), BLOCK, axis=-1)[..., :codes.shape[-2]]
    return np.asarray(codes, dtype=np.float64) * s[..., None]


def decode_with_bound(q, k, v, u, b, offsets, seq_lens, mode, v_scale=None):
    """Decode attention in fp64 and what bounds a kernel's rounding of it.

    q [S, N, Hq, d], k, v [S, Hkv, L, d], u [S, N or 1, L, r], b [N, r, Hkv d].
    Returns (out, a_v, a_z, floor): a_v = sum_t p |v|, a_z = sum_t p |U| |B| per output element, the sizes that a
    relative error of each weight p multiplies, and floor = max_t (p s_t) sum_t |v / s_t| with the value scales s_t
    of v_scale [S, Hkv, blocks] (0 without them), what an error of each weight p s_t relative to the row's
    largest multiplies.
    """
    S, N, Hq, d = q.shape
    Hkv, r = k.shape[1], u.shape[-1]
    G = Hq // Hkv
    out, a_v, a_z, floor = (np.zeros((S, N, Hq, d)) for _ in range(4))
    for s in range(S):
        n = int(seq_lens[s])
        if n == 0:
            continue
        for i in range(N):
            ui = np.array(u[s, i if mode == 0 else 0, :n])
            ui[:max(0, int(offsets[s, i]))] = 0.0
            for h in range(Hq):
                g = h // G
                w = (k[s, g, :n] @ q[s, i, h]) / math.sqrt(d)
                p = np.exp(w - w.max())
                p /= p.sum()
                bg = b[i][:, g * d:(g + 1) * d]
                out[s, i, h] = p @ v[s, g, :n] + (p @ ui) @ bg
                a_v[s, i, h] = p @ np.abs(v[s, g, :n])
                a_z[s, i, h] = (p @ np.abs(ui)) @ np.abs(bg)
                if v_scale is not None:
                    st = np.repeat(v_scale[s, g], BLOCK)[:n, None]
                    codes = np.divide(np.abs(v[s, g, :n]), st, out=np.zeros((n, d)), where=st > 0)
                    floor[s, i, h] = (p * st[:, 0]).max() * codes.sum(axis=0)
    return out, a_v, a_z, floor
