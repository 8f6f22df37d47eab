"""Plain fp64 definitions of the 8-bit paged cache (test infrastructure only).

A cache holds codes (e4m3 or int8, one byte) and one scale per group of 16
consecutive slots of a page and kv head, K and V apart; value = code * scale.

* ``q8_round``   rounds a value to a code: nearest, ties to even, at most the
                 largest code.
* ``q8_values``  code bytes -> float64 code values.
* ``q8_bytes``   float64 code values -> code bytes.
* ``q8_append``  the append's quantisation rule, group by group.
"""

from __future__ import annotations

import numpy as np

GROUP = 16
TOP = {"e4m3": 448.0, "int8": 127.0}
MIN_EXP, MAX_EXP = -64, 63


def q8_round(x, fmt):
    """float64 -> the float64 value of the nearest code (ties to even)."""
    x = np.asarray(x, np.float64)
    x = np.clip(x, -TOP[fmt], TOP[fmt])
    if fmt == "int8":
        return np.rint(x)
    _, e = np.frexp(np.where(x == 0, 1.0, np.abs(x)))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)   # 3 fraction bits, subnormals below 2^-6
    return np.clip(np.rint(x / step) * step, -TOP[fmt], TOP[fmt])


def q8_values(codes, fmt):
    """Code bytes (uint8) -> float64; the e4m3 NaN pattern gives NaN."""
    b = np.asarray(codes, np.uint8)
    if fmt == "int8":
        return b.view(np.int8).astype(np.float64)
    e = ((b >> 3) & 15).astype(np.int64)
    m = (b & 7).astype(np.float64)
    mag = np.where(e == 0, np.ldexp(m, -9), np.ldexp(8 + m, e - 10))
    mag = np.where((b & 0x7F) == 0x7F, np.nan, mag)
    return np.where(b & 0x80, -mag, mag)


def q8_bytes(values, fmt):
    """float64 code values -> code bytes (values must be codes)."""
    v = np.asarray(values, np.float64)
    if fmt == "int8":
        return v.astype(np.int8).view(np.uint8)
    a = np.abs(v)
    _, e = np.frexp(np.where(a == 0, 1.0, a))
    sub = a < 2.0 ** -6
    field = np.where(sub, 0, e + 6)
    frac = np.where(sub, a * 2.0 ** 9, np.ldexp(a, 4 - e) - 8)
    return ((np.signbit(v).astype(np.uint8) << 7)
            | (field.astype(np.uint8) << 3) | frac.astype(np.uint8))


def q8_scale_exponent(amax, fmt):
    """Smallest e in [MIN_EXP, MAX_EXP] with amax <= TOP * 2^e (MAX_EXP beyond)."""
    for e in range(MIN_EXP, MAX_EXP):
        if amax <= TOP[fmt] * 2.0 ** e:
            return e
    return MAX_EXP


def q8_append(values, slots, codes, scales, fmt):
    """Append values [T, H, D] (float64) at `slots` into codes [NB, bs, H, D]
    (uint8) and scales [NB, bs // 16, H] (float); returns copies.

    Per group and head: amax over the finite appended values; the scale is
    2^e where slot 0 is among them, else the larger of 2^e and the stored one
    (outside 2^-64 .. 2^63: 2^-64), and the other codes follow a grown scale.
    NaN appends as 0.  Slots outside the cache append nothing.
    """
    y = np.asarray(values, np.float64)
    nb, bs, H, D = codes.shape
    c = q8_values(codes, fmt).reshape(nb * bs // GROUP, GROUP, H, D)
    s = np.array(scales, np.float64).reshape(nb * bs // GROUP, H)
    groups = {}
    for t, slot in enumerate(np.asarray(slots).tolist()):
        if 0 <= slot < nb * bs:
            groups.setdefault(slot // GROUP, []).append((slot % GROUP, t))
    for g, members in groups.items():
        offs = [o for o, _ in members]
        rest = [o for o in range(GROUP) if o not in offs]
        for h in range(H):
            rows = y[[t for _, t in members], h]
            finite = np.abs(rows[np.isfinite(rows)])
            new = 2.0 ** q8_scale_exponent(finite.max() if finite.size else 0.0, fmt)
            if 0 not in offs:
                old = s[g, h] if 2.0 ** MIN_EXP <= s[g, h] <= 2.0 ** MAX_EXP else 2.0 ** MIN_EXP
                new = max(new, old)
                if new > old:
                    c[g, rest, h] = q8_round(c[g, rest, h] * (old / new), fmt)
            s[g, h] = new
            c[g, offs, h] = q8_round(np.where(np.isnan(rows), 0.0, rows) / new, fmt)
    return c.reshape(codes.shape), s.reshape(scales.shape)
