"""Float64 definitions of the rotary operator and the 8-bit paged cache."""
from __future__ import annotations

import math

import numpy as np

PAGE = 64
MIN_EXP, MAX_EXP = -100, 100


def rope_frequencies(span, n_rot, theta=10000.0, scaling="plain", factor=1.0, original=0.0,
                     turns_lo=1.0, turns_hi=32.0):
    """Angle per position of each turned pair."""
    if scaling == "raised":
        theta = theta * factor ** (span / (span - 2))
    out = []
    for j in range(n_rot):
        g = theta ** (-2.0 * j / span)
        if scaling == "linear":
            g /= factor
        if scaling == "parts":
            turns = original * g / (2.0 * math.pi)
            w = min(1.0, max(0.0, (turns - turns_lo) / (turns_hi - turns_lo)))
            g = (1.0 - w) * g / factor + w * g
        out.append(g)
    return np.array(out, dtype=np.float64)


def rope(x, positions, freq, layout="half", span=None, magnitude=1.0, inverse=False):
    """x [rows, heads, dim] turned at positions [rows]; rows at negative positions are returned as they are."""
    x = np.array(x, dtype=np.float64)
    span = x.shape[-1] if span is None else span
    for t in range(x.shape[0]):
        if positions[t] < 0:
            continue
        for j, f in enumerate(freq):
            a, b = (j, j + span // 2) if layout == "half" else (2 * j, 2 * j + 1)
            ang = float(positions[t]) * f
            c, s = magnitude * math.cos(ang), magnitude * math.sin(ang)
            if inverse:
                s = -s
            x0, x1 = x[t, :, a].copy(), x[t, :, b].copy()
            x[t, :, a], x[t, :, b] = x0 * c - x1 * s, x0 * s + x1 * c
    return x


def e4m3_values():
    """Value of each of the 256 codes (NaN for the two NaN codes)."""
    v = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        mag = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            mag = math.nan
        v[code] = -mag if code & 128 else mag
    return v


VALUES = e4m3_values()


def e4m3_codes(x):
    """Code of the nearest value, ties to the even code, 448 at most; NaN as 0."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    pos = VALUES[:127]
    hi = np.minimum(np.searchsorted(pos, a), 126)
    lo = np.maximum(hi - 1, 0)
    up, down = pos[hi] - a, a - pos[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (pick | np.where(np.signbit(x) & ~np.isnan(x), 128, 0)).astype(np.uint8)


def block_scale(x):
    """Least power of two with every finite |x| <= 448 of it, within the scales' range."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    a = a[np.isfinite(a)]
    top = a.max() if a.size else 0.0
    e = MIN_EXP
    while e < MAX_EXP and 448.0 * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


def append(codes, scales, block, table_row, L, rows):
    """Stores rows [n, H, D] (float64, turned) at positions L.. in place.

    codes [P, H, PAGE, D] uint8, scales [P, H, PAGE // block] float32."""
    n, H, _ = rows.shape
    pos = L
    while pos < L + n:
        first = pos // block * block
        end = min(first + block, L + n)
        page, slot = int(table_row[first // PAGE]), first % PAGE
        for h in range(H):
            new = rows[pos - L:end - L, h]
            scale = block_scale(new)
            if pos > first:
                was = float(scales[page, h, slot // block])
                scale = max(scale, was)
                if scale > was:
                    held = slice(slot, slot + pos - first)
                    codes[page, h, held] = e4m3_codes(VALUES[codes[page, h, held]] * (was / scale))
            codes[page, h, slot + pos - first:slot + end - first] = e4m3_codes(new / scale)
            scales[page, h, slot // block] = scale
        pos = end


def attention(q, k_codes, k_scales, v_codes, v_scales, block, table_row, L, q_offset, kv_extra, window,
              scale=None):
    """q [n, Hq, D] (float64, turned) at positions L + q_offset + i.

    Returns (out [n, Hq, D], spread, mass, tail, of the same shape): the result, and
    what bounds the effect of small errors of the weights and scores: spread =
    sum_j p_j e_j |v_j - out|, mass = sum_j p_j |v_j|, tail = keys * max_j p_j *
    max |v|, with e_j = scale * sum_d |q_d k_jd| the size of the products in score j."""
    n, Hq, D = q.shape
    H = k_codes.shape[1]
    G = Hq // H
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out, spread, mass, tail = (np.zeros((n, Hq, D)) for _ in range(4))
    for i in range(n):
        p = L + q_offset + i
        hi = min(p, L + kv_extra - 1)
        lo = max(0, p - window + 1) if window > 0 else 0
        j = np.arange(lo, hi + 1)
        pages = np.asarray(table_row)[j // PAGE] if j.size else np.zeros(0, dtype=int)
        ok = (pages >= 0) & (pages < k_codes.shape[0])
        j, pages = j[ok], pages[ok]
        if j.size == 0:
            continue
        slot = j % PAGE
        for h in range(H):
            k = VALUES[k_codes[pages, h, slot]] * k_scales[pages, h, slot // block, None].astype(np.float64)
            v = VALUES[v_codes[pages, h, slot]] * v_scales[pages, h, slot // block, None].astype(np.float64)
            for g in range(G):
                x = q[i, h * G + g]
                s = scale * (k @ x)
                w = np.exp(s - s.max())
                w /= w.sum()
                o = w @ v
                e = scale * (np.abs(k) @ np.abs(x))
                out[i, h * G + g] = o
                spread[i, h * G + g] = (w * e) @ np.abs(v - o)
                mass[i, h * G + g] = w @ np.abs(v)
                tail[i, h * G + g] = j.size * w.max() * np.abs(v).max()
    return out, spread, mass, tail
