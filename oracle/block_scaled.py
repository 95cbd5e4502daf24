"""Plain CPU statement of the FP8 cache with block scales and of rotary positions (numpy, float64).

TEST INFRASTRUCTURE ONLY, like the rest of this package: it shares no code with the CUDA library.
The writer follows the header's definition step by step, a block at a time; the quotients and products named
there are float32 operations (numpy's are IEEE), the rounding to E4M3 is a search for the nearest value,
ties to the even code.  Attention is float64 over exactly the tokens a row sees.  Angles of rotary positions
are reduced in exact rationals.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from .fp4 import E4M3, nearest_code

MIN_EXP, MAX_EXP = -60, 120
# 1 / 2 pi to 2^-160
INV_2PI = 1 / (2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459"))


def scale_ok(s):
    s = np.asarray(s)
    with np.errstate(all="ignore"):
        return np.isfinite(s) & (s >= 2.0 ** MIN_EXP) & (s <= 2.0 ** MAX_EXP) & (np.frexp(s)[0] == 0.5)


def power_for(a: float) -> float:
    """The smallest power of two, 2^-60 at least, with 448 times it not below a."""
    k = MIN_EXP
    while 448.0 * 2.0 ** k < a:
        k += 1
    return 2.0 ** k


def decode(codes: np.ndarray) -> np.ndarray:
    """uint8 -> float64 (0x7F and 0xFF NaN)."""
    v = np.append(E4M3, np.nan)[codes & 0x7F]
    return np.where(codes >= 0x80, -v, v)


def encode(y: np.ndarray) -> np.ndarray:
    """float32 -> codes: to nearest even, saturating, NaN to sign | 0x7F."""
    y = np.asarray(y, np.float32)
    with np.errstate(all="ignore"):
        mag = np.minimum(np.where(np.isnan(y), 0.0, np.abs(y.astype(np.float64))), 448.0)
    code = np.where(np.isnan(y), 0x7F, nearest_code(mag, E4M3))
    return (code | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def write(x: np.ndarray, codes: np.ndarray, scales: np.ndarray, slots: np.ndarray):
    """Rows x (float32 [n, n_kv, hd]) into codes [nb, bs, n_kv, hd] and scales [nb, stride]; returns (a slot was out
    of range, an old scale that counts was not valid).  No slot twice."""
    nb, bs, n_kv, _ = codes.shape
    ok = (slots >= 0) & (slots < nb * bs)
    bad_scale = False
    rows_of = {}
    for i in np.nonzero(ok)[0]:
        rows_of.setdefault(int(slots[i]) // bs, []).append(int(i))
    with np.errstate(all="ignore"):
        for b, rows in rows_of.items():
            off = slots[rows] % bs
            others = np.setdiff1d(np.arange(bs), off)
            for h in range(n_kv):
                r = np.asarray(x[rows, h], np.float32)
                mag = np.abs(r)
                a = float(mag[np.isfinite(mag)].max(initial=0.0))
                old = np.float32(0) if (off == 0).any() else scales[b, h]
                if old != 0 and not scale_ok(old):
                    bad_scale = True
                    continue
                s = max(old, np.float32(power_for(a)))
                if s > old and old > 0:
                    c = codes[b, others, h]
                    up = encode(decode(c).astype(np.float32) * (old / s))
                    codes[b, others, h] = np.where((c & 0x7F) == 0x7F, c, up)
                scales[b, h] = s
                y = r / s
                y = np.where(np.isnan(r), np.copysign(np.float32(np.nan), r), y)
                codes[b, off, h] = encode(y)
    return bool(np.any(~ok & (slots != -1))), bad_scale


def dequant(codes: np.ndarray, scales: np.ndarray, slots: np.ndarray):
    """float32 rows dec(code) * scale; slots out of range and scales that are not valid give zeros."""
    nb, bs, n_kv, _ = codes.shape
    ok = (slots >= 0) & (slots < nb * bs)
    at = np.where(ok, slots, 0)
    s = scales[at // bs, :n_kv]
    with np.errstate(all="ignore"):
        out = decode(codes[at // bs, at % bs]).astype(np.float32) * s[..., None]
    return np.where((ok[:, None] & scale_ok(s))[..., None], out, np.float32(0))


def attention(q: np.ndarray, qsl: np.ndarray, kc, vc, ks, vs, block_tables, seq_lens, causal=True, sm_scale=0.0):
    """(out, weight, reach), float64: attention of each sequence's queries (its last tokens when causal, else queries
    that see all of it); weight = sum_t p_t |v_t| / sum_t p_t, reach [rows, n_q] = the largest sm |q| . |k_t|,
    the sizes that rounding errors go by.  A token in a block outside the pool or without valid scales is
    not there.  Rows that see nothing are zero."""
    n_q, hd = q.shape[1:]
    nb, bs, n_kv, _ = kc.shape
    group = n_q // n_kv
    sm = sm_scale if sm_scale > 0 else 1.0 / np.sqrt(hd)
    out, weight, reach = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
    for i, length in enumerate(np.asarray(seq_lens).tolist()):
        r0, n = int(qsl[i]), int(qsl[i + 1] - qsl[i])
        if n == 0 or length <= 0:
            continue
        t = np.arange(length)
        blk = block_tables[i, t // bs]
        there = (blk >= 0) & (blk < nb)
        for h in range(n_kv):
            kscale = np.where(there, ks[np.where(there, blk, 0), h], np.nan).astype(np.float64)
            vscale = np.where(there, vs[np.where(there, blk, 0), h], np.nan).astype(np.float64)
            with np.errstate(all="ignore"):
                good = there & scale_ok(kscale) & scale_ok(vscale)
            th = t[good]
            kr = decode(kc[blk[good], th % bs, h]) * kscale[good, None]
            vr = decode(vc[blk[good], th % bs, h]) * vscale[good, None]
            for j in range(n):
                sees = th <= length - n + j if causal else np.ones(len(th), bool)
                if not sees.any():
                    continue
                heads = slice(h * group, (h + 1) * group)
                x = sm * (q[r0 + j, heads] @ kr[sees].T)
                p = np.exp(x - x.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                out[r0 + j, heads] = p @ vr[sees]
                weight[r0 + j, heads] = p @ np.abs(vr[sees])
                reach[r0 + j, heads] = sm * (np.abs(q[r0 + j, heads]) @ np.abs(kr[sees]).T).max(-1)
    return out, weight, reach


def angle(position: int, frequency: float) -> float:
    """position * frequency reduced to [0, 2 pi)."""
    turns = int(position) * Fraction(float(frequency)) * INV_2PI
    return 2 * math.pi * float(turns - math.floor(turns))


def rotary(x: np.ndarray, positions, frequencies, interleaved=False, magnitude=1.0, transpose=False):
    """float64 [n, heads, hd]: the pairs of the first 2 len(frequencies) dims turned by their angles."""
    half = len(frequencies)
    t = np.array([[angle(p, f) for f in frequencies] for p in positions]).reshape(len(positions), 1, half)
    c, s = magnitude * np.cos(t), magnitude * np.sin(t) * (-1 if transpose else 1)
    x = np.asarray(x, np.float64)
    out = x.copy()
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = x[..., first], x[..., second]
    out[..., first], out[..., second] = a * c - b * s, a * s + b * c
    return out
