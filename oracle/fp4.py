"""Plain CPU statement of the 4-bit paged cache and of the page operations (numpy, float64).

TEST INFRASTRUCTURE ONLY, like the rest of this package: it shares no code with the CUDA library.
The writer follows the header's definition step by step: the quotients and the product named
there are float32 operations (numpy's are IEEE), the roundings to E4M3 and E2M1 are searches for
the nearest value, ties to the even code.  Attention is float64 over exactly the tokens a row
sees.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m * 2.0 ** -9) if e == 0 else 2.0 ** (e - 7) * (1 + m / 8)
                 for e in range(16) for m in range(8)][:127])  # code = index; 127 is NaN


def nearest_code(x: np.ndarray, values: np.ndarray) -> np.ndarray:
    """Index of the nearest of the ascending values (x >= 0, float64), halfway to the even
    index, above the last one the last."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(values, x, side="left"), 1, len(values) - 1)
    lo = hi - 1
    dl, dh = x - values[lo], values[hi] - x
    up = (dl > dh) | ((dl == dh) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def bf16_to_f32(u16: np.ndarray) -> np.ndarray:
    return (u16.astype(np.uint32) << 16).view(np.float32)


def quantize(x: np.ndarray, s: float):
    """float32 [..., hd] -> (codes uint8 [..., hd/2], scale bytes uint8 [..., hd/16])."""
    x = np.asarray(x, np.float32)
    s = np.float32(s)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    with np.errstate(all="ignore"):
        a = np.abs(g).max(-1)
        nan = np.isnan(g).any(-1)
        t = (a / np.abs(s)) / np.float32(6.0)
        assert t.dtype == np.float32
        b = nearest_code(np.minimum(np.where(nan, 0.0, t).astype(np.float64), 448.0), E4M3)
        d = E4M3[b].astype(np.float32) * np.abs(s)
        assert d.dtype == np.float32
        q = np.abs(g) / np.where(d == 0, np.float32(1), d)[..., None]
        q = np.where(d[..., None] == 0, np.float32(0), q)
        q = np.where(np.isinf(g), np.float32(6), q)
        code = nearest_code(np.minimum(np.where(np.isnan(q), 0.0, q).astype(np.float64), 6.0), E2M1)
    code = code + 8 * ((g < 0) != (s < 0))
    code = np.where(nan[..., None], 0, code).astype(np.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), np.where(nan, 0x7F, b).astype(np.uint8)


def write(x: np.ndarray, codes: np.ndarray, scales: np.ndarray, slots: np.ndarray, s: float) -> bool:
    """Rows x (float32 [n, n_kv, hd]) into codes [nb, bs, n_kv, hd/2] and scales [nb, n_kv, bs,
    hd/16]; returns whether a slot was out of range."""
    nb, bs = codes.shape[:2]
    ok = (slots >= 0) & (slots < nb * bs)
    c, b = quantize(x[ok], s)
    blk, off = slots[ok] // bs, slots[ok] % bs
    codes[blk, off] = c
    scales[blk, :, off] = b
    return bool(np.any(~ok & (slots != -1)))


def scale_values(scales: np.ndarray) -> np.ndarray:
    """E4M3 bytes -> float64 (0x7F and 0xFF NaN)."""
    v = np.append(E4M3, np.nan)[scales & 0x7F]
    return np.where(scales >= 0x80, -v, v)


def code_values(codes: np.ndarray) -> np.ndarray:
    """uint8 [..., n] -> float64 [..., 2n]"""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    return np.where(c >= 8, -E2M1[c & 7], E2M1[c & 7])


def rows(codes: np.ndarray, scales: np.ndarray, slots: np.ndarray) -> np.ndarray:
    """code * B of the rows at `slots`: float64 [n, n_kv, hd] (the layer's scalar left out)."""
    bs = codes.shape[1]
    v = code_values(codes[slots // bs, slots % bs])
    b = scale_values(scales[slots // bs, :, slots % bs])
    return (v.reshape(*b.shape, 16) * b[..., None]).reshape(v.shape)


def dequant(codes: np.ndarray, scales: np.ndarray, slots: np.ndarray, s: float) -> np.ndarray:
    """float32 rows code * (B * s), each product a float product; slots out of range give zeros."""
    nb, bs, n_kv, half = codes.shape
    ok = (slots >= 0) & (slots < nb * bs)
    at = np.where(ok, slots, 0)
    v = code_values(codes[at // bs, at % bs]).astype(np.float32)
    with np.errstate(all="ignore"):
        d = scale_values(scales[at // bs, :, at % bs]).astype(np.float32) * np.float32(s)
        out = (v.reshape(*d.shape, 16) * d[..., None]).reshape(v.shape)
    return np.where(ok[:, None, None], out, np.float32(0))


def attention(q: np.ndarray, qsl: np.ndarray, kc, vc, kg, vg, block_tables, seq_lens, ks: float,
              vs: float, sm_scale: float = 0.0):
    """Causal attention of each sequence's last n_b tokens: (out, weight), float64 [rows, n_q,
    hd]; weight is sum_t p_t |v_t| / sum_t p_t, the size that rounding errors of the weights go
    by.  A token in a block outside the pool is not there.  Rows that see nothing are zero."""
    n_q, hd = q.shape[1:]
    nb, bs, n_kv, _ = kc.shape
    group = n_q // n_kv
    sm = sm_scale if sm_scale > 0 else 1.0 / np.sqrt(hd)
    out = np.zeros(q.shape)
    weight = np.zeros(q.shape)
    for i, length in enumerate(np.asarray(seq_lens).tolist()):
        r0, n = int(qsl[i]), int(qsl[i + 1] - qsl[i])
        if n == 0 or length == 0:
            continue
        t = np.arange(length)
        blk = block_tables[i, t // bs]
        there = (blk >= 0) & (blk < nb)
        t, blk = t[there], blk[there].astype(np.int64)
        slot = blk * bs + t % bs
        kr, vr = rows(kc, kg, slot), rows(vc, vg, slot)
        for j in range(n):
            sees = t <= length - n + j
            if not sees.any():
                continue
            for h in range(n_kv):
                qh = q[r0 + j, h * group:(h + 1) * group]
                x = sm * ks * (qh @ kr[sees, h].T)
                p = np.exp(x - x.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                out[r0 + j, h * group:(h + 1) * group] = vs * (p @ vr[sees, h])
                weight[r0 + j, h * group:(h + 1) * group] = abs(vs) * (p @ np.abs(vr[sees, h]))
    return out, weight


def copy_blocks(caches, src, dst):
    """The copies in place; returns whether a pair was refused."""
    nb = caches[0].shape[0]
    bad = [not (0 <= s < nb and 0 <= d < nb) for s, d in zip(src, dst)]
    refused = any(b and s != -1 and d != -1 for b, s, d in zip(bad, src, dst))
    pairs = [(s, d) for b, s, d in zip(bad, src, dst) if not b and s != d]
    written = [d for _, d in pairs]
    old = [c.copy() for c in caches]
    for s, d in pairs:
        if written.count(d) > 1 or s in written:
            refused = True
            continue
        for c, o in zip(caches, old):
            c[d] = o[s]
    return refused


def compact(caches, block_tables, seq_lens, block_size):
    """The moves in place; returns (new tables, used blocks, whether something was flagged)."""
    nb = caches[0].shape[0]
    most = block_tables.shape[1] * block_size
    new = np.full(block_tables.shape, -1, np.int32)
    flagged = False
    live = []
    for i, length in enumerate(np.asarray(seq_lens).tolist()):
        flagged |= length < 0 or length > most
        length = min(max(length, 0), most)
        for e in range(-(-length // block_size)):
            b = int(block_tables[i, e])
            if 0 <= b < nb:
                live.append((i, e, b))
            else:
                flagged = True
    used = sorted({b for _, _, b in live})
    n = len(used)
    to = dict(zip([b for b in used if b >= n], [b for b in range(n) if b not in set(used)]))
    for c in caches:
        old = c.copy()
        for s, d in to.items():
            c[d] = old[s]
    for i, e, b in live:
        new[i, e] = to.get(b, b)
    return new, n, flagged
