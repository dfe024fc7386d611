"""Plain 64-bit oracle of kvo_append_tokens, kvo_index_scores and kvo_attend.

numpy only, one token, query or row at a time, from the definitions in
include/kvo.h.  Shares no code with the library.
"""
from __future__ import annotations

import math

import numpy as np

ROW, LATENT, ROPE, KEY, GROUP = 656, 512, 64, 128, 64


# ------------------------------------------------------------ number formats
def bf16_bits(x) -> np.ndarray:
    """float64 -> bf16 bits, one rounding to nearest even (through an exact split, not through float32)."""
    x = np.asarray(x, np.float64)
    out = np.empty(x.shape, np.uint16)
    flat, o = x.ravel(), out.ravel()
    for i, v in enumerate(flat):
        sign = 0x8000 if math.copysign(1.0, v) < 0 else 0
        a = abs(v)
        if math.isnan(a):
            o[i] = 0x7FC0
        elif a == 0:
            o[i] = sign
        elif math.isinf(a):
            o[i] = sign | 0x7F80
        else:
            e = max(math.frexp(a)[1] - 1, -126)
            m = int(np.rint(a / 2.0 ** (e - 7)))     # 8 significant bits; a / 2^k is exact
            if m == 256:
                m, e = 128, e + 1
            bits = 0x7F80 if e > 127 else m if m < 128 else ((e + 127) << 7) + (m - 128)
            o[i] = sign | bits
    return out


def bf16_value(bits) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_value(bits) -> np.ndarray:
    b = np.asarray(bits, np.uint8).astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((b & 127) == 127, np.nan, v)
    return np.where(b & 128, -v, v)


_E4M3 = e4m3_value(np.arange(127))                   # ascending positive values


def e4m3_bits(x: float) -> int:
    """Round to the nearest e4m3, ties to the even significand, saturating."""
    a = min(abs(x), 448.0)
    hi = int(np.searchsorted(_E4M3, a))
    if hi and (hi > 126 or _E4M3[hi] != a):
        lo = hi - 1
        d = (a - _E4M3[lo]) - (_E4M3[hi] - a)
        hi = lo if d < 0 or (d == 0 and lo % 2 == 0) else hi
    return hi | (128 if math.copysign(1.0, x) < 0 else 0)


# -------------------------------------------------------------------- append
_FP16 = np.arange(0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64)   # ascending, finite


def latent_group(x):
    """(int8[64], fp16 scale bits) of one group of 64 finite values."""
    x = np.asarray(x, np.float64)
    if not np.isfinite(x).all():
        return np.zeros(GROUP, np.int8), 0x7E00
    bits = min(int(np.searchsorted(127.0 * _FP16, np.abs(x).max())), 0x7BFF)
    s = _FP16[bits]
    if s == 0:
        return np.zeros(GROUP, np.int8), 0
    return np.clip(np.rint(x / s), -127, 127).astype(np.int8), bits


def rotate(rope, pos: int, inv_freq, interleaved: bool) -> np.ndarray:
    """The 64 rotated values in 64 bits (the angle reduced exactly)."""
    from fractions import Fraction
    two_pi = Fraction(2) * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    x = np.asarray(rope, np.float64)
    out = np.empty(ROPE)
    for i in range(ROPE // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + ROPE // 2)
        turn = Fraction(float(inv_freq[i])) * pos / two_pi
        angle = float((turn - math.floor(turn)) * two_pi)
        c, s = math.cos(angle), math.sin(angle)
        out[a], out[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
    return out


def key_e4m3(key):
    """(uint8[128], float factor) of one key."""
    k = np.asarray(key, np.float64)
    if not np.isfinite(k).all():
        return np.zeros(KEY, np.uint8), math.nan
    e = -100
    while 448.0 * 2.0 ** e < np.abs(k).max():
        e += 1
    return np.array([e4m3_bits(v / 2.0 ** e) for v in k], np.uint8), 2.0 ** e


# --------------------------------------------------------------- cache rows
def row_of(table, blocks, block_rows, sequences, s, p):
    """Row number of position p of sequence s, or None where there is none."""
    b, r = divmod(p, block_rows)
    if table is None:
        return s * block_rows + r if b == 0 and s < sequences else None
    if b >= table.shape[1]:
        return None
    i = int(table[s, b])
    return i * block_rows + r if 0 <= i < blocks else None


def row_values(row) -> tuple:
    """(latent[512], rope[64]): the bf16 values a 656-byte row stands for, in 64 bits."""
    row = np.ascontiguousarray(row, np.uint8)
    q = row[:LATENT].view(np.int8).astype(np.float64)
    s = row[LATENT:LATENT + 16].view(np.float16).astype(np.float64)
    with np.errstate(invalid="ignore"):
        product = (q.reshape(8, GROUP) * s[:, None]).ravel()
    latent = np.empty(LATENT)
    fin = np.isfinite(product)
    latent[~fin] = product[~fin]
    # int8 * fp16 has 19 significant bits: float32 holds it, and rounds to bf16 once
    f = product[fin].astype(np.float32).view(np.uint32).astype(np.uint64)
    f = (f + 0x7FFF + ((f >> 16) & 1)) >> 16
    latent[fin] = bf16_value(f.astype(np.uint16))
    return latent, bf16_value(row[LATENT + 16:].view(np.uint16))


# -------------------------------------------------------------------- score
def index_scores(q, w, keys, factors, rows, lens, block):
    """q [nq, H, 128], w [nq, H], keys [*, 128], factors [*] in 64 bits;
    rows[t][j] = the key of query t's position j or None; returns (scores,
    bound): bound is sum_h |w_h| sum_d |q_d k_d| of the same entries."""
    nq = len(lens)
    n = max(len(r) for r in rows)
    score, size = np.full((nq, n), -np.inf), np.zeros((nq, n))
    for t in range(nq):
        for j in range(min(n, max(0, lens[t]))):
            r = rows[t][j]
            if r is None:
                continue
            with np.errstate(invalid="ignore"):
                dots = q[t] @ keys[r]
                score[t, j] = factors[r] * (w[t] * np.where(dots < 0, 0.0, dots)).sum()
            size[t, j] = abs(factors[r]) * (np.abs(w[t]) * (np.abs(q[t]) @ np.abs(keys[r]))).sum()
    if block == 1:
        return score, size
    cols = -(-n // block)
    out, mag = np.full((nq, cols), -np.inf), np.zeros((nq, cols))
    for b in range(cols):
        part = score[:, b * block:(b + 1) * block]
        out[:, b] = np.where(np.isnan(part), -np.inf, part).max(1)
        mag[:, b] = np.nan_to_num(size[:, b * block:(b + 1) * block]).max(1)
    return out, mag


# ------------------------------------------------------------------- attend
def positions_of(sel, sel_block, length, rows):
    """The visible positions of one query, in list order."""
    if sel is None:
        return list(range(max(0, min(length, rows))))
    out = []
    for u in sel:
        if u >= 0:
            out += [p for p in range(int(u) * sel_block, (int(u) + 1) * sel_block) if p < length]
    return out


def attend(q, scale, rows):
    """q [H, 576] against a list of 656-byte rows: (out [H, 512], lse [H],
    spread [H, 512] = sum p |v|, size [H] = max_j scale * sum |q k|)."""
    heads = q.shape[0]
    if not rows:
        return (np.zeros((heads, LATENT)), np.full(heads, -np.inf), np.zeros((heads, LATENT)), np.zeros(heads))
    vals = [row_values(r) for r in rows]
    lat = np.stack([v[0] for v in vals])
    key = np.concatenate([lat, np.stack([v[1] for v in vals])], 1)
    z = scale * (q @ key.T)
    top = z.max(1, keepdims=True)
    p = np.exp(z - top)
    total = p.sum(1, keepdims=True)
    p /= total
    size = abs(scale) * (np.abs(q) @ np.abs(key).T).max(1)
    return p @ lat, (np.log(total) + top)[:, 0], p @ np.abs(lat), size
