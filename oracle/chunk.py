"""New tokens of a batch over a paged cache, float64, by definition: the append (norm,
rotary positions, the write into the pages, 8-bit quantisation) and causal attention of
packed chunks.

Rows are packed: sequence b owns rows offsets[b] .. offsets[b+1]-1 of q / k / v, the i-th
of them at logical position S_b + i.  Logical token t lives in physical page
page_table[b][t // 16], slot t % 16.  An 8-bit pool holds e4m3 codes [P][16][Hkv][D] and
scales [P][Hkv][16]; an element stands for code * scale.
"""
from __future__ import annotations

import math

import numpy as np

PS = 16
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -100
# 1 / (2 pi) as an integer times 2^-200, from 2 pi to 70 decimal places
_TWO_PI = 62831853071795864769252867665590057683943387987502116419498891846156328  # x 10^-70
_INV_TWO_PI_200 = (10 ** 70 << 200) // _TWO_PI


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits, no
    infinities, 0x7f and 0xff NaN."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = math.nan
        out[c] = -v if c & 128 else v
    return out


def to_e4m3(x) -> np.ndarray:
    """Codes of |x| <= 448 rounded to nearest, ties to the even code; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    mag = e4m3_values()[:127]                      # increasing
    a = np.abs(x)
    hi = np.searchsorted(mag, a).clip(0, 126)
    lo = (hi - 1).clip(0)
    below, above = a - mag[lo], mag[hi] - a
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == mag[hi], hi, code)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantise(x):
    """Codes and scales of rows [..., D]: scale = max |x| / 448, at least 2^-100."""
    x = np.asarray(x, dtype=np.float64)
    big = np.abs(x).max(-1)
    scale = np.where(big / E4M3_MAX < SCALE_MIN, SCALE_MIN, big / E4M3_MAX)
    with np.errstate(invalid="ignore"):
        return to_e4m3(x / scale[..., None]), scale


def angle(position: int, inv_freq: float) -> float:
    """position * inv_freq modulo a turn, in radians, from whole-number arithmetic."""
    m, e = math.frexp(float(inv_freq))
    whole, exp = int(m * 2 ** 53), e - 53          # inv_freq = whole * 2^exp
    turns = int(position) * whole * _INV_TWO_PI_200   # x 2^(exp - 200)
    shift = 200 - exp
    return (turns & ((1 << shift) - 1)) / (1 << shift) * 2 * math.pi


def norm(x, weight, eps: float) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def rotate(x, position: int, inv_freq, interleaved: bool, rope_scale: float = 1.0) -> np.ndarray:
    """Heads [H][D] of one token."""
    x = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        w = angle(position, inv_freq[j])
        c, s = math.cos(w) * rope_scale, math.sin(w) * rope_scale
        x[:, a], x[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
    return x


def append(q, k, v, page_table, prefix_lens, offsets, num_pages: int, *, positions=None, q_norm=None, k_norm=None,
           eps: float = 1e-6, inv_freq=(), interleaved: bool = False, rope_scale: float = 1.0):
    """What the append writes: {row: q heads}, {(page, slot): (k heads, v heads)} in float64.

    Rows of no sequence, rows with a negative position, rows whose slot lies outside the
    page table and rows whose page lies outside the pool are in neither."""
    q_rows, slots = {}, {}
    for b in range(len(prefix_lens)):
        o0, o1 = int(offsets[b]), int(offsets[b + 1])
        S = int(prefix_lens[b])
        if not 0 <= o0 <= o1 <= len(q):
            continue
        for t in range(o0, o1):
            at = S + t - o0
            pos = at if positions is None else int(positions[t])
            if pos < 0 or S < 0 or at >= page_table.shape[1] * PS:
                continue
            page = int(page_table[b, at // PS])
            if not 0 <= page < num_pages:
                continue
            qt, kt = np.asarray(q[t], dtype=np.float64), np.asarray(k[t], dtype=np.float64)
            if q_norm is not None:
                qt = norm(qt, q_norm, eps)
            if k_norm is not None:
                kt = norm(kt, k_norm, eps)
            q_rows[t] = rotate(qt, pos, inv_freq, interleaved, rope_scale)
            slots[(page, at % PS)] = (rotate(kt, pos, inv_freq, interleaved, rope_scale),
                                      np.asarray(v[t], dtype=np.float64))
    return q_rows, slots


def attend(q, K, V, seen):
    """q [H][D] of one token, K / V [L][Hkv][D], seen [L] -> (out [H][D], spread [H][D],
    reach [H]): the attention, sum_t w_t |V_t| and the largest sum_d |q_d K_td| / sqrt(D) of
    the tokens that the row sees (what rounding errors of its terms scale with)."""
    H, D = q.shape
    G = H // K.shape[1]
    out, spread, reach = np.empty((H, D)), np.empty((H, D)), np.empty(H)
    for h in range(H):
        k, v = K[seen, h // G], V[seen, h // G]
        s = k @ q[h] / math.sqrt(D)
        with np.errstate(invalid="ignore"):
            w = np.exp(s - s.max())
            w = w / w.sum()
            out[h], spread[h] = w @ v, w @ np.abs(v)
        reach[h] = (np.abs(k) @ np.abs(q[h])).max() / math.sqrt(D)
    return out, spread, reach


def chunk_attention(q, k_pages, v_pages, page_table, prefix_lens, offsets):
    """Causal attention of packed rows q [T][Hq][D] over float64 pools [P][16][Hkv][D].
    Returns (out, spread, reach) of attend for every row, NaN where a row has none."""
    T, H, D = q.shape
    out, spread, reach = np.full((T, H, D), np.nan), np.full((T, H, D), np.nan), np.full((T, H), np.nan)
    for b in range(len(prefix_lens)):
        o0, o1, S = int(offsets[b]), int(offsets[b + 1]), int(prefix_lens[b])
        if not 0 <= o0 <= o1 <= T:
            continue
        if S < 0 or S + o1 - o0 > page_table.shape[1] * PS:
            out[o0:o1] = spread[o0:o1] = reach[o0:o1] = 0
            continue
        t = np.arange(S + o1 - o0)
        pages = np.asarray(page_table[b])[t // PS]
        K, V = k_pages[pages, t % PS], v_pages[pages, t % PS]
        for i in range(o1 - o0):
            out[o0 + i], spread[o0 + i], reach[o0 + i] = attend(q[o0 + i], K, V, t <= S + i)
    return out, spread, reach


def dequantise(codes, scales) -> np.ndarray:
    """Codes [P][16][Hkv][D] (uint8) and scales [P][Hkv][16] -> float64 pool."""
    return e4m3_values()[codes] * np.asarray(scales, dtype=np.float64).transpose(0, 2, 1)[..., None]
