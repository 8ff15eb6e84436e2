"""Plain float64 forms of the 4-bit cache and of attention with a window on the CPU -- test infrastructure only.

Definitions (include/gqa_decode.h, "several position axes; the 4-bit cache; windows"), element by element:

* sixteen elements with the largest magnitude ``m``: the scale ``min(m / 6, 10240)`` rounded to the nearest number whose
  binary16 form has a lower byte of 0 (ties to the even upper byte), and the codes of ``x / scale``, the nearest of
  0, 0.5, 1, 1.5, 2, 3, 4, 6 with its sign (ties to the even code); with a NaN or an infinity: the scale byte 0x7f;
* the bytes of a (block, head): K codes, V codes (two in a byte, the even element in the low four bits), K scales, V
  scales; the 16-byte chunk ``c`` of row ``r`` of the codes at chunk ``c ^ (r // 2 % 4)`` (d_head 128) or
  ``c ^ (r // 4 % 2)`` (d_head 64);
* a token at place ``p`` sees the keys ``j <= p`` with ``j > p - window`` or ``j < sinks``.

Scales and codes are found by comparing with every number there is; nothing here is shared with the library or with the
benchmark's plain forms.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np
import torch

from .gqa_oracle import normalize, partial_rows

__all__ = ["MAGNITUDES", "scale_value", "scale_byte", "encode", "put_row", "get_row", "gather_kv4", "sees", "decode_window",
           "turn_rows"]

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def scale_value(byte: int) -> float:
    """The binary16 number with this upper byte and a lower byte of 0."""
    e, f = byte >> 2 & 31, byte & 3
    if e == 31:
        return math.nan if f else math.inf
    return math.ldexp(f, -16) if e == 0 else math.ldexp(4 + f, e - 17)


_SCALES = [Fraction(scale_value(b)) for b in range(0x7c)]


def scale_byte(top: float) -> int:
    if not math.isfinite(top):
        return 0x7f
    want = min(Fraction(top) / 6, Fraction(10240))
    return min(range(len(_SCALES)), key=lambda b: (abs(_SCALES[b] - want), b & 1))


def encode(x: float, scale: float) -> int:
    """Code of one finite element."""
    sign = 8 if math.copysign(1.0, x) < 0 else 0
    if scale == 0:
        return sign
    z = abs(Fraction(x)) / Fraction(scale)
    return sign + min(range(8), key=lambda c: (abs(Fraction(MAGNITUDES[c]) - z), c & 1))


def _chunk(row: int, c: int, D: int) -> int:
    return c ^ (row // 2 % 4 if D == 128 else row // 4 % 2)


def code_offset(row: int, e: int, D: int, bs: int, which: int) -> int:
    """Byte offset of element e's code; which: 0 K, 1 V."""
    byte = e // 2
    return which * bs * (D // 2) + row * (D // 2) + _chunk(row, byte // 16, D) * 16 + byte % 16


def scale_offset(row: int, e: int, D: int, bs: int, which: int) -> int:
    return bs * D + which * bs * (D // 16) + row * (D // 16) + e // 16


def row_offsets(row: int, D: int, bs: int, which: int) -> list:
    """Every byte of a row."""
    return sorted({code_offset(row, e, D, bs, which) for e in range(D)} | {scale_offset(row, e, D, bs, which) for e in range(D)})


def put_row(cache, slot: int, head: int, which: int, x, D: int, bs: int) -> None:
    """Store one float64 row in ``cache`` (numpy uint8 (num_blocks, h_kv, bytes))."""
    blk, row = divmod(int(slot), bs)
    for g in range(0, D, 16):
        part = [float(v) for v in x[g:g + 16]]
        b = scale_byte(max(abs(v) for v in part) if all(math.isfinite(v) for v in part) else math.nan)
        cache[blk, head, scale_offset(row, g, D, bs, which)] = b
        for i in range(0, 16, 2):
            codes = [encode(v, scale_value(b)) if b != 0x7f else (8 if math.copysign(1.0, v) < 0 else 0) for v in part[i:i + 2]]
            cache[blk, head, code_offset(row, g + i, D, bs, which)] = codes[0] + 16 * codes[1]


def get_row(cache, slot: int, head: int, which: int, D: int, bs: int) -> np.ndarray:
    blk, row = divmod(int(slot), bs)
    out = np.empty(D)
    for e in range(D):
        c = int(cache[blk, head, code_offset(row, e, D, bs, which)]) >> (4 * (e % 2)) & 15
        s = int(cache[blk, head, scale_offset(row, e, D, bs, which)])
        out[e] = math.nan if s >= 0x7c else (-1 if c & 8 else 1) * MAGNITUDES[c & 7] * scale_value(s)
    return out


def gather_kv4(cache, table, n: int, D: int, bs: int):
    """K and V ``(n, h_kv, D)`` float64 of one sequence (entries of the table that are no block: zeros)."""
    hk = cache.shape[1]
    out = np.zeros((2, n, hk, D))
    mags = np.array(MAGNITUDES + tuple(-m for m in MAGNITUDES))
    scales = np.array([scale_value(b) if b < 0x7c else math.nan for b in range(256)])
    e = np.arange(D)
    for w in (0, 1):
        for r in range(min(bs, n)):
            at = np.arange(r, n, bs)
            ids = np.asarray(table)[at // bs]
            ok = (ids >= 0) & (ids < cache.shape[0])
            blk = cache[np.where(ok, ids, 0)]
            codes = blk[:, :, [code_offset(r, int(i), D, bs, w) for i in e]] >> (4 * (e % 2)).astype(np.uint8) & 15
            s = blk[:, :, [scale_offset(r, int(i), D, bs, w) for i in e]]
            out[w, at] = np.where(ok[:, None, None], mags[codes] * scales[s], 0.0)
    return out[0], out[1]


def sees(place: int, key: int, window: int, sinks: int) -> bool:
    return key <= place and (window == 0 or key > place - window or key < sinks)


def decode_window(q, kv, lens, h_q: int, h_kv: int, D: int, scale: float, causal: bool = False, window: int = 0,
                  sinks: int = 0):
    """``(O, A, l, top)`` as kv8_oracle.decode_kv8; ``kv(b, n)``: K and V ``(n, h_kv, D)`` of sequence b."""
    q = torch.as_tensor(np.asarray(q, dtype=np.float64))
    N, T, _ = q.shape
    o, a = torch.zeros(N, T, h_q, D, dtype=torch.float64), torch.zeros(N, T, h_q, D, dtype=torch.float64)
    ls, top = torch.zeros(N, T, h_q, dtype=torch.float64), torch.zeros(N, dtype=torch.float64)
    q = q.reshape(N, T, h_q, D)
    G = h_q // h_kv
    for b in range(N):
        n = int(lens[b])
        if n <= 0:
            continue
        k, v = (torch.from_numpy(np.ascontiguousarray(x)) for x in kv(b, n))
        for t in range(T):
            place = n - T + t if causal else n - 1
            keys = torch.arange(max(place + 1, 0))
            if window:
                keys = keys[(keys > place - window) | (keys < sinks)]
            if len(keys) == 0:
                continue
            for g in range(h_kv):
                hs = slice(g * G, (g + 1) * G)
                kk, vv = k[keys, g], v[keys, g]
                _, l, acc = partial_rows(q[b, t, hs], kk, vv, scale)
                o[b, t, hs] = normalize(l, acc)
                a[b, t, hs] = normalize(l, partial_rows(q[b, t, hs], kk, vv.abs(), scale)[2])
                ls[b, t, hs] = l
                top[b] = max(float(top[b]), float(vv.abs().max()))
    return o.reshape(N, T, -1), a.reshape(N, T, -1), ls, top


def turn_rows(y, cos_sin, positions, pair_axes, interleaved: bool) -> np.ndarray:
    """Rotation of ``y (T, heads, D)`` float64 by positions ``(axes, T)``: pair i by the row of its own axis."""
    out = np.array(y, dtype=np.float64)
    half = cos_sin.shape[1] // 2
    for t in range(out.shape[0]):
        for i in range(half):
            p = int(positions[int(pair_axes[i])][t])
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = float(cos_sin[p][i]), float(cos_sin[p][half + i])
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
    return out
