"""Plain float64 forms of the cache operators on the CPU -- test infrastructure only.

Definitions (include/gqa_decode.h, "filling a cache; the 8-bit cache"), element by element:

* a head's row after the norm: ``x_i * (mean(x^2) + eps)^(-1/2) * w_i``; after the rotation of its pairs
  ``(a, b)``: ``(a cos - b sin, b cos + a sin)``, pairs ``(i, i + rot/2)`` or ``(2i, 2i + 1)``;
* a row ``x`` in 8 bits: the codes ``e4m3(x * 2^-k)``, nearest even, ``k`` the smallest integer with
  ``max|x| <= 448 * 2^k`` (at least -126), and the exponent byte ``k + 127``;
* the bytes of a (block, head): K codes, V codes, K exponents, V exponents; the 16-byte chunk ``c`` of row
  ``r`` at chunk ``c ^ (r % 8)`` (d_head 128) or ``c ^ (r // 2 % 4)`` (d_head 64).

Codes are found by searching the table of their values, offsets by plain integer arithmetic on one row at a
time; nothing here is shared with the library or with the benchmark's plain forms.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np
import torch

from .gqa_oracle import partial_rows, normalize

__all__ = ["code_values", "encode", "exponent", "head_rows", "row_offsets", "put_row", "get_row", "gather_kv8",
           "decode_kv8"]


def code_values() -> np.ndarray:
    """Value of each e4m3 byte: 1 sign, 4 exponent (bias 7), 3 fraction bits; 0x7f and 0xff are NaN."""
    out = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out.append(math.nan if c & 127 == 127 else (-v if c & 128 else v))
    return np.array(out)


_VALUES = code_values()
_POSITIVE = _VALUES[:127]            # ascending
_MIDDLES = (_POSITIVE[1:] + _POSITIVE[:-1]) / 2


def encode(x) -> np.ndarray:
    """e4m3 bytes of float64 values: nearest, ties to the even code, beyond 448 saturated, NaN kept."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    lo = np.searchsorted(_MIDDLES, a, side="left")     # ties stay below
    tie = (lo < 126) & (a == _MIDDLES[np.minimum(lo, 125)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo).astype(np.uint8)
    code = np.where(np.isnan(x), 127, code).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7)


def exponent(top: float) -> int:
    """Exponent byte of a row whose largest magnitude is ``top``."""
    if math.isinf(top):
        return 247
    k = -126
    while Fraction(top) > Fraction(448) * Fraction(2) ** k:
        k += 1
    return k + 127


def head_rows(x, heads: int, weight, eps: float, cos_sin, positions, interleaved: bool) -> np.ndarray:
    """Norm and rotation of ``x (T, heads*D)``; float64 ``(T, heads, D)``."""
    x = np.asarray(x, dtype=np.float64)
    y = x.reshape(x.shape[0], heads, -1).copy()
    if weight is not None:
        y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    if cos_sin is None:
        return y
    half = cos_sin.shape[1] // 2
    out = y.copy()
    for t, p in enumerate(positions):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = float(cos_sin[p, i]), float(cos_sin[p, half + i])
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
    return out


def row_offsets(row: int, D: int, bs: int, which: int) -> np.ndarray:
    """Byte offsets of the D codes of a row; which: 0 K, 1 V."""
    turn = row % 8 if D == 128 else row // 2 % 4
    return np.array([which * bs * D + row * D + ((i // 16) ^ turn) * 16 + i % 16 for i in range(D)])


def put_row(cache, slot: int, head: int, which: int, x, D: int, bs: int) -> None:
    """Store one float64 row in ``cache`` (numpy uint8 (num_blocks, h_kv, bytes))."""
    x = np.asarray(x, dtype=np.float64)
    finite = x[~np.isnan(x)]
    e = exponent(float(np.abs(finite).max()) if finite.size else 0.0)
    blk, row = divmod(int(slot), bs)
    cache[blk, head, row_offsets(row, D, bs, which)] = encode(x * 2.0 ** (127 - e))
    cache[blk, head, 2 * bs * D + which * bs + row] = e


def get_row(cache, slot: int, head: int, which: int, D: int, bs: int) -> np.ndarray:
    blk, row = divmod(int(slot), bs)
    e = int(cache[blk, head, 2 * bs * D + which * bs + row])
    return _VALUES[cache[blk, head, row_offsets(row, D, bs, which)]] * 2.0 ** (e - 127)


def gather_kv8(cache, table, n: int, D: int, bs: int):
    """K and V ``(n, h_kv, D)`` float64 of one sequence."""
    hk = cache.shape[1]
    out = np.empty((2, n, hk, D))
    rows = {(r, w): row_offsets(r, D, bs, w) for r in range(min(bs, n)) for w in (0, 1)}
    for w in (0, 1):
        for r in range(min(bs, n)):
            at = np.arange(r, n, bs)
            blk = cache[np.asarray(table)[at // bs]]
            e = blk[:, :, 2 * bs * D + w * bs + r].astype(np.int64)
            out[w, at] = _VALUES[blk[:, :, rows[r, w]]] * (2.0 ** (e - 127.0))[..., None]
    return out[0], out[1]


def decode_kv8(q, cache, tables, lens, h_q: int, h_kv: int, D: int, scale: float, bs: int, causal: bool = False):
    """``(O, A, l, top)``: the output ``(N, T_q, h_q*D)``, the same softmax weights on |V|, the softmax sums
    relative to the largest score ``(N, T_q, h_q)`` and the largest |V| of each sequence."""
    q = torch.as_tensor(np.asarray(q, dtype=np.float64))
    N, T, _ = q.shape
    o, a = torch.zeros(N, T, h_q, D, dtype=torch.float64), torch.zeros(N, T, h_q, D, dtype=torch.float64)
    ls, top = torch.zeros(N, T, h_q, dtype=torch.float64), torch.zeros(N, dtype=torch.float64)
    q = q.reshape(N, T, h_q, D)
    for b in range(N):
        n = int(lens[b])
        if n <= 0:
            continue
        k, v = (torch.from_numpy(x) for x in gather_kv8(cache, tables[b], n, D, bs))
        top[b] = v.abs().max()
        G = h_q // h_kv
        for t in range(T):
            end = n - T + t + 1 if causal else n
            if end <= 0:
                continue
            for g in range(h_kv):
                hs = slice(g * G, (g + 1) * G)
                _, l, acc = partial_rows(q[b, t, hs], k[:end, g], v[:end, g], scale)
                o[b, t, hs] = normalize(l, acc)
                a[b, t, hs] = normalize(l, partial_rows(q[b, t, hs], k[:end, g], v[:end, g].abs(), scale)[2])
                ls[b, t, hs] = l
    return o.reshape(N, T, -1), a.reshape(N, T, -1), ls, top
