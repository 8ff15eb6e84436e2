"""The 4-bit cache's oracle against its definition, and what the C entry points and the binding refuse (no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv4_oracle as k4


@pytest.fixture(scope="module")
def b():
    from decode_attention_03_gb300 import build
    build.build()
    import decode_attention_03_gb300._binding as binding
    return binding


# ---------------------------------------------------------------- the oracle
def test_scales_are_binary16_numbers_with_a_lower_byte_of_0():
    half = (np.arange(0x80, dtype=np.uint16) << 8).view(np.float16).astype(np.float64)
    for byte in range(0x80):
        v = k4.scale_value(byte)
        assert v == half[byte] or (math.isnan(v) and math.isnan(half[byte]))
    assert k4.scale_byte(0.0) == 0 and k4.scale_byte(1e300) == k4.scale_byte(61440.0) and k4.scale_value(k4.scale_byte(1e9)) == 10240
    assert k4.scale_value(k4.scale_byte(6.0)) == 1.0
    assert k4.scale_value(k4.scale_byte(6.75)) == 1.0 and k4.scale_value(k4.scale_byte(8.25)) == 1.5     # ties: the even byte
    assert k4.scale_value(k4.scale_byte(6 * 2.0 ** -17)) == 0.0 and k4.scale_value(k4.scale_byte(6.1 * 2.0 ** -17)) == 2.0 ** -16
    assert k4.scale_byte(math.inf) == k4.scale_byte(math.nan) == 0x7f


def test_codes_are_the_nearest_and_ties_are_even():
    assert [k4.encode(x, 1.0) for x in (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 100.0)] == [0, 2, 2, 4, 4, 6, 6, 7]
    assert [k4.encode(x, 1.75) for x in (-0.4375, 1.3125, -8.75)] == [8, 2, 14] and k4.encode(-0.0, 1.0) == 8
    assert k4.encode(-3.0, 0.0) == 8
    rng = np.random.default_rng(0)
    for x in rng.standard_normal(200) * 3:
        c = k4.encode(float(x), 0.875)
        v = (-1 if c & 8 else 1) * k4.MAGNITUDES[c & 7] * 0.875
        assert all(abs(v - x) <= abs(s * m * 0.875 - x) for m in k4.MAGNITUDES for s in (1, -1))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
def test_every_byte_of_a_block_has_one_place(D, bs):
    seen = []
    for w in (0, 1):
        for r in range(bs):
            codes = [k4.code_offset(r, e, D, bs, w) for e in range(D)]
            assert codes[0::2] == codes[1::2]
            seen += codes[0::2] + sorted({k4.scale_offset(r, e, D, bs, w) for e in range(D)})
    assert sorted(seen) == list(range(bs * (D + D // 8)))


def test_rows_come_back():
    rng = np.random.default_rng(1)
    for D, bs in ((64, 8), (128, 32)):
        cache = np.zeros((3, 2, bs * (D + D // 8)), dtype=np.uint8)
        rows = {}
        for slot in rng.permutation(2 * bs)[:11]:
            for h in range(2):
                for w in (0, 1):
                    x = rng.standard_normal(D) * 10.0 ** rng.integers(-3, 4)
                    k4.put_row(cache, slot, h, w, x, D, bs)
                    rows[slot, h, w] = x
        for (slot, h, w), x in rows.items():
            got = k4.get_row(cache, slot, h, w, D, bs)
            # half of the widest step, a third of the largest magnitude's 6 units, or 1/8 of it cut off by the scale's rounding
            top = np.repeat(np.abs(x).reshape(-1, 16).max(1), 16)
            assert (np.abs(got - x) <= top / 6 * 1.125 + 1e-12).all()
        k, v = k4.gather_kv4(cache, [1, 0, -1], 2 * bs + 3, D, bs)
        assert (k[2 * bs:] == 0).all()
        for (slot, h, w), x in rows.items():
            at = (slot - bs) % (2 * bs)
            np.testing.assert_array_equal((k, v)[w][at, h], k4.get_row(cache, slot, h, w, D, bs))


def test_attention_with_a_window_against_plain_softmax():
    rng = np.random.default_rng(2)
    n, hq, hk, D = 23, 4, 2, 16
    k, v = rng.standard_normal((2, n, hk, D))
    q = rng.standard_normal((1, 3, hq * D))
    for window, sinks, causal in ((0, 0, True), (5, 0, True), (5, 2, False), (1, 4, True), (50, 3, True)):
        o, a, l, top = k4.decode_window(q, lambda b, m: (k[:m], v[:m]), [n], hq, hk, D, 0.3, causal, window, sinks)
        for t in range(3):
            p = n - 3 + t if causal else n - 1
            keys = [j for j in range(n) if k4.sees(p, j, window, sinks)]
            assert p in keys and (window == 0 or len([j for j in keys if j >= sinks]) <= window)
            for h in range(hq):
                s = 0.3 * k[keys, h // 2] @ q[0, t, h * D:(h + 1) * D]
                w = np.exp(s - s.max())
                np.testing.assert_allclose(o[0, t, h * D:(h + 1) * D], w @ v[keys, h // 2] / w.sum(), atol=1e-12)
    assert (k4.decode_window(q, lambda b, m: (k[:m], v[:m]), [2], hq, hk, D, 0.3, True, 4)[0][0, 0] == 0).all()


def test_turns_by_several_axes():
    rng = np.random.default_rng(3)
    cs = np.concatenate([np.cos(rng.random((9, 4))), np.sin(rng.random((9, 4)))], 1)
    y = rng.standard_normal((2, 1, 8))
    pos, axes = [[3, 8], [0, 5]], [0, 1, 1, 0]
    for inter in (False, True):
        got = k4.turn_rows(y, cs, pos, axes, inter)
        for t in range(2):
            for i in range(4):
                a, b = (2 * i, 2 * i + 1) if inter else (i, i + 4)
                z = complex(y[t, 0, a], y[t, 0, b]) * complex(cs[pos[axes[i]][t], i], cs[pos[axes[i]][t], 4 + i])
                np.testing.assert_allclose([got[t, 0, a], got[t, 0, b]], [z.real, z.imag], atol=1e-15)


# ---------------------------------------------------------------- helpers and refusals
def _p(n=1 << 12):
    buf = ctypes.create_string_buffer(n + 64)
    return buf, (ctypes.addressof(buf) + 15) & ~15


def test_block_bytes(b):
    assert b.gqa_kv4_block_bytes(16, 128) == 16 * 144 and b.gqa_kv4_block_bytes(8, 64) == 8 * 72
    assert b.gqa_kv4_block_bytes(12, 128) == 0 and b.gqa_kv4_block_bytes(16, 96) == 0
    eight = {b.gqa_kv8_block_bytes(bs, d) for bs in (8, 16, 32, 64) for d in (64, 128)}
    for bs in (8, 16, 32, 64):
        for d in (64, 128):
            n = b.gqa_kv4_block_bytes(bs, d)
            assert n % 16 == 0 and n not in eight          # a bulk copy's size; the two caches are told apart by it
    assert b.gqa_kv4_cache(4, 16, 2, 128, device="cpu").shape == (4, 2, 16 * 144)
    with pytest.raises(b.GQAError):
        b.gqa_kv4_cache(4, 12, 2, 128, device="cpu")


def test_pair_axes(b):
    assert b.gqa_pair_axes([2, 3, 1], device="cpu").tolist() == [0, 0, 1, 1, 1, 2]
    assert b.gqa_pair_axes([4, 2, 3], in_turn=True, device="cpu").tolist() == [0, 1, 2, 0, 1, 2, 0, 2, 0]
    assert b.gqa_pair_axes([24, 20, 20], in_turn=True, device="cpu").tolist() == [0, 1, 2] * 20 + [0] * 4
    assert b.gqa_pair_axes([5], device="cpu").dtype == torch.uint8
    for bad in ([], [3, -1], [1] * 33):
        with pytest.raises(ValueError):
            b.gqa_pair_axes(bad, device="cpu")


def test_append_refusals(b):
    _b, p = _p()
    good = dict(q=p, k=p, v=p, q_out=p, q_stride=1024, k_stride=256, v_stride=256, q_out_stride=1024, q_weight=p,
                k_weight=p, cos_sin=p, positions=p, slots=p, k_cache=p, v_cache=None, num_tokens=0, h_q=8, h_kv=2,
                d_head=128, max_position=16, rot_dim=128, interleaved=0, num_blocks=4, block_size=16,
                cache_layout=b.GQA_CACHE_KV4, bf16=0, eps=1e-6)

    def call(axes=p, n=3, ws=p, wsb=256, **kw):
        return b.lib.gqa_append_axes(b.gqa_append_args(**{**good, **kw}), axes, n, ws, wsb, None)

    INV = b.GQA_ERR_INVALID_ARG
    assert call() == b.GQA_OK and call(axes=None, n=1) == b.GQA_OK and call(n=32) == b.GQA_OK
    assert b.lib.gqa_append_axes(None, p, 1, p, 256, None) == INV
    for bad in [dict(n=0), dict(n=33), dict(n=-1), dict(axes=None, n=2), dict(cache_layout=5), dict(cache_layout=3),
                dict(block_size=24), dict(num_tokens=1, k_cache=None), dict(num_tokens=1, k_cache=p + 8),
                dict(num_tokens=1, ws=None), dict(num_blocks=1 << 27), dict(rot_dim=4)]:
        assert call(**bad) == INV, bad
    assert call(num_tokens=1, wsb=8) == b.GQA_ERR_WORKSPACE and call(d_head=32) == b.GQA_ERR_UNSUPPORTED


def test_decode_and_read_refusals(b):
    _b, p = _p()
    INV, UNS, WSP = b.GQA_ERR_INVALID_ARG, b.GQA_ERR_UNSUPPORTED, b.GQA_ERR_WORKSPACE

    def kv4(q=p, cache=p, N=1, T=1, mb=4, nb=4, bs=16, hq=8, hk=2, d=128, scale=0.1, w=0, s=0, ws=p, wsb=1 << 30, status=None,
            o=p, tab=p, lens=p):
        return b.lib.gqa_decode_kv4(q, cache, tab, lens, o, N, T, mb, nb, bs, hq, hk, d, scale, w, s, ws, wsb, status, None, None)

    def rows(q=p, cache=p, v=p, N=1, T=1, mb=4, nb=4, bs=16, hq=8, hk=2, d=128, scale=0.1, w=8, s=0, ws=p, wsb=1 << 30,
             status=None, o=p, tab=p, lens=p):
        return b.lib.gqa_decode_window(q, cache, v, tab, lens, o, N, T, mb, nb, bs, hq, hk, d, scale, w, s, ws, wsb, status, None,
                                       None)

    for dec in (kv4, rows):
        assert dec(N=0) == b.GQA_OK
        for bad in [dict(N=-1), dict(N=65536), dict(T=0), dict(mb=0), dict(nb=-1), dict(bs=24), dict(hq=7), dict(hk=0),
                    dict(scale=math.inf), dict(scale=math.nan), dict(q=None), dict(q=p + 2), dict(cache=p + 8),
                    dict(cache=None), dict(ws=None), dict(ws=p + 8), dict(status=p + 4), dict(mb=1 << 27, bs=16), dict(w=-1),
                    dict(s=-1), dict(o=None), dict(tab=p + 2), dict(lens=None)]:
            assert dec(**bad) == INV, bad
        assert dec(d=80) == UNS and dec(hq=130, hk=2) == UNS and dec(hq=8, hk=1, T=9) == UNS
        assert dec(wsb=255) == WSP
    assert rows(v=None) == INV and rows(v=p + 8) == INV
    assert b.gqa_decode_window_workspace_size(1, 1, 9, 2, 128) == 0
    assert b.gqa_decode_window_workspace_size(1, 1, 8, 2, 128, b.GQA_CACHE_VLLM) == 0

    def read(cache=p, k=p, v=p, N=1, n=16, mb=4, nb=4, bs=16, hk=2, d=128, ws=p, wsb=256, begins=None):
        return b.lib.gqa_kv4_read(cache, p, p, begins, k, v, N, n, mb, nb, bs, hk, d, ws, wsb, None, None)

    assert read(N=0) == b.GQA_OK and read(n=0) == b.GQA_OK
    for bad in [dict(N=-1), dict(n=-1), dict(n=1 << 31), dict(k=None, v=None), dict(k=p + 2), dict(cache=None),
                dict(bs=0), dict(mb=0), dict(ws=None), dict(begins=p + 2)]:
        assert read(**bad) == INV, bad
    assert read(d=256) == UNS and read(wsb=0) == WSP


def test_binding_refuses_what_is_not_on_a_gpu(b):
    x = torch.zeros(4, 256, dtype=torch.float16)
    i = torch.zeros(4, dtype=torch.int64)
    cache, tab = torch.zeros(2, 2, 16 * 144, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.int32)
    pool = torch.zeros(2, 16, 256, dtype=torch.float16)
    with pytest.raises(ValueError):
        b.gqa_append(x, x, x, 2, 2, i, cache, positions=tab.view(1, 4), pair_axes=i.byte())
    with pytest.raises(ValueError):
        b.gqa_decode_kv4(x, cache, tab, i.int(), 2, 2)
    with pytest.raises(ValueError):
        b.gqa_decode_window(x, pool, pool, tab, i.int(), 2, 2, window=4)
    with pytest.raises(ValueError):
        b.gqa_kv4_read(cache, tab, i.int(), 128, 16)
