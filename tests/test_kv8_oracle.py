"""The float64 oracle of the cache operators pinned by hand, and the host-side refusals of
gqa_append, gqa_decode_kv8 and gqa_kv8_read (no GPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv8_oracle as ko


@pytest.fixture(scope="module")
def b():
    from decode_attention_03_gb300 import build
    build.build()
    import decode_attention_03_gb300._binding as binding
    return binding


# ---------------------------------------------------------------- oracle pins
def test_code_values_are_e4m3():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ko.code_values(), v)
    assert ko.code_values()[0x7e] == 448.0 and ko.code_values()[1] == 2.0 ** -9


def test_encode_nearest_even():
    v = ko.code_values()
    for x, want in [(0.0, 0.0), (448.0, 448.0), (1e9, 448.0), (-1e9, -448.0), (17.0, 16.0), (19.0, 20.0),
                    (17.0001, 18.0), (2.0 ** -10, 0.0), (3 * 2.0 ** -10, 2 * 2.0 ** -9), (-0.3, -0.3125)]:
        assert v[ko.encode(x)] == want, x
    x = np.concatenate([np.random.default_rng(0).standard_normal(20000) * 50, np.linspace(-448, 448, 9999)])
    t = torch.from_numpy(x).float()
    want = t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ko.encode(t.double().numpy()), want)
    assert math.isnan(v[ko.encode(math.nan)])


def test_exponent_is_the_smallest_that_holds():
    assert ko.exponent(0.0) == 1 and ko.exponent(448.0) == 127 and ko.exponent(448.0000001) == 128
    assert ko.exponent(224.0) == 126 and ko.exponent(1.75) == 119 and ko.exponent(math.inf) == 247
    assert ko.exponent(3.38e38) == 247 and ko.exponent(2.0 ** -133) == 1


def test_rotation_and_norm_by_hand():
    x = np.array([[3.0, 4.0, 0.0, 0.0, 1.0, 0.0, 0.0, 2.0]])
    cs = np.array([[0.0, 1.0, 1.0, 0.0]])          # first pair a quarter turn, second none
    y = ko.head_rows(x, 1, None, 0.0, cs, [0], False)[0, 0]
    np.testing.assert_array_equal(y, [0.0, 4.0, 3.0, 0.0, 1.0, 0.0, 0.0, 2.0])
    y = ko.head_rows(x, 1, None, 0.0, cs, [0], True)[0, 0]
    np.testing.assert_array_equal(y, [-4.0, 3.0, 0.0, 0.0, 1.0, 0.0, 0.0, 2.0])
    y = ko.head_rows(np.array([[3.0, 4.0]]), 1, [2.0, 1.0], 0.0, None, None, False)[0, 0]
    np.testing.assert_allclose(y, [6 / math.sqrt(12.5), 4 / math.sqrt(12.5)])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 64])
def test_rows_fill_a_block_without_overlap(D, bs):
    at = np.concatenate([ko.row_offsets(r, D, bs, w) for r in range(bs) for w in (0, 1)])
    assert sorted(at) == list(range(2 * bs * D))
    rng = np.random.default_rng(1)
    cache = np.full((3, 2, bs * (2 * D + 2)), 0x7F, dtype=np.uint8)
    rows = {}
    for slot in range(bs, 2 * bs):
        for h in (0, 1):
            for w in (0, 1):
                x = rng.standard_normal(D) * 10.0 ** rng.integers(-3, 4)
                ko.put_row(cache, slot, h, w, x, D, bs)
                rows[slot, h, w] = x
    assert (cache[[0, 2]] == 0x7F).all()
    k, v = ko.gather_kv8(cache, [1], bs, D, bs)
    for (slot, h, w), x in rows.items():
        got = ko.get_row(cache, slot, h, w, D, bs)
        np.testing.assert_array_equal(got, (k, v)[w][slot - bs, h])
        assert (np.abs(got - x) <= np.maximum(np.abs(x) * 2.0 ** -4, np.abs(x).max() / 224 * 2.0 ** -10)).all()


def test_decode_kv8_against_plain_softmax():
    rng = np.random.default_rng(2)
    D, bs, hq, hk = 64, 8, 4, 2
    cache = np.zeros((5, hk, bs * (2 * D + 2)), dtype=np.uint8)
    table, n = [3, 0, 2], 19
    for j in range(n):
        for h in range(hk):
            for w in (0, 1):
                ko.put_row(cache, table[j // bs] * bs + j % bs, h, w, rng.standard_normal(D), D, bs)
    q = rng.standard_normal((1, 2, hq * D))
    o, a, l, top = ko.decode_kv8(q, cache, [table], [n], hq, hk, D, 0.125, bs, causal=True)
    k, v = ko.gather_kv8(cache, table, n, D, bs)
    for t in range(2):
        for h in range(hq):
            end = n - 1 + t
            s = 0.125 * k[:end, h // 2] @ q[0, t, h * D:(h + 1) * D]
            p = np.exp(s - s.max())
            np.testing.assert_allclose(o[0, t, h * D:(h + 1) * D], p @ v[:end, h // 2] / p.sum(), atol=1e-12)
            np.testing.assert_allclose(l[0, t, h], p.sum())
    assert (a >= o.abs()).all() and float(top[0]) == np.abs(v).max()
    assert (ko.decode_kv8(q, cache, [table], [1], hq, hk, D, 0.125, bs, causal=True)[0][0, 0] == 0).all()


# ---------------------------------------------------------------- refusals
def _p(n=1 << 12):
    buf = ctypes.create_string_buffer(n + 64)
    return buf, (ctypes.addressof(buf) + 15) & ~15


def test_block_bytes(b):
    assert b.gqa_kv8_block_bytes(16, 128) == 16 * 258 and b.gqa_kv8_block_bytes(8, 64) == 8 * 130
    assert b.gqa_kv8_block_bytes(12, 128) == 0 and b.gqa_kv8_block_bytes(16, 96) == 0
    for bs in (8, 16, 32, 64):
        for d in (64, 128):
            assert b.gqa_kv8_block_bytes(bs, d) % 16 == 0        # a bulk copy's size


def test_append_refusals(b):
    _b, p = _p()
    good = dict(q=p, k=p, v=p, q_out=p, q_stride=1024, k_stride=256, v_stride=256, q_out_stride=1024, q_weight=p,
                k_weight=p, cos_sin=p, positions=p, slots=p, k_cache=p, v_cache=p, num_tokens=0, h_q=8, h_kv=2,
                d_head=128, max_position=16, rot_dim=128, interleaved=0, num_blocks=4, block_size=16, cache_layout=2,
                bf16=0, eps=1e-6)

    def call(ws=p, wsb=256, **kw):
        return b.lib.gqa_append(b.gqa_append_args(**{**good, **kw}), ws, wsb, None)

    assert call() == b.GQA_OK                                    # no tokens: nothing to do
    INV, UNS, WSP = b.GQA_ERR_INVALID_ARG, b.GQA_ERR_UNSUPPORTED, b.GQA_ERR_WORKSPACE
    assert b.lib.gqa_append(None, p, 256, None) == INV
    one = dict(num_tokens=1)
    for bad in [dict(num_tokens=-1), dict(h_q=-1), dict(h_kv=0), dict(h_q=7), dict(num_blocks=-1),
                dict(block_size=12), dict(num_blocks=1 << 27), dict(cache_layout=3), dict(cache_layout=-1),
                dict(eps=-1.0), dict(eps=math.nan), dict(rot_dim=12), dict(rot_dim=136), dict(rot_dim=0),
                dict(max_position=0), dict(positions=None), dict(cos_sin=p + 4),
                {**one, "k": None}, {**one, "v": p + 2}, {**one, "q": None}, {**one, "q_out": None},
                {**one, "slots": None}, {**one, "k_cache": None}, {**one, "cache_layout": 0, "v_cache": None},
                {**one, "q_stride": 1023}, {**one, "q_stride": 1016}, {**one, "k_stride": 0}, {**one, "v_stride": 260},
                {**one, "q_out_stride": 8}, {**one, "q_weight": p + 8}, {**one, "ws": None}]:
        assert call(**bad) == INV, bad
    assert call(d_head=96) == UNS
    assert call(num_tokens=1, wsb=255) == WSP


def test_decode_and_read_refusals(b):
    _b, p = _p()
    INV, UNS, WSP = b.GQA_ERR_INVALID_ARG, b.GQA_ERR_UNSUPPORTED, b.GQA_ERR_WORKSPACE

    def dec(q=p, cache=p, N=1, T=1, mb=4, nb=4, bs=16, hq=8, hk=2, d=128, scale=0.1, ws=p, wsb=1 << 30):
        return b.lib.gqa_decode_kv8(q, cache, p, p, p, N, T, mb, nb, bs, hq, hk, d, scale, ws, wsb, None, None)

    assert dec(N=0) == b.GQA_OK
    for bad in [dict(N=-1), dict(N=65536), dict(T=0), dict(mb=0), dict(nb=-1), dict(bs=24), dict(hq=7), dict(hk=0),
                dict(scale=math.inf), dict(q=None), dict(q=p + 2), dict(cache=p + 8), dict(ws=None),
                dict(mb=1 << 27, bs=16)]:
        assert dec(**bad) == INV, bad
    assert dec(d=80) == UNS and dec(hq=130, hk=2) == UNS and dec(hq=8, hk=1, T=9) == UNS
    assert dec(wsb=255) == WSP
    assert b.gqa_decode_kv8_workspace_size(1, 1, 9, 2, 128) == 0

    def read(cache=p, k=p, v=p, N=1, n=16, mb=4, nb=4, bs=16, hk=2, d=128, ws=p, wsb=256, begins=None):
        return b.lib.gqa_kv8_read(cache, p, p, begins, k, v, N, n, mb, nb, bs, hk, d, ws, wsb, None, None)

    assert read(N=0) == b.GQA_OK and read(n=0) == b.GQA_OK
    for bad in [dict(N=-1), dict(n=-1), dict(n=1 << 31), dict(k=None, v=None), dict(k=p + 2), dict(cache=None),
                dict(bs=0), dict(mb=0), dict(ws=None), dict(begins=p + 2)]:
        assert read(**bad) == INV, bad
    assert read(d=256) == UNS and read(wsb=0) == WSP


def test_binding_refuses_what_is_not_on_a_gpu(b):
    x = torch.zeros(4, 256, dtype=torch.float16)
    i = torch.zeros(4, dtype=torch.int64)
    cache = torch.zeros(2, 2, 16 * 258, dtype=torch.uint8)
    with pytest.raises(ValueError):
        b.gqa_append(x, x, x, 2, 2, i, cache)
    with pytest.raises(ValueError):
        b.gqa_decode_kv8(x, cache, torch.zeros(4, 1, dtype=torch.int32), i.int(), 2, 2)
    with pytest.raises(ValueError):
        b.gqa_kv8_read(cache, torch.zeros(4, 1, dtype=torch.int32), i.int(), 128, 16)
    with pytest.raises(b.GQAError):
        b.gqa_kv8_cache(4, 12, 2, 128, device="cpu")
    assert b.gqa_kv8_cache(4, 16, 2, 128, device="cpu").shape == (4, 2, 16 * 258)
