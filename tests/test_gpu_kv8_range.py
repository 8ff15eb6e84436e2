"""gqa_decode_kv8 where weights and value scales lie far apart: keys that take all the weight, values of very
different size, infinities, values that the causal tail hides.

Tolerance, for every output element, with A = sum p|v| / l of that element and u the half step of the output's type:
u|o| + 4 * 2^-11 A + half the smallest subnormal.  2^-11 A is the rounding of the weights to f16, another the fp32 sums
and ex2 (as in test_gpu_kv8.py).  The rest is for weights below f16's normal range.  A weight is stored times 2^11 and
the scale of its value over the largest one so far, as long as the scales lie within 2^10: it is off by at most
2^-25 2^-11 = 2^-36 of the largest weight with the largest scale.  The cases here that stay in that form have no weight
below 2^-26 of the largest and equal scales: 2^-10 A.  Beyond, a range of scales is taken by itself in every tile, relative to the
row's largest weight there: 2^-29 of it.  The tolerance has no term with the number of keys or the largest value."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import kv8_oracle as ko

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}
# (D, h_q, h_kv, T_q): 4, 8, 12, 24, 32, 40 and 64 query rows for a KV head
SHAPES = [(128, 4, 1, 1), (64, 16, 2, 1), (64, 12, 1, 1), (128, 12, 1, 2), (128, 16, 1, 2), (64, 40, 1, 1), (128, 16, 1, 4)]


@pytest.fixture(scope="module")
def gqa():
    from decode_attention_03_gb300 import build
    build.build()
    import decode_attention_03_gb300._binding as b
    assert torch.cuda.is_available()
    return b


def gen(seed):
    return torch.Generator().manual_seed(seed)


def npy(t):
    return t.double().cpu().numpy()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows_to_cache(k, k_exp, v, v_exp, bs, seed, room=0):
    """(cache, table (1, blocks + room)) of one sequence: codes (n, h_kv, D) and exponent bytes (n, h_kv)."""
    n, hk, D = k.shape
    nb = -(-n // bs)
    tab = np.random.default_rng(seed).permutation(nb + 1)[:nb].astype(np.int32)
    cache = np.full((nb + 1, hk, bs * (2 * D + 2)), 0x7F, dtype=np.uint8)
    for w, (codes, exps) in enumerate(((k, k_exp), (v, v_exp))):
        for r in range(min(bs, n)):
            at = np.arange(r, n, bs)
            cache[tab[at // bs][:, None, None], np.arange(hk)[None, :, None], ko.row_offsets(r, D, bs, w)] = codes[at]
            cache[tab[at // bs], :, 2 * bs * D + w * bs + r] = exps[at]
    return cache, np.pad(tab, (0, room), constant_values=-1)[None]


def keys(n, hk, D, seed):
    """K codes of zero: every key's logit is 0.  V codes of normal positive and negative values, a mean above 0."""
    rng = np.random.default_rng(seed)
    v = ko.encode(rng.standard_normal((n, hk, D)) * 60 + 60)
    return np.zeros((n, hk, D), np.uint8), np.full((n, hk), 120, np.uint8), v, np.full((n, hk), 120, np.uint8)


def signs(D, heads, T, seed):
    """Queries of +-1, the same pattern for all heads and tokens: with K = c * pattern the logit is c * sqrt(D)."""
    s = np.where(np.random.default_rng(seed).standard_normal(D) < 0, -1.0, 1.0)
    return s, torch.from_numpy(np.tile(s, (1, T, heads)))


def aligned_key(k, k_exp, j, s, logit):
    """Gives key j about the logit asked for, with a code that is exact."""
    D = len(s)
    c = float(ko.code_values()[ko.encode(logit / math.sqrt(D))])
    k[j] = ko.encode(s * c)
    k_exp[j] = 127
    return c * math.sqrt(D)


def check(gqa, cache, tab, n, q, hq, hk, D, bs, elem, causal=False, skip=(), where=""):
    q = q.to(DT[elem])
    o = gqa.gqa_decode_kv8(q.cuda(), dev(cache), dev(tab), torch.tensor([n], dtype=torch.int32, device="cuda"), hq, hk,
                           causal=causal)
    ref, a, _, _ = ko.decode_kv8(npy(q), cache, tab, [n], hq, hk, D, D ** -0.5, bs, causal)
    o = o.double().cpu().reshape(ref.shape)
    ok = torch.ones(D, dtype=torch.bool)
    ok[list(skip)] = False
    ok = ok.repeat(hq).expand_as(ref) & (ref.abs() < torch.finfo(DT[elem]).max * 0.99)
    tol = U[elem] * ref.abs() + 4 * 2.0 ** -11 * a + TINY[elem]
    err = (o - ref).abs()
    assert torch.isfinite(o[ok]).all(), where
    bad = ok & (err > tol)
    assert not bad.any(), f"{where}: {int(bad.sum())} of {int(ok.sum())} out, worst {float((err / a)[bad].max()):.3e} of A"


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("empty_exponent", [1, 120])
@pytest.mark.parametrize("n,at", [(1 << 20, 123), (5000, 4999), (70, 0)])
def test_a_key_without_value_that_takes_the_weight(gqa, n, at, empty_exponent, elem):
    """One key 2^26 above the rest whose values are zero, as gqa_append stores them (exponent 1) or with another
    exponent: what is left is the others' sum."""
    D, hq, bs = 64, 4, 64
    k, ke, v, ve = keys(n, 1, D, n)
    s, q = signs(D, hq, 1, 3)
    logit = aligned_key(k, ke, at, s, 18.0)
    assert 25.5 < logit * math.log2(math.e) < 26
    v[at], ve[at] = 0, empty_exponent
    check(gqa, *rows_to_cache(k, ke, v, ve, bs, 4), n, q, hq, 1, D, bs, elem)


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("gap,logit", [(16, 18.0), (26, 18.0), (26, 26.0), (26, 9.0), (60, 40.0), (60, 56.0), (110, 64.0)])
@pytest.mark.parametrize("D,hq,hk,T", SHAPES)
def test_the_key_that_takes_the_weight_has_small_values(gqa, D, hq, hk, T, gap, logit, elem):
    """Its V exponent is `gap` below that of the others, whose weight is next to nothing."""
    bs = 16
    for n, at in ((700, 350), (9000, 8999), (40, 0)):
        for room in (0, 2000):                            # the short and the general form
            k, ke, v, ve = keys(n, hk, D, n + D)
            s, q = signs(D, hq, T, 5)
            aligned_key(k, ke, at, s, logit)
            ve[at] -= gap
            ve[n // 3] -= 3
            check(gqa, *rows_to_cache(k, ke, v, ve, bs, 6, room), n, q, hq, hk, D, bs, elem, where=f"{n} {at} {room}")


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("up", [12, 30, 127])
@pytest.mark.parametrize("D,hq,hk,T", SHAPES)
def test_one_large_row_leaves_the_other_columns(gqa, D, hq, hk, T, up, elem):
    """A V row whose one large value sets its exponent (127: what an infinity leaves) and whose others are zero, with the
    weight of any other key: only that column knows of it."""
    bs, col = 32, 17
    for n, at in ((700, 40), (6000, 5000), (33, 32)):
        for room in (0, 1000):
            k, ke, v, ve = keys(n, hk, D, n + D + 1)
            v[at] = 0
            v[at, :, col] = 0x7E
            ve[at] += up
            q = torch.randn(1, T, hq * D, generator=gen(7))
            check(gqa, *rows_to_cache(k, ke, v, ve, bs, 8, room), n, q, hq, hk, D, bs, elem, skip=[col],
                  where=f"{n} {at} {room}")


@pytest.mark.parametrize("elem", ["f16", "bf16"])
def test_large_and_infinite_values_through_the_cache(gqa, elem):
    """65504 and an infinity among values of size 1, stored by gqa_append: their columns aside, nothing changes."""
    D, hq, hk, bs, n = 128, 8, 2, 16, 300
    g = gen(9)
    x = torch.randn(n, 2 * hk * D, generator=g)
    x[200, hk * D + 5] = 65504.0
    x[77, hk * D + D + 9] = math.inf
    x = x.to(DT[elem]).cuda()
    cache = gqa.gqa_kv8_cache(n // bs + 1, bs, hk, D)
    gqa.gqa_append(None, x[:, :hk * D], x[:, hk * D:], hq, hk, torch.arange(n, device="cuda"), cache)
    tab = np.arange(n // bs + 1, dtype=np.int32)[None]
    host = cache.cpu().numpy()
    assert host[77 // bs, 1, 2 * bs * D + bs + 77 % bs] == 247
    q = torch.randn(1, 1, hq * D, generator=g)
    check(gqa, host, tab, n, q, hq, hk, D, bs, elem, skip=[5, 9])


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("up", [14, 40, 100])
@pytest.mark.parametrize("D,hq,hk,T", [(128, 2, 1, 4), (64, 4, 1, 6), (128, 8, 1, 4), (64, 8, 1, 8), (128, 4, 2, 3)])
def test_large_values_that_the_causal_tail_hides(gqa, D, hq, hk, T, up, elem):
    """The newest tokens' V rows are larger than all before: the tokens that do not see them do not notice."""
    bs = 16
    for n in (6000, 400, 33, T + 2):
        for room in (0, 2000):
            k, ke, v, ve = keys(n, hk, D, n + up)
            ve[n - 2:] += up
            q = torch.randn(1, T, hq * D, generator=gen(10))
            check(gqa, *rows_to_cache(k, ke, v, ve, bs, 11, room), n, q, hq, hk, D, bs, elem, causal=True,
                  where=f"{n} {room}")


@pytest.mark.parametrize("elem", ["f16", "bf16"])
def test_scales_of_any_order(gqa, elem):
    """V exponents drawn from 60 .. 200, from tile to tile in ranges of their own, weights of any size."""
    D, hq, hk, bs, n = 64, 8, 2, 8, 2500
    rng = np.random.default_rng(12)
    for room in (0, 3000):
        k, ke, v, ve = keys(n, hk, D, 13)
        k[:] = ko.encode(rng.standard_normal(k.shape) * 100)
        ve[:] = np.clip(120 + (rng.standard_normal((n // 100, hk)) * 30).astype(int).repeat(100, 0) +
                        rng.integers(-8, 8, (n, hk)), 60, 125)
        q = torch.randn(1, 1, hq * D, generator=gen(14)) * 3
        check(gqa, *rows_to_cache(k, ke, v, ve, bs, 15, room), n, q, hq, hk, D, bs, elem)


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("D,hq,hk,T", [(128, 2, 1, 4), (64, 8, 2, 2), (128, 8, 1, 3), (64, 2, 1, 8), (128, 8, 1, 4),
                                       (64, 4, 1, 16), (128, 6, 1, 7), (64, 1, 1, 40)])
def test_not_a_number_that_the_causal_tail_hides(gqa, D, hq, hk, T, elem):
    """NaN in values of the newest tokens: it spoils its column for the tokens that see it, and for no other."""
    for bs in (8, 64):
        for n in (5000, 33, 64, T + 1, max(T - 2, 2)):        # the tail in one tile or two, or longer than the sequence
            for room in (0, 4000):
                k, ke, v, ve = keys(n, hk, D, n + T)
                for back, col in ((1, 5), (2, 40), (min(T, n) // 2 + 1, 11), (min(T + 3, n), 23)):
                    v[n - back, 0, col] = 0x7F if back % 2 else 0xFF
                if n > 100:
                    ve[n - 1] += 20
                    ve[n // 2] -= 3
                cache, tab = rows_to_cache(k, ke, v, ve, bs, 16, room)
                q = torch.randn(1, T, hq * D, generator=gen(17)).to(DT[elem])
                o = gqa.gqa_decode_kv8(q.cuda(), dev(cache), dev(tab), torch.tensor([n], dtype=torch.int32).cuda(), hq,
                                       hk, causal=True).double().cpu()
                ref, a, _, _ = ko.decode_kv8(npy(q), cache, tab, [n], hq, hk, D, D ** -0.5, bs, True)
                where = f"{bs} {n} {room}"
                assert torch.equal(o.isnan(), ref.isnan()), where
                err, tol = (o - ref).abs(), U[elem] * ref.abs() + 4 * 2.0 ** -11 * a + TINY[elem]
                assert not (err > tol).any(), where


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("D,hq,hk,T", SHAPES)
def test_pieces_of_values_of_any_one_size(gqa, D, hq, hk, T, elem):
    """A last tile whose only key has the largest exponent that an infinity leaves, or the smallest, behind tiles of ordinary
    ones: its worker has seen no other scale.  And sequences of one scale throughout, from the smallest to the largest."""
    bs = 16
    for n, last, rest in ((1633, 247, 120), (1633, 1, 120), (97, 247, 120), (1633, 30, 30), (4097, 2, 2), (1633, 215, 215),
                          (1633, 235, 235), (1633, 63, 63), (1633, 64, 64), (1633, 191, 191), (1633, 192, 192)):
        for room in (0, 3000):
            k, ke, v, ve = keys(n, hk, D, n + last)
            ve[:] = rest
            ve[n - 1] = last
            q = torch.randn(1, T, hq * D, generator=gen(25))
            check(gqa, *rows_to_cache(k, ke, v, ve, bs, 26, room), n, q, hq, hk, D, bs, elem, where=f"{n} {last} {rest} {room}")
