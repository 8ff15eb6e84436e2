"""gqa_decode_kv4 and gqa_decode_window at the ends of the numbers' ranges, against the float64 oracle.

Weights.  Six visible keys whose values nearly cancel, so that |o| is far below A = sum p|v| / l and the weights' rounding
stands out.  Queries have one element, 1, so that a score is one element of its key, exactly.  Then, relative to A: logits
of at most 2^2 in log2 units, factor and product rounded, 2^-21; ex2 2^-22; l, the products' sums and the quotient 2^-20; in
all below 2^-18.  The weights: two f16 numbers 2^-22, two bf16 numbers 2^-16, one f16 number 2^-12.

Range.  Scales of the 4-bit cache over all bytes it writes, values of 16 bits over many powers of two, queries of any size
with a scale that keeps sum |q||k| * scale at 2^5.  Tolerance: the output's rounding u|o|; weights 2^-12 A at most; scores (2^5 *
128 terms * 2^-24, in log2 units) and sums 2^-11 A; weights near f16's smallest 2^-36 of the row's largest each, taken twice.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import kv4_oracle as k4
from test_gpu_window import DT, TINY, Case, U, gen, gqa, npy, queries  # noqa: F401  (gqa: a fixture)

HK, D, SEEN = 4, 128, 6
WEIGHTS = {("kv4", "f16"): 2.0 ** -22, ("rows", "f16"): 2.0 ** -22, ("rows", "bf16"): 2.0 ** -16, ("kv4", "bf16"): 2.0 ** -12}


def rounded(x, elem):
    return x.to(DT[elem]).double()


def cancelling(kind, elem, n, seed):
    """A sequence of n tokens whose last SEEN values nearly cancel under the weights of one query head for each KV head."""
    c = Case(kind, elem, [n], D, HK, 16, seed)
    q = torch.zeros(1, 1, HK, D)
    q[..., 3] = 1
    k = c.kv(0, n)[0]
    g = np.random.default_rng(seed)
    v = g.uniform(32, 60, (SEEN, HK, D)) * g.choice([-1.0, 1.0], (SEEN, HK, D))
    w = np.exp(k[n - SEEN:, :, 3])
    last = int(np.argmax(w.sum(1)))
    for key in [i for i in range(SEEN) if i != last] + [last]:
        at = n - SEEN + key
        blk, row = int(c.tab[0, at // 16]), at % 16
        if key == last:
            rest = np.delete(c.kv(0, n)[1][n - SEEN:], last, 0)
            v[last] = -(np.delete(w, last, 0)[..., None] * rest).sum(0) / w[last][:, None]
        for h in range(HK):
            if kind == "kv4":
                k4.put_row(c.cache.numpy(), blk * 16 + row, h, 1, v[key, h], D, 16)
            else:
                c.v[blk, row, h * D:(h + 1) * D] = torch.from_numpy(v[key, h]).to(DT[elem])
    return c, q.reshape(1, 1, -1).to(DT[elem])


def bounds(c, q, n, elem, kind):
    ref, a, _, _ = k4.decode_window(npy(q), c.kv, [n], HK, HK, D, 1.0, False, SEEN, 0)
    return ref, U[elem] * ref.abs() + (WEIGHTS[kind, elem] + 2.0 ** -18) * a + TINY[elem]


@pytest.mark.parametrize("kind,elem", WEIGHTS)
def test_one_rounding_of_the_weights_would_show(kind, elem):
    """On the CPU: with weights of one 16-bit number where the calls keep two, the bounds below do not hold."""
    if (kind, elem) == ("kv4", "bf16"):
        return
    c, q = cancelling(kind, elem, 40, 5)
    ref, tol = bounds(c, q, 40, elem, kind)
    k, v = (torch.from_numpy(x[-SEEN:]) for x in c.kv(0, 40))
    p = (k[:, :, 3] - k[:, :, 3].max(0).values).exp()
    one = rounded(p * 2048, elem) / 2048
    two = one + rounded((p - one) * 2048, elem) / 2048
    for w, holds in ((one, False), (two, True)):
        o = (w[..., None] * v).sum(0) / p.sum(0)[:, None]
        err = (o.reshape(-1) - ref.reshape(-1)).abs()
        out = (err > tol.reshape(-1)).double().mean()
        assert out == 0 if holds else out > 0.1, (kind, elem, float(out))


@pytest.mark.gpu
@pytest.mark.parametrize("kind,elem", WEIGHTS)
@pytest.mark.parametrize("n", [SEEN, 40, 5000])
def test_weights_are_as_exact_as_stated(gqa, kind, elem, n):  # noqa: F811
    for seed in (5, 6, 7):
        c, q = cancelling(kind, elem, n, seed)
        ref, tol = bounds(c, q, n, elem, kind)
        err = (c.run(gqa, q, HK, scale=1.0, window=SEEN).double().cpu() - ref).abs()
        assert (err <= tol).all(), (kind, elem, n, float((err / tol).max()))
    assert gqa.gqa_status_check() == gqa.GQA_OK


SHAPES = [(128, 8, 2, 1), (64, 8, 2, 2), (128, 16, 1, 1), (64, 24, 1, 1), (128, 16, 2, 4), (64, 64, 1, 1)]      # D, hq, hk, T
LENS = [[300], [700, 33, 129] * 8]


def check_range(gqa, c, q, hq, window):  # noqa: F811
    D = c.D
    k = max(np.abs(c.kv(b, n)[0]).sum(-1).max() for b, n in enumerate(c.lens))
    scale = float(torch.tensor(32.0 / (float(q.double().abs().max()) * k)).float())
    assert 2.0 ** -120 < scale < 2.0 ** 120
    o = c.run(gqa, q, hq, scale=scale, causal=True, window=window, sinks=3).double().cpu()
    ref, a, l, top = k4.decode_window(npy(q), c.kv, c.lens, hq, c.hk, D, scale, True, window, 3)
    n = torch.tensor(c.lens, dtype=torch.float64)
    low = (n * 2.0 ** -35 * top)[:, None, None] / l.clamp(min=1.0)
    tol = U[c.elem] * ref.abs() + (2.0 ** -12 + 2.0 ** -11) * a + low.repeat_interleave(D, -1) + TINY[c.elem]
    err = (o - ref).abs()
    assert torch.isfinite(o).all() and (err <= tol).all(), float((err / tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("D,hq,hk,T", SHAPES)
def test_scales_of_the_4_bit_cache(gqa, elem, lens, D, hq, hk, T):  # noqa: F811
    """Every scale byte that is written, 0 and the subnormal ones too: K's, V's, and both."""
    bs = 16
    for which in ("k", "v", "both"):
        c = Case("kv4", elem, lens, D, hk, bs, 30 + D + hq)
        some = torch.randint(0, 0x72, c.cache[..., bs * D:].shape, generator=gen(31)).byte()
        half = bs * D // 16
        if which != "v":
            c.cache[..., bs * D:bs * D + half] = some[..., :half]
        if which != "k":
            c.cache[..., bs * D + half:] = some[..., half:]
        for window in (0, 100):
            check_range(gqa, c, queries(elem, len(lens), T, hq * D, 32), hq, window)
    assert gqa.gqa_status_check() == gqa.GQA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["kv4", "rows"])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("D,hq,hk,T", SHAPES)
def test_queries_of_any_size(gqa, kind, lens, D, hq, hk, T):  # noqa: F811
    """bfloat16 queries from 2^-120 (16-bit pools: 2^-100, so that fp32 holds their products) to 2^100; over the 4-bit cache
    they become f16 by a power of two for each row."""
    c = Case(kind, "bf16", lens, D, hk, 16, 33 + D + hq)
    for e in (-120 if kind == "kv4" else -100, -60, 40, 100):
        q = (torch.randn(len(lens), T, hq * D, generator=gen(34), dtype=torch.float64) * 2.0 ** e).bfloat16()
        if e > -60:      # rows of very different sizes: one of each four far below the others
            q.view(len(lens), T, hq, D)[:, :, ::4] *= 2.0 ** -30
        for window in (0, 100):
            check_range(gqa, c, q, hq, window)
    assert gqa.gqa_status_check() == gqa.GQA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("elem,lo,hi", [("f16", -14, 13), ("bf16", -100, 100)])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("D,hq,hk,T", SHAPES)
def test_values_and_keys_of_16_bits(gqa, elem, lo, hi, lens, D, hq, hk, T):  # noqa: F811
    """Keys and values over many powers of two, one for each token."""
    c = Case("rows", elem, lens, D, hk, 16, 35 + D + hq)
    g = gen(36)
    nb = c.k.shape[0]
    for name in ("k", "v"):
        by = 2.0 ** torch.randint(lo, hi, (nb, 16, 1), generator=g).double()
        x = (torch.randn(nb, 16, hk * D, generator=g, dtype=torch.float64).clamp(-3.9, 3.9) * by).to(DT[elem])
        setattr(c, name, x)
    q = queries(elem, len(lens), T, hq * D, 37)
    for window in (0, 100):
        check_range(gqa, c, q, hq, window)
    assert gqa.gqa_status_check() == gqa.GQA_OK
