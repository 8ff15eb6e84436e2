"""Attention whose logits are far from 0 in size (2^26 and more), as one outlier channel of queries and keys makes them.

Only channel 0 of queries and keys is not 0, so that fp32 holds every score q.k exactly, and logits are either equal or so far
apart that the smaller one's weight is 0: the output is the mean of the values of the row's largest keys.

Tolerance: the output's rounding u|o| (f16 2^-11, bf16 2^-8), the weights' 2^-11 A at most (A: the mean of |v|), fp32 sums 2^-18 A.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def gqa():
    from decode_attention_03_gb300 import build
    build.build()
    import decode_attention_03_gb300._binding as b
    assert torch.cuda.is_available()
    return b


def case(elem, D, hk, G, T, n, seed, same):
    """Queries (T, hk*G*D), keys and values (n, hk*D): `same`: every key alike, else a few that are the largest."""
    g = torch.Generator().manual_seed(seed)
    top = 60000.0 if elem == "f16" else 2.0 ** 60
    q, k = torch.zeros(T, hk * G, D), torch.zeros(n, hk, D)
    q[:, :, 0] = top * (0.3 + 0.7 * torch.rand(T, hk * G, generator=g))
    if same:
        k[:, :, 0] = -37000.0
    else:
        k[:, :, 0] = 37000.0 * torch.tensor([-0.5, 0.0, 0.25])[torch.randint(0, 3, (n, hk), generator=g)]
        for h in range(hk):
            k[torch.randperm(n, generator=g)[:5], h, 0] = 37000.0
    v = torch.randn(n, hk, D, generator=g)
    return q.reshape(T, -1).to(DT[elem]), k.reshape(n, -1).to(DT[elem]), v.reshape(n, -1).to(DT[elem])


def pools(gqa, op, k, v, hk, D, bs):
    """The tokens in the cache of `op`, in a shuffled order of blocks: its arrays, the table, and the keys and values held."""
    n, nb = k.shape[0], -(-k.shape[0] // bs)
    order = torch.randperm(nb, generator=torch.Generator().manual_seed(3))
    at = torch.arange(n)
    slots = (order[at // bs] * bs + at % bs).cuda()
    tab, lens = order.int()[None].cuda(), torch.tensor([n]).int().cuda()
    k, v = k.cuda(), v.cuda()
    if op == "rows":
        cache = [torch.zeros(nb, bs, hk * D, dtype=k.dtype, device="cuda") for _ in range(2)]
    else:
        cache = [(gqa.gqa_kv4_cache if op == "kv4" else gqa.gqa_kv8_cache)(nb, bs, hk, D)]
    gqa.gqa_append(None, k, v, hk, hk, slots, *cache)
    if op != "rows":
        k, v = (gqa.gqa_kv4_read if op == "kv4" else gqa.gqa_kv8_read)(*cache, tab, lens, D, n, dtype=k.dtype)
        k, v = k[0], v[0]
    return cache, tab, lens, k.double().cpu(), v.double().cpu()


def check(o, k, v, hk, G, D, elem, sign):
    """o (T, hk*G*D): the mean of the values whose key is the largest, in the scale's sign, of its head."""
    k0, v = k.reshape(-1, hk, D)[:, :, 0] * sign, v.reshape(-1, hk, D)
    o = o.double().cpu().reshape(-1, hk, G, D)
    assert torch.isfinite(o).all()
    for h in range(hk):
        best = v[k0[:, h] == k0[:, h].max(), h]
        ref, a = best.mean(0), best.abs().mean(0)
        err = (o[:, h] - ref).abs()
        assert (err <= U[elem] * ref.abs() + (2.0 ** -11 + 2.0 ** -18) * a).all(), (h, float(err.max()))


ROWS = [(2, 1), (4, 4), (8, 3), (16, 2), (5, 8), (8, 8)]      # query heads of a KV head, new tokens: 2 to 64 query rows


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("op", ["rows", "kv4", "kv8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,T", ROWS)
def test_paged_calls(gqa, elem, op, D, G, T):
    hk, bs = 2, 16
    for n, same, sign in ((1000, False, 1), (1000, False, -1), (700, True, 1), (9000, False, 1)):
        q, k, v = case(elem, D, hk, G, T, n, G + T + n, same)
        cache, tab, lens, k, v = pools(gqa, op, k, v, hk, D, bs)
        call = {"rows": lambda *a, **kw: gqa.gqa_decode_window(*a, window=0, **kw), "kv4": gqa.gqa_decode_kv4, "kv8": gqa.gqa_decode_kv8}[op]
        for scale in (D ** -0.5, 2.0 ** 20):
            o = call(q.cuda()[None], *cache, tab, lens, hk * G, hk, sign * scale)
            check(o[0], k, v, hk, G, D, elem, sign)
    assert gqa.gqa_status_check() == gqa.GQA_OK


def test_8_bit_values_far_apart(gqa):
    """The same where a token's values are 0, so that the exponents of its sequence lie far apart."""
    D, hk, G, bs = 128, 2, 4, 16
    for n in (1000, 9000):
        q, k, v = case("f16", D, hk, G, 1, n, n, False)
        v[::64] = 0
        cache, tab, lens, k, v = pools(gqa, "kv8", k, v, hk, D, bs)
        o = gqa.gqa_decode_kv8(q.cuda()[None], *cache, tab, lens, hk * G, hk)
        check(o[0], k, v, hk, G, D, "f16", 1)


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,T", ROWS + [(16, 8)])
def test_contiguous_calls(gqa, elem, D, G, T):
    """gqa_decode: mma.sync kernels below 16 query rows, tcgen05 from there on."""
    hk = 2
    for n, same, sign in ((1000, False, 1), (1000, False, -1), (700, True, 1), (9000, False, 1)):
        q, k, v = case(elem, D, hk, G, T, n, G + T + n, same)
        for scale in (D ** -0.5, 2.0 ** 20):
            o = gqa.gqa_decode(q.cuda()[None], k.cuda()[None], v.cuda()[None], hk * G, hk, sign * scale)
            check(o[0], k.double(), v.double(), hk, G, D, elem, sign)
