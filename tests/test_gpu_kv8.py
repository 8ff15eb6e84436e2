"""GPU parity of the cache operators -- gqa_append, gqa_decode_kv8, gqa_kv8_read -- against the float64
oracle (oracle/kv8_oracle.py).

Tolerances, from half steps u = finfo.eps / 2 (f16 2^-11, bf16 2^-8, fp32 2^-24):
* append, 16-bit outputs: one rounding of y, u|y| + half the smallest subnormal, and the fp32 steps before it.
  Those are at most 12 roundings of quantities no larger than |a| + |b| (the pair before the rotation):
  2^-20 (|a| + |b|).
* append, 8 bits: half an e4m3 step, 2^-4 |x| or 2^-10 below the smallest normal, in units of the row's
  scale, plus the same fp32 term.  A value within the fp32 term of the border of two codes may take either.
* read: a code times a power of two has 4 significant bits: the one rounding, to 16 bits, is the oracle's; equal.
* decode: the output's rounding u|o|; P rounded to f16 for the MMA: 2^-11 A, A = sum p|v| / l; a weight p 2^kv
  below f16's normal range is off by at most 2^-25 of the range, for n keys n 2^-25 2 max|V| / l;
  and the fp32 sums, ex2 (2 ulp) and scores: another 2^-11 A, generous for scores below 2^6 in size.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import kv8_oracle as ko

pytestmark = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}


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


def table(max_pos, rot, seed=0):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def append_case(elem, D, hq, hk, T, seed, norm=True, rot=None, max_pos=50):
    g = gen(seed)
    dt = DT[elem]
    rot = D if rot is None else rot
    qkv = torch.randn(T, (hq + 2 * hk) * D, generator=g).to(dt)
    c = dict(elem=elem, D=D, hq=hq, hk=hk, T=T, qkv=qkv, q=qkv[:, :hq * D], k=qkv[:, hq * D:(hq + hk) * D],
             v=qkv[:, (hq + hk) * D:], qw=None, kw=None, cs=None,
             pos=torch.randint(0, max_pos, (T,), generator=g).int())
    if norm:
        c["qw"] = (1 + 0.3 * torch.randn(D, generator=g)).to(dt)
        c["kw"] = (1 + 0.3 * torch.randn(D, generator=g)).to(dt)
    if rot:
        c["cs"] = table(max_pos, rot)
    return c


def cuda(t):
    return None if t is None else t.cuda()


def run_append(gqa, c, slots, k_cache, v_cache=None, inter=False, eps=1e-5, **kw):
    qkv = c["qkv"].cuda()
    n = c["hq"] * c["D"], c["hk"] * c["D"]
    q = gqa.gqa_append(qkv[:, :n[0]] if c["hq"] else None, qkv[:, n[0]:n[0] + n[1]], qkv[:, n[0] + n[1]:], c["hq"],
                       c["hk"], slots.cuda(), k_cache, v_cache, positions=c["pos"].cuda(), cos_sin=cuda(c["cs"]),
                       interleaved=inter, q_weight=cuda(c["qw"]), k_weight=cuda(c["kw"]), eps=eps, **kw)
    torch.cuda.synchronize()
    return q


def rows_of(c, x, w, heads, inter, eps=1e-5):
    """The oracle's rows (T, heads, D) and the fp32 term of their tolerance."""
    cs, pos = (None, None) if c["cs"] is None else (npy(c["cs"]), c["pos"].tolist())
    w = None if w is None else npy(w)
    y = ko.head_rows(npy(x), heads, w, eps, cs, pos, inter)
    n = ko.head_rows(npy(x), heads, w, eps, None, None, inter)
    size = np.abs(n)
    if cs is not None:
        half = cs.shape[1] // 2
        i = np.arange(half)
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        both = size[..., a] + size[..., b]
        size[..., a] = both
        size[..., b] = both
    return y, size * 2.0 ** -20


def close16(got, y, fp32, elem, where):
    got = npy(got).reshape(y.shape)
    err = np.abs(got - y)
    bad = err > U[elem] * np.abs(y) + TINY[elem] + fp32
    assert not bad.any(), f"{where}: {bad.sum()} of {bad.size} out, worst {err[bad].max():.3e}"


def close8(got, y, fp32, where):
    """got: values held in 8 bits, rows along the last axis."""
    top = np.abs(y).max(-1, keepdims=True)
    unit = 2.0 ** np.maximum(np.ceil(np.log2(np.maximum(top, 1e-300) / 448.0 * (1 - 2.0 ** -20))), -126)
    err = np.abs(got - y)
    # a maximum within the fp32 term of 448 * 2^k may take the next scale: the subnormal step doubles
    bad = err > np.maximum(np.abs(y) * 2.0 ** -4, unit * 2.0 ** -9) + 2 * fp32
    assert not bad.any(), f"{where}: {bad.sum()} of {bad.size} out, worst {err[bad].max():.3e}"
    assert (np.abs(got) <= 448 * 2 * unit).all()


def slots_for(T, num_blocks, bs, seed, skip=0):
    s = torch.randperm(num_blocks * bs, generator=gen(seed))[:T]
    if skip:
        s[torch.randperm(T, generator=gen(seed + 1))[:skip]] = -1 - torch.arange(skip) * 1000
    return s


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("D,hq,hk,rot,inter", [(128, 8, 2, 128, False), (128, 6, 3, 64, False), (128, 4, 4, 128, True),
                                               (64, 8, 2, 64, False), (64, 7, 1, 8, True), (64, 10, 5, 48, False),
                                               (128, 32, 8, 24, True), (128, 5, 1, 0, False)])
@pytest.mark.parametrize("layout,bs,T", [("rows", 16, 37), ("vllm", 8, 70), ("kv8", 32, 53), ("kv8", 8, 1)])
def test_append(gqa, elem, D, hq, hk, rot, inter, layout, bs, T):
    c = append_case(elem, D, hq, hk, T, 100 + D + hq + T, norm=(hq + T) % 4 != 1, rot=rot)
    nb = (T + bs - 1) // bs + 3
    slots = slots_for(T, nb, bs, 7, skip=T // 9)
    dt = DT[elem]
    if layout == "kv8":
        caches = [torch.full((nb, hk, bs * (2 * D + 2)), 0x5A, dtype=torch.uint8, device="cuda")]
    elif layout == "rows":
        caches = [torch.full((nb, bs, hk * D), 7.0, dtype=dt, device="cuda") for _ in range(2)]
    else:
        caches = [torch.full((nb, hk, D // 8, bs, 8), 7.0, dtype=dt, device="cuda"),
                  torch.full((nb, hk, D, bs), 7.0, dtype=dt, device="cuda")]
    q = run_append(gqa, c, slots, *caches, inter=inter)
    y, f = rows_of(c, c["q"], c["qw"], hq, inter)
    close16(q, y, f, elem, "q_out")
    k, fk = rows_of(c, c["k"], c["kw"], hk, inter)
    v, fv = npy(c["v"]).reshape(T, hk, D), np.zeros((T, hk, D))
    kept = [(t, int(s)) for t, s in enumerate(slots) if s >= 0]
    ts, ss = np.array([t for t, _ in kept]), np.array([s for _, s in kept])
    if layout == "kv8":
        got = caches[0].cpu().numpy()
        untouched = np.ones_like(got, dtype=bool)
        for w, (y, f) in enumerate(((k, fk), (v, fv))):
            held = np.stack([[ko.get_row(got, s, h, w, D, bs) for h in range(hk)] for s in ss])
            close8(held, y[ts], f[ts], f"cache {w}")
            for s in ss:
                blk, row = divmod(int(s), bs)
                untouched[blk][:, ko.row_offsets(row, D, bs, w)] = False
                untouched[blk][:, 2 * bs * D + w * bs + row] = False
            if w == 1:                                            # V is exact until the one rounding
                want = got.copy()
                for t, s in kept:
                    for h in range(hk):
                        ko.put_row(want, s, h, 1, v[t, h], D, bs)
                np.testing.assert_array_equal(got, want)
        assert (got[untouched] == 0x5A).all()
        return
    flat = []
    for i, x in enumerate(caches):
        x = x.float().cpu()
        if layout == "vllm":
            x = x.permute(0, 3, 1, 2, 4) if i == 0 else x.permute(0, 3, 1, 2)
        flat.append(x.reshape(nb * bs, hk, D))
    close16(flat[0][ss], k[ts], fk[ts], elem, "k cache")
    assert torch.equal(flat[1][ss], c["v"].float().view(T, hk, D)[ts])
    rest = np.setdiff1d(np.arange(nb * bs), ss)
    assert all((x[rest] == 7.0).all() for x in flat)


def test_append_many_tokens_wide_model(gqa):
    """Enough work for the largest launch shape; an odd head count leaves part of a warp idle."""
    for D, hq, hk, T in [(128, 33, 11, 1500), (64, 63, 9, 2100)]:
        c = append_case("bf16", D, hq, hk, T, 300 + D)
        cache = gqa.gqa_kv8_cache(T // 16 + 2, 16, hk, D)
        slots = torch.randperm(T + 9, generator=gen(3))[:T]
        q = run_append(gqa, c, slots, cache)
        y, f = rows_of(c, c["q"], c["qw"], hq, False)
        close16(q, y, f, "bf16", "q_out")
        got = cache.cpu().numpy()
        k, fk = rows_of(c, c["k"], c["kw"], hk, False)
        some = np.arange(0, T, 7)
        held = np.stack([[ko.get_row(got, int(slots[t]), h, 0, D, 16) for h in range(hk)] for t in some])
        close8(held, k[some], fk[some], "k")


def test_append_in_place_and_without_queries(gqa):
    c = append_case("f16", 128, 8, 2, 19, 5)
    cache = gqa.gqa_kv8_cache(4, 16, 2, 128)
    slots = torch.arange(19)
    want = run_append(gqa, c, slots, cache)
    qkv = c["qkv"].cuda()
    c2 = gqa.gqa_kv8_cache(4, 16, 2, 128)
    q = qkv[:, :1024]
    out = gqa.gqa_append(q, qkv[:, 1024:1280], qkv[:, 1280:], 8, 2, slots.cuda(), c2, positions=c["pos"].cuda(),
                         cos_sin=c["cs"].cuda(), q_weight=c["qw"].cuda(), k_weight=c["kw"].cuda(), eps=1e-5, q_out=q)
    assert out.data_ptr() == qkv.data_ptr() and torch.equal(out, want) and torch.equal(c2, cache)
    assert torch.equal(qkv[:, 1024:].cpu(), c["qkv"][:, 1024:])
    c3 = gqa.gqa_kv8_cache(4, 16, 2, 128)
    assert gqa.gqa_append(None, qkv[:, 1024:1280], qkv[:, 1280:], 8, 2, slots.cuda(), c3, positions=c["pos"].cuda(),
                          cos_sin=c["cs"].cuda(), k_weight=c["kw"].cuda(), eps=1e-5) is None
    assert torch.equal(c3, cache)
    empty = qkv[:0]
    assert gqa.gqa_append(empty[:, :1024], empty[:, 1024:1280], empty[:, 1280:], 8, 2, slots[:0].cuda(), c3).shape == (0, 1024)


def test_append_rows_of_any_size(gqa):
    """Zeros, the borders of a scale, the smallest and largest values, infinities and NaN."""
    D, bs = 64, 8
    big = 3.0e38
    rows = [torch.zeros(D), torch.full((D,), 448.0), torch.full((D,), 449.0), torch.full((D,), 3.5),
            torch.linspace(-1e-39, 1e-39, D), torch.linspace(-big, big, D), torch.tensor([math.inf] + [1.0] * (D - 1)),
            torch.tensor([math.nan, -2.0] + [0.5] * (D - 2)), torch.full((D,), math.nan),
            torch.tensor([448.0] + [2.0 ** -9 * (i % 5) / 2 for i in range(D - 1)]), torch.full((D,), -0.0),
            2.0 ** torch.arange(-40, 24).float()]
    x = torch.stack(rows).bfloat16()
    T = len(rows)
    cache = gqa.gqa_kv8_cache(2, bs, 1, D)
    gqa.gqa_append(None, x.cuda(), x.cuda(), 1, 1, torch.arange(T).cuda(), cache)
    want = np.zeros((2, 1, bs * (2 * D + 2)), dtype=np.uint8)
    for t in range(T):
        for w in (0, 1):
            ko.put_row(want, t, 0, w, npy(x[t]), D, bs)
    got = cache.cpu().numpy()
    nan = np.isnan(ko.code_values())
    same = (got == want) | (nan[got] & nan[want])
    assert same.all(), np.argwhere(~same)[:5]


def test_append_reports_bad_slots_and_positions(gqa):
    D, bs, hk = 128, 16, 2
    c = append_case("f16", D, 8, hk, 6, 11)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    cache = torch.full((2, hk, bs * (2 * D + 2)), 9, dtype=torch.uint8, device="cuda")
    slots = torch.tensor([0, 5, 32, -1, 31, 1 << 40])
    good = run_append(gqa, c, slots, cache, workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
    got = cache.cpu().numpy()
    rows = sorted({r for r in range(32) if (got[r // bs, 0, ko.row_offsets(r % bs, D, bs, 0)] != 9).any()})
    assert rows == [0, 5, 31]
    c["pos"] = torch.tensor([0, 50, 3, -1, 2, 49]).int()          # the table has 50 rows
    q = torch.full((6, 8 * D), 3.0, dtype=torch.float16, device="cuda")
    cache.fill_(9)
    run_append(gqa, c, torch.arange(6), cache, workspace_tensor=ws, q_out=q)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
    got = cache.cpu().numpy()
    rows = sorted({r for r in range(32) if (got[r // bs, 0, ko.row_offsets(r % bs, D, bs, 0)] != 9).any()})
    assert rows == [0, 2, 4, 5]
    assert (q[[1, 3]] == 3.0).all() and torch.equal(q[[0, 2, 4, 5]] == 3.0, torch.zeros(4, 1024, dtype=torch.bool).cuda())
    assert good.shape == (6, 8 * D)


@pytest.mark.parametrize("D,hk,bs", [(128, 8, 32), (64, 3, 8), (128, 1, 16), (64, 21, 64)])
@pytest.mark.parametrize("T,start,holes", [(1, 0, ()), (8, 8, ()), (200, 0, ()), (333, 5, ()), (97, 16, (3, 40, 41, 96)),
                                           (30, 7, (0,))])
def test_append_values_into_vllm_rows_in_order(gqa, D, hk, bs, T, start, holes):
    """Tokens of a prompt, whose slots follow one another, from an even or odd place on, with padding among them: the
    values are where the layout has them, bit for bit, and nothing else is written."""
    nb = (T + start) // bs + 2
    order = torch.randperm(nb, generator=gen(T))
    at = torch.arange(start, start + T)
    slots = order[at // bs] * bs + at % bs
    slots[list(holes)] = -1
    x = torch.randn(T, 2 * hk * D, generator=gen(T + 1)).half()
    x[0, -1] = math.nan
    k, v = torch.full((nb, hk, D // 8, bs, 8), 3.0).half().cuda(), torch.full((nb, hk, D, bs), 3.0).half().cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    xc = x.cuda()
    gqa.gqa_append(None, xc[:, :hk * D], xc[:, hk * D:], hk, hk, slots.cuda(), k, v, workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
    keep = slots >= 0
    want_k, want_v = torch.full(k.shape, 3.0).half(), torch.full(v.shape, 3.0).half()
    b, r = (slots // bs)[keep], (slots % bs)[keep]
    want_k[b, :, :, r] = x[keep, :hk * D].view(-1, hk, D // 8, 8)
    want_v[b, :, :, r] = x[keep, hk * D:].view(-1, hk, D)
    assert torch.equal(k.cpu().view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(v.cpu().view(torch.int16), want_v.view(torch.int16))


@pytest.mark.parametrize("layout,D,hq,hk,T,bs,rot,inter,norm,elem", [
    ("kv8", 128, 4, 2, 20011, 16, 128, False, True, "bf16"), ("rows", 128, 64, 8, 5003, 32, 64, False, True, "bf16"),
    ("vllm", 64, 4, 2, 20003, 8, 24, True, True, "f16"), ("kv8", 64, 3, 3, 10009, 64, 0, False, True, "f16"),
    ("rows", 128, 8, 4, 11000, 8, 24, False, False, "f16"), ("kv8", 128, 2, 1, 19999, 8, 128, True, True, "f16")])
def test_append_warps_with_several_tokens(gqa, layout, D, hq, hk, T, bs, rot, inter, norm, elem):
    """Calls with more tokens than the GPU has warps give what calls of few tokens give, bit for bit, padding and bad
    slots and positions among them; in place too."""
    c = append_case(elem, D, hq, hk, T, 400 + T, norm=norm, rot=rot)
    nb, dt, g = T // bs + 2, DT[elem], gen(T)
    slots = slots_for(T, nb, bs, 9, skip=T // 5)
    slots[torch.randperm(T, generator=g)[:20]] = nb * bs + 7
    bad = torch.randperm(T, generator=g)[:30] if rot else torch.zeros(0, dtype=torch.long)
    c["pos"][bad] = torch.tensor([50, -1, 1 << 30] * 10)[:len(bad)].int()
    part = lambda x, i: None if x is None else x[i:i + 1500]

    def caches():
        if layout == "kv8":
            return [torch.full((nb, hk, bs * (2 * D + 2)), 0x5A, dtype=torch.uint8, device="cuda")]
        if layout == "rows":
            return [torch.full((nb, bs, hk * D), 3.0, dtype=dt, device="cuda") for _ in range(2)]
        return [torch.full((nb, hk, D // 8, bs, 8), 3.0, dtype=dt, device="cuda"),
                torch.full((nb, hk, D, bs), 3.0, dtype=dt, device="cuda")]

    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want, small = torch.full((T, hq * D), 5.0, dtype=dt, device="cuda"), caches()
    for i in range(0, T, 1500):
        p = dict(c, **{n: part(c[n], i) for n in ("qkv", "pos")})
        run_append(gqa, p, slots[i:i + 1500], *small, inter=inter, q_out=want[i:i + 1500], workspace_tensor=ws)
    gqa.gqa_workspace_check(ws)
    once, whole = torch.full_like(want, 5.0), caches()
    run_append(gqa, c, slots, *whole, inter=inter, q_out=once, workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
    assert torch.equal(once, want) and all(torch.equal(a, b) for a, b in zip(whole, small))
    assert (once[bad] == 5.0).all()
    qkv, again = c["qkv"].cuda(), caches()
    n = hq * D
    gqa.gqa_append(qkv[:, :n], qkv[:, n:n + hk * D], qkv[:, n + hk * D:], hq, hk, slots.cuda(), *again,
                   positions=c["pos"].cuda(), cos_sin=cuda(c["cs"]), interleaved=inter, q_weight=cuda(c["qw"]),
                   k_weight=cuda(c["kw"]), eps=1e-5, q_out=qkv[:, :n], workspace_tensor=ws)
    keep = torch.ones(T, dtype=torch.bool)
    keep[bad] = False
    assert torch.equal(qkv[keep, :n], want[keep]) and torch.equal(qkv[:, n:].cpu(), c["qkv"][:, n:])
    assert torch.equal(qkv[bad, :n].cpu(), c["qkv"][bad, :n])
    assert all(torch.equal(a, b) for a, b in zip(again, small))


# ---------------------------------------------------------------- a cache as one finds it
def make_cache(lens, D, hk, bs, seed, spread=3, tail=True, extra=2):
    """(cache, tables) numpy: values of normal size, scales spread over 2^spread, NaN codes and 255 exponents
    in every row that no sequence owns."""
    rng = np.random.default_rng(seed)
    need = [(n + bs - 1) // bs for n in lens]
    nb, mb = sum(need) + extra, max(max(need), 1)
    perm = rng.permutation(nb)
    tab = np.full((len(lens), mb), -1, dtype=np.int32)
    cache = np.empty((nb, hk, bs * (2 * D + 2)), dtype=np.uint8)
    x = rng.standard_normal((nb, hk, 2 * bs * D)) * 96
    cache[..., :2 * bs * D] = ko.encode(x)
    cache[..., 2 * bs * D:] = rng.integers(119 - spread, 121, (nb, hk, 2 * bs))
    used = np.zeros((nb, bs), dtype=bool)
    at = 0
    for b, n in enumerate(lens):
        tab[b, :need[b]] = perm[at:at + need[b]]
        for j in range(need[b]):
            used[perm[at + j], :min(bs, n - j * bs)] = True
        at += need[b]
    if tail:
        for blk, row in np.argwhere(~used):
            for w in (0, 1):
                cache[blk][:, ko.row_offsets(row, D, bs, w)] = 0x7F
                cache[blk][:, 2 * bs * D + w * bs + row] = 0xFF
    return cache, tab


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ---------------------------------------------------------------- read
@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("D,hk,bs", [(128, 8, 16), (128, 1, 8), (64, 2, 64), (64, 3, 32), (128, 3, 64), (64, 5, 8)])
def test_read(gqa, elem, D, hk, bs):
    lens = [0, 1, bs - 1, bs, bs + 1, 100, 33]
    cache, tab = make_cache(lens, D, hk, bs, 21 + D + hk)
    for begins, n in [(None, 100), (None, 17), ([0, 0, 3, 1, bs, 90, 40], 23)]:
        k = torch.full((len(lens), n, hk * D), 5.0, dtype=DT[elem], device="cuda")
        v = k.clone()
        bt = None if begins is None else dev(np.array(begins, dtype=np.int32))
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        gqa.gqa_kv8_read(dev(cache), dev(tab), dev(np.array(lens, np.int32)), D, begins=bt, k_out=k, v_out=v,
                         workspace_tensor=ws)
        assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
        only = gqa.gqa_kv8_read(dev(cache), dev(tab), dev(np.array(lens, np.int32)), D, begins=bt,
                                v_out=torch.full_like(v, 5.0))
        assert only[0] is None and torch.equal(only[1], v)
        for b, L in enumerate(lens):
            s = 0 if begins is None else begins[b]
            m = max(0, min(n, L - s))
            want = ko.gather_kv8(cache, tab[b], L, D, bs) if L else None
            for w, got in ((0, k), (1, v)):
                if m:
                    ref = torch.from_numpy(want[w][s:s + m]).to(DT[elem]).reshape(m, -1)
                    assert torch.equal(got[b, :m].cpu(), ref), (b, w)
                assert (got[b, m:] == 5.0).all()


def test_read_defaults_and_reports(gqa):
    lens = [20, 40]
    cache, tab = make_cache(lens, 64, 2, 16, 30)
    k, v = gqa.gqa_kv8_read(dev(cache), dev(tab), dev(np.array(lens, np.int32)), 64, 64)
    assert k.dtype == torch.float16 and k.shape == (2, 64, 128) and (k[0, 20:] == 0).all()
    assert torch.equal(k[1, :40].cpu(), torch.from_numpy(ko.gather_kv8(cache, tab[1], 40, 64, 16)[0]).half().view(40, -1))
    with pytest.raises(ValueError):
        gqa.gqa_kv8_read(dev(cache), dev(tab), dev(np.array(lens, np.int32)), 64)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    bad = tab.copy()
    bad[0, 1] = cache.shape[0]
    out = torch.full((2, 64, 128), 5.0, dtype=torch.float16, device="cuda")
    gqa.gqa_kv8_read(dev(cache), dev(bad), dev(np.array(lens, np.int32)), 64, k_out=out, workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
    assert torch.equal(out[0, :16], k[0, :16]) and (out[0, 16:] == 5.0).all() and torch.equal(out[1, :40], k[1, :40])
    for ln, bg in [([-1, 40], None), ([20, 1000], None), ([20, 40], [0, -3])]:
        out.fill_(5.0)
        gqa.gqa_kv8_read(dev(cache), dev(tab), dev(np.array(ln, np.int32)), 64, k_out=out, workspace_tensor=ws,
                         begins=None if bg is None else dev(np.array(bg, np.int32)))
        assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG


def test_read_into_outputs_on_16_byte_borders(gqa):
    """Outputs whose addresses are multiples of 16 bytes, but not of 32."""
    D, hk, bs, n = 128, 3, 16, 50
    cache, tab = make_cache([n, 20], D, hk, bs, 31)
    big = torch.full((2, 2 * n * hk * D + 8), 5.0, dtype=torch.float16, device="cuda")
    k, v = (x[8:].view(2, n, hk * D) for x in big)
    assert k.data_ptr() % 32 == 16
    gqa.gqa_kv8_read(dev(cache), dev(tab), dev(np.array([n, 20], np.int32)), D, k_out=k, v_out=v)
    wk, wv = gqa.gqa_kv8_read(dev(cache), dev(tab), dev(np.array([n, 20], np.int32)), D, n)
    assert torch.equal(k[0], wk[0]) and torch.equal(v[0], wv[0]) and torch.equal(v[1, :20], wv[1, :20])
    assert (big[:, :8] == 5.0).all() and (k[1, 20:] == 5.0).all()


# ---------------------------------------------------------------- decode
def check_decode(o, cache, tab, lens, q, hq, hk, D, scale, bs, causal, elem, where):
    ref, a, l, top = ko.decode_kv8(npy(q).reshape(len(lens), -1, hq * D), cache, tab, lens, hq, hk, D, scale, bs, causal)
    o = o.double().cpu().reshape(ref.shape)
    n = torch.tensor([max(int(x), 0) for x in lens], dtype=torch.float64)
    low = (n * 2.0 ** -25 * 2 * top)[:, None, None] / l.clamp(min=1.0)
    tol = U[elem] * ref.abs() + 2 * 2.0 ** -11 * a + low.repeat_interleave(D, -1) + TINY[elem]
    err = (o - ref).abs()
    assert torch.isfinite(o).all(), where
    assert not (err > tol).any(), f"{where}: {int((err > tol).sum())} out, worst {float((err - tol).max()):.3e}"
    none = (l == 0).repeat_interleave(D, -1)
    assert (o[none] == 0).all(), where


def run_decode(gqa, cache, tab, lens, q, hq, hk, **kw):
    o = gqa.gqa_decode_kv8(q.cuda(), dev(cache), dev(tab), dev(np.asarray(lens, np.int32)), hq, hk, **kw)
    torch.cuda.synchronize()
    return o


def edge_lens(bs):
    return [0, 1, 2, 31, 32, 33, bs - 1, bs, bs + 1, 64, 65, 127, 129, 511, 700, 0, 1025]


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("D,hq,hk,T,causal", [(128, 32, 8, 1, False), (64, 8, 2, 1, False), (128, 2, 2, 1, True),
                                              (128, 7, 1, 2, True), (64, 6, 2, 5, True), (64, 64, 2, 1, False),
                                              (128, 64, 1, 1, False), (128, 16, 2, 8, True), (64, 24, 1, 2, False),
                                              (128, 40, 1, 1, False)])
def test_decode_edges(gqa, elem, bs, D, hq, hk, T, causal):
    lens = edge_lens(bs)
    cache, tab = make_cache(lens, D, hk, bs, 40 + bs + hq)
    q = torch.randn(len(lens), T, hq * D, generator=gen(bs + hq + T)).to(DT[elem])
    ws = torch.zeros(gqa.gqa_decode_kv8_workspace_size(len(lens), T, hq, hk, D), dtype=torch.uint8, device="cuda")
    o = run_decode(gqa, cache, tab, lens, q, hq, hk, causal=causal, workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
    check_decode(o, cache, tab, lens, q, hq, hk, D, D ** -0.5, bs, causal, elem, f"bs {bs}")


@pytest.mark.parametrize("lens", [[1], [9000], [5000, 3, 8191], [200] * 40])
@pytest.mark.parametrize("hq,hk,D", [(4, 1, 128), (16, 2, 64), (32, 1, 128)])
def test_decode_split_over_long_sequences(gqa, lens, hq, hk, D):
    cache, tab = make_cache(lens, D, hk, 16, 50 + hq)
    q = torch.randn(len(lens), hq * D, generator=gen(9)).to(torch.float16)
    o = run_decode(gqa, cache, tab, lens, q, hq, hk)
    assert o.shape == q.shape
    check_decode(o, cache, tab, lens, q, hq, hk, D, D ** -0.5, 16, False, "f16", f"{lens[:3]}")
    again = run_decode(gqa, cache, tab, lens, q, hq, hk)
    assert torch.equal(o, again)


def test_decode_more_sequences_than_one_launch_takes(gqa):
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 40, 2500).tolist()
    cache, tab = make_cache(lens, 64, 1, 8, 60, tail=False)
    q = torch.randn(2500, 2 * 64, generator=gen(10)).to(torch.bfloat16)
    o = run_decode(gqa, cache, tab, lens, q, 2, 1)
    check_decode(o, cache, tab, lens, q, 2, 1, 64, 0.125, 8, False, "bf16", "2500 sequences")


@pytest.mark.parametrize("elem", ["f16", "bf16"])
def test_decode_scales_far_apart(gqa, elem):
    """V rows of very different size, growing and shrinking along the sequence; K rows that dominate; queries
    of any size in bf16."""
    D, hk, bs, n = 128, 2, 16, 1500
    cache, tab = make_cache([n, n, n], D, hk, bs, 70, spread=0)
    ex = 2 * bs * D
    for b in range(3):
        for j in range(n):
            kv = {0: 100 + 30 * j // n, 1: 130 - 30 * j // n, 2: 127 - (j % 23)}[b]
            cache[tab[b, j // bs], :, ex + bs + j % bs] = kv
    for b, j in ((0, 1200), (1, 40), (2, 777)):                    # one key far above the others
        cache[tab[b, j // bs], :, ex + j % bs] = 123
    q = torch.randn(3, 8 * D, generator=gen(12))
    if elem == "bf16":
        q = q * torch.tensor([1e-20, 1.0, 300.0])[:, None]
    q = q.to(DT[elem])
    for scale in (D ** -0.5, 0.5, 0.0):
        o = run_decode(gqa, cache, tab, [n] * 3, q, 8, hk, scale=scale / (300 if elem == "bf16" else 1))
        check_decode(o, cache, tab, [n] * 3, q, 8, hk, D, scale / (300 if elem == "bf16" else 1), bs, False, elem,
                     f"scale {scale}")


def test_decode_one_key_far_away_takes_everything(gqa):
    """A key whose score is above every other by far more than fp32 holds returns its value."""
    D, bs, n = 64, 16, 3000
    cache, tab = make_cache([n], D, 1, bs, 80)
    q = torch.ones(1, 4 * D).half()
    for j in (0, 31, 32, 1777, 2999):
        c = cache.copy()
        off = ko.row_offsets(j % bs, D, bs, 0)
        c[tab[0, j // bs], 0, off] = 0x7E                          # 448 everywhere
        c[tab[0, j // bs], 0, 2 * bs * D + j % bs] = 127
        o = run_decode(gqa, c, tab, [n], q, 4, 1)
        v = torch.from_numpy(ko.get_row(c, int(tab[0, j // bs]) * bs + j % bs, 0, 1, D, bs))
        assert torch.equal(o.view(4, D).cpu(), v.half().expand(4, D)), j


def test_f16_outputs_are_as_exact_as_their_rounding(gqa):
    """With the weights in two f16 numbers the error of an f16 output is its own rounding: relative L2 at most 1.2 of
    what rounding the oracle's result to f16 gives (weights in one f16 number: about 1.4)."""
    for D, hq, hk, bs, T in [(128, 32, 8, 16, 1), (64, 8, 2, 16, 1), (128, 16, 1, 32, 2)]:
        lens = [900, 400, 1300]
        cache, tab = make_cache(lens, D, hk, bs, 95)
        q = torch.randn(3, T, hq * D, generator=gen(14)).half()
        o = run_decode(gqa, cache, tab, lens, q, hq, hk)
        ref = ko.decode_kv8(npy(q), cache, tab, lens, hq, hk, D, D ** -0.5, bs)[0]
        own = float((o.double().cpu() - ref).norm() / ref.norm())
        least = float((ref.half().double() - ref).norm() / ref.norm())
        assert own <= 1.2 * least, (own, least)


def test_not_a_number_stays_in_its_row(gqa):
    """A NaN query spoils its own row, a NaN value its column for the heads that share it, an infinite query its
    row; nothing else changes."""
    D, hq, hk, bs, n = 128, 8, 2, 16, 500
    cache, tab = make_cache([n], D, hk, bs, 96)
    q = torch.randn(1, hq * D, generator=gen(15)).half()
    want = run_decode(gqa, cache, tab, [n], q, hq, hk).view(hq, D)
    bad = q.clone()
    bad[0, 3 * D + 5] = math.nan
    bad[0, 6 * D + 9] = math.inf
    o = run_decode(gqa, cache, tab, [n], bad, hq, hk).view(hq, D)
    assert o[[3, 6]].isnan().all()
    keep = [0, 1, 2, 4, 5, 7]
    assert torch.equal(o[keep], want[keep])
    c = cache.copy()
    j, col = 333, 77
    c[tab[0, j // bs], 1, ko.row_offsets(j % bs, D, bs, 1)[col]] = 0x7F
    o = run_decode(gqa, c, tab, [n], q, hq, hk).view(hq, D)
    assert o[4:, col].isnan().all()
    o[4:, col] = want[4:, col]
    assert torch.equal(o, want)


def test_one_call_shapes_on_one_workspace(gqa):
    """The cached workspace grows and serves calls of other shapes, in any order."""
    cases = []
    for i, (hq, hk, D, lens) in enumerate([(4, 2, 64, [70]), (64, 1, 128, [900, 33]), (32, 8, 128, [1200] * 5),
                                           (2, 2, 64, [31] * 30)]):
        cache, tab = make_cache(lens, D, hk, 16, 150 + i)
        q = torch.randn(len(lens), hq * D, generator=gen(70 + i)).half()
        cases.append((cache, tab, lens, q, hq, hk))
    s = torch.cuda.Stream()
    want = None
    for _ in range(2):
        got = []
        for cache, tab, lens, q, hq, hk in cases + cases[::-1]:
            x = q.cuda(), dev(cache), dev(tab), dev(np.array(lens, np.int32))
            torch.cuda.synchronize()
            got.append(gqa.gqa_decode_kv8(*x, hq, hk, stream=s))
            torch.cuda.synchronize()
        assert want is None or all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(got[:4], got[:3:-1]))
        want = got
    for (cache, tab, lens, q, hq, hk), o in zip(cases, want):
        D = q.shape[1] // hq
        check_decode(o, cache, tab, lens, q, hq, hk, D, D ** -0.5, 16, False, "f16", f"{hq}")


def test_decode_shared_blocks(gqa):
    """Sequences that share their prefix's blocks."""
    D, bs, hk = 128, 16, 2
    cache, tab = make_cache([96, 40], D, hk, bs, 90)
    t = np.stack([tab[0], tab[0]])
    t[1, 4:] = tab[1, :2]
    lens = [96, 80]
    cache[tab[1, 0]] = cache[tab[0, 1]]
    q = torch.randn(2, 8 * D, generator=gen(13)).half()
    o = run_decode(gqa, cache, t, lens, q, 8, hk)
    check_decode(o, cache, t, lens, q, 8, hk, D, D ** -0.5, bs, False, "f16", "shared")


def test_decode_reports_bad_blocks_and_lengths(gqa):
    D, bs, hk = 64, 16, 2
    lens = [100, 40, 70]
    cache, tab = make_cache(lens, D, hk, bs, 100)
    q = torch.randn(3, 8 * D, generator=gen(14)).half()
    ws = torch.zeros(gqa.gqa_decode_kv8_workspace_size(3, 1, 8, hk, D), dtype=torch.uint8, device="cuda")
    for what in ("id", "negative id", "long", "negative length"):
        t, ln = tab.copy(), list(lens)
        if what == "id":
            t[1, 1] = cache.shape[0]
        elif what == "negative id":
            t[1, 2] = -7
        else:
            ln[1] = 10 ** 6 if what == "long" else -5
        if what == "long":
            t[1] = t[0]
        o = run_decode(gqa, cache, t, ln, q, 8, hk, workspace_tensor=ws)
        assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG, what
        ok = [0, 2]
        check_decode(o[ok], cache, t[ok], [lens[i] for i in ok], q[ok], 8, hk, D, D ** -0.5, bs, False, "f16", what)
        if what == "negative length":
            assert (o[1] == 0).all()
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK


@pytest.mark.parametrize("hq,worker", [(16, 3), (64, 1), (256, 0)])
def test_decode_timeout_is_reported_not_hung(gqa, hq, worker):
    """A worker whose second tile never comes (one warp, two and four warps on a ring)."""
    D, hk, bs = 128, 4, 16
    lens = [4000] * 8
    cache, tab = make_cache(lens, D, hk, bs, 105)
    q = torch.randn(8, hq * D, generator=gen(15)).half()
    ws = torch.zeros(gqa.gqa_decode_kv8_workspace_size(8, 1, hq, hk, D), dtype=torch.uint8, device="cuda")
    run_decode(gqa, cache, tab, lens, q, hq, hk, workspace_tensor=ws, timeout_us=20000, test_stall_cta=worker)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_TIMEOUT
    o = run_decode(gqa, cache, tab, lens, q, hq, hk, workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
    check_decode(o[:2], cache, tab[:2], lens[:2], q[:2], hq, hk, D, D ** -0.5, bs, False, "f16", "after a timeout")


# ---------------------------------------------------------------- short units: one launch of clusters
# The table's width decides: the short form leaves the workspace behind its header alone, the other one notes its cut
# units there.
SHORT = [  # D, hq, hk, T, bs, sequences, blocks of the table -> CTAs of a unit, tiles of a worker
    (128, 16, 8, 1, 32, 16, 64),     # 1, 8
    (64, 16, 8, 1, 64, 16, 32),      # 1, 8
    (128, 8, 8, 1, 32, 18, 8),       # 1, 1
    (128, 32, 4, 1, 16, 10, 32),     # 2, 1
    (64, 60, 5, 1, 8, 4, 125),       # 4, 1
    (64, 8, 2, 1, 16, 1, 256),       # 8, 2
    (128, 8, 1, 4, 8, 5, 520),       # 8, 3, 32 rows
    (128, 16, 4, 12, 16, 8, 80),     # 2, 5, two warps on a ring of four
    (64, 80, 2, 1, 32, 12, 72),      # 4, 5: two warps on a ring of eight
    (64, 64, 1, 1, 8, 3, 21),        # 2, 1: the last CTA has part of its workers
    (128, 24, 2, 2, 16, 6, 100),     # 8, 1, 24 rows
    (64, 7, 1, 3, 32, 20, 60),       # 4, 2, 21 rows
    (128, 40, 1, 1, 16, 9, 64),      # 8, 1, 40 rows
    (64, 48, 2, 2, 8, 8, 240),       # 4, 4, 48 rows, a ring of two warps goes round
]


def short_case(D, hq, hk, T, bs, N, blocks, seed):
    full = blocks * bs
    lens = ([full, 0, 1, full - 1, 33, full // 2 + 5, 64, full - 33, 32, full // 3] * 2)[:N]
    cache, tab = make_cache(lens, D, hk, bs, seed)
    tab = np.ascontiguousarray(np.pad(tab, ((0, 0), (0, blocks)))[:, :blocks])
    return cache, tab, lens, torch.randn(N, T, hq * D, generator=gen(seed)).half()


def wide(tab, bs, keys=20000):
    """The same table, with room for more keys than the short form takes."""
    return np.ascontiguousarray(np.pad(tab, ((0, 0), (0, keys // bs - tab.shape[1]))))


def marked(gqa, N, T, hq, hk, D):
    ws = torch.full((gqa.gqa_decode_kv8_workspace_size(N, T, hq, hk, D),), 0xA5, dtype=torch.uint8, device="cuda")
    ws[:256] = 0
    return ws


def untouched(ws):
    return bool((ws[256:] == 0xA5).all())


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D,hq,hk,T,bs,N,blocks", SHORT)
def test_decode_of_short_units_in_one_launch(gqa, D, hq, hk, T, bs, N, blocks, causal):
    cache, tab, lens, q = short_case(D, hq, hk, T, bs, N, blocks, 160 + hq + T)
    for t, short in ((tab, True), (wide(tab, bs), False)):
        ws = marked(gqa, N, T, hq, hk, D)
        o = run_decode(gqa, cache, t, lens, q, hq, hk, causal=causal, workspace_tensor=ws)
        assert untouched(ws) == short
        assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
        check_decode(o, cache, t, lens, q, hq, hk, D, D ** -0.5, bs, causal, "f16", f"short {short}")
        assert torch.equal(o, run_decode(gqa, cache, t, lens, q, hq, hk, causal=causal, workspace_tensor=ws))


@pytest.mark.parametrize("D,hq,hk,T,bs,N,blocks,worker", [(128, 16, 8, 1, 32, 16, 64, 3), (128, 16, 4, 12, 16, 8, 80, 1),
                                                          (64, 8, 2, 1, 16, 1, 256, 9)])
def test_timeout_of_short_units(gqa, D, hq, hk, T, bs, N, blocks, worker):
    """A worker whose second tile never comes: alone in its CTA, with two warps on a ring, in a cluster."""
    cache, tab, lens, q = short_case(D, hq, hk, T, bs, N, blocks, 170)
    ws = marked(gqa, N, T, hq, hk, D)
    run_decode(gqa, cache, tab, lens, q, hq, hk, workspace_tensor=ws, timeout_us=20000, test_stall_cta=worker)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_TIMEOUT
    o = run_decode(gqa, cache, tab, lens, q, hq, hk, workspace_tensor=ws)
    assert untouched(ws) and gqa.gqa_workspace_check(ws) == gqa.GQA_OK
    check_decode(o, cache, tab, lens, q, hq, hk, D, D ** -0.5, bs, False, "f16", "after a timeout")


@pytest.mark.parametrize("short", [True, False])
def test_both_forms_keep_not_a_number_in_its_row_and_report(gqa, short):
    D, hq, hk, bs = 128, 8, 2, 16
    lens = [700, 300]
    cache, tab = make_cache(lens, D, hk, bs, 97)
    tab = tab if short else wide(tab, bs)
    q = torch.randn(2, hq * D, generator=gen(16)).half()
    ws = marked(gqa, 2, 1, hq, hk, D)
    want = run_decode(gqa, cache, tab, lens, q, hq, hk, workspace_tensor=ws)
    assert untouched(ws) == short
    bad = q.clone()
    bad[0, 3 * D + 5] = math.nan
    bad[1, 6 * D + 9] = math.inf
    c = cache.copy()
    j, col = 650, 77
    c[tab[0, j // bs], 1, ko.row_offsets(j % bs, D, bs, 1)[col]] = 0x7F
    o = run_decode(gqa, c, tab, lens, bad, hq, hk).view(2, hq, D)
    assert o[0, 3].isnan().all() and o[1, 6].isnan().all() and o[0, 4:, col].isnan().all()
    w = want.view(2, hq, D).clone()
    w[0, 3], w[1, 6], w[0, 4:, col] = o[0, 3], o[1, 6], o[0, 4:, col]
    assert torch.equal(o.nan_to_num(9.0), w.nan_to_num(9.0))
    for at, what in (((1, 2), cache.shape[0]), ((1, 3), -1)):
        t = tab.copy()
        t[at] = what
        o = run_decode(gqa, cache, t, lens, q, hq, hk, workspace_tensor=ws)
        assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
        assert torch.equal(o[0], want[0])
    for n in (10 ** 6, -3):
        o = run_decode(gqa, cache, tab, [700, n] if n < 0 else [n, 300], q, hq, hk, workspace_tensor=ws)
        assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
        i = 0 if n < 0 else 1
        check_decode(o[i:i + 1], cache, tab[i:i + 1], lens[i:i + 1], q[i:i + 1], hq, hk, D, D ** -0.5, bs, False, "f16",
                     f"length {n}")
        assert n > 0 or (o[1] == 0).all()


def test_short_units_replayed_with_other_lengths(gqa):
    """A captured call of clusters follows the lengths, ids and queries that its tensors hold at the replay."""
    D, hq, hk, T, bs, N, blocks = SHORT[5]
    cache, tab, _, q = short_case(*SHORT[5], 180)
    x = [q.cuda(), dev(cache), dev(tab), dev(np.array([blocks * bs], np.int32))]
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(x[0])
    with torch.cuda.stream(s):
        gqa.gqa_decode_kv8(*x, hq, hk, out=out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        gqa.gqa_decode_kv8(*x, hq, hk, out=out)
    for n in (blocks * bs, 0, 1, 777, 4000):
        x[0].copy_(torch.randn(q.shape, generator=gen(n)).half())
        x[3].fill_(n)
        out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        check_decode(out, cache, tab, [n], x[0].cpu(), hq, hk, D, D ** -0.5, bs, False, "f16", f"{n} keys")


def test_bounds_checked_build_of_both_forms(gqa):
    from decode_attention_03_gb300 import build
    lib = gqa.open_library(build.build(checked=True))
    raw = torch.cuda.current_stream().cuda_stream
    for i, (D, hq, hk, T, bs, N, blocks) in enumerate(SHORT):
        cache, tab, lens, q = short_case(D, hq, hk, T, bs, N, blocks, 190 + i)
        for t, short in ((tab, True), (wide(tab, bs), False)):
            ws = marked(gqa, N, T, hq, hk, D)
            x = [q.cuda(), dev(cache), dev(t), dev(np.array(lens, np.int32))]
            o = torch.full_like(x[0], math.nan)
            assert lib.gqa_decode_kv8(*(y.data_ptr() for y in x), o.data_ptr(), N, T, t.shape[1], cache.shape[0], bs, hq,
                                      hk, D, D ** -0.5, ws.data_ptr(), ws.numel(), raw, None) == 0
            assert untouched(ws) == short
            assert lib.gqa_workspace_check(ws.data_ptr(), raw) == 0
            check_decode(o, cache, t, lens, q, hq, hk, D, D ** -0.5, bs, False, "f16", f"{SHORT[i]} {short}")


def test_timeout_before_a_unit_that_nobody_notes(gqa):
    """The last worker, which has the end of a long sequence and a sequence of one tile, gives up before the latter; the
    workspace holds anything at all behind its header, and the merge reads nothing outside of it."""
    D, hq, hk, bs = 128, 4, 1, 16
    lens = [100000, 5]
    tiles = sum((n + 31) // 32 for n in lens)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    share = -(-tiles // (8 * sms))
    last = (tiles - 1) // share
    assert tiles - last * share == 3                         # two tiles of the long one, then the short one's
    cache, tab = make_cache(lens, D, hk, bs, 106, tail=False)
    q = torch.randn(2, hq * D, generator=gen(16)).half()
    for junk in (0x5A, 0xFF, 0x7F, 0x00, 0x80):
        ws = torch.full((gqa.gqa_decode_kv8_workspace_size(2, 1, hq, hk, D),), junk, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        run_decode(gqa, cache, tab, lens, q, hq, hk, workspace_tensor=ws, timeout_us=20000, test_stall_cta=last)
        assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_TIMEOUT
        o = run_decode(gqa, cache, tab, lens, q, hq, hk, workspace_tensor=ws)
        assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
    check_decode(o, cache, tab, lens, q, hq, hk, D, D ** -0.5, bs, False, "f16", "after a timeout")


def test_offsets_past_32_bits(gqa):
    """Blocks behind the first 4 GiB of a cache, written, attended to and read back."""
    D, hk, bs, hq = 128, 8, 64, 32
    nb = (5 << 30) // (hk * bs * 258)
    cache = torch.empty(nb, hk, bs * 258, dtype=torch.uint8, device="cuda")
    ids = [nb - 1, 3, nb - 2]
    n = 3 * bs - 5
    c = append_case("bf16", D, hq, hk, n, 15)
    slots = torch.tensor([ids[j // bs] * bs + j % bs for j in range(n)])
    q = run_append(gqa, c, slots, cache)[-1:].contiguous()
    tab = torch.tensor([ids], dtype=torch.int32, device="cuda")
    small = cache[ids].cpu().numpy()
    st = np.arange(3, dtype=np.int32)[None]
    k, fk = rows_of(c, c["k"], c["kw"], hk, False)
    got, gv = ko.gather_kv8(small, st[0], n, D, bs)
    close8(got, k, fk, "k")
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    o = gqa.gqa_decode_kv8(q, cache, tab, ln, hq, hk)
    check_decode(o, small, st, [n], q, hq, hk, D, D ** -0.5, bs, False, "bf16", "past 4 GiB")
    kr, vr = gqa.gqa_kv8_read(cache, tab, ln, D, n, dtype=torch.bfloat16)
    assert torch.equal(kr[0].cpu(), torch.from_numpy(got).bfloat16().view(n, -1))
    assert torch.equal(vr[0].cpu(), torch.from_numpy(gv).bfloat16().view(n, -1))
    del cache
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("elem", ["f16", "bf16"])
def test_prompt_then_steps_then_verification(gqa, elem):
    """Prompts of different length enter the cache in padded chunks, single tokens follow, then 3 speculated
    tokens are verified; every attention against the oracle on the cache's bytes and, through the read-back,
    against gqa_decode."""
    D, hq, hk, bs = 128, 16, 4, 16
    prompts = [70, 5, 33]
    N, mb = 3, 8
    cache = gqa.gqa_kv8_cache(N * mb, bs, hk, D)
    tab = torch.randperm(N * mb, generator=gen(16)).view(N, mb).int()
    kept = [[] for _ in range(N)]

    def tokens(rows):
        """rows: (sequence or -1, position) of every token of a call."""
        c = append_case(elem, D, hq, hk, len(rows), 17 + sum(map(len, kept)) + len(rows), max_pos=mb * bs)
        c["pos"] = torch.tensor([max(p, 0) for _, p in rows]).int()
        slots = torch.tensor([int(tab[b, p // bs]) * bs + p % bs if b >= 0 else -1 for b, p in rows])
        out = run_append(gqa, c, slots, cache)
        k, fk = rows_of(c, c["k"], c["kw"], hk, False)
        for i, (b, _) in enumerate(rows):
            if b >= 0:
                kept[b].append((k[i], fk[i], npy(c["v"])[i].reshape(hk, D)))
        return out

    tokens([(b, p) if p < n else (-1, 0) for b, n in enumerate(prompts) for p in range(max(prompts))])
    lens = list(prompts)
    for new in (1, 1, 3):
        q = tokens([(b, lens[b] + i) for b in range(N) for i in range(new)]).view(N, new, -1)
        lens = [n + new for n in lens]
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        o = gqa.gqa_decode_kv8(q, cache, tab.cuda(), ln, hq, hk, causal=True)
        host = cache.cpu().numpy()
        check_decode(o, host, tab.numpy(), lens, q, hq, hk, D, D ** -0.5, bs, True, elem, f"{new} new")
    for b in range(N):
        k, v = ko.gather_kv8(host, tab[b].numpy(), lens[b], D, bs)
        close8(k, np.stack([x[0] for x in kept[b]]), np.stack([x[1] for x in kept[b]]), "k")
        close8(v, np.stack([x[2] for x in kept[b]]), 0 * v, "v")
    k, v = gqa.gqa_kv8_read(cache, tab.cuda(), ln, D, max(lens), dtype=DT[elem])
    for b in range(N):
        n = lens[b]
        o16 = gqa.gqa_decode(q[b:b + 1].contiguous(), k[b:b + 1, :n].contiguous(), v[b:b + 1, :n].contiguous(), hq, hk,
                             causal=True)
        torch.testing.assert_close(o16[0].float(), o[b].float(), rtol=4 * U[elem], atol=8e-3)


def test_append_into_the_16_bit_caches_then_decode(gqa):
    """What gqa_append writes is what gqa_decode_paged and gqa_decode_paged_vllm read."""
    D, hq, hk, bs, n = 128, 16, 4, 16, 150
    c = append_case("f16", D, hq, hk, n, 18, max_pos=n)
    c["pos"] = torch.arange(n).int()
    nb = 12
    tab = torch.randperm(nb, generator=gen(19))[:10].int()
    slots = tab.long()[torch.arange(n) // bs] * bs + torch.arange(n) % bs
    rows = [torch.zeros(nb, bs, hk * D, dtype=torch.float16, device="cuda") for _ in range(2)]
    vllm = [torch.zeros(nb, hk, D // 8, bs, 8, dtype=torch.float16, device="cuda"),
            torch.zeros(nb, hk, D, bs, dtype=torch.float16, device="cuda")]
    q = run_append(gqa, c, slots, *rows)[-1:].contiguous()
    run_append(gqa, c, slots, *vllm)
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    o1 = gqa.gqa_decode_paged(q, *rows, tab[None].cuda(), ln, hq, hk, max_seq_len=n, head_group=4)
    o2 = gqa.gqa_decode_paged_vllm(q, *vllm, tab[None].cuda(), ln, hq, hk, max_seq_len=n, head_group=4)
    assert torch.equal(o1, o2)
    k = rows_of(c, c["k"], c["kw"], hk, False)[0]
    y = rows_of(c, c["q"], c["qw"], hq, False)[0][-1]
    v = npy(c["v"]).reshape(n, hk, D)
    for h in range(hq):
        s = k[:, h // 4] @ y[h] / math.sqrt(D)
        p = np.exp(s - s.max())
        np.testing.assert_allclose(npy(o1)[0, h * D:(h + 1) * D], p @ v[:, h // 4] / p.sum(), atol=6e-3)


# ---------------------------------------------------------------- graphs, streams, arguments
def test_graphs_replay_and_do_not_share(gqa):
    """Two graphs captured one after the other hold workspaces of their own: replayed side by side on two
    streams they give what the eager calls give; a replay sees the inputs as they are then."""
    D, hq, hk, bs = 128, 16, 4, 16
    lens = [900, 65, 3000]
    cache, tab = make_cache(lens, D, hk, bs, 110)
    cache, tab, ln = dev(cache), dev(tab), dev(np.array(lens, np.int32))
    q = [torch.randn(3, hq * D, generator=gen(20 + i)).half().cuda() for i in range(2)]
    x = [torch.randn(3, 2 * hk * D, generator=gen(30 + i)).half().cuda() for i in range(2)]
    caches = [cache.clone() for _ in range(2)]
    slots = torch.stack([tab[b, (n - 1) // bs].long() * bs + (n - 1) % bs for b, n in enumerate(lens)])

    def step(i, qq):
        gqa.gqa_append(None, x[i][:, :hk * D], x[i][:, hk * D:], hq, hk, slots, caches[i])
        o = gqa.gqa_decode_kv8(qq, caches[i], tab, ln, hq, hk)
        k, v = gqa.gqa_kv8_read(caches[i], tab, ln, D, 64)
        return o, k, v

    want = [[t.clone() for t in step(i, q[i])] for i in range(2)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(i, q[i]))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        caches[i].copy_(cache)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, w) for a, w in zip(outs[i], want[i])), i
    q[0].copy_(q[1])
    x[0].copy_(x[1])
    torch.cuda.synchronize()
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, w) for a, w in zip(outs[0], want[1]))


def test_other_streams(gqa):
    """Calls on a stream given by argument, several at once."""
    D, hq, hk, bs = 64, 8, 2, 16
    lens = [400, 1000]
    cache, tab = make_cache(lens, D, hk, bs, 120)
    cache, tab, ln = dev(cache), dev(tab), dev(np.array(lens, np.int32))
    q = [torch.randn(2, hq * D, generator=gen(40 + i)).half().cuda() for i in range(4)]
    want = [gqa.gqa_decode_kv8(x, cache, tab, ln, hq, hk) for x in q]
    wk, wv = gqa.gqa_kv8_read(cache, tab, ln, D, 1000)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for _ in range(5):
        for i, s in enumerate(streams):
            handle = s if i % 2 else s.cuda_stream
            got.append((i, gqa.gqa_decode_kv8(q[i], cache, tab, ln, hq, hk, stream=handle)))
            k, v = gqa.gqa_kv8_read(cache, tab, ln, D, 1000, stream=handle)
            got.append((None, (k, v)))
    torch.cuda.synchronize()
    for i, o in got:
        assert torch.equal(o, want[i]) if i is not None else torch.equal(o[0], wk) and torch.equal(o[1], wv)


def test_other_calls_on_the_same_stream_keep_their_counters(gqa):
    """gqa_decode folding in its last CTA counts arrivals in its workspace: a gqa_decode_kv8 in between
    must not leave anything there."""
    D, hq, hk, bs = 128, 8, 2, 16
    lens = [3000, 50, 700]
    cache, tab = make_cache(lens, D, hk, bs, 140)
    q = torch.randn(3, hq * D, generator=gen(60)).half().cuda()
    k = torch.randn(3, 4000, hk * D, generator=gen(61)).half().cuda()
    v = torch.randn(3, 4000, hk * D, generator=gen(62)).half().cuda()
    want = gqa.gqa_decode(q[:, None], k, v, hq, hk, n_splits=9, merge_mode=1)
    x = dev(cache), dev(tab), dev(np.array(lens, np.int32))
    first = gqa.gqa_decode_kv8(q, *x, hq, hk)
    for _ in range(3):
        assert torch.equal(gqa.gqa_decode_kv8(q, *x, hq, hk), first)
        o = gqa.gqa_decode(q[:, None], k, v, hq, hk, n_splits=9, merge_mode=2)
        torch.testing.assert_close(o, want, rtol=2e-3, atol=1e-4)
    o = gqa.gqa_decode_kv8(q, *x, hq, hk)
    assert torch.equal(o, first)
    check_decode(o, cache, tab, lens, q.cpu(), hq, hk, D, D ** -0.5, bs, False, "f16", "after gqa_decode")


def test_status_of_calls_without_a_workspace(gqa):
    """The status word of the stream's own small workspace, eager and replayed; larger workspaces do not move it."""
    D, hk = 64, 2
    x = torch.randn(3, hk * D, generator=gen(60)).half().cuda()
    cache, slots = gqa.gqa_kv8_cache(2, 16, hk, D), torch.tensor([0, 5, 31]).cuda()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        gqa.gqa_append(None, x, x, 0, hk, slots, cache)
        status = gqa.workspace(256, use="status")
        assert gqa.gqa_workspace_check(status) == gqa.GQA_OK
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            gqa.gqa_append(None, x, x, 0, hk, slots, cache)
        gqa.workspace(1 << 22)
        graph.replay()
        assert gqa.gqa_workspace_check(status) == gqa.GQA_OK
        slots[1] = 32
        graph.replay()
        assert gqa.workspace(256, use="status") is status
        assert gqa.gqa_workspace_check(status) == gqa.GQA_ERR_INVALID_ARG
        table = torch.tensor([[0, 7]], dtype=torch.int32, device="cuda")
        gqa.gqa_kv8_read(cache, table, torch.tensor([20], dtype=torch.int32, device="cuda"), D, 20)
        assert gqa.gqa_workspace_check(status) == gqa.GQA_ERR_INVALID_ARG


def test_binding_checks(gqa):
    D, hq, hk, bs = 64, 8, 2, 16
    cache = gqa.gqa_kv8_cache(4, bs, hk, D)
    x = torch.zeros(3, (hq + 2 * hk) * D, dtype=torch.float16, device="cuda")
    q, k, v = x[:, :512], x[:, 512:640], x[:, 640:]
    s = torch.arange(3, device="cuda")
    pos, cs = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(4, 64, device="cuda")
    gqa.gqa_append(q, k, v, hq, hk, s, cache, positions=pos, cos_sin=cs)
    pool = torch.zeros(4, bs, hk * D, dtype=torch.float16, device="cuda")
    for args, kw in [((q, k, v[:2], hq, hk, s, cache), {}), ((q.bfloat16(), k, v, hq, hk, s, cache), {}),
                     ((q, k, v, hq, hk, s.int(), cache), {}), ((q, k, v, hq, hk, s[:2], cache), {}),
                     ((q, k, v, hq, hk, s, cache, pool), {}), ((q, k, v, hq, hk, s, pool), {}),
                     ((q, k, v, hq, hk, s, pool, pool[:3]), {}), ((q, k, v, hq, hk, s, cache[:, :, :-1]), {}),
                     ((q, k, v, hq, hk, s, cache), dict(cos_sin=cs)),
                     ((q, k, v, hq, hk, s, cache), dict(cos_sin=cs.half(), positions=pos)),
                     ((q, k, v, hq, hk, s, cache), dict(cos_sin=cs, positions=pos.long())),
                     ((q, k, v, hq, hk, s, cache), dict(q_weight=torch.zeros(32, dtype=torch.float16, device="cuda"))),
                     ((q, k, v, hq, hk, s.cpu(), cache), {}),
                     ((q, torch.zeros(256, 3, dtype=torch.float16, device="cuda").t()[:, ::2], v, hq, hk, s, cache), {})]:
        with pytest.raises(ValueError):
            gqa.gqa_append(*args, **kw)
    with pytest.raises(gqa.GQAError):
        gqa.gqa_append(q, k.expand(3, 128)[:1].expand(3, 128), v, hq, hk, s, cache)     # rows on top of one another
    tab, ln = torch.zeros(3, 1, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")
    qc = q.contiguous()
    gqa.gqa_decode_kv8(qc, cache, tab, ln, hq, hk)
    for args in [(q, cache, tab, ln), (qc, cache.half(), tab, ln), (qc, cache, tab.long(), ln), (qc, cache, tab, ln[:2]),
                 (qc, cache, tab[:2], ln), (qc.float(), cache, tab, ln), (qc, cache[:, :1], tab, ln)]:
        with pytest.raises(ValueError):
            gqa.gqa_decode_kv8(*args, hq, hk)
    with pytest.raises(gqa.GQAError):
        gqa.gqa_decode_kv8(qc.view(1, 3, -1).repeat(1, 6, 1), cache, tab[:1], ln[:1], hq, hk)   # G * T_q = 72
    with pytest.raises(ValueError):
        gqa.gqa_kv8_read(cache, tab, ln, D, k_out=torch.zeros(3, 4, 64, dtype=torch.float16, device="cuda"))


# ---------------------------------------------------------------- the bounds-checked build
def test_bounds_checked_build(gqa):
    from decode_attention_03_gb300 import build
    lib = gqa.open_library(build.build(checked=True))
    raw = torch.cuda.current_stream().cuda_stream
    for D, hq, hk, bs, T in [(128, 32, 8, 16, 1), (64, 8, 2, 64, 3), (128, 64, 1, 8, 1), (64, 15, 1, 32, 1)]:
        lens = edge_lens(bs)
        N = len(lens)
        cache, tab = make_cache(lens, D, hk, bs, 130 + D)
        q = torch.randn(N, T, hq * D, generator=gen(50)).half()
        x = [q.cuda(), dev(cache), dev(tab), dev(np.array(lens, np.int32))]
        o = torch.full_like(x[0], math.nan)
        n = lib.gqa_decode_kv8_workspace_size(N, T, hq, hk, D)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        assert lib.gqa_decode_kv8(*(t.data_ptr() for t in x), o.data_ptr(), N, T, tab.shape[1], cache.shape[0], bs, hq,
                                  hk, D, D ** -0.5, ws.data_ptr(), n, raw, None) == 0
        assert lib.gqa_workspace_check(ws.data_ptr(), raw) == 0
        check_decode(o, cache, tab, lens, q, hq, hk, D, D ** -0.5, bs, False, "f16", "checked")
        k = torch.zeros(N, 700, hk * D, dtype=torch.float16, device="cuda")
        assert lib.gqa_kv8_read(x[1].data_ptr(), x[2].data_ptr(), x[3].data_ptr(), None, k.data_ptr(), k.data_ptr(), N,
                                700, tab.shape[1], cache.shape[0], bs, hk, D, ws.data_ptr(), n, raw, None) == 0
        assert lib.gqa_workspace_check(ws.data_ptr(), raw) == 0
        for layout in (0, 1, 2):
            t = 29
            h = torch.randn(t, hk * D, generator=gen(51)).half().cuda()
            pools = [torch.zeros(4 * bs * hk * (2 * D + 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
            s = torch.arange(4 * bs - 29, 4 * bs, device="cuda")
            a = gqa.gqa_append_args(0, h.data_ptr(), h.data_ptr(), 0, 0, hk * D, hk * D, 0, 0, 0, 0, 0, s.data_ptr(),
                                    pools[0].data_ptr(), pools[1].data_ptr(), t, 0, hk, D, 0, 0, 0, 4, bs, layout, 0,
                                    1e-6)
            assert lib.gqa_append(a, ws.data_ptr(), n, raw) == 0
            assert lib.gqa_workspace_check(ws.data_ptr(), raw) == 0
