"""GPU parity of filling the 4-bit cache, of reading it back and of rotary positions with several axes, against the float64
oracle (oracle/kv4_oracle.py).

Tolerances, from half steps u = finfo.eps / 2 (f16 2^-11, bf16 2^-8, fp32 2^-24):
* 16-bit outputs: one rounding of y, u|y| + half the smallest subnormal, and the fp32 steps before it: at most 12
  roundings of quantities no larger than |a| + |b| (the pair before the rotation): f = 2^-20 (|a| + |b|).
* 4 bits: the scale of sixteen elements is one that some maximum within f of theirs has, and with that scale every code
  lies between those of y - f and y + f.  V is not rotated: its scales and codes are the oracle's, bit for bit (x has at
  most 11 bits and a scale 3, so x / s in fp32 is on a border of two codes exactly when x / s is).
* read: what is held has 5 significant bits: equal.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import kv4_oracle as k4
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


def cuda(t):
    return None if t is None else t.cuda()


def table(max_pos, rot):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def case(elem, D, hq, hk, T, seed, norm=True, rot=None, axes=1, in_turn=False, max_pos=50, gqa=None):
    """axes 0: the one-axis call, positions (T)."""
    g, dt, rot = gen(seed), DT[elem], D if rot is None else rot
    qkv = (torch.randn(T, (hq + 2 * hk) * D, generator=g) * torch.exp(torch.randn(T, 1, generator=g))).to(dt)
    n = hq * D, hk * D
    c = dict(elem=elem, D=D, hq=hq, hk=hk, T=T, qkv=qkv, q=qkv[:, :n[0]], k=qkv[:, n[0]:n[0] + n[1]], v=qkv[:, n[0] + n[1]:],
             qw=None, kw=None, cs=None, pos=None, axes=None)
    if norm:
        c["qw"] = (1 + 0.3 * torch.randn(D, generator=g)).to(dt)
        c["kw"] = (1 + 0.3 * torch.randn(D, generator=g)).to(dt)
    if rot:
        c["cs"] = table(max_pos, rot)
        c["pos"] = torch.randint(0, max_pos, (max(axes, 1), T), generator=g).int()
        c["axes"] = torch.randint(0, max(axes, 1), (rot // 2,), generator=g).byte()
        if axes > 1 and not in_turn:
            c["axes"] = c["axes"].sort().values
        if axes == 0:
            c["pos"], c["axes"] = c["pos"][0], None
    return c


def run(gqa, c, slots, *caches, inter=False, **kw):
    qkv = c["qkv"].cuda()
    n = c["hq"] * c["D"], c["hk"] * c["D"]
    q = gqa.gqa_append(qkv[:, :n[0]] if c["hq"] else None, qkv[:, n[0]:n[0] + n[1]], qkv[:, n[0] + n[1]:], c["hq"], c["hk"],
                       slots.cuda(), *caches, positions=cuda(c["pos"]), cos_sin=cuda(c["cs"]), pair_axes=cuda(c["axes"]),
                       interleaved=inter, q_weight=cuda(c["qw"]), k_weight=cuda(c["kw"]), eps=1e-5, **kw)
    torch.cuda.synchronize()
    return q


def rows_of(c, x, w, heads, inter):
    """The oracle's rows (T, heads, D) and their fp32 term."""
    n = ko.head_rows(npy(x), heads, None if w is None else npy(w), 1e-5, None, None, inter)
    size = np.abs(n)
    if c["cs"] is None:
        return n, size * 2.0 ** -20
    pos = c["pos"].view(-1, c["T"]).tolist()
    half = c["cs"].shape[1] // 2
    axes = [0] * half if c["axes"] is None else c["axes"].tolist()
    y = k4.turn_rows(n, npy(c["cs"]), pos, axes, inter)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
    size[..., a] = size[..., b] = size[..., a] + size[..., b]
    return y, size * 2.0 ** -20


def close16(got, y, f, elem, where):
    err = np.abs(npy(got).reshape(y.shape) - y)
    bad = err > U[elem] * np.abs(y) + TINY[elem] + f
    assert not bad.any(), f"{where}: {bad.sum()} of {bad.size} out, worst {err[bad].max():.3e}"


def signed(code):
    return (-1.0 if code & 8 else 1.0) * k4.MAGNITUDES[code & 7]


def close4(cache, slot, h, y, f, D, bs, where):
    """A K row of the cache against 64-bit values with fp32 terms."""
    blk, row = divmod(int(slot), bs)
    for g in range(0, D, 16):
        p, e = y[g:g + 16], f[g:g + 16]
        byte = int(cache[blk, h, k4.scale_offset(row, g, D, bs, 0)])
        lo, hi = np.maximum(np.abs(p) - e, 0).max(), (np.abs(p) + e).max()
        assert k4.scale_byte(lo) <= byte <= k4.scale_byte(hi), where
        s = k4.scale_value(byte)
        got = k4.get_row(cache, slot, h, 0, D, bs)[g:g + 16]
        for i in range(16):
            # (the codes of values within the fp32 term and one rounding of the quotient)
            d = e[i] + abs(p[i]) * 2.0 ** -23
            assert signed(k4.encode(p[i] - d, s)) * s <= got[i] <= signed(k4.encode(p[i] + d, s)) * s, where


def slots_for(T, num_blocks, bs, seed, skip=0):
    s = torch.randperm(num_blocks * bs, generator=gen(seed))[:T]
    if skip:
        s[torch.randperm(T, generator=gen(seed + 1))[:skip]] = -1 - torch.arange(skip) * 1000
    return s


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("D,hq,hk,rot,inter,axes", [(128, 8, 2, 128, False, 0), (128, 6, 3, 64, False, 3), (128, 4, 4, 128, True, 2),
                                                    (64, 8, 2, 64, False, 4), (64, 7, 1, 8, True, 0), (64, 10, 5, 48, False, 1),
                                                    (128, 32, 8, 24, True, 3), (128, 5, 1, 0, False, 0), (64, 4, 2, 16, False, 2),
                                                    (128, 3, 3, 96, False, 32), (64, 0, 2, 40, False, 3),
                                                    (128, 2, 1, 112, True, 3)])
@pytest.mark.parametrize("bs,T", [(32, 23), (8, 1), (64, 9), (16, 17)])
def test_append(gqa, elem, D, hq, hk, rot, inter, axes, bs, T):
    c = case(elem, D, hq, hk, T, 100 + D + hq + T, norm=(hq + T) % 4 != 1, rot=rot, axes=axes, in_turn=bs > 16)
    nb = (T + bs - 1) // bs + 3
    slots = slots_for(T, nb, bs, 7, skip=T // 9)
    cache = torch.full((nb, hk, bs * (D + D // 8)), 0x5A, dtype=torch.uint8, device="cuda")
    q = run(gqa, c, slots, cache, inter=inter)
    if hq:
        close16(q, *rows_of(c, c["q"], c["qw"], hq, inter), elem, "q_out")
    k, fk = rows_of(c, c["k"], c["kw"], hk, inter)
    v = npy(c["v"]).reshape(T, hk, D)
    got = cache.cpu().numpy()
    want, there = got.copy(), np.zeros_like(got, dtype=bool)
    for t, s in enumerate(slots.tolist()):
        if s < 0:
            continue
        for h in range(hk):
            close4(got, s, h, k[t, h], fk[t, h], D, bs, f"k of token {t}, head {h}")
            k4.put_row(want, s, h, 1, v[t, h], D, bs)
            for w in (0, 1):
                there[s // bs, h, k4.row_offsets(s % bs, D, bs, w)] = True
    np.testing.assert_array_equal(got, want)
    assert (got[~there] == 0x5A).all()


@pytest.mark.parametrize("layout", ["rows", "vllm", "kv8"])
@pytest.mark.parametrize("elem,D,hq,hk,rot,inter,axes,T", [("f16", 128, 8, 2, 128, False, 3, 41), ("bf16", 64, 4, 4, 24, True, 2, 20),
                                                           ("bf16", 128, 3, 1, 64, False, 4, 1), ("f16", 64, 12, 4, 64, True, 32, 70)])
def test_axes_into_the_other_caches(gqa, layout, elem, D, hq, hk, rot, inter, axes, T):
    bs, dt = 16, DT[elem]
    c = case(elem, D, hq, hk, T, 200 + T, rot=rot, axes=axes, in_turn=True)
    nb = T // bs + 2
    slots = slots_for(T, nb, bs, 3)
    if layout == "kv8":
        caches = [gqa.gqa_kv8_cache(nb, bs, hk, D)]
    elif layout == "rows":
        caches = [torch.zeros(nb, bs, hk * D, dtype=dt, device="cuda") for _ in range(2)]
    else:
        caches = [torch.zeros(nb, hk, D // 8, bs, 8, dtype=dt, device="cuda"), torch.zeros(nb, hk, D, bs, dtype=dt, device="cuda")]
    q = run(gqa, c, slots, *caches, inter=inter)
    close16(q, *rows_of(c, c["q"], c["qw"], hq, inter), elem, "q_out")
    k, f = rows_of(c, c["k"], c["kw"], hk, inter)
    if layout == "kv8":
        got = caches[0].cpu().numpy()
        held = np.stack([[ko.get_row(got, s, h, 0, D, bs) for h in range(hk)] for s in slots.tolist()])
        top = np.abs(k).max(-1, keepdims=True)
        # half an e4m3 step, or its subnormal one, 2^-10 of a scale that is at most twice the largest magnitude's 448th
        assert (np.abs(held - k) <= np.maximum(np.abs(k) * 2.0 ** -4, top / 224 * 2.0 ** -9) + 2 * f).all()
        return
    x = caches[0].float().cpu()
    x = (x.permute(0, 3, 1, 2, 4) if layout == "vllm" else x).reshape(nb * bs, hk, D)[slots]
    close16(x, k, f, elem, "k cache")
    x = caches[1].float().cpu()
    x = (x.permute(0, 3, 1, 2) if layout == "vllm" else x).reshape(nb * bs, hk, D)[slots]
    assert torch.equal(x, c["v"].float().view(T, hk, D))


def test_axes_that_agree_are_one_axis(gqa):
    """Text: all axes have the same position, and the bits of the one-axis call come out, whatever turns a pair."""
    for layout, T in (("kv4", 300), ("rows", 3000)):
        c = case("bf16", 128, 8, 2, T, 5, axes=0)
        make = (lambda: [gqa.gqa_kv4_cache(T // 16 + 1, 16, 2, 128)]) if layout == "kv4" else \
            (lambda: [torch.zeros(T // 16 + 1, 16, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2)])
        one = make()
        q = run(gqa, c, torch.arange(T), *one)
        for axes in (gqa.gqa_pair_axes([16, 24, 24], device="cpu"), gqa.gqa_pair_axes([24, 20, 20], in_turn=True, device="cpu")):
            c3, three = dict(c, pos=c["pos"].expand(3, -1).contiguous(), axes=axes), make()
            assert torch.equal(run(gqa, c3, torch.arange(T), *three), q)
            assert all(torch.equal(a, b) for a, b in zip(one, three))


@pytest.mark.parametrize("layout,D,hq,hk,T,bs,rot,inter,elem,axes", [
    ("kv4", 128, 4, 2, 20011, 16, 128, False, "bf16", 3), ("kv4", 64, 3, 3, 10009, 64, 24, False, "f16", 2),
    ("kv4", 128, 64, 8, 5003, 32, 64, True, "bf16", 0), ("rows", 128, 8, 4, 11000, 8, 128, False, "f16", 3),
    ("vllm", 64, 4, 2, 20003, 8, 64, True, "bf16", 4), ("kv8", 128, 2, 1, 19999, 8, 128, False, "f16", 3)])
def test_append_warps_with_several_tokens(gqa, layout, D, hq, hk, T, bs, rot, inter, elem, axes):
    """Calls with more tokens than the GPU has warps give what calls of few tokens give, bit for bit, padding and bad slots
    and positions (on any axis) among them."""
    c = case(elem, D, hq, hk, T, 400 + T, rot=rot, axes=axes, in_turn=True)
    nb, dt, g = T // bs + 2, DT[elem], gen(T)
    slots = slots_for(T, nb, bs, 9, skip=T // 5)
    slots[torch.randperm(T, generator=g)[:20]] = nb * bs + 7
    bad = torch.randperm(T, generator=g)[:30]
    pos = c["pos"].view(-1, T)
    pos[torch.arange(30) % pos.shape[0], bad] = torch.tensor([50, -1, 1 << 30] * 10).int()

    def caches():
        if layout in ("kv8", "kv4"):
            n = 2 * D + 2 if layout == "kv8" else D + D // 8
            return [torch.full((nb, hk, bs * n), 0x5A, dtype=torch.uint8, device="cuda")]
        if layout == "rows":
            return [torch.full((nb, bs, hk * D), 3.0, dtype=dt, device="cuda") for _ in range(2)]
        return [torch.full((nb, hk, D // 8, bs, 8), 3.0, dtype=dt, device="cuda"),
                torch.full((nb, hk, D, bs), 3.0, dtype=dt, device="cuda")]

    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    want, small = torch.full((T, hq * D), 5.0, dtype=dt, device="cuda"), caches()
    for i in range(0, T, 1500):
        part = dict(c, qkv=c["qkv"][i:i + 1500], pos=c["pos"][..., i:i + 1500].contiguous())
        run(gqa, part, slots[i:i + 1500], *small, inter=inter, q_out=want[i:i + 1500], workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
    once, whole = torch.full_like(want, 5.0), caches()
    run(gqa, c, slots, *whole, inter=inter, q_out=once, workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
    assert torch.equal(once, want) and all(torch.equal(a, b) for a, b in zip(whole, small))
    assert (once[bad] == 5.0).all()


def test_append_rows_of_any_size(gqa):
    """Zeros, the borders of a scale and of codes, the smallest and largest values, infinities and NaN."""
    D, bs = 64, 8
    big = 3.0e38
    edge = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    rows = [torch.zeros(D), torch.full((D,), 61440.0), torch.full((D,), 70000.0), torch.linspace(-1e-39, 1e-39, D),
            torch.linspace(-big, big, D), torch.tensor([math.inf] + [1.0] * (D - 1)), torch.tensor([math.nan, -2.0] + [0.5] * (D - 2)),
            torch.full((D,), math.nan), torch.full((D,), -0.0), 2.0 ** torch.arange(-40, 24).float(),
            torch.cat([edge * s for s in (1.0, -1.25, 1.5, -1.75, 2.0, 3.5, -5.0, 1.0)]),
            torch.linspace(-6 * 2.0 ** -15, 6 * 2.0 ** -16, D), torch.cat([torch.full((16,), x) for x in (6.75, 8.25, 9.75, 11.25)]),
            torch.cat([torch.full((16,), x * 2.0 ** -17) for x in (6.0, 6.0625, 9.0, 18.0)])]
    x = torch.stack(rows).bfloat16()
    T = len(rows)
    cache = gqa.gqa_kv4_cache(2, bs, 1, D)
    gqa.gqa_append(None, x.cuda(), x.cuda(), 1, 1, torch.arange(T).cuda(), cache)
    want = np.zeros((2, 1, bs * (D + D // 8)), dtype=np.uint8)
    for t in range(T):
        for w in (0, 1):
            k4.put_row(want, t, 0, w, npy(x[t]), D, bs)
    got = cache.cpu().numpy()
    for t in range(T):
        for w in (0, 1):
            np.testing.assert_array_equal(k4.get_row(got, t, 0, w, D, bs), k4.get_row(want, t, 0, w, D, bs), err_msg=f"row {t}")
            s = [k4.scale_offset(t % bs, e, D, bs, w) for e in range(0, D, 16)]
            np.testing.assert_array_equal(got[t // bs, 0, s], want[t // bs, 0, s])
    k, v = gqa.gqa_kv4_read(cache, torch.tensor([[0, 1]]).int().cuda(), torch.tensor([T]).int().cuda(), D, T, dtype=torch.bfloat16)
    assert torch.equal(k.isnan(), v.isnan()) and bool(k[0, 5, :16].isnan().all()) and not bool(k[0, 5, 16:].isnan().any())
    assert (k[0, 2] == 61440.0).all()


def test_append_reports(gqa):
    D, bs, hk = 128, 16, 2
    c = case("f16", D, 8, hk, 6, 11, axes=3, in_turn=True)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    fresh = lambda: torch.full((2, hk, bs * (D + D // 8)), 9, dtype=torch.uint8, device="cuda")

    def written(cache):
        got = cache.cpu().numpy()
        return sorted({r for r in range(32) if (got[r // bs, 0, k4.row_offsets(r % bs, D, bs, 0)] != 9).any()})

    cache = fresh()
    run(gqa, c, torch.tensor([0, 5, 32, -1, 31, 1 << 40]), cache, workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG and gqa.gqa_workspace_check(ws) == gqa.GQA_OK
    assert written(cache) == [0, 5, 31]
    c["pos"][1, 1], c["pos"][2, 3], cache = 50, -1, fresh()
    q = torch.full((6, 8 * D), 3.0, dtype=torch.float16, device="cuda")
    run(gqa, c, torch.arange(6), cache, workspace_tensor=ws, q_out=q)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
    assert written(cache) == [0, 2, 4, 5] and (q[[1, 3]] == 3.0).all() and not (q[[0, 2, 4, 5]] == 3.0).all(1).any()
    c["axes"][63], cache = 3, fresh()          # there are three axes: no token is taken
    q.fill_(3.0)
    run(gqa, c, torch.arange(6), cache, workspace_tensor=ws, q_out=q)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG and written(cache) == [] and (q == 3.0).all()


@pytest.mark.parametrize("layout", ["rows", "vllm", "kv8", "kv4"])
@pytest.mark.parametrize("T", [5, 40])
def test_a_pair_on_an_axis_that_is_none(gqa, layout, T):
    """No query, key or value is written, into any cache, and the call reports."""
    D, hk, bs, nb = 64, 2, 8, 8
    c = case("f16", D, 4, hk, T, 12, axes=2)
    c["axes"][7] = 2
    if layout in ("kv8", "kv4"):
        caches = [torch.full((nb, hk, bs * (2 * D + 2 if layout == "kv8" else D + D // 8)), 9, dtype=torch.uint8, device="cuda")]
    elif layout == "rows":
        caches = [torch.full((nb, bs, hk * D), 3.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    else:
        caches = [torch.full(s, 3.0, dtype=torch.float16, device="cuda") for s in ((nb, hk, D // 8, bs, 8), (nb, hk, D, bs))]
    before, q = [x.clone() for x in caches], torch.full((T, 4 * D), 3.0, dtype=torch.float16, device="cuda")
    assert gqa.gqa_status_check() == gqa.GQA_OK
    run(gqa, c, torch.arange(T), *caches, q_out=q)
    assert gqa.gqa_status_check() == gqa.GQA_ERR_INVALID_ARG
    assert (q == 3.0).all() and all(torch.equal(a, b) for a, b in zip(caches, before))


def test_append_in_place_and_no_tokens(gqa):
    c = case("f16", 128, 8, 2, 19, 5, axes=3)
    cache, again = gqa.gqa_kv4_cache(4, 16, 2, 128), gqa.gqa_kv4_cache(4, 16, 2, 128)
    want = run(gqa, c, torch.arange(19), cache)
    qkv = c["qkv"].cuda()
    q, k, v = qkv[:, :1024], qkv[:, 1024:1280], qkv[:, 1280:]
    kw = dict(positions=c["pos"].cuda(), cos_sin=c["cs"].cuda(), pair_axes=c["axes"].cuda(), q_weight=c["qw"].cuda(),
              k_weight=c["kw"].cuda(), eps=1e-5)
    out = gqa.gqa_append(q, k, v, 8, 2, torch.arange(19).cuda(), again, q_out=q, **kw)
    assert out.data_ptr() == qkv.data_ptr() and torch.equal(out, want) and torch.equal(again, cache)
    kw["positions"] = kw["positions"][:, :0].contiguous()
    assert gqa.gqa_append(q[:0], k[:0], v[:0], 8, 2, torch.arange(0).cuda(), again, **kw).shape == (0, 1024)
    assert torch.equal(again, cache)


def test_binding_checks_of_append(gqa):
    c = case("f16", 64, 4, 2, 5, 5, axes=3)
    cache, slots = gqa.gqa_kv4_cache(2, 16, 2, 64), torch.arange(5)
    for bad in (dict(pos=c["pos"][0]), dict(pos=c["pos"][:, :4].contiguous()), dict(axes=c["axes"][:31].contiguous()),
                dict(axes=c["axes"].int()), dict(cs=None), dict(pos=c["pos"].t()), dict(pos=c["pos"].long()),
                dict(pos=torch.zeros(33, 5).int()), dict(pos=torch.zeros(0, 5).int()), dict(axes=None)):
        with pytest.raises(ValueError):
            run(gqa, dict(c, **bad), slots, cache)
    with pytest.raises(ValueError):
        run(gqa, c, slots, cache, cache)
    for shape in ((2, 3, 16 * 72), (2, 2, 16 * 72 + 1)):
        with pytest.raises((ValueError, gqa.GQAError)):
            run(gqa, c, slots, torch.zeros(shape, dtype=torch.uint8, device="cuda"))


# ---------------------------------------------------------------- read
def random_cache(nb, hk, bs, D, seed):
    """Any codes, any finite scales."""
    g = gen(seed)
    cache = torch.randint(0, 256, (nb, hk, bs * (D + D // 8)), generator=g).byte()
    cache[..., bs * D:] = torch.randint(0, 0x72, (nb, hk, bs * D // 8), generator=g).byte()     # up to 6 * 10240
    return cache.numpy()


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("D,hk,bs", [(128, 8, 16), (128, 1, 8), (64, 2, 64), (64, 3, 32), (128, 3, 64), (64, 5, 8)])
def test_read(gqa, elem, D, hk, bs):
    lens, begins = [0, 1, bs, 3 * bs + 5, 40, 100], [0, 0, bs - 1, bs + 3, 40, 90]
    need = [(n + bs - 1) // bs for n in lens]
    cache = random_cache(sum(need) + 2, hk, bs, D, 30 + D)
    ids = torch.randperm(sum(need), generator=gen(1)).tolist()
    tab = np.full((len(lens), max(need)), -1, np.int32)
    for b, m in enumerate(need):
        tab[b, :m] = [ids.pop() for _ in range(m)]
    d = lambda x: torch.from_numpy(np.asarray(x)).cuda()
    for bg, count in (([0] * 6, 104), (begins, 20)):
        k, v = (torch.full((6, count, hk * D), 5.0, dtype=DT[elem], device="cuda") for _ in range(2))
        out = gqa.gqa_kv4_read(d(cache), d(tab), d(np.array(lens, np.int32)), D, begins=d(np.array(bg, np.int32)), k_out=k, v_out=v)
        assert out[0] is k and out[1] is v
        only = gqa.gqa_kv4_read(d(cache), d(tab), d(np.array(lens, np.int32)), D, begins=d(np.array(bg, np.int32)),
                                v_out=torch.full_like(v, 5.0))
        assert only[0] is None and torch.equal(only[1], v)
        for b, n in enumerate(lens):
            wk, wv = k4.gather_kv4(cache, tab[b], n, D, bs)
            m = max(min(n - bg[b], count), 0)
            for x, w in ((k, wk), (v, wv)):
                np.testing.assert_array_equal(npy(x[b, :m]).reshape(m, hk, D), w[bg[b]:bg[b] + m])
                assert (x[b, m:] == 5.0).all()
    assert gqa.gqa_status_check() == gqa.GQA_OK


def test_read_reports_and_defaults(gqa):
    D, hk, bs = 64, 2, 16
    cache = torch.from_numpy(random_cache(4, hk, bs, D, 3)).cuda()
    tab = torch.tensor([[0, 4, 1], [2, -1, 3]]).int().cuda()
    lens, ws = torch.tensor([40, 10]).int().cuda(), torch.zeros(256, dtype=torch.uint8, device="cuda")
    k, v = gqa.gqa_kv4_read(cache, tab, lens, D, 48, workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
    wk, _ = k4.gather_kv4(cache.cpu().numpy(), [0, -1, 1], 40, D, bs)
    np.testing.assert_array_equal(npy(k[0, :40]).reshape(40, hk, D), wk)
    assert k.dtype == torch.float16 and (k[0, 40:] == 0).all() and (k[1, 10:] == 0).all()
    for n, bg in ((-3, 0), (1000, 40), (10, -1)):
        gqa.gqa_kv4_read(cache, torch.zeros_like(tab), torch.tensor([n, 10]).int().cuda(), D, 8,
                         begins=torch.tensor([bg, 0]).int().cuda(), workspace_tensor=ws)
        assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG, (n, bg)
    big = torch.full((2, 8 + 2 * 40 * hk * D), 5.0, dtype=torch.float16, device="cuda")
    k2, v2 = (x[8:].view(2, 40, hk * D) for x in big)                 # on a border of 16 bytes, not of 32
    tab[0, 1] = 2
    gqa.gqa_kv4_read(cache, tab, lens, D, k_out=k2, v_out=v2)
    wk, wv = k4.gather_kv4(cache.cpu().numpy(), [0, 2, 1], 40, D, bs)
    np.testing.assert_array_equal(npy(k2[0]).reshape(40, hk, D), wk)
    np.testing.assert_array_equal(npy(v2[0]).reshape(40, hk, D), wv)
    assert (big[:, :8] == 5.0).all() and (k2[1, 10:] == 5.0).all()
