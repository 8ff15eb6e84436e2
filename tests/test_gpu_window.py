"""GPU parity of gqa_decode_kv4 and gqa_decode_window against the float64 oracle (oracle/kv4_oracle.py).

Tolerances, from half steps u = finfo.eps / 2 (f16 2^-11, bf16 2^-8), with A = sum p|v| / l:
* the output's rounding, u|o|;
* the weights: rounded to f16 once (kv4, bf16 calls) 2^-12 A, else to two 16-bit numbers, less; below f16's normal range
  (2^-14 in units of 2^-11 of the row's largest) off by at most 2^-36 of it, for n keys n 2^-36 max|V| / l, of which
  n 2^-25 2 max|V| / l is the generous form;
* fp32 sums, ex2 (2 ulp) and scores: 2^-11 A, generous for scores below 2^6 in size.
"""
from __future__ import annotations

import math
import threading

import numpy as np
import pytest
import torch

from oracle import kv4_oracle as k4

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


class Case:
    """A cache of either kind, on the CPU: pools of blocks in any order, a table with -1 past a sequence's blocks."""

    def __init__(self, kind, elem, lens, D, hk, bs, seed, extra=2):
        self.kind, self.elem, self.lens, self.D, self.hk, self.bs = kind, elem, list(lens), D, hk, bs
        need = [(max(n, 0) + bs - 1) // bs for n in lens]
        nb = sum(need) + extra
        g = gen(seed)
        if kind == "kv4":
            self.cache = torch.randint(0, 256, (nb, hk, bs * (D + D // 8)), generator=g).byte()
            self.cache[..., bs * D:] = torch.randint(0x2a, 0x38, (nb, hk, bs * D // 8), generator=g).byte()
        else:
            self.k, self.v = (torch.randn(nb, bs, hk * D, generator=g).to(DT[elem]) for _ in range(2))
        ids = torch.randperm(nb, generator=g).tolist()
        self.tab = np.full((len(lens), max(need + [1])), -1, np.int32)
        for b, m in enumerate(need):
            self.tab[b, :m] = [ids.pop() for _ in range(m)]

    def kv(self, b, n):
        if self.kind == "kv4":
            return k4.gather_kv4(self.cache.numpy(), self.tab[b], n, self.D, self.bs)
        at = np.arange(n)
        ids = self.tab[b][at // self.bs]
        ok = (ids >= 0) & (ids < self.k.shape[0])
        rows = np.where(ok, ids, 0) * self.bs + at % self.bs
        return [np.where(ok[:, None, None], npy(x).reshape(-1, self.hk, self.D)[rows], 0.0) for x in (self.k, self.v)]

    def nan_row(self, b, j, k=True, v=True, value=math.nan):
        """Key j of sequence b holds `value` (kv4: NaN) in K and/or V, in every head."""
        blk, row = int(self.tab[b, j // self.bs]), j % self.bs
        if self.kind == "kv4":
            for w, on in enumerate((k, v)):
                if on:
                    for e in range(0, self.D, 16):
                        self.cache[blk, :, k4.scale_offset(row, e, self.D, self.bs, w)] = 0x7f
        else:
            for x, on in ((self.k, k), (self.v, v)):
                if on:
                    x[blk, row] = value

    def run(self, gqa, q, hq, tab=None, lens=None, **kw):
        tab = torch.from_numpy(np.ascontiguousarray(self.tab if tab is None else tab)).cuda()
        ln = torch.tensor(self.lens if lens is None else lens, dtype=torch.int32).cuda()
        if self.kind == "kv4":
            o = gqa.gqa_decode_kv4(q.cuda(), self.cache.cuda(), tab, ln, hq, self.hk, **kw)
        else:
            kw.setdefault("window", 0)
            o = gqa.gqa_decode_window(q.cuda(), self.k.cuda(), self.v.cuda(), tab, ln, hq, self.hk, **kw)
        torch.cuda.synchronize()
        return o

    def workspace(self, gqa, N, T, hq):
        n = gqa.gqa_decode_window_workspace_size(N, T, hq, self.hk, self.D, gqa.GQA_CACHE_KV4 if self.kind == "kv4" else gqa.GQA_CACHE_ROWS)
        assert n > 0
        return torch.zeros(n, dtype=torch.uint8, device="cuda")

    def check(self, o, q, hq, where="", some=None, scale=None, causal=False, window=0, sinks=0):
        D, some = self.D, list(range(len(self.lens))) if some is None else some
        q = npy(q).reshape(len(self.lens), -1, hq * D)[some]
        lens = [self.lens[i] for i in some]
        ref, a, l, top = k4.decode_window(q, lambda b, n: self.kv(some[b], n), lens, hq, self.hk, D,
                                          D ** -0.5 if scale is None else scale, causal, window, sinks)
        o = o.double().cpu().reshape(len(self.lens), -1, hq * D)[some]
        n = torch.tensor([max(int(x), 0) for x in lens], dtype=torch.float64)
        low = (n * 2.0 ** -25 * 2 * top)[:, None, None] / l.clamp(min=1.0)
        tol = U[self.elem] * ref.abs() + (2.0 ** -12 + 2.0 ** -11) * a + low.repeat_interleave(D, -1) + TINY[self.elem]
        err = (o - ref).abs()
        assert torch.isfinite(o).all(), where
        assert not (err > tol).any(), f"{where}: {int((err > tol).sum())} out, worst {float((err - tol).max()):.3e}"
        assert (o[(l == 0).repeat_interleave(D, -1)] == 0).all(), where


def queries(elem, N, T, width, seed):
    return torch.randn(N, T, width, generator=gen(seed)).to(DT[elem])


KINDS = ["kv4", "rows"]
# D, hq, hk, T, causal: each class of query rows, with one, two, three and four n-tiles, and two warps on a ring
SHAPES = [(128, 32, 8, 1, False), (64, 8, 2, 1, True), (128, 7, 1, 2, True), (64, 6, 2, 5, True), (64, 64, 2, 1, False),
          (128, 48, 2, 1, True), (128, 16, 2, 8, True), (64, 24, 1, 2, False), (128, 40, 1, 1, False), (64, 12, 2, 4, True),
          (128, 4, 4, 3, False)]
WINDOWS = [(0, 0), (1, 0), (33, 0), (32, 1), (40, 70), (100, 4), (5, 33), (4000, 4)]


def edge_lens(bs):
    return [0, 1, 2, 31, 32, 33, bs - 1, bs, bs + 1, 64, 65, 127, 129, 511, 700, 0, 1025]


# ---------------------------------------------------------------- values
@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("D,hq,hk,T,causal", SHAPES)
def test_edges(gqa, elem, kind, bs, D, hq, hk, T, causal):
    lens = edge_lens(bs)
    c = Case(kind, elem, lens, D, hk, bs, 40 + bs + hq)
    q = queries(elem, len(lens), T, hq * D, bs + hq + T)
    ws = c.workspace(gqa, len(lens), T, hq)
    for window, sinks in WINDOWS:
        o = c.run(gqa, q, hq, causal=causal, window=window, sinks=sinks, workspace_tensor=ws)
        assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
        c.check(o, q, hq, f"window {window}, sinks {sinks}", causal=causal, window=window, sinks=sinks)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens", [[1], [9000], [5000, 3, 8191], [200] * 40, [300]])
@pytest.mark.parametrize("hq,hk,D,elem", [(4, 1, 128, "bf16"), (16, 2, 64, "f16"), (32, 1, 128, "f16")])
def test_split_over_long_sequences(gqa, kind, lens, hq, hk, D, elem):
    c = Case(kind, elem, lens, D, hk, 16, 50 + len(lens))
    q = queries(elem, len(lens), 1, hq * D, 9)
    for window, sinks in ((0, 0), (3000, 5), (777, 100), (64, 0)):
        o = c.run(gqa, q, hq, window=window, sinks=sinks)
        c.check(o, q, hq, f"window {window}", window=window, sinks=sinks)
        assert torch.equal(o, c.run(gqa, q, hq, window=window, sinks=sinks))          # the same call, the same bits
    assert gqa.gqa_status_check() == gqa.GQA_OK


@pytest.mark.parametrize("kind", KINDS)
def test_more_sequences_than_one_launch_takes(gqa, kind):
    lens = [(7 * i) % 90 for i in range(1500)]
    c = Case(kind, "f16", lens, 64, 1, 8, 60)
    q = queries("f16", 1500, 1, 2 * 64, 3)
    o = c.run(gqa, q, 2, window=20, sinks=2)
    c.check(o, q, 2, window=20, sinks=2)


@pytest.mark.parametrize("kind", KINDS)
def test_scale_of_any_sign_and_size(gqa, kind):
    c = Case(kind, "bf16", [200, 70], 128, 2, 16, 61)
    q = queries("bf16", 2, 1, 8 * 128, 4)
    for scale in (-0.1, 0.0, 1e-3, 0.3):
        c.check(c.run(gqa, q, 8, scale=scale, window=100), q, 8, f"scale {scale}", scale=scale, window=100)


def test_window_of_everything_is_no_window(gqa):
    for kind in KINDS:
        c = Case(kind, "f16", [700, 40], 128, 2, 16, 62)
        q = queries("f16", 2, 2, 8 * 128, 5)
        full = c.run(gqa, q, 8, causal=True)
        for window, sinks in ((704, 0), (1 << 40, 1 << 40), (700, 3), (650, 60)):
            assert torch.equal(c.run(gqa, q, 8, causal=True, window=window, sinks=sinks), full), (kind, window)


@pytest.mark.parametrize("elem", ["f16", "bf16"])
def test_full_attention_agrees_with_the_paged_call(gqa, elem):
    c = Case("rows", elem, [900, 1, 333], 128, 4, 16, 63)
    q = queries(elem, 3, 1, 16 * 128, 6)
    o = c.run(gqa, q, 16, window=0)
    p = gqa.gqa_decode_paged(q[:, 0].cuda(), c.k.cuda(), c.v.cuda(), torch.from_numpy(c.tab).cuda(),
                             torch.tensor(c.lens).int().cuda(), 16, 4, max_seq_len=1024)
    c.check(p[:, None], q, 16)
    c.check(o, q, 16)


def test_f16_outputs_are_as_exact_as_their_rounding(gqa):
    """Weights in two numbers: beside the output's own half step little is lost."""
    for kind, elem in (("kv4", "f16"), ("rows", "f16"), ("rows", "bf16")):
        c = Case(kind, elem, [3000], 128, 2, 16, 64)
        q = queries(elem, 1, 1, 8 * 128, 7)
        ref, a, _, _ = k4.decode_window(npy(q), c.kv, c.lens, 8, 2, 128, 128 ** -0.5, False, 2000, 4)
        err = (c.run(gqa, q, 8, window=2000, sinks=4).double().cpu() - ref).abs()
        # two numbers of the weight: 2^-22 (bf16: 2^-16) A; fp32 scores and sums: 2^-18 A
        assert (err <= U[elem] * ref.abs() + (2.0 ** -15 + 2.0 ** -18) * a + TINY[elem]).all(), (kind, elem)


# ---------------------------------------------------------------- masked places
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", [8, 16, 64])
@pytest.mark.parametrize("N", [1, 30])
def test_what_no_token_sees_reaches_nothing(gqa, kind, bs, N):
    """NaN in every key that is hidden, behind the last one, and no block at all where none of a block's keys is seen."""
    D, hq, hk, T, window, sinks = 128, 8, 2, 3, 50, 5
    c = Case(kind, "bf16", [1000, 313, 60, 3][:N] if N < 4 else [1000, 313, 60, 3] + [400 + i for i in range(N - 4)], D, hk, bs, 70)
    q = queries("bf16", N, T, hq * D, 8)
    o = c.run(gqa, q, hq, causal=True, window=window, sinks=sinks)
    c.check(o, q, hq, causal=True, window=window, sinks=sinks)
    tab = c.tab.copy()
    for b, n in enumerate(c.lens):
        first = max(n - T - window + 1, 0)
        for j in range(sinks, first):
            c.nan_row(b, j)
        for j in range(n, (n + bs - 1) // bs * bs):
            c.nan_row(b, j)
        for blk in range(tab.shape[1]):
            if blk * bs >= sinks and (blk + 1) * bs <= first or blk * bs >= n:
                tab[b, blk] = [-1, 1 << 30, -(1 << 31), c.tab.max() + 50][(b + blk) % 4]
    ws = c.workspace(gqa, N, T, hq)
    again = c.run(gqa, q, hq, tab=tab, causal=True, window=window, sinks=sinks, workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
    assert torch.equal(again, o)


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,hq,hk,T", [(128, 2, 1, 4), (64, 8, 2, 2), (128, 8, 1, 3), (64, 2, 1, 8), (128, 8, 1, 4), (64, 16, 2, 5),
                                       (128, 12, 1, 5)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_what_some_tokens_see_reaches_only_them(gqa, elem, kind, D, hq, hk, T, value):
    """A key that the oldest tokens see no more, or the newest alone see, holds NaN or an infinity."""
    if kind == "kv4" and value == math.inf:
        pytest.skip("the 4-bit cache holds no infinity")
    window, sinks = 70, 3
    for lens in ([300], [300, 45, 700] * 20):
        c = Case(kind, elem, lens, D, hk, 16, 80 + D)
        q = queries(elem, len(lens), T, hq * D, 9)
        clean = c.run(gqa, q, hq, causal=True, window=window, sinks=sinks)
        n = lens[0]
        for j, sees in ((n - 1, lambda t: t == T - 1), (n - 2, lambda t: t >= T - 2), (n - T - window + 1, lambda t: t == 0),
                        (n - T - window + 2, lambda t: t <= 1)):
            keep = [x.clone() for x in ((c.cache,) if kind == "kv4" else (c.k, c.v))]
            c.nan_row(0, j, k=False, value=value)
            o = c.run(gqa, q, hq, causal=True, window=window, sinks=sinks)
            for t in range(T):
                if sees(t):
                    assert not torch.isfinite(o[0, t]).any(), (j, t)
                else:      # (other products of the tile's values: not the same bits)
                    ref, a, _, _ = k4.decode_window(npy(q[:1, t:t + 1]), lambda b, m: [np.nan_to_num(x, posinf=0.0) for x in c.kv(0, m)],
                                                    [n - T + t + 1], hq, hk, D, D ** -0.5, True, window, sinks)
                    assert ((o[0, t].double().cpu() - ref[0, 0]).abs() <= U[elem] * ref.abs()[0, 0] + 2.0 ** -10 * a.reshape(-1)
                            + TINY[elem]).all(), (j, t)
            assert torch.equal(o[1:], clean[1:])
            if kind == "kv4":
                c.cache = keep[0]
            else:
                c.k, c.v = keep


@pytest.mark.parametrize("kind", KINDS)
def test_not_a_number_stays_in_its_row(gqa, kind):
    D, hq, hk = 64, 8, 2
    for lens in ([100], [100] * 90):
        c = Case(kind, "f16", lens, D, hk, 16, 81)
        q = queries("f16", len(lens), 1, hq * D, 10)
        q[0, 0, 3 * D + 5] = math.nan                       # one query head
        o = c.run(gqa, q, hq, window=40)
        nan = torch.isnan(o[0, 0]).view(hq, D)
        assert nan[3].all() and not nan[[0, 1, 2, 4, 5, 6, 7]].any() and torch.isfinite(o[1:]).all()
        q[0, 0, 3 * D + 5] = 0
        c.nan_row(0, 80, v=False)                           # a key that is seen
        o = c.run(gqa, q, hq, window=40)
        assert torch.isnan(o[0]).all() and torch.isfinite(o[1:]).all()
        c.nan_row(0, 50)                                    # and one that is not
        assert torch.isnan(c.run(gqa, q, hq, window=20)[0]).all()       # keys 80 .. 99
        assert torch.isfinite(c.run(gqa, q, hq, window=19)).all()


@pytest.mark.parametrize("kind", KINDS)
def test_tokens_that_see_no_key(gqa, kind):
    """More new tokens than keys: the oldest see none."""
    for lens in ([3], [3, 0, 1, 40] * 20):
        c = Case(kind, "f16", lens, 64, 2, 8, 82)
        q = queries("f16", len(lens), 5, 4 * 64, 11)
        for window, sinks in ((0, 0), (2, 1), (7, 0)):
            out = torch.full_like(q, 7.0).cuda()
            o = c.run(gqa, q, 4, causal=True, window=window, sinks=sinks, out=out)
            assert o is out and (o[0, :2] == 0).all()
            c.check(o, q, 4, causal=True, window=window, sinks=sinks)


# ---------------------------------------------------------------- reports
@pytest.mark.parametrize("kind", KINDS)
def test_reports_bad_blocks_and_lengths(gqa, kind):
    D, bs, hk = 64, 16, 2
    lens = [100, 40, 70]
    c = Case(kind, "f16", lens, D, hk, bs, 100)
    q = queries("f16", 3, 1, 8 * D, 14)
    ws = c.workspace(gqa, 3, 1, 8)
    nb = (c.cache if kind == "kv4" else c.k).shape[0]
    for what in ("id", "negative id", "sink's id", "long", "negative length"):
        t, ln = c.tab.copy(), list(lens)
        if what in ("id", "negative id"):
            t[1, 1 if what == "id" else 2] = nb if what == "id" else -7
        elif what == "sink's id":
            t[1, 0] = nb
        else:
            ln[1] = 10 ** 6 if what == "long" else -5
        if what == "long":
            t[1] = t[0]
        o = c.run(gqa, q, 8, tab=t, lens=ln, window=30, sinks=2, workspace_tensor=ws)
        assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG, what
        c.check(o, q, 8, what, some=[0, 2], window=30, sinks=2)
        if what == "negative length":
            assert (o[1] == 0).all()
    c.run(gqa, q, 8, tab=c.tab, window=30, sinks=2, workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("hq,N,lens,worker", [(16, 8, 4000, 3), (160, 8, 4000, 1), (8, 1, 8000, 1)])
def test_timeout_is_reported_not_hung(gqa, kind, hq, N, lens, worker):
    """A worker whose second tile never comes: one warp, two warps on a ring, the short form."""
    c = Case(kind, "f16", [lens] * N, 128, 4, 16, 105)
    q = queries("f16", N, 1, hq * 128, 15)
    ws = c.workspace(gqa, N, 1, hq)
    tab = c.tab if N > 1 else np.ascontiguousarray(c.tab[:, :lens // 16 + 1])
    c.run(gqa, q, hq, tab=tab, workspace_tensor=ws, timeout_us=20000, test_stall_cta=worker)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_TIMEOUT
    o = c.run(gqa, q, hq, tab=tab, workspace_tensor=ws)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
    c.check(o, q, hq, some=[0])


# ---------------------------------------------------------------- both forms of the launch
SHORT = [  # D, hq, hk, T, bs, sequences, blocks of the table
    (128, 16, 8, 1, 32, 16, 64), (64, 16, 8, 1, 64, 16, 32), (128, 8, 8, 1, 32, 18, 8), (128, 32, 4, 1, 16, 10, 32),
    (64, 60, 5, 1, 8, 4, 125), (64, 8, 2, 1, 16, 1, 256), (128, 8, 1, 4, 8, 5, 260), (128, 16, 4, 12, 16, 8, 40),
    (64, 80, 2, 1, 32, 12, 36), (64, 64, 1, 1, 8, 3, 21), (128, 24, 2, 2, 16, 6, 50), (64, 7, 1, 3, 32, 20, 30),
    (128, 40, 1, 1, 16, 9, 64), (64, 48, 2, 2, 8, 8, 120)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,hq,hk,T,bs,N,blocks", SHORT)
def test_both_forms(gqa, kind, D, hq, hk, T, bs, N, blocks):
    """A table that bounds the sequences takes the short form where they are few, a wide one the general form, a window the
    short one again; the values are the same."""
    full = blocks * bs
    lens = ([full, 0, 1, full - 1, 33, full // 2 + 5, 64, full - 33, 32, full // 3] * 2)[:N]
    c = Case(kind, "f16", lens, D, hk, bs, 160 + hq + T)
    tab = np.ascontiguousarray(np.pad(c.tab, ((0, 0), (0, blocks)), constant_values=-1)[:, :blocks])
    wide = np.ascontiguousarray(np.pad(tab, ((0, 0), (0, 40000 // bs)), constant_values=-1))
    q = queries("f16", N, T, hq * D, 16)
    for window, sinks in ((0, 0), (full // 3, 4)):
        for t in (tab, wide):
            for causal in (False, True):
                ws = c.workspace(gqa, N, T, hq)
                ws[256:] = 0xA5
                o = c.run(gqa, q, hq, tab=t, causal=causal, window=window, sinks=sinks, workspace_tensor=ws)
                assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
                c.check(o, q, hq, causal=causal, window=window, sinks=sinks)


# ---------------------------------------------------------------- streams, graphs, threads, devices' memory
@pytest.mark.parametrize("kind", KINDS)
def test_graphs_replay_with_other_lengths_and_do_not_share(gqa, kind):
    D, hq, hk, bs = 128, 8, 2, 16
    c = Case(kind, "bf16", [5000, 900, 3000], D, hk, bs, 110)
    pools = [x.cuda() for x in ((c.cache,) if kind == "kv4" else (c.k, c.v))]
    tab = torch.from_numpy(c.tab).cuda()
    call = gqa.gqa_decode_kv4 if kind == "kv4" else gqa.gqa_decode_window
    graphs = []
    for i in range(2):
        q, lens = queries("bf16", 3, 1, hq * D, 20 + i), torch.tensor(c.lens).int().cuda()
        qd, s = q.cuda(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            o = call(qd, *pools, tab, lens, hq, hk, window=1500, sinks=4)
        graphs.append((g, q, qd, lens, o))
    streams = [torch.cuda.Stream() for _ in graphs]
    for new in ([5000, 900, 3000], [17, 900, 2999], [0, 1, 4]):
        c.lens = new
        for _, _, _, lens, _ in graphs:
            lens.copy_(torch.tensor(new).int())
        torch.cuda.synchronize()
        for _ in range(5):
            for (g, *_), s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for _, q, _, _, o in graphs:
            c.check(o, q, hq, str(new), window=1500, sinks=4)
    assert gqa.gqa_status_check() == gqa.GQA_OK


@pytest.mark.parametrize("kind", KINDS)
def test_other_streams_and_threads(gqa, kind):
    D, hq, hk, bs = 64, 8, 2, 16
    c = Case(kind, "f16", [3000, 70, 5000], D, hk, bs, 111)
    qs = [queries("f16", 3, 1, hq * D, 30 + i) for i in range(4)]
    want = [c.run(gqa, q, hq, window=900, sinks=3) for q in qs]
    pools = [x.cuda() for x in ((c.cache,) if kind == "kv4" else (c.k, c.v))]
    tab, lens = torch.from_numpy(c.tab).cuda(), torch.tensor(c.lens).int().cuda()
    call = gqa.gqa_decode_kv4 if kind == "kv4" else gqa.gqa_decode_window
    dev = [q.cuda() for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = [call(q, *pools, tab, lens, hq, hk, window=900, sinks=3, stream=s) for q, s in zip(dev, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    wrong = []

    def work(i):
        s = streams[0]                                   # all on one stream, with its workspace
        with torch.cuda.stream(s):
            for _ in range(50):
                o = call(dev[i], *pools, tab, lens, hq, hk, window=900, sinks=3)
                s.synchronize()
                if not torch.equal(o, want[i]):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


def test_calls_of_both_kinds_and_sizes_in_turn(gqa):
    """The stream's workspace grows, and serves other shapes, other row classes and the other calls between."""
    cases = [(Case("kv4", "f16", [4000, 50], 128, 2, 16, 112), 8), (Case("rows", "bf16", [2000] * 3, 64, 1, 8, 113), 40),
             (Case("rows", "f16", [9000], 128, 1, 32, 114), 64), (Case("kv4", "bf16", [700] * 50, 64, 4, 64, 115), 8)]
    for _ in range(2):
        for c, hq in cases:
            q = queries(c.elem, len(c.lens), 1, hq * c.D, 31)
            c.check(c.run(gqa, q, hq, window=600, sinks=9), q, hq, some=[0], window=600, sinks=9)
    assert gqa.gqa_status_check() == gqa.GQA_OK


def test_status_of_calls_without_a_workspace(gqa):
    assert gqa.gqa_status_check() == gqa.GQA_OK
    for kind in KINDS:
        c = Case(kind, "f16", [100, 40], 64, 2, 16, 116)
        t = c.tab.copy()
        t[0, 5] = -9
        q = queries("f16", 2, 1, 8 * 64, 32)
        c.run(gqa, q, 8, tab=t, window=50)
        assert gqa.gqa_status_check() == gqa.GQA_ERR_INVALID_ARG and gqa.gqa_status_check() == gqa.GQA_OK


@pytest.mark.parametrize("kind", KINDS)
def test_offsets_past_32_bits(gqa, kind):
    D, hk, hq, bs = 128, 8, 16, 64
    row = hk * (D + D // 8) if kind == "kv4" else hk * D          # bytes, or elements, of a token in one array
    nb = (1 << 32) // (row * bs) + 50
    n, tail = 40 * bs, list(range(nb - 40, nb))
    c = Case(kind, "bf16", [n], D, hk, bs, 117)
    tab = np.array([tail], np.int32)
    small = c.tab[0]
    q = queries("bf16", 1, 1, hq * D, 33)
    tabd, lens = torch.from_numpy(tab).cuda(), torch.tensor([n]).int().cuda()
    if kind == "kv4":
        big = torch.zeros(nb, hk, bs * (D + D // 8), dtype=torch.uint8, device="cuda")
        big[nb - 40:] = c.cache[small].cuda()
        o = gqa.gqa_decode_kv4(q.cuda(), big, tabd, lens, hq, hk, window=2000, sinks=4)
        k, _ = gqa.gqa_kv4_read(big, tabd, lens, D, n)
        np.testing.assert_array_equal(npy(k[0, ::97]).reshape(-1, hk, D), c.kv(0, n)[0][::97])
        x = torch.randn(3, 2 * hk * D, generator=gen(1)).bfloat16().cuda()
        slots = torch.tensor([nb * bs - 1, nb * bs - 70, 5]).cuda()
        gqa.gqa_append(None, x[:, :hk * D], x[:, hk * D:], hk, hk, slots, big)
        t3 = torch.tensor([[nb - 1], [nb - 2], [0]]).int().cuda()
        back, _ = gqa.gqa_kv4_read(big, t3, torch.tensor([64, 64, 64]).int().cuda(), D, 64, dtype=torch.bfloat16)
        other = gqa.gqa_kv4_cache(1, 8, hk, D)
        gqa.gqa_append(None, x[:, :hk * D], x[:, hk * D:], hk, hk, torch.arange(3).cuda(), other)
        want, _ = gqa.gqa_kv4_read(other, torch.tensor([[0]]).int().cuda(), torch.tensor([3]).int().cuda(), D, 3, dtype=torch.bfloat16)
        assert torch.equal(torch.stack([back[0, 63], back[1, 58], back[2, 5]]), want[0])
    else:
        pools = []
        for x in (c.k, c.v):
            big = torch.zeros(nb, bs, hk * D, dtype=torch.bfloat16, device="cuda")
            big[nb - 40:] = x[small].cuda()
            pools.append(big)
        o = gqa.gqa_decode_window(q.cuda(), *pools, tabd, lens, hq, hk, window=2000, sinks=4)
    c.check(o, q, hq, window=2000, sinks=4)
    assert gqa.gqa_status_check() == gqa.GQA_OK


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("elem", ["f16", "bf16"])
def test_prompt_with_pictures_then_steps_then_verification(gqa, elem):
    """Tokens with three position axes go into the 4-bit cache and into 16-bit pools, and every step attends to what is there
    under a window; the cache read back is what the attention saw."""
    D, hq, hk, bs, blocks, rot = 64, 8, 2, 16, 24, 64
    g, dt = gen(90), DT[elem]
    cs = torch.rand(500, rot // 2, generator=g) * 6.28
    cs = torch.cat([cs.cos(), cs.sin()], 1).float().cuda()
    axes = gqa.gqa_pair_axes([12, 10, 10], in_turn=True)
    w = (1 + 0.1 * torch.randn(D, generator=g)).to(dt).cuda()
    cache = gqa.gqa_kv4_cache(blocks, bs, hk, D)
    pools = [torch.zeros(blocks, bs, hk * D, dtype=dt, device="cuda") for _ in range(2)]
    tab = torch.randperm(blocks, generator=g)[None].int()
    have = 0
    for new in (250, 1, 1, 4, 3):
        qkv = torch.randn(new, (hq + 2 * hk) * D, generator=g).to(dt).cuda()
        pos = torch.stack([torch.arange(have, have + new), torch.arange(new) // 8 + have, torch.arange(new) % 8 + have]).int().cuda()
        at = torch.arange(have, have + new)
        slots = (tab[0, at // bs].long() * bs + at % bs).cuda()
        parts = qkv[:, :hq * D], qkv[:, hq * D:(hq + hk) * D], qkv[:, (hq + hk) * D:]
        kw = dict(positions=pos, cos_sin=cs, pair_axes=axes, q_weight=w, k_weight=w)
        q = gqa.gqa_append(*parts, hq, hk, slots, cache, **kw)
        assert torch.equal(q, gqa.gqa_append(*parts, hq, hk, slots, *pools, **kw))
        have += new
        if new > 8:
            continue
        lens = torch.tensor([have]).int().cuda()
        for kind in KINDS:
            c = Case.__new__(Case)
            c.kind, c.elem, c.lens, c.D, c.hk, c.bs, c.tab = kind, elem, [have], D, hk, bs, tab.numpy()
            if kind == "kv4":
                c.cache = cache.cpu()
                o = gqa.gqa_decode_kv4(q[None], cache, tab.cuda(), lens, hq, hk, causal=True, window=60, sinks=4)
                k, v = gqa.gqa_kv4_read(cache, tab.cuda(), lens, D, have, dtype=dt)
                for x, y in zip((k, v), c.kv(0, have)):
                    np.testing.assert_array_equal(npy(x[0]).reshape(have, hk, D), y)
            else:
                c.k, c.v = (x.cpu() for x in pools)
                o = gqa.gqa_decode_window(q[None], *pools, tab.cuda(), lens, hq, hk, causal=True, window=60, sinks=4)
            c.check(o, q[None].cpu(), hq, f"{kind} {have}", causal=True, window=60, sinks=4)
    assert gqa.gqa_status_check() == gqa.GQA_OK


def test_binding_checks(gqa):
    c4, c16 = Case("kv4", "f16", [100], 128, 2, 16, 1), Case("rows", "f16", [100], 128, 2, 16, 1)
    q = queries("f16", 1, 1, 8 * 128, 1)
    for c in (c4, c16):
        for bad in (dict(window=-1), dict(sinks=-1), dict(window=3.5), dict(out=torch.zeros(1, 2, 1024).half().cuda()),
                    dict(causal=torch.ones(2)), dict(timeout_us=-1), dict(scale="x"),
                    dict(workspace_tensor=torch.zeros(256, dtype=torch.uint8))):
            with pytest.raises((ValueError, TypeError)):
                c.run(gqa, q, 8, **bad)
        with pytest.raises(gqa.GQAError):
            c.run(gqa, q, 8, workspace_tensor=torch.zeros(256, dtype=torch.uint8, device="cuda"))
        with pytest.raises(ValueError):
            c.run(gqa, q.float(), 8)
        with pytest.raises(gqa.GQAError):
            c.run(gqa, torch.zeros(1, 17, 8 * 128).half(), 8)               # 68 rows
    tab, lens = torch.from_numpy(c4.tab).cuda(), torch.tensor([100]).int().cuda()
    with pytest.raises(ValueError):
        gqa.gqa_decode_kv4(q.cuda(), gqa.gqa_kv8_cache(8, 16, 2, 128), tab, lens, 8, 2)
    with pytest.raises(ValueError):
        gqa.gqa_decode_kv8(q.cuda(), c4.cache.cuda(), tab, lens, 8, 2)
    with pytest.raises(ValueError):
        gqa.gqa_decode_window(q.cuda(), c16.k.cuda(), c16.v.cuda().bfloat16(), tab, lens, 8, 2, window=4)
    with pytest.raises(ValueError):
        gqa.gqa_decode_window(q.cuda(), c16.k.cuda(), c16.v.cuda()[:, :8], tab, lens, 8, 2, window=4)
    with pytest.raises(ValueError):
        gqa.gqa_decode_kv4(q.cuda(), c4.cache.cuda(), tab.long(), lens, 8, 2)


def test_bounds_checked_build(gqa):
    """The same calls through the checked library: no offset leaves its buffer."""
    import ctypes

    from decode_attention_03_gb300 import build
    lib = gqa.open_library(build.build(checked=True))
    assert lib.gqa_build_flags() == gqa.GQA_BUILD_BOUNDS_CHECK
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    opt = gqa._opts(causal=True)
    for D, hq, hk, T, bs, lens, window, sinks in [(128, 8, 2, 3, 16, [1000, 0, 33, 64], 100, 5), (64, 6, 3, 1, 8, [7, 513, 90], 0, 0),
                                                  (128, 64, 2, 2, 64, [3000, 129], 700, 40), (64, 8, 1, 4, 32, [95], 33, 1),
                                                  (128, 4, 1, 1, 16, [5000] * 200, 900, 4)]:
        N = len(lens)
        q = queries("f16", N, T, hq * D, 40)
        for kind in KINDS:
            c = Case(kind, "f16", lens, D, hk, bs, 118)
            ws = c.workspace(gqa, N, T, hq)
            qd, o = q.cuda(), torch.empty_like(q).cuda()
            tab, ln = torch.from_numpy(c.tab).cuda(), torch.tensor(lens).int().cuda()
            pools = [x.cuda() for x in ((c.cache,) if kind == "kv4" else (c.k, c.v))]
            call = lib.gqa_decode_kv4 if kind == "kv4" else lib.gqa_decode_window
            st = call(p(qd), *map(p, pools), p(tab), p(ln), p(o), N, T, c.tab.shape[1], pools[0].shape[0], bs, hq, hk, D, D ** -0.5,
                      window, sinks, p(ws), ws.numel(), None, None, ctypes.byref(opt))
            torch.cuda.synchronize()
            assert st == gqa.GQA_OK and lib.gqa_workspace_check(p(ws), None) == gqa.GQA_OK, (D, kind)
            c.check(o, q, hq, some=range(min(N, 4)), causal=True, window=window, sinks=sinks)
            if kind == "kv4":
                k, v = (torch.zeros(N, max(lens), hk * D, dtype=torch.float16, device="cuda") for _ in range(2))
                st = lib.gqa_kv4_read(p(pools[0]), p(tab), p(ln), None, p(k), p(v), N, max(lens), c.tab.shape[1], pools[0].shape[0],
                                      bs, hk, D, p(ws), 256, None, ctypes.byref(gqa._opts()))
                torch.cuda.synchronize()
                assert st == gqa.GQA_OK and lib.gqa_workspace_check(p(ws), None) == gqa.GQA_OK
                np.testing.assert_array_equal(npy(v[0, :lens[0]]).reshape(-1, hk, D), c.kv(0, lens[0])[1])
    T, D, hq, hk, bs = 300, 64, 6, 3, 8
    g = gen(41)
    qkv = torch.randn(T, (hq + 2 * hk) * D, generator=g).half().cuda()
    cs, pos = torch.rand(20, 40, generator=g).cuda(), torch.randint(0, 20, (3, T), generator=g).int().cuda()
    axes, slots = torch.randint(0, 3, (20,), generator=g).byte().cuda(), torch.arange(T).cuda()
    cache, q_out = gqa.gqa_kv4_cache(T // bs + 1, bs, hk, D), torch.empty(T, hq * D, dtype=torch.float16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    n, w = (hq + 2 * hk) * D, torch.ones(D).half().cuda()
    a = gqa.gqa_append_args(q=p(qkv), k=p(qkv[:, hq * D:]), v=p(qkv[:, (hq + hk) * D:]), q_out=p(q_out), q_stride=n, k_stride=n,
                            v_stride=n, q_out_stride=hq * D, q_weight=p(w), k_weight=p(w), cos_sin=p(cs), positions=p(pos),
                            slots=p(slots), k_cache=p(cache), v_cache=None, num_tokens=T, h_q=hq, h_kv=hk, d_head=D, max_position=20,
                            rot_dim=40, interleaved=0, num_blocks=cache.shape[0], block_size=bs, cache_layout=gqa.GQA_CACHE_KV4,
                            bf16=0, eps=1e-6)
    assert lib.gqa_append_axes(ctypes.byref(a), p(axes), 3, p(ws), 256, None) == gqa.GQA_OK
    assert lib.gqa_workspace_check(p(ws), None) == gqa.GQA_OK
    again = torch.zeros_like(cache)
    q2 = gqa.gqa_append(qkv[:, :hq * D], qkv[:, hq * D:(hq + hk) * D], qkv[:, (hq + hk) * D:], hq, hk, slots, again, positions=pos,
                        cos_sin=cs, pair_axes=axes, q_weight=w, k_weight=w)
    assert torch.equal(again, cache) and torch.equal(q2, q_out)


def test_the_first_call_of_a_process_is_captured(gqa):
    """Nothing of the library was called before on the device: the capture makes everything that it needs."""
    import os
    import subprocess
    import sys
    code = """
import torch, decode_attention_03_gb300 as gqa
dev = "cuda"
cache = gqa.gqa_kv4_cache(4, 16, 2, 128)
pools = [torch.zeros(4, 16, 256, dtype=torch.float16, device=dev) for _ in range(2)]
x, q = torch.randn(3, 512, device=dev).half(), torch.randn(1, 1024, device=dev).half()
slots, tab = torch.arange(3, device=dev), torch.arange(4, dtype=torch.int32, device=dev)[None]
ln = torch.tensor([3], dtype=torch.int32, device=dev)
cs = torch.rand(9, 128, device=dev)
kw = dict(positions=torch.randint(0, 9, (3, 3), device=dev).int(), cos_sin=cs, pair_axes=gqa.gqa_pair_axes([16, 24, 24]))
back = [torch.zeros(1, 8, 256, dtype=torch.float16, device=dev) for _ in range(2)]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    gqa.gqa_append(None, x[:, :256], x[:, 256:], 2, 2, slots, cache, **kw)
    gqa.gqa_append(None, x[:, :256], x[:, 256:], 2, 2, slots, *pools, **kw)
    a = gqa.gqa_decode_kv4(q, cache, tab, ln, 8, 2, window=2, sinks=1)
    b = gqa.gqa_decode_window(q, *pools, tab, ln, 8, 2, window=2, sinks=1)
    gqa.gqa_kv4_read(cache, tab, ln, 128, k_out=back[0], v_out=back[1])
g.replay()
assert gqa.gqa_status_check() == gqa.GQA_OK
assert torch.equal(a, gqa.gqa_decode_kv4(q, cache, tab, ln, 8, 2, window=2, sinks=1))
assert torch.equal(b, gqa.gqa_decode_window(q, *pools, tab, ln, 8, 2, window=2, sinks=1))
k, v = gqa.gqa_kv4_read(cache, tab, ln, 128, 8)
assert torch.equal(k, back[0]) and torch.equal(v, back[1]) and bool((k != 0).any())
tab[0, 0] = 4
g.replay()
assert gqa.gqa_status_check() == gqa.GQA_ERR_INVALID_ARG and gqa.gqa_status_check() == gqa.GQA_OK
print("captured first")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("kind", KINDS)
def test_no_sequences_and_no_keys(gqa, kind):
    c = Case(kind, "bf16", [0, 0, 0], 128, 2, 16, 119)
    q = queries("bf16", 3, 2, 8 * 128, 50)
    for window in (0, 5):
        for causal in (False, True):
            out = torch.full_like(q, 7.0).cuda()
            assert (c.run(gqa, q, 8, causal=causal, window=window, sinks=1, out=out) == 0).all()
    wide = np.full((3, 4000), -1, np.int32)                  # the general form
    assert (c.run(gqa, q, 8, tab=wide, window=0) == 0).all()
    none = c.run(gqa, q[:0], 8, tab=np.zeros((0, 4), np.int32), lens=[])
    assert none.shape == (0, 2, 8 * 128) and gqa.gqa_status_check() == gqa.GQA_OK


@pytest.mark.parametrize("seed", range(40))
def test_random_configurations(gqa, seed):
    import random
    r = random.Random(1000 + seed)
    kind, elem, D, bs = r.choice(KINDS), r.choice(["f16", "bf16"]), r.choice([64, 128]), r.choice([8, 16, 32, 64])
    hk = r.choice([1, 2, 3, 5, 8])
    G = r.choice([1, 2, 3, 4, 5, 7, 8, 16])
    T = r.randint(1, max(1, min(9, 64 // G)))
    N = r.choice([1, 2, 5, 17, 60])
    top = r.choice([40, 300, 2500]) if N < 60 else 300
    lens = [r.randint(0, top) for _ in range(N)]
    c = Case(kind, elem, lens, D, hk, bs, 2000 + seed)
    q = queries(elem, N, T, G * hk * D, 3000 + seed)
    some = r.sample(range(N), min(N, 6))
    for _ in range(3):
        window, sinks, causal = r.choice([0, 1, r.randint(1, 60), r.randint(1, top)]), r.choice([0, 1, 4, r.randint(0, top)]), r.random() < 0.6
        ws = c.workspace(gqa, N, T, G * hk)
        o = c.run(gqa, q, G * hk, causal=causal, window=window, sinks=sinks, workspace_tensor=ws)
        assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
        c.check(o, q, G * hk, f"window {window}, sinks {sinks}, causal {causal}", some=some, causal=causal, window=window, sinks=sinks)
