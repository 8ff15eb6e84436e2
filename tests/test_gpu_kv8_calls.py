"""How the cache operators are called: host threads on one stream, empty calls, captured calls and where their reports go,
arguments that are no numbers."""
from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

from oracle import kv8_oracle as ko

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gqa():
    from decode_attention_03_gb300 import build
    build.build()
    import decode_attention_03_gb300._binding as b
    assert torch.cuda.is_available()
    return b


def gen(seed):
    return torch.Generator().manual_seed(seed)


def sequences(gqa, lens, hk, D, bs, seed, room=0):
    """(cache, tables, lens) on the GPU: random keys and values, written by gqa_append."""
    need = [-(-n // bs) for n in lens]
    nb, wide = sum(need) + 1, max(max(need), 1) + room
    order = torch.randperm(nb, generator=gen(seed)).int()
    tab = torch.full((len(lens), wide), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        tab[b, :n] = order[at:at + n]
        at += n
    slots = torch.cat([tab[b, torch.arange(n) // bs].long() * bs + torch.arange(n) % bs for b, n in enumerate(lens)])
    x = torch.randn(len(slots), 2 * hk * D, generator=gen(seed + 1)).half().cuda()
    cache = gqa.gqa_kv8_cache(nb, bs, hk, D)
    gqa.gqa_append(None, x[:, :hk * D], x[:, hk * D:], hk, hk, slots.cuda(), cache)
    return cache, tab.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- host threads
def test_threads_on_one_stream(gqa):
    """Four host threads decode on the default stream, with its workspace, calls of one launch and of two: each gets what
    it gets alone."""
    cases = []
    for i, (lens, hq, hk, D, room) in enumerate([([3000, 500, 9000], 8, 2, 128, 0), ([3000, 500, 9000], 8, 2, 128, 0),
                                                 ([7000] * 6, 32, 8, 64, 0), ([200, 100], 4, 1, 128, 4000)]):
        x = sequences(gqa, lens, hk, D, 16, 200 + 7 * i, room)
        q = torch.randn(len(lens), hq * D, generator=gen(300 + i)).half().cuda()
        cases.append((q, *x, hq, hk))
    for c in cases:                        # the stream's workspace has its final size
        gqa.gqa_decode_kv8(*c)
    torch.cuda.synchronize()
    want = [gqa.gqa_decode_kv8(*c) for c in cases]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(cases))

    def work(i):
        torch.cuda.set_device(want[i].device)
        out = [torch.empty_like(want[i]) for _ in range(250)]
        start.wait()
        for o in out:
            gqa.gqa_decode_kv8(*cases[i], out=o)
        torch.cuda.synchronize()
        bad.append((i, sum(not torch.equal(o, want[i]) for o in out)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sorted(bad) == [(i, 0) for i in range(len(cases))]


# ---------------------------------------------------------------- calls without tokens
@pytest.mark.parametrize("layout", ["rows", "vllm", "kv8"])
def test_append_of_no_tokens(gqa, layout):
    """An empty call with norms and rotation is a no-op, as one without them."""
    D, hq, hk, bs = 128, 8, 2, 16
    x = torch.zeros(0, (hq + 2 * hk) * D, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    shapes = {"rows": [(4, bs, hk * D)] * 2, "vllm": [(4, hk, D // 8, bs, 8), (4, hk, D, bs)], "kv8": []}[layout]
    caches = [torch.full(s, 3.0, dtype=torch.bfloat16, device="cuda") for s in shapes] or \
        [torch.full((4, hk, bs * (2 * D + 2)), 9, dtype=torch.uint8, device="cuda")]
    before = [c.clone() for c in caches]
    none = dict(positions=torch.zeros(0, dtype=torch.int32, device="cuda"), cos_sin=torch.zeros(16, D, device="cuda"),
                q_weight=w, k_weight=w)
    for kw in ({}, none, dict(none, interleaved=True)):
        for q in (x[:, :hq * D], None):
            out = gqa.gqa_append(q, x[:, hq * D:(hq + hk) * D], x[:, (hq + hk) * D:], hq, hk,
                                 torch.zeros(0, dtype=torch.int64, device="cuda"), *caches, **kw)
            assert out is None if q is None else out.shape == (0, hq * D)
    assert all(torch.equal(a, b) for a, b in zip(caches, before))


# ---------------------------------------------------------------- arguments
def test_flags_that_are_neither_true_nor_false(gqa):
    """Refused before anything is launched."""
    D, hq, hk, bs = 64, 8, 2, 16
    x = torch.randn(3, (hq + 2 * hk) * D, generator=gen(1)).half().cuda()
    cache = gqa.gqa_kv8_cache(2, bs, hk, D)
    pos, cs = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones(4, D, device="cuda")
    slots = torch.arange(3, device="cuda")
    for flag in (torch.zeros(2), np.zeros(3)):
        with pytest.raises(ValueError, match="interleaved"):
            gqa.gqa_append(None, x[:, :hk * D], x[:, :hk * D], hq, hk, slots, cache, positions=pos, cos_sin=cs,
                           interleaved=flag)
        with pytest.raises(ValueError, match="causal"):
            gqa.gqa_decode_kv8(x[:, :hq * D].contiguous(), cache, slots.int().view(3, 1), pos, hq, hk, causal=flag)
    torch.cuda.synchronize()
    assert (cache == 0).all()
