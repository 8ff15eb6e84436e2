"""How the cache operators are called: host threads on one stream, empty calls, captured calls and where their reports go,
arguments that are no numbers."""
from __future__ import annotations

import ctypes
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


@pytest.mark.parametrize("paged", [False, True])
def test_threads_on_one_stream_over_16_bit_caches(gqa, paged):
    """The same for the calls over contiguous and paged caches that fold their splits in a second launch."""
    D, hq, hk, bs, n, raw = 128, 8, 2, 16, 4096, torch.cuda.current_stream().cuda_stream
    size = max(gqa.gqa_paged_workspace_size(2, hq, hk, D, n, 512), gqa.gqa_decode_workspace_size(2, 1, n, hq, hk, D, 9))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    opt = ctypes.byref(gqa._opts(9, 1))
    calls, want, held = [], [], []
    for i in range(4):
        q = torch.randn(2, hq * D, generator=gen(500 + i)).half().cuda()
        k, v = (torch.randn(2, n, hk * D, generator=gen(510 + 2 * i + w)).half().cuda() for w in (0, 1))
        tab = torch.arange(2 * n // bs, dtype=torch.int32, device="cuda")
        ln = torch.full((2,), n - 100 * i, dtype=torch.int32, device="cuda")
        held += [q, k, v, tab, ln]
        at = [x.data_ptr() for x in (q, k, v, tab, ln)]
        if paged:
            calls.append(lambda out, p=at: gqa.lib.gqa_decode_paged(*p, out.data_ptr(), 2, n // bs, 2 * n // bs, bs, 512, hq,
                                                                    hk, D, D ** -0.5, n, ws.data_ptr(), size, raw))
        else:
            calls.append(lambda out, p=at: gqa.lib.gqa_decode_ex(*p[:3], out.data_ptr(), 2, 1, n, hq, hk, D, D ** -0.5,
                                                                 ws.data_ptr(), size, raw, opt))
        want.append(torch.empty_like(q))
        assert calls[i](want[i]) == gqa.GQA_OK
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(calls))

    def work(i):
        torch.cuda.set_device(want[i].device)
        out = [torch.empty_like(want[i]) for _ in range(2000)]
        start.wait()
        for o in out:
            calls[i](o)
        torch.cuda.synchronize()
        bad.append((i, sum(not torch.equal(o, want[i]) for o in out)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert sorted(bad) == [(i, 0) for i in range(len(calls))]


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


# ---------------------------------------------------------------- reports of calls without a workspace
def step(gqa, slots, x, cache, tab, lens, q, hq, hk, D, **kw):
    """One layer of a decode step: append, attention, and a look at the first tokens."""
    gqa.gqa_append(None, x[:, :hk * D], x[:, hk * D:], hk, hk, slots, cache)
    o = gqa.gqa_decode_kv8(q, cache, tab, lens, hq, hk, **kw)
    return o, gqa.gqa_kv8_read(cache, tab, lens, D, 8)[0]


def step_case(gqa, room=0, seed=400, lens=(900, 70, 3000)):
    D, hq, hk, bs = 128, 8, 2, 16
    cache, tab, ln = sequences(gqa, lens, hk, D, bs, seed, room)
    x = torch.randn(len(lens), 2 * hk * D, generator=gen(seed + 2)).half().cuda()
    q = torch.randn(len(lens), hq * D, generator=gen(seed + 3)).half().cuda()
    slots = torch.stack([tab[b, (n - 1) // bs].long() * bs + (n - 1) % bs for b, n in enumerate(lens)])
    return slots, x, cache, tab, ln, q, hq, hk, D


@pytest.mark.parametrize("room", [0, 2000])
def test_reports_of_replayed_calls(gqa, room):
    """Captured on a stream that had no call before: bad slots, blocks and lengths of a replay are reported, and the graph
    holds the library's kernels alone."""
    case = step_case(gqa, room)
    slots, cache, tab, ln = case[0], case[2], case[3], case[4]
    want = step(gqa, *case)
    torch.cuda.synchronize()
    assert gqa.gqa_status_check() == gqa.GQA_OK
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        got = step(gqa, *case)
    side = torch.cuda.Stream()

    def replay():
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        return gqa.gqa_status_check()

    assert replay() == gqa.GQA_OK and all(torch.equal(a, b) for a, b in zip(got, want))
    for t, at, bad in ((slots, 1, 1 << 40), (tab, (2, 5), cache.shape[0]), (ln, 0, -4)):
        keep = t[at].clone()
        t[at] = bad
        assert replay() == gqa.GQA_ERR_INVALID_ARG
        t[at] = keep
        assert replay() == gqa.GQA_OK and all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_timeout_of_a_replayed_call_is_reported(gqa):
    case = step_case(gqa, 0, 410, [90000, 30000])
    tiles = 2 * (-(-90000 // 32) - (-30000 // 32))
    assert tiles > 2 * 8 * torch.cuda.get_device_properties(0).multi_processor_count       # a worker has a second tile
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        step(gqa, *case, timeout_us=20000, test_stall_cta=0)
    torch.cuda.synchronize()
    assert gqa.gqa_status_check() == gqa.GQA_OK
    graph.replay()
    assert gqa.gqa_status_check() == gqa.GQA_ERR_TIMEOUT
    assert gqa.gqa_status_check() == gqa.GQA_OK


def test_captured_calls_make_no_other_nodes(gqa):
    """A captured append, decode and read are as many nodes as they are launches: nothing is filled beside them."""
    if not hasattr(torch.cuda.CUDAGraph, "raw_cuda_graph"):
        pytest.skip("this torch does not give the captured graph away")
    nodes_of = ctypes.CDLL("libcuda.so.1").cuGraphGetNodes
    for room, kernels in ((0, 3), (2000, 4)):
        case = step_case(gqa, room)
        out = torch.empty_like(case[5])
        back = [torch.zeros(3, 8, 256, dtype=torch.float16, device="cuda") for _ in range(2)]
        graph, s = torch.cuda.CUDAGraph(keep_graph=True), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=s):
            slots, x, cache, tab, ln, q, hq, hk, D = case
            gqa.gqa_append(None, x[:, :hk * D], x[:, hk * D:], hk, hk, slots, cache)
            gqa.gqa_decode_kv8(q, cache, tab, ln, hq, hk, out=out)
            gqa.gqa_kv8_read(cache, tab, ln, D, k_out=back[0], v_out=back[1])
        n = ctypes.c_size_t(0)
        assert nodes_of(ctypes.c_void_p(graph.raw_cuda_graph()), None, ctypes.byref(n)) == 0
        assert n.value == kernels


def test_the_first_call_of_a_process_is_captured(gqa):
    """Nothing of the library was called before on the device: the capture makes everything that it needs."""
    import os
    import subprocess
    import sys
    code = """
import torch, decode_attention_03_gb300 as gqa
cache = gqa.gqa_kv8_cache(4, 16, 2, 128)
x = torch.randn(3, 512, device="cuda").half()
q = torch.randn(1, 1024, device="cuda").half()
slots = torch.arange(3, device="cuda")
tab = torch.arange(4, dtype=torch.int32, device="cuda")[None]
ln = torch.tensor([3], dtype=torch.int32, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    gqa.gqa_append(None, x[:, :256], x[:, 256:], 2, 2, slots, cache)
    o = gqa.gqa_decode_kv8(q, cache, tab, ln, 8, 2)
g.replay()
assert gqa.gqa_status_check() == gqa.GQA_OK
assert torch.equal(o, gqa.gqa_decode_kv8(q, cache, tab, ln, 8, 2))
slots[2] = 64
g.replay()
assert gqa.gqa_status_check() == gqa.GQA_ERR_INVALID_ARG and gqa.gqa_status_check() == gqa.GQA_OK
print("captured first")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_a_report_outlives_a_larger_call(gqa):
    """The stream's workspace grows between the report and the check."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        slots, x, cache, tab, ln, q, hq, hk, D = step_case(gqa, 2000, 420)
        tab[0, 3] = -2
        gqa.gqa_decode_kv8(q, cache, tab, ln, hq, hk)
        gqa.gqa_decode_kv8(torch.zeros(1, 8, 8 * D, dtype=torch.float16, device="cuda"), cache, tab[1:2], ln[1:2], 8, hk)
        assert gqa.gqa_workspace_check(gqa.workspace(256, use="status")) == gqa.GQA_ERR_INVALID_ARG
    assert gqa.gqa_status_check() == gqa.GQA_OK


def test_decode_with_a_status_word_of_its_own(gqa):
    """gqa_decode_kv8_status: the workspace is scratch from its first byte on."""
    _, _, cache, tab, ln, q, hq, hk, D = step_case(gqa, 2000, 430)
    want = gqa.gqa_decode_kv8(q, cache, tab, ln, hq, hk)
    ws = torch.full((gqa.gqa_decode_kv8_workspace_size(3, 1, hq, hk, D),), 0xC3, dtype=torch.uint8, device="cuda")
    status = torch.zeros(256, dtype=torch.uint8, device="cuda")
    raw = torch.cuda.current_stream().cuda_stream

    def call(out, table):
        return gqa.lib.gqa_decode_kv8_status(q.data_ptr(), cache.data_ptr(), table.data_ptr(), ln.data_ptr(), out.data_ptr(), 3,
                                             1, tab.shape[1], cache.shape[0], 16, hq, hk, D, D ** -0.5, ws.data_ptr(),
                                             ws.numel(), status.data_ptr(), raw, None)

    out = torch.empty_like(q)
    assert call(out, tab) == gqa.GQA_OK
    assert gqa.gqa_workspace_check(status) == gqa.GQA_OK and torch.equal(out, want)
    bad = tab.clone()
    bad[2, 0] = 1 << 20
    assert call(out, bad) == gqa.GQA_OK
    assert gqa.gqa_workspace_check(status) == gqa.GQA_ERR_INVALID_ARG and bool((ws[:256] == 0xC3).all())
