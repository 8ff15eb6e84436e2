"""A wait limit of one microsecond: calls go through as they would with a longer one (a limit below the memory's latency would
let a kernel leave while its copies are on their way)."""
from __future__ import annotations

import pytest
import torch

from test_gpu_window import KINDS, Case, gqa, queries  # noqa: F401  (gqa: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,hq", [([700], 8), ([3000, 50, 900] * 10, 8), ([1000] * 8, 64)])
def test_paged_calls(gqa, kind, lens, hq):  # noqa: F811
    c = Case(kind, "f16", lens, 128, 2, 16, 5)
    q = queries("f16", len(lens), 1, hq * 128, 6)
    ws = c.workspace(gqa, len(lens), 1, hq)
    o = c.run(gqa, q, hq, workspace_tensor=ws, timeout_us=1)
    assert gqa.gqa_workspace_check(ws) == gqa.GQA_OK
    assert torch.equal(o, c.run(gqa, q, hq))
    if kind == "rows":
        args = [c.k.cuda(), c.v.cuda(), torch.from_numpy(c.tab).cuda(), torch.tensor(lens).int().cuda(), hq, 2]
        p = gqa.gqa_decode_paged(q[:, 0].cuda(), *args, max_seq_len=3000, timeout_us=1)
        assert torch.equal(p, gqa.gqa_decode_paged(q[:, 0].cuda(), *args, max_seq_len=3000))


@pytest.mark.parametrize("hq", [8, 64])
def test_contiguous_and_8_bit_calls(gqa, hq):  # noqa: F811
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(1, 2048, 2 * 128, generator=g).half().cuda() for _ in range(2))
    q = torch.randn(1, 1, hq * 128, generator=g).half().cuda()
    assert torch.equal(gqa.gqa_decode(q, k, v, hq, 2, timeout_us=1), gqa.gqa_decode(q, k, v, hq, 2))
    cache, tab, lens = gqa.gqa_kv8_cache(128, 16, 2, 128), torch.arange(128).int()[None].cuda(), torch.tensor([2048]).int().cuda()
    gqa.gqa_append(None, k[0], v[0], hq, 2, torch.arange(2048).cuda(), cache)
    assert torch.equal(gqa.gqa_decode_kv8(q, cache, tab, lens, hq, 2, timeout_us=1), gqa.gqa_decode_kv8(q, cache, tab, lens, hq, 2))
    assert gqa.gqa_status_check() == gqa.GQA_OK
