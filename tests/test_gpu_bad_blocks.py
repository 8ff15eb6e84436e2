"""Blocks with a bad id that some token sees: gqa_decode_kv4 and gqa_decode_window take their keys and values for zeros,
whatever was computed before, and report them.  Values against the float64 oracle, as tests/test_gpu_window.py."""
from __future__ import annotations

import pytest
import torch

from test_gpu_window import KINDS, Case, gqa, queries  # noqa: F401  (gqa: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("D,hq,hk,T", [(128, 8, 2, 1), (64, 8, 2, 2), (128, 32, 2, 1), (64, 24, 1, 1), (128, 16, 2, 4), (64, 64, 1, 1)])
def test_keys_of_bad_blocks_are_zeros(gqa, elem, kind, bs, D, hq, hk, T):  # noqa: F811
    before = Case(kind, elem, [3000] * 20, D, hk, bs, 7)          # leaves its keys in the rings
    for lens in ([900], [1500, 70, 900, 333] * 6):
        c = Case(kind, elem, lens, D, hk, bs, 8)
        q = queries(elem, len(lens), T, hq * D, 9)
        nb = (c.cache if kind == "kv4" else c.k).shape[0]
        for b, n in enumerate(lens):
            blocks = (n + bs - 1) // bs
            for j in (blocks - 1, blocks // 2, blocks // 2 + 1, 3 * blocks // 4):
                c.tab[b, j] = [nb, -7, 1 << 30, -(1 << 31)][(b + j) % 4]
        c.tab[0, 0] = -1
        ws = c.workspace(gqa, len(lens), T, hq)
        for window, sinks in ((0, 0), (400, 5)):
            before.run(gqa, queries(elem, 20, T, hq * D, 10), hq)
            o = c.run(gqa, q, hq, causal=True, window=window, sinks=sinks, workspace_tensor=ws)
            assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
            c.check(o, q, hq, f"window {window}", causal=True, window=window, sinks=sinks)
            assert torch.equal(o, c.run(gqa, q, hq, causal=True, window=window, sinks=sinks, workspace_tensor=ws))
            assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
