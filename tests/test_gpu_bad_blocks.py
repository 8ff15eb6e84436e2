"""Blocks with a bad id that some token sees: gqa_decode_kv4, gqa_decode_window and gqa_decode_kv8 take their keys and values for
zeros, whatever was computed before, and report them.  Values against the float64 oracles, as the other tests of these calls."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import test_gpu_kv8 as kv8
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


@pytest.mark.parametrize("elem", ["f16", "bf16"])
@pytest.mark.parametrize("bs", [8, 16, 32, 64])
@pytest.mark.parametrize("D,hq,hk,T", [(128, 8, 2, 1), (64, 8, 2, 2), (128, 32, 2, 1), (64, 24, 1, 1), (128, 16, 2, 4), (64, 64, 1, 1)])
def test_keys_of_bad_blocks_of_the_8_bit_cache_are_zeros(gqa, elem, bs, D, hq, hk, T):  # noqa: F811
    old, old_tab = kv8.make_cache([3000] * 20, D, hk, bs, 7)
    for lens in ([900], [1500, 70, 900, 333] * 6):
        cache, tab = kv8.make_cache(lens, D, hk, bs, 8)
        q = queries(elem, len(lens), T, hq * D, 9)
        for b, n in enumerate(lens):
            blocks = (n + bs - 1) // bs
            for j in (blocks - 1, blocks // 2, blocks // 2 + 1, 3 * blocks // 4):
                tab[b, j] = [cache.shape[0], -7, 1 << 30, -(1 << 31)][(b + j) % 4]
        tab[0, 0] = -1
        zeros = np.zeros_like(cache[:1])                # a block of rows of zeros, for the oracle
        zeros[..., 2 * bs * D:] = 1
        held, held_tab = np.concatenate([cache, zeros]), np.where((tab < 0) | (tab >= len(cache)), len(cache), tab)
        ws = torch.zeros(gqa.gqa_decode_kv8_workspace_size(len(lens), T, hq, hk, D), dtype=torch.uint8, device="cuda")
        kv8.run_decode(gqa, old, old_tab, [3000] * 20, queries(elem, 20, T, hq * D, 10), hq, hk)
        for causal in (True, False):
            o = kv8.run_decode(gqa, cache, tab, lens, q, hq, hk, causal=causal, workspace_tensor=ws)
            assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
            kv8.check_decode(o, held, held_tab, lens, q, hq, hk, D, D ** -0.5, bs, causal, elem, f"causal {causal}")
            assert torch.equal(o, kv8.run_decode(gqa, cache, tab, lens, q, hq, hk, causal=causal, workspace_tensor=ws))
            assert gqa.gqa_workspace_check(ws) == gqa.GQA_ERR_INVALID_ARG
