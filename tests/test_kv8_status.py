"""Host-side refusals of gqa_decode_kv8_status (no GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def b():
    from decode_attention_03_gb300 import build
    build.build()
    import decode_attention_03_gb300._binding as binding
    return binding


def test_refusals(b):
    buf = ctypes.create_string_buffer(4096 + 64)
    p = (ctypes.addressof(buf) + 15) & ~15

    def dec(N=1, T=1, hq=8, hk=2, d=128, ws=p, wsb=1 << 30, status=p):
        return b.lib.gqa_decode_kv8_status(p, p, p, p, p, N, T, 4, 4, 16, hq, hk, d, 0.1, ws, wsb, status, None, None)

    assert dec(N=0) == b.GQA_OK
    for bad in [dict(status=None), dict(status=p + 4), dict(ws=None), dict(N=-1), dict(hq=7)]:
        assert dec(**bad) == b.GQA_ERR_INVALID_ARG, bad
    assert dec(d=80) == b.GQA_ERR_UNSUPPORTED and dec(wsb=255) == b.GQA_ERR_WORKSPACE
