"""Bounded waits of the kernels, by their sources: a warp whose lanes shuffle, vote or synchronise after a wait gives it up
as a whole.  (A lane that alone went on, or alone left, would wait for the others for ever; that is not tried on a GPU.)"""
import os

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_attention_03_gb300", "csrc")


def waits(name):
    with open(os.path.join(CSRC, name)) as f:
        return [s.strip() for s in f if "mbar_wait_bounded(" in s]


def test_cache_decode_kernels_vote():
    """In the kernels over the caches every wait that decides something is a vote; the others are for copies in flight."""
    for name in ("gqa_kv8_decode.cuh", "gqa_win.cuh"):
        for line in waits(name):
            assert line.startswith("ptx::mbar_wait_bounded(") or "__all_sync(" in line, (name, line)


def test_the_limit_has_one_origin():
    """Every call's limit goes through the function that keeps it above the memory's latency."""
    found = 0
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh")):
            continue
        with open(os.path.join(CSRC, name)) as f:
            for line in f:
                if "timeout_ns = " in line:
                    assert "wait_limit_ns(opt.timeout_us)" in line, (name, line)
                    found += 1
    assert found == 4
