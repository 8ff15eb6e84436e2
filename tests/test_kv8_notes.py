"""The notes by which the workers of gqa_decode_kv8 tell its merge kernel what to fold: the checks of csrc/kv8_notes.h, compiled
for the host, let no note through whose addresses lie outside of the output or the workspace, and every note that a worker
writes (no GPU)."""
import itertools
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_attention_03_gb300", "csrc")
PROGRAM = """
#include <cstdio>
#include "kv8_notes.h"
int main() {
  gqa::Kv8Note n;
  int workers, sequences, heads;
  while (std::scanf("%d %d %d %d %d %d %d", &n.pieces, &n.first, &n.b, &n.g, &workers, &sequences, &heads) == 7) {
    const bool ok = gqa::kv8_note_ok(n, workers, sequences, heads);
    std::printf("%d", ok ? 1 : 0);
    if (ok)
      for (int i = 0; i < n.pieces; ++i) std::printf(" %d", gqa::kv8_slot(n, i));
    std::printf("\\n");
  }
}
"""


@pytest.fixture(scope="module")
def follow(tmp_path_factory):
    d = tmp_path_factory.mktemp("notes")
    (d / "notes.cpp").write_text(PROGRAM)
    exe = str(d / "notes")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "notes.cpp"), "-o", exe], check=True)

    def run(lines):
        text = "\n".join(" ".join(map(str, x)) for x in lines)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        return [[int(v) for v in x.split()] for x in out]
    return run


def test_no_note_leads_outside(follow):
    big = [-2 ** 31, -2 ** 31 + 1, -1, 2 ** 30, 2 ** 31 - 2, 2 ** 31 - 1]
    cases = []
    for workers, sequences, heads in [(1, 1, 1), (2, 3, 1), (5, 1, 2), (7, 4, 3)]:
        for p, f in itertools.product(list(range(0, workers + 3)) + big, list(range(0, 2 * workers + 3)) + big):
            cases.append((p, f, 0, heads - 1, workers, sequences, heads))
        for b, g in itertools.product(list(range(0, sequences + 2)) + big, list(range(0, heads + 2)) + big):
            cases.append((2, 0, b, g, workers, sequences, heads))
    good = 0
    for c, got in zip(cases, follow(cases)):
        p, f, b, g, workers, sequences, heads = c
        inside = p >= 2 and 0 <= b < sequences and 0 <= g < heads and f >= 0 and (f & ~1) + 2 * (p - 1) < 2 * workers
        assert got[0] == inside, c
        if inside:
            assert all(0 <= s < 2 * workers for s in got[1:]) and len(set(got[1:])) == p, c
            good += 1
    assert good > 50


def test_every_note_of_a_worker_is_followed(follow):
    """The workers' shares and notes restated: the slots of a unit are those that its pieces went to."""
    rng = np.random.default_rng(1)
    cases, want = [], []
    for _ in range(60):
        workers, heads = int(rng.integers(2, 40)), int(rng.integers(1, 4))
        tiles = rng.integers(0, 30, int(rng.integers(1, 8))).tolist()
        units = [(b, g, n) for b, n in enumerate(tiles) for g in range(heads) if n]
        total = sum(n for _, _, n in units)
        if total == 0:
            continue
        share = -(-total // workers)
        start = np.concatenate([[0], np.cumsum([n for _, _, n in units])])
        for w in range(workers):
            f0 = w * share
            if f0 >= total:
                continue
            u = int(np.searchsorted(start, f0, side="right")) - 1
            b, g, n = units[u]
            t = f0 - int(start[u])
            if not 0 < t <= share:
                continue
            cases.append((1 + -(-(n - t) // share), 2 * (w - 1) + (1 if t < share else 0), b, g, workers, len(tiles), heads))
            slots = []
            for x in range(w - 1, workers):             # the workers that have tiles of this unit
                lo, hi = max(x * share, int(start[u])), min((x + 1) * share, int(start[u + 1]))
                if lo < hi:
                    slots.append(2 * x if lo == x * share else 2 * x + 1)
            want.append(slots)
    assert len(cases) > 100
    for c, got, slots in zip(cases, follow(cases), want):
        assert got == [1] + slots, (c, got, slots)
