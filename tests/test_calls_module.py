"""The extension module of the cache operators belongs to one torch and one Python: the rest of the binding works without it,
and a module that was built for another torch is refused by name (no GPU)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROBE = """
import sys, torch
sys.path.insert(0, {root!r})
{before}
import decode_attention_03_gb300 as gqa
assert gqa.gqa_version() > 0 and gqa.gqa_kv8_block_bytes(16, 128) == 16 * 258
assert callable(gqa.gqa_decode) and callable(gqa.gqa_decode_paged)
x, i = torch.zeros(4, 256, dtype=torch.float16), torch.zeros(4, dtype=torch.int64)
cache = torch.zeros(2, 2, 16 * 258, dtype=torch.uint8)
for _ in range(2):
    try:
        gqa.gqa_append(None, x, x, 2, 2, i, cache, workspace_tensor=cache)
    except Exception as e:
        print(type(e).__name__, e)
"""


@pytest.fixture(scope="module")
def build():
    from decode_attention_03_gb300 import build
    build.build()
    return build


def probe(root, before=""):
    r = subprocess.run([sys.executable, "-c", PROBE.format(root=root, before=before)], capture_output=True, text=True,
                       cwd=root, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    return r.stdout.splitlines()


def package_without(build, tmp_path, skip):
    to = tmp_path / "decode_attention_03_gb300"
    to.mkdir()
    for name in os.listdir(build.PKG):
        if not name.startswith("__pycache__") and not name.startswith(skip):
            (to / name).symlink_to(os.path.join(build.PKG, name))
    return str(tmp_path)


def test_the_module_is_used_where_it_fits(build):
    lines = probe(ROOT)
    assert len(lines) == 2 and all(x.startswith("ValueError") and "CUDA" in x for x in lines), lines


def test_without_the_module_the_other_calls_work(build, tmp_path):
    lines = probe(package_without(build, tmp_path, "_calls"))
    assert len(lines) == 2 and all(x.startswith("ImportError") and "rebuild" in x for x in lines), lines


def test_a_module_for_another_torch_is_named(build):
    lines = probe(ROOT, "torch.__version__ = '1.0.0'")
    assert len(lines) == 2 and all(x.startswith("ImportError") and "1.0.0" in x and build.torch_version() in x for x in lines)


def test_another_torch_or_python_builds_it_anew(build, tmp_path, monkeypatch):
    assert build.calls_up_to_date()
    monkeypatch.setattr(build, "torch_version", lambda: "1.0.0")
    assert not build.calls_up_to_date()
    monkeypatch.undo()
    assert build.calls_up_to_date()
    monkeypatch.setattr(build.sys, "version", "3.99")
    assert not build.calls_up_to_date()
