"""Builds of the extension with the calls from Python: which one is current, and
what works without it."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def compiled(monkeypatch, tmp_path):
    """Builds into a folder of the test with a compiler that only writes its output; the outputs it was asked for."""
    from nvfp4_precision_b200 import build
    done = []

    def run(cmd, check):
        done.append(os.path.basename(cmd[cmd.index("-o") + 1]).split(".so")[0])
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", run)
    return done


def test_the_extension_is_built_again_for_another_torch_or_python(compiled, monkeypatch):
    import torch

    from nvfp4_precision_b200 import build
    first = build.build_calls()
    assert os.path.exists(first) and len(compiled) == 1
    assert build.build_calls() == first and len(compiled) == 1
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    second = build.build_calls()
    assert second != first and len(compiled) == 2
    monkeypatch.setattr(sys.implementation, "cache_tag", "cpython-999")
    third = build.build_calls()
    assert third not in (first, second) and len(compiled) == 3
    assert build.build_calls(force=True) == third and len(compiled) == 4


def test_the_library_is_built_before_the_extension(monkeypatch):
    from nvfp4_precision_b200 import build
    order = []
    monkeypatch.setattr(build, "build_library", lambda *a: order.append("library"))
    monkeypatch.setattr(build, "build_calls", lambda *a: order.append("extension"))
    build.build()
    assert order == ["library", "extension"]


def test_the_attention_does_without_the_extension():
    """Import and the attention's entry points need the library alone; a linear layer says what is missing."""
    from nvfp4_precision_b200 import build
    build.build()
    code = ("import torch\n"
            "from nvfp4_precision_b200 import build\n"
            "build.calls_path = lambda: '/nonexistent/_calls.so'\n"
            "from nvfp4_precision_b200 import fp4attn as fa\n"
            "assert fa.fp4attn_workspace_bytes(1, 2, 300) > 0\n"
            "for call in (lambda: fa.fp4attn_norm_gate(torch.zeros(4, 64)),\n"
            "             lambda: fa.fp4attn_dequant_rows(torch.zeros(4, 32), torch.zeros(512))):\n"
            "    try:\n"
            "        call()\n"
            "    except ImportError as e:\n"
            "        assert 'build it' in str(e)\n"
            "    else:\n"
            "        raise SystemExit('no error')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
