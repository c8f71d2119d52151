"""What build.py needs, and when it builds again."""
import os
import subprocess
import sys
import textwrap

import pytest

import io_aware_exact_06_gb300 as fa
from io_aware_exact_06_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_library_needs_no_torch():
    """Without torch the library is built all the same, and its calls work."""
    build.build()
    script = textwrap.dedent(f"""
        import sys
        sys.path.insert(0, {ROOT!r})
        sys.modules["torch"] = None  # import torch raises
        from io_aware_exact_06_gb300 import build
        assert build.build() == build.LIB
        import io_aware_exact_06_gb300 as fa
        assert fa.attn_fwd_tree_workspace(2, 10, 8, 4, 128, 8, 4096, 8) > 0
        print("ok")
    """)
    out = subprocess.run([sys.executable, "-c", script], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and "ok" in out.stdout, out.stderr[-2000:]


def test_the_module_belongs_to_one_torch(monkeypatch):
    """The module built against this torch is not loaded into another one."""
    torch = pytest.importorskip("torch")
    build.build()
    monkeypatch.setattr(fa, "_serve", None)
    monkeypatch.setattr(torch, "__version__", "9.9.9+other")
    with pytest.raises(RuntimeError, match="not built"):
        fa._native()
    monkeypatch.undo()
    assert fa._native() is fa._native()
