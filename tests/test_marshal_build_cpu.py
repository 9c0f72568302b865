"""When the argument marshalling of the small calls is built and loaded."""
from __future__ import annotations

import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_does_without_it():
    """A host without a compiler or torch's headers still has dispatch and combine; the small calls say what is missing."""
    r = subprocess.run([sys.executable, "-c", textwrap.dedent("""
        from combine_moe_get_gb300 import build

        def build_marshal(force=False):
            raise RuntimeError("no host compiler")
        build.build_marshal = build_marshal
        import torch
        from combine_moe_get_gb300 import binding as moe
        assert moe.moe_get_layout_workspace_size(128, 64, 8) > 0
        try:
            moe.moe_topk_gate(torch.zeros(4, 8), 2, status=torch.zeros(1, dtype=torch.int32))
        except RuntimeError as e:
            assert "no host compiler" in str(e)
        else:
            raise AssertionError("no error")
        """)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_another_torch_gets_a_build_of_its_own(monkeypatch):
    import torch

    from combine_moe_get_gb300 import build
    here = build.build_marshal()
    assert build.build_marshal() == here                    # not built again

    def run(cmd, **kw):
        raise RuntimeError("built again")
    monkeypatch.setattr(torch, "__version__", "0.0")
    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="built again"):
        build.build_marshal()
